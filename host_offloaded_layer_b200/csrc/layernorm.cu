// LayerNorm forward and backward over bf16 rows.
//
//   mean = sum_j x_j / H, rstd = 1 / sqrt(sum_j (x_j - mean)^2 / H + eps), xh = (x - mean) rstd, y = xh g + b
//   w = dy g, dx = rstd (w - mean_j(w) - xh mean_j(w xh)) + dres, dg = sum_rows dy xh, db = sum_rows dy
//
// Both are bound by HBM: the forward has to move 4 bytes an element, the backward 6 (8 with dres). So every
// element is read once: a group of W warps holds a whole row in registers, which also lets the variance be
// taken of x - mean (a second sum over registers, exact for rows whose mean is large against their spread).
// The backward's column sums dg and db come from the same pass: a thread owns the same columns of every row
// its group visits and keeps their sums in registers; a group adds its sums to the CTA's in shared memory, a
// CTA leaves one partial row, and a second small kernel adds the partial rows in a fixed order. No atomics:
// the result depends on the sizes alone.
//
// Rows come through a ring in shared memory that cp.async fills some rows ahead; a thread copies exactly the
// 16-byte vectors that it reads, so the ring needs no barrier, and what is in flight does not cost registers.
// The arithmetic is packed (two fp32 a register pair): unpacked, the forward was bound by instruction issue
// (72% of the slots at 2.2 TB/s of reads).
//
// Rows of any alignment take this path. A group's vectors are the 16-byte granules of memory that lie whole in
// its rows; where H or the row stride is odd, rows start at different places in their first granule, and that
// place (`shift`, in elements) repeats every 8 rows: groups step by multiples of 8 rows, so that each sees one
// shift and its threads keep their columns. The up to 14 elements of a row in front of its first and behind its
// last whole granule go to lanes of the group's last warp, one each, in plain loads and stores. (Only operands
// whose rows lie differently in their granules go an element at a time.)
//
// The times beside the variants below compare two builds as each choice was made. The kernels now, between events:
// forward 98304 x 3584 in 232 us, 32768 x 5120 in 126, 100000 x 1153 in 99; backward 98304 x 3584 in 366, 32768 x 5120
// in 188, 8192 x 3584 with dres in 52, 32768 x 5113 in 289, 100000 x 1153 in 158.
#include <algorithm>

#include "mt_internal.h"
#include "tcgen05.cuh"
#include "vec.cuh"

namespace mt {
namespace {

using namespace vec;

constexpr int SMS = 148;            // the partial rows of dg and db are counted for a whole B200, so that sums do not depend on the device
constexpr int DEPTH = 3;            // stages of a ring: two in flight, one being read
constexpr int MAX_H_REG = 8192;     // the widest row that 16 warps of two vectors a thread hold
constexpr int MAX_H = 1 << 28;      // and the widest of all, so that columns and their doubles count in 32 bits

__device__ __forceinline__ void group_bar(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Sums of N values over the W warps of this thread's group, in every thread. red: [32 warps][N] floats of the
// group, a buffer that the next call does not use (two in turn: a warp that runs ahead writes the other one).
template <int N>
__device__ __forceinline__ void group_sums(float (&v)[N], int W, int warp_in_group, int bar_id, float* red) {
  warp_sums<N>(v);
  if (W == 1) return;
  const int lane = threadIdx.x & 31;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < N; ++i) red[warp_in_group * N + i] = v[i];
  }
  group_bar(bar_id, W * 32);
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = lane < W ? red[lane * N + i] : 0.f;
  warp_sums<N>(v);
}

// 16 bytes from global to shared memory.
__device__ __forceinline__ void copy_async(uint32_t dst, const void* p) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(p) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// `bytes` (a multiple of 16) from global to shared memory, counted by the barrier at `bar`; all 16-byte aligned.
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* p, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(p),
               "r"(bytes), "r"(bar)
               : "memory");
}

__device__ __forceinline__ void lds128(uint32_t at, uint32_t (&w)[4]) {
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at) : "memory");
}

// 1 / sqrt(v): the fast approximation (2 units in the last place) and one Newton step; not where that is 0 or infinite
// (a variance that left fp32, or none and no eps), which the step would make NaN.
// (1 / sqrtf(v) in its place: 98304 x 3584 in 248 us, against 227.)
__device__ __forceinline__ float inv_sqrt(float v) {
  const float r = rsqrtf(v);
  const float c = fmaf(-v * r, r, 1.0f);
  return c == c ? fmaf(0.5f * r, c, r) : r;
}

// s / H: the product with the rounded 1 / H, and what it leaves of s divided likewise. Without that the mean of a row of
// equal elements is a step beside them, which a small spread and eps make visible (H = 3584, elements of 1000, eps = 1e-6:
// xh = 0.09 in place of 0). An infinite sum stays as it is. (s / H as one operation: 98304 x 3584 in 245 us, against 229.)
__device__ __forceinline__ float row_mean(float s, float inv_h, float h) {
  const float m = s * inv_h, left = fmaf(-m, h, s);
  return left == left ? fmaf(left, inv_h, m) : m;
}

// A thread's NV vectors of a row whose first element is the shift-th of its granule: vector t + k T holds the
// columns col[k] .. col[k] + 7, all in the row, or is absent. EDGE: rows may have elements outside their whole
// granules; edge is the column of one that this lane has, or -1. (A mask for partial vectors instead, in the threads
// that hold them, made their warp the one that its group waits for: 100000 x 1153 took 159 us, against 97.)
template <int NV, bool EDGE>
struct Cols {
  int col[NV], edge;
  bool there[NV];
  __device__ __forceinline__ Cols(int t, int T, int shift, int H) {
    const int head = EDGE ? min((8 - shift) & 7, H) : 0, tail = EDGE ? (H - head) & 7 : 0;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      col[k] = head + 8 * (t + k * T);
      there[k] = col[k] + 8 <= H;
    }
    const int e = t - (T - 32);
    edge = !EDGE || e < 0 || e >= head + tail ? -1 : e < head ? e : H - tail + (e - head);
  }
  __device__ __forceinline__ bool any(int k) const { return there[k]; }
  __device__ __forceinline__ bool has_edge() const { return EDGE && edge >= 0; }
  // Starts the copy of a vector of the row.
  __device__ __forceinline__ void fetch(int k, uint32_t dst, const __nv_bfloat16* row) const {
    if (any(k)) copy_async(dst, row + col[k]);  // an absent one's place in the ring holds zeros from the start
  }
  __device__ __forceinline__ void store(int k, __nv_bfloat16* row, const uint32_t (&w)[4]) const {
    if (any(k)) *reinterpret_cast<uint4*>(row + col[k]) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  // Zeros for the absent vectors of `slots` places of the ring, `pitch` bytes apart.
  __device__ __forceinline__ void clear_absent(uint32_t ring, int T, int slots, uint32_t pitch) const {
#pragma unroll
    for (int k = 0; k < NV; ++k)
      if (!any(k))
        for (int i = 0; i < slots; ++i)
          asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(ring + i * pitch + k * T * 16), "r"(0) : "memory");
  }
  // bf16 values of a vector over the columns (gain or bias), `fill` where there are none
  __device__ __forceinline__ void gather(int k, const __nv_bfloat16* p, float fill, f2 (&v)[4]) const {
    const bool have = p && any(k);
    if (!EDGE && have && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
      uint32_t w[4];
      words(__ldg(reinterpret_cast<const uint4*>(p + col[k])), w);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = f2_of(w[i]);
      return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = f2_make(have ? __bfloat162float(p[col[k] + 2 * i]) : fill, have ? __bfloat162float(p[col[k] + 2 * i + 1]) : fill);
  }
  __device__ __forceinline__ float gather_edge(const __nv_bfloat16* p, float fill) const {
    return p && has_edge() ? __bfloat162float(p[edge]) : fill;
  }
};

// A bf16 element's bits, and their value: apart, so that a load in flight is not waited for where it is issued (the
// forward of 100000 x 1153: 97 us, against 126).
__device__ __forceinline__ uint32_t bits(const __nv_bfloat16* p) { return *reinterpret_cast<const uint16_t*>(p); }
__device__ __forceinline__ float as_f32(uint32_t b) { return __uint_as_float(b << 16); }

// The group's place: rows first, first + stride, ... of one shift.
__device__ __forceinline__ int row_shift(const void* base, int64_t ld, int64_t row) {
  return static_cast<int>((reinterpret_cast<uintptr_t>(base) / 2 + static_cast<uint64_t>(row) * static_cast<uint64_t>(ld)) & 7);
}

struct LnFwd {
  const __nv_bfloat16* x;
  const __nv_bfloat16 *g, *b;
  __nv_bfloat16* y;
  float *mean, *rstd;
  int64_t ld_x, ld_y, rows, stride;  // stride: rows from one of a group's to its next; hop: elements, likewise
  int64_t hop_x, hop_y;
  int H, W;
  float eps, inv_h, h;
};

// R rows at a time: one exchange of R sums serves them. Two, where registers allow; rows of 4097 to 5120 would leave
// one CTA of 320 threads on an SM then, so they go one at a time in two (32768 x 5120: 125 us, against 142 with one
// vector a thread and 640 threads). A ring that bulk copies fill, as the backward's, was slower here (98304 x 3584:
// 249 us against 227).
template <int NV, int R, bool EDGE, int THREADS, int CTAS>
__global__ void __launch_bounds__(THREADS, CTAS) layernorm_fwd_kernel(const __grid_constant__ LnFwd a) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float red[2][32 * R];
  const int warp = threadIdx.x >> 5, W = a.W, T = W * 32;
  const int group = warp / W, wig = warp - group * W, groups = blockDim.x / T;
  const int t = threadIdx.x - group * T;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * groups + group;
  if (first >= a.rows) return;  // whole groups leave; nothing below waits for another group
  const Cols<NV, EDGE> cols(t, T, row_shift(a.x, a.ld_x, first), a.H);
  const uint32_t slice = static_cast<uint32_t>(T) * NV * 16;
  const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(smem)) + group * (DEPTH * R * slice) + t * 16;
  const uint32_t ring_end = ring + DEPTH * R * slice;
  f2 gain[NV][4], bias[NV][4];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    cols.gather(k, a.g, 1.f, gain[k]);
    cols.gather(k, a.b, 0.f, bias[k]);
  }
  cols.clear_absent(ring, T, DEPTH * R, slice);
  const float edge_gain = cols.gather_edge(a.g, 1.f), edge_bias = cols.gather_edge(a.b, 0.f);
  int64_t next = first;  // the row to fetch next
  const __nv_bfloat16* x_row = a.x + first * a.ld_x;
  auto fill = [&](uint32_t to) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (next < a.rows) {
#pragma unroll
        for (int k = 0; k < NV; ++k) cols.fetch(k, to + r * slice + k * T * 16, x_row);
      }
      next += a.stride;
      x_row += a.hop_x;
    }
    copy_commit();
  };
  const __nv_bfloat16* edge_at = a.x + first * a.ld_x + cols.edge;  // edge elements are read one turn ahead
  uint32_t next_edge[R];
  auto fetch_edge = [&](int64_t row) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      next_edge[r] = cols.has_edge() && row + r * a.stride < a.rows ? bits(edge_at) : 0;
      if (EDGE) edge_at += a.hop_x;
    }
  };
  fetch_edge(first);
  __nv_bfloat16* out = a.y + first * a.ld_y;
  uint32_t to = ring, at = ring;
  for (int s = 0; s < DEPTH - 1; ++s, to += R * slice) fill(to);
  for (int64_t row0 = first; row0 < a.rows; row0 += R * a.stride) {
    fill(to);
    to += R * slice;
    if (to == ring_end) to = ring;
    asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 1) : "memory");
    f2 x[R][NV][4];
    float s[R], edge[R];
#pragma unroll
    for (int r = 0; r < R; ++r) edge[r] = as_f32(next_edge[r]);
    fetch_edge(row0 + R * a.stride);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      f2 sum = 0;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        uint32_t w[4];
        lds128(at + r * slice + k * T * 16, w);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[r][k][i] = f2_of(w[i]);
          sum = f2_add(sum, x[r][k][i]);
        }
      }
      s[r] = f2_sum(sum);
      if (EDGE) s[r] += edge[r];
    }
    at += R * slice;
    if (at == ring_end) at = ring;
    group_sums<R>(s, W, wig, 1 + group, red[0] + group * W * R);
    float q[R], mean[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      mean[r] = row_mean(s[r], a.inv_h, a.h);
      f2 sum = 0;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const f2 neg = f2_both(cols.any(k) ? -mean[r] : 0.f);  // absent vectors stay zero
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[r][k][i] = f2_add(x[r][k][i], neg);
          sum = f2_fma(x[r][k][i], x[r][k][i], sum);
        }
      }
      q[r] = f2_sum(sum);
      if (EDGE) {  // no branch: zeros in the other lanes
        edge[r] -= cols.has_edge() ? mean[r] : 0.f;
        q[r] = fmaf(edge[r], edge[r], q[r]);
      }
    }
    group_sums<R>(q, W, wig, 1 + group, red[1] + group * W * R);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t row = row0 + r * a.stride;
      if (row >= a.rows) continue;
      const float rstd = inv_sqrt(fmaf(q[r], a.inv_h, a.eps));
      if (t == 0) {
        if (a.mean) a.mean[row] = mean[r];
        if (a.rstd) a.rstd[row] = rstd;
      }
      const f2 rs = f2_both(rstd);
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = f2_pack(f2_fma(f2_mul(x[r][k][i], rs), gain[k][i], bias[k][i]));
        cols.store(k, out, w);
      }
      if (cols.has_edge()) out[cols.edge] = __float2bfloat16_rn(fmaf(edge[r] * rstd, edge_gain, edge_bias));
      out += a.hop_y;
    }
  }
}

// Rows wider than the registers of a CTA hold, and operands whose rows lie differently in their granules: one
// CTA a row, three passes over it (the second and third from L1 or L2), an element at a time.
__global__ void __launch_bounds__(1024, 1) layernorm_fwd_wide_kernel(LnFwd a) {
  __shared__ float red[2][32];
  const int wig = threadIdx.x >> 5;
  const float inv_h = 1.0f / static_cast<float>(a.H);
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const __nv_bfloat16* x = a.x + row * a.ld_x;
    float s[1] = {0.f}, q[1] = {0.f};
    for (int j = threadIdx.x; j < a.H; j += blockDim.x) s[0] += __bfloat162float(x[j]);
    group_sums<1>(s, blockDim.x >> 5, wig, 1, red[0]);
    const float mean = row_mean(s[0], inv_h, static_cast<float>(a.H));
    for (int j = threadIdx.x; j < a.H; j += blockDim.x) {
      const float c = __bfloat162float(x[j]) - mean;
      q[0] = fmaf(c, c, q[0]);
    }
    group_sums<1>(q, blockDim.x >> 5, wig, 1, red[1]);
    const float rstd = 1.0f / sqrtf(q[0] * inv_h + a.eps);
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
    for (int j = threadIdx.x; j < a.H; j += blockDim.x) {
      float o = (__bfloat162float(x[j]) - mean) * rstd;
      if (a.g) o *= __bfloat162float(a.g[j]);
      if (a.b) o += __bfloat162float(a.b[j]);
      a.y[row * a.ld_y + j] = __float2bfloat16_rn(o);
    }
  }
}

struct LnBwd {
  const __nv_bfloat16* dy;  // dy, dres and dx may be the same rows
  const __nv_bfloat16* x;
  const __nv_bfloat16* g;
  const float *mean, *rstd;
  const __nv_bfloat16* dres;
  __nv_bfloat16* dx;
  float* part;  // [gridDim.x][2][H]: partial dg and db, unless the grid is one CTA
  float *dg, *db;
  int64_t ld_dy, ld_x, ld_dres, ld_dx, rows, stride;
  int64_t hop_dy, hop_x, hop_dres, hop_dx;
  int H, W, slots;
  float inv_h;
  int32_t* err;
};

// The column sums of the CTA's groups into the CTA's partial row, or with one CTA into dg and db. sums: [groups][2H]
// in shared memory (groups may hold other columns, their sums meet by column), added in group order. One group after
// the other into a single row took 256 x 256 from 4.8 to 8.6 us.
template <int NV, bool EDGE>
__device__ __forceinline__ void leave_sums(const LnBwd& a, const Cols<NV, EDGE>& cols, float* sums, int group, int groups,
                                           const f2 (&dg)[NV][4], const f2 (&db)[NV][4], float edge_dg, float edge_db) {
  if (!a.dg && !a.db) return;
  // one group of whole vectors of 16-byte aligned rows: its registers are the partial row
  const bool direct = !EDGE && groups == 1 && gridDim.x > 1;
  float* pg = direct ? a.part + static_cast<int64_t>(blockIdx.x) * 2 * a.H : sums + group * 2 * a.H;
  float* pb = pg + a.H;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    if (!cols.any(k)) continue;
    float vg[8], vb[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f2_split(dg[k][i], vg[2 * i], vg[2 * i + 1]);
      f2_split(db[k][i], vb[2 * i], vb[2 * i + 1]);
    }
    if (!EDGE) {
#pragma unroll
      for (int i = 0; i < 8; i += 4) {
        *reinterpret_cast<float4*>(pg + cols.col[k] + i) = make_float4(vg[i], vg[i + 1], vg[i + 2], vg[i + 3]);
        *reinterpret_cast<float4*>(pb + cols.col[k] + i) = make_float4(vb[i], vb[i + 1], vb[i + 2], vb[i + 3]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        pg[cols.col[k] + i] = vg[i];
        pb[cols.col[k] + i] = vb[i];
      }
    }
  }
  if (cols.has_edge()) {
    pg[cols.edge] = edge_dg;
    pb[cols.edge] = edge_db;
  }
  if (direct) return;
  const int n = 2 * a.H;
  auto leave = [&](int j, float v) {
    if (j < a.H) {
      if (a.dg) a.dg[j] = v;
    } else if (a.db) {
      a.db[j - a.H] = v;
    }
  };
  __syncthreads();
  for (int j = threadIdx.x; j < n; j += blockDim.x) {
    float v = sums[j];
    for (int gi = 1; gi < groups; ++gi) v += sums[gi * n + j];
    if (gridDim.x == 1)
      leave(j, v);
    else
      a.part[static_cast<int64_t>(blockIdx.x) * n + j] = v;
  }
}

// The same with the thread's places worked out anew, rather than kept in registers over the rows (32768 x 5120, one row
// at a time: 177 us against 199, which spilled a register; with two rows at a time the registers are better used than
// freed, 32768 x 3584: 123 us against 133).
template <int NV, bool EDGE>
__device__ __forceinline__ void leave_sums_anew(const LnBwd& a, float* sums, const f2 (&dg)[NV][4], const f2 (&db)[NV][4],
                                                float edge_dg, float edge_db) {
  int tid;
  asm volatile("mov.u32 %0, %%tid.x;" : "=r"(tid));
  const int T = a.W * 32, group = tid / T, groups = blockDim.x / T;
  const int shift = EDGE ? row_shift(a.x, a.ld_x, static_cast<int64_t>(blockIdx.x) * groups + group) : 0;
  leave_sums<NV, EDGE>(a, Cols<NV, EDGE>(tid - group * T, T, shift, a.H), sums, group, groups, dg, db, edge_dg, edge_db);
}

// Both backward kernels subtract the mean before they scale: x rstd - mean rstd, one instruction less, would be off by half a
// step of mean rstd, which rows far from zero against their spread have in every xh and in dg (98304 x 3584: 366 us, against
// 359; 32768 x 5120: 189 against 183).
//
// Rows with elements outside their whole granules: a row at a time, the next ones in flight.
template <int NV, bool RES, int THREADS, int CTAS>
__global__ void __launch_bounds__(THREADS, CTAS) layernorm_bwd_kernel(const __grid_constant__ LnBwd a) {
  constexpr int TENSORS = RES ? 3 : 2;
  extern __shared__ __align__(16) uint8_t smem[];  // the groups' rings; [groups][2][H] sums after the rows
  __shared__ float red[2][32 * 2];
  const int warp = threadIdx.x >> 5, W = a.W, T = W * 32;
  const int group = warp / W, wig = warp - group * W, groups = blockDim.x / T;
  const int t = threadIdx.x - group * T;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * groups + group;
  const Cols<NV, true> cols(t, T, row_shift(a.x, a.ld_x, first), a.H);
  const uint32_t slice = static_cast<uint32_t>(T) * NV * 16;  // one row of one operand
  const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(smem)) + group * (DEPTH * TENSORS * slice) + t * 16;
  const uint32_t ring_end = ring + DEPTH * TENSORS * slice;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  f2 dg[NV][4], db[NV][4], gain[NV][4];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    cols.gather(k, a.g, 1.f, gain[k]);
#pragma unroll
    for (int i = 0; i < 4; ++i) dg[k][i] = db[k][i] = 0;
  }
  cols.clear_absent(ring, T, DEPTH * TENSORS, slice);
  int64_t next = first;  // the row to fetch next
  const __nv_bfloat16 *dy_row = a.dy + first * a.ld_dy, *x_row = a.x + first * a.ld_x, *res_row = a.dres + first * a.ld_dres;
  auto fill = [&](uint32_t to) {
    if (next < a.rows) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const uint32_t dst = to + k * T * 16;
        cols.fetch(k, dst, dy_row);
        cols.fetch(k, dst + slice, x_row);
        if (RES) cols.fetch(k, dst + 2 * slice, res_row);
      }
    }
    next += a.stride;
    dy_row += a.hop_dy;
    x_row += a.hop_x;
    if (RES) res_row += a.hop_dres;
    copy_commit();
  };
  // edge elements are read one turn ahead
  const float edge_gain = cols.gather_edge(a.g, 1.f);
  float edge_dg = 0.f, edge_db = 0.f;
  uint32_t next_dy = 0, next_x = 0, next_res = 0;
  const __nv_bfloat16 *edge_dy_at = dy_row + cols.edge, *edge_x_at = x_row + cols.edge, *edge_res_at = res_row + cols.edge;
  auto fetch_edge = [&](int64_t row) {
    const bool live = cols.has_edge() && row < a.rows;
    next_dy = live ? bits(edge_dy_at) : 0;
    next_x = live ? bits(edge_x_at) : 0;
    if (RES) next_res = live ? bits(edge_res_at) : 0;
    edge_dy_at += a.hop_dy;
    edge_x_at += a.hop_x;
    if (RES) edge_res_at += a.hop_dres;
  };
  fetch_edge(first);
  __nv_bfloat16* out = a.dx + first * a.ld_dx;
  uint32_t to = ring;
  for (int s = 0; s < DEPTH - 1; ++s, to += TENSORS * slice) fill(to);
  float next_mean = 0.f, next_rstd = 0.f;
  if (first < a.rows) {
    next_mean = a.mean[first];
    next_rstd = a.rstd[first];
  }
  uint32_t at = ring;
  int buf = 0;
  for (int64_t row = first; row < a.rows; row += a.stride) {
    const float mean = next_mean, rstd = next_rstd;
    if (row + a.stride < a.rows) {
      next_mean = a.mean[row + a.stride];
      next_rstd = a.rstd[row + a.stride];
    }
    const float edge_dy = as_f32(next_dy), edge_x = as_f32(next_x), edge_res = as_f32(next_res);
    fetch_edge(row + a.stride);
    fill(to);
    to += TENSORS * slice;
    if (to == ring_end) to = ring;
    asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 1) : "memory");
    f2 s0 = 0, s1 = 0;
    const f2 rs = f2_both(rstd), off = f2_both(-mean);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      uint32_t d[4], x[4];
      lds128(at + k * T * 16, d);
      lds128(at + slice + k * T * 16, x);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f2 dv = f2_of(d[i]), xh = f2_mul(f2_add(f2_of(x[i]), off), rs), w = f2_mul(dv, gain[k][i]);
        s0 = f2_add(s0, w);
        s1 = f2_fma(w, xh, s1);
        dg[k][i] = f2_fma(dv, xh, dg[k][i]);
        db[k][i] = f2_add(db[k][i], dv);
      }
    }
    // absent vectors and the edge elements of other lanes hold dy = 0, which adds nothing to any sum
    float s[2] = {f2_sum(s0), f2_sum(s1)};
    const float edge_w = edge_dy * edge_gain, edge_xh = (edge_x - mean) * rstd;
    s[0] += edge_w;
    s[1] = fmaf(edge_w, edge_xh, s[1]);
    edge_dg = fmaf(edge_dy, edge_xh, edge_dg);
    edge_db += edge_dy;
    group_sums<2>(s, W, wig, 1 + group, red[buf] + group * W * 2);
    buf ^= 1;
    // dx = rstd w - rstd c1 - (x - mean) (rstd rstd c2) + dres, from the ring again: registers that held w and xh meanwhile would spill
    const f2 k1 = f2_both(-rstd * (s[0] * a.inv_h)), k2 = f2_both(-rstd * (rstd * (s[1] * a.inv_h)));
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      uint32_t o[4], r[4], d[4], x[4];
      lds128(at + k * T * 16, d);
      lds128(at + slice + k * T * 16, x);
      if (RES) lds128(at + 2 * slice + k * T * 16, r);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f2 v = f2_fma(f2_add(f2_of(x[i]), off), k2, k1);
        v = f2_fma(f2_mul(f2_of(d[i]), gain[k][i]), rs, v);
        if (RES) v = f2_add(v, f2_of(r[i]));
        o[i] = f2_pack(v);
      }
      cols.store(k, out, o);
    }
    if (cols.has_edge()) {
      const float v = fmaf(edge_w, rstd, -rstd * (s[0] * a.inv_h) - edge_xh * (rstd * (s[1] * a.inv_h)));
      out[cols.edge] = __float2bfloat16_rn(RES ? v + edge_res : v);
    }
    out += a.hop_dx;
    at += TENSORS * slice;
    if (at == ring_end) at = ring;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
  leave_sums_anew<NV, true>(a, reinterpret_cast<float*>(smem), dg, db, edge_dg, edge_db);
}

// A warp's way out of the rows from `row` on when a wait ran out (the error word is set): it only keeps the group's barriers
// going, one a turn. The first warp of a group, which fills the ring, no longer does, and sees that what is in flight
// lands before the CTA leaves (filled so far: the ring, and R rows in each turn from the second on). Apart from the kernel,
// whose registers it would cost otherwise (98304 x 3584: 357 us, against 391 inside and 349 with the outcome unused).
template <int R>
__device__ __noinline__ void give_up(int64_t rows, int64_t stride, int64_t row, int W, int slots, uint32_t full) {
  const int warp = threadIdx.x >> 5, group = warp / W, groups = blockDim.x / (W * 32);
  for (int64_t left = row; W > 1 && left < rows; left += R * stride) group_bar(1 + group, W * 32);
  if (threadIdx.x == group * W * 32) {
    const int64_t first = static_cast<int64_t>(blockIdx.x) * groups + group;
    const int64_t turns = (row - first) / (R * stride), all = (rows - first + stride - 1) / stride;
    tc::drain_ring(full, static_cast<uint32_t>(min(all, slots + R * max(turns - 1, int64_t(0)))), slots);
  }
  __syncthreads();  // the one behind the rows
  asm volatile("exit;");
}

// Rows of whole granules: R rows of a group at a time, through a ring of `slots` rows (a multiple of R, 2 R at least:
// the slots of the R rows before are filled while R are worked on) that bulk copies fill (one an
// operand and row, issued by the group's first thread, which spares the others the addresses and the instructions).
// One exchange of sums serves the R rows; what the second half of the work needs is read from the ring again rather
// than held in registers meanwhile: spilled registers would go to an L1 that the rings leave small.
constexpr int MAX_SLOTS = 8;
template <int NV, int R, bool RES, int THREADS, int CTAS>
__global__ void __launch_bounds__(THREADS, CTAS) layernorm_bwd_bulk_kernel(const __grid_constant__ LnBwd a) {

  constexpr int TENSORS = RES ? 3 : 2;
  extern __shared__ __align__(16) uint8_t smem[];  // the groups' rings; [groups][2][H] sums after the rows
  __shared__ float red[2][32 * 2 * R];
  __shared__ uint64_t full_bars[8][MAX_SLOTS];
  __shared__ int abort_word;
  const int warp = threadIdx.x >> 5, W = a.W, T = W * 32;
  const int group = warp / W, wig = warp - group * W, groups = blockDim.x / T;
  const int t = threadIdx.x - group * T;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * groups + group;
  const Cols<NV, false> cols(t, T, 0, a.H);
  const uint32_t slice = static_cast<uint32_t>(T) * NV * 16, slot_bytes = TENSORS * slice;
  const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(smem)) + group * a.slots * slot_bytes + t * 16;
  const uint32_t full = tc::smem_u32(&full_bars[group][0]);
  if (t == 0)
    for (int s = 0; s < a.slots; ++s) tc::mbar_init(full + 8 * s, 1);
  if (threadIdx.x == 0) abort_word = 0;
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // into slot s, by the group's first thread
  auto fill = [&](int64_t row, int s) {
    if (t == 0 && row < a.rows) {
      const uint32_t bytes = static_cast<uint32_t>(a.H) * 2, to = ring + s * slot_bytes, bar = full + 8 * s;
      tc::mbar_expect_tx(bar, bytes * TENSORS);
      bulk_copy(to, a.dy + row * a.ld_dy, bytes, bar);
      bulk_copy(to + slice, a.x + row * a.ld_x, bytes, bar);
      if (RES) bulk_copy(to + 2 * slice, a.dres + row * a.ld_dres, bytes, bar);
    }
  };
  for (int s = 0; s < a.slots; ++s) fill(first + s * a.stride, s);  // its own barriers: initialised by this thread
  f2 dg[NV][4], db[NV][4], gain[NV][4];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    cols.gather(k, a.g, 1.f, gain[k]);
#pragma unroll
    for (int i = 0; i < 4; ++i) dg[k][i] = db[k][i] = 0;
  }
  cols.clear_absent(ring, T, a.slots * TENSORS, slice);  // behind what a copy writes
  __syncthreads();
  float next_mean[R], next_rstd[R];
  auto stats = [&](int64_t row) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const bool live = row + r * a.stride < a.rows;
      next_mean[r] = live ? a.mean[row + r * a.stride] : 0.f;
      next_rstd[r] = live ? a.rstd[row + r * a.stride] : 0.f;
    }
  };
  stats(first);
  int slot = 0, buf = 0;  // a.slots is a multiple of R
  uint32_t phase = 0;
  __nv_bfloat16* out = a.dx + first * a.ld_dx;
  for (int64_t row = first; row < a.rows; row += R * a.stride) {
    float s[2 * R];
    f2 rs[R], off[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      rs[r] = f2_both(next_rstd[r]);
      off[r] = f2_both(-next_mean[r]);
    }
    stats(row + R * a.stride);
    const uint32_t at = ring + slot * slot_bytes;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      f2 s0 = 0, s1 = 0;
      if (row + r * a.stride < a.rows) {
        const uint32_t bar = full + 8 * (slot + r);
        if (!__all_sync(0xffffffffu, tc::mbar_try(bar, phase)) &&  // bounded
            !tc::warp_wait(bar, phase, &abort_word, a.err, DEV_ERR_TIMEOUT_PRODUCER))
          give_up<R>(a.rows, a.stride, row, W, a.slots, full);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
          uint32_t d[4], x[4];
          lds128(at + r * slot_bytes + k * T * 16, d);
          lds128(at + r * slot_bytes + slice + k * T * 16, x);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const f2 dv = f2_of(d[i]), xh = f2_mul(f2_add(f2_of(x[i]), off[r]), rs[r]), w = f2_mul(dv, gain[k][i]);
            s0 = f2_add(s0, w);
            s1 = f2_fma(w, xh, s1);
            dg[k][i] = f2_fma(dv, xh, dg[k][i]);
            db[k][i] = f2_add(db[k][i], dv);
          }
        }
      }
      s[2 * r] = f2_sum(s0);
      s[2 * r + 1] = f2_sum(s1);
    }
    group_sums<2 * R>(s, W, wig, 1 + group, red[buf] + group * W * 2 * R);
    buf ^= 1;
    // the whole group is behind the rows before these: their slots take the rows a ring's length after them
    if (row != first) {
      const int before = slot == 0 ? a.slots - R : slot - R;
#pragma unroll
      for (int r = 0; r < R; ++r) fill(row + (a.slots - R + r) * a.stride, before + r);
    }
    slot += R;
    if (slot == a.slots) {
      slot = 0;
      phase ^= 1;
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (row + r * a.stride < a.rows) {
        // dx = rstd w - rstd c1 - (x - mean) (rstd rstd c2) + dres
        float rstd, same;
        f2_split(rs[r], rstd, same);
        const f2 k1 = f2_both(-rstd * (s[2 * r] * a.inv_h)), k2 = f2_both(-rstd * (rstd * (s[2 * r + 1] * a.inv_h)));
#pragma unroll
        for (int k = 0; k < NV; ++k) {
          uint32_t o[4], q[4], d[4], x[4];
          lds128(at + r * slot_bytes + k * T * 16, d);
          lds128(at + r * slot_bytes + slice + k * T * 16, x);
          if (RES) lds128(at + r * slot_bytes + 2 * slice + k * T * 16, q);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            f2 v = f2_fma(f2_add(f2_of(x[i]), off[r]), k2, k1);
            v = f2_fma(f2_mul(f2_of(d[i]), gain[k][i]), rs[r], v);
            if (RES) v = f2_add(v, f2_of(q[i]));
            o[i] = f2_pack(v);
          }
          cols.store(k, out, o);
        }
      }
      out += a.hop_dx;
    }
  }
  __syncthreads();
  if (*static_cast<volatile int*>(&abort_word)) return;  // no column sums of rows that did not arrive
  if constexpr (R == 1)
    leave_sums_anew<NV, false>(a, reinterpret_cast<float*>(smem), dg, db, 0.f, 0.f);
  else
    leave_sums<NV, false>(a, cols, reinterpret_cast<float*>(smem), group, groups, dg, db, 0.f, 0.f);
}

// dg and db from `parts` partial rows of 2H floats: 32 columns a block, 32 threads a column, each the sum of
// every 32nd row, added in order. Launched ahead of the pass's end (its CTAs start as that one's leave): `part` is still written
// then, so it is no const __restrict__, whose loads may go by the non-coherent path and ahead of the wait.
constexpr int REDUCE_Y = 32;
__global__ void __launch_bounds__(32 * REDUCE_Y) layernorm_bwd_reduce_kernel(const float* part, int parts, int H, float* dg,
                                                                             float* db) {
  __shared__ float red[REDUCE_Y][32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int64_t j = static_cast<int64_t>(blockIdx.x) * 32 + lane, cols = 2 * static_cast<int64_t>(H);
  float v = 0.f;
  if (j < cols) {
#pragma unroll 10
    for (int p = y; p < parts; p += REDUCE_Y) v += part[p * cols + j];
  }
  red[y][lane] = v;
  __syncthreads();
  if (y == 0 && j < cols) {
#pragma unroll
    for (int k = 1; k < REDUCE_Y; ++k) v += red[k][lane];
    if (j < H) {
      if (dg) dg[j] = v;
    } else if (db) {
      db[j - H] = v;
    }
  }
}

// Rows wider than the registers of a CTA hold, and operands whose rows lie differently in their granules: the
// column sums in a kernel of their own (before dx, which may overwrite dy), then dx a row at a time, the second
// pass from L1 or L2.
__global__ void __launch_bounds__(1024, 1) layernorm_bwd_wide_dx_kernel(LnBwd a) {
  __shared__ float red[2][64];
  const int wig = threadIdx.x >> 5;
  const float inv_h = 1.0f / static_cast<float>(a.H);
  int buf = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const __nv_bfloat16 *dy = a.dy + row * a.ld_dy, *x = a.x + row * a.ld_x;
    const float mean = a.mean[row], rstd = a.rstd[row];
    float s[2] = {0.f, 0.f};
    for (int j = threadIdx.x; j < a.H; j += blockDim.x) {
      const float w = __bfloat162float(dy[j]) * (a.g ? __bfloat162float(a.g[j]) : 1.f);
      s[0] += w;
      s[1] = fmaf(w, (__bfloat162float(x[j]) - mean) * rstd, s[1]);
    }
    group_sums<2>(s, blockDim.x >> 5, wig, 1, red[buf]);
    buf ^= 1;
    for (int j = threadIdx.x; j < a.H; j += blockDim.x) {
      const float w = __bfloat162float(dy[j]) * (a.g ? __bfloat162float(a.g[j]) : 1.f);
      const float xh = (__bfloat162float(x[j]) - mean) * rstd;
      const float r = a.dres ? __bfloat162float(a.dres[row * a.ld_dres + j]) : 0.f;
      a.dx[row * a.ld_dx + j] = __float2bfloat16_rn(fmaf(rstd, w - s[0] * inv_h - xh * (s[1] * inv_h), r));
    }
  }
}

__global__ void __launch_bounds__(256) layernorm_bwd_wide_cols_kernel(LnBwd a) {
  const int64_t j = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (j >= a.H) return;
  float dg = 0.f, db = 0.f;
  for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    const float d = __bfloat162float(a.dy[row * a.ld_dy + j]);
    dg = fmaf(d, (__bfloat162float(a.x[row * a.ld_x + j]) - a.mean[row]) * a.rstd[row], dg);
    db += d;
  }
  a.part[static_cast<int64_t>(blockIdx.y) * 2 * a.H + j] = dg;
  a.part[static_cast<int64_t>(blockIdx.y) * 2 * a.H + a.H + j] = db;
}

// Whether the rows of all operands lie alike in their 16-byte granules, and how often their place repeats.
struct Granules {
  uintptr_t base, ld;
  bool alike = true;
  Granules(const void* p, int64_t l) : base(reinterpret_cast<uintptr_t>(p) & 15), ld(static_cast<uintptr_t>(l) & 7) {}
  void add(const void* p, int64_t l) {
    if (p && ((reinterpret_cast<uintptr_t>(p) & 15) != base || (static_cast<uintptr_t>(l) & 7) != ld)) alike = false;
  }
  int period() const { return ld == 0 ? 1 : ld % 4 == 0 ? 2 : ld % 2 == 0 ? 4 : 8; }
  bool shifted() const { return base != 0 || ld != 0; }
};

// A pass's groups: W warps of NV vectors a thread, `groups` to a CTA, `ctas` CTAs; rings of smem bytes in all.
struct Shape {
  int nv, W, groups, threads, ctas;
  int64_t smem;
};

// threads_sm: threads of an SM that the pass's registers allow; rows_stage, tensors: rows and operands of a stage.
// Works on a whole B200's 148 SMs whatever the device, so that results do not depend on it.
Shape shape_of(int64_t rows, int H, const Granules& g, int one_vec, int threads_sm, int rows_stage, int tensors) {
  Shape s;
  const int vecs = std::max(1, H / 8);  // whole granules of a row at most
  s.nv = vecs <= one_vec ? 1 : 2;
  s.W = (vecs + 32 * s.nv - 1) / (32 * s.nv);
  s.groups = std::max(1, 8 / s.W);
  s.threads = s.groups * s.W * 32;
  int resident = std::max(1, threads_sm / s.threads);
  // more groups in one CTA of all the threads (three warps: five groups, against two CTAs of two; forward of
  // 100000 x 1160: 95 us against 107)
  if (s.W * 32 <= threads_sm / 2 && threads_sm / (s.W * 32) > resident * s.groups) {
    s.groups = threads_sm / (s.W * 32);
    s.threads = s.groups * s.W * 32;
    resident = 1;
  }
  const int64_t want = (rows + s.groups - 1) / s.groups;
  const int64_t most = static_cast<int64_t>(SMS) * resident;
  int64_t ctas = std::min(want, most), up = ctas;
  // the groups' stride has to be a multiple of the period: more CTAs, or fewer where more would not be resident
  while (up * s.groups % g.period()) ++up;
  while (up > most && ctas * s.groups % g.period()) --ctas;
  s.ctas = static_cast<int>(up > most ? ctas : up);
  s.smem = static_cast<int64_t>(s.threads) * s.nv * 16 * rows_stage * tensors * DEPTH;
  return s;
}

Shape bwd_shape(int64_t rows, int H, const Granules& g, bool res) {
  if (g.shifted() || H % 8) {
    // Rows with elements outside their whole granules, registers of 128 a thread with two vectors: two CTAs of up to
    // 256 threads, rows of up to 4096. Up to 5120, one vector a thread and 640 threads of 96 registers keep more warps
    // on the SM (32768 x 5113: 279 us, against 374 with two vectors).
    const int vecs = std::max(1, H / 8);  // whole granules of a row at most
    return shape_of(rows, H, g, vecs > 512 && vecs <= 640 ? 640 : 32, 512, 1, res ? 3 : 2);
  }
  // whole granules: 128 registers a thread, 512 threads an SM; or, rows of 4097 to 5120, two CTAs of up to 320 threads of
  // 96 (32768 x 5120: 177 us, against 204 with one CTA of 128)
  const Shape s = shape_of(rows, H, g, 32, 512, 1, res ? 3 : 2);
  return s.threads > 256 && s.threads <= 320 ? shape_of(rows, H, g, 32, 640, 1, res ? 3 : 2) : s;
}

template <int NV, int R, bool EDGE, int THREADS, int CTAS>
mt_status fwd_go(const LnFwd& a, const Shape& s, cudaStream_t st) {
  static SmemOptIn opt;
  if (s.smem > 40 * 1024) MT_TRY(opt.raise(reinterpret_cast<const void*>(layernorm_fwd_kernel<NV, R, EDGE, THREADS, CTAS>)));
  layernorm_fwd_kernel<NV, R, EDGE, THREADS, CTAS><<<s.ctas, s.threads, s.smem, st>>>(a);
  return launch_check("layernorm_fwd_kernel");
}

template <bool EDGE>
mt_status fwd_shape_go(const LnFwd& a, const Shape& s, cudaStream_t st) {
  if (s.nv == 1) return fwd_go<1, 2, EDGE, 256, 2>(a, s, st);
  if (s.threads <= 256) return fwd_go<2, 2, EDGE, 256, 2>(a, s, st);
  return s.threads <= 320 ? fwd_go<2, 1, EDGE, 320, 2>(a, s, st) : fwd_go<2, 2, EDGE, 512, 1>(a, s, st);
}

// Threads of a CTA that walks a row an element at a time.
int wide_threads(int H) { return std::min(1024, std::max(32, (H + 127) / 128 * 32)); }

mt_status layernorm_fwd_launch(LnFwd a, cudaStream_t st) {
  Granules g(a.x, a.ld_x);
  g.add(a.y, a.ld_y);
  if (!g.alike || a.H > MAX_H_REG) {
    const int64_t grid = std::min<int64_t>(a.rows, static_cast<int64_t>(num_sms()) * 2048 / wide_threads(a.H));
    layernorm_fwd_wide_kernel<<<static_cast<unsigned>(grid), wide_threads(a.H), 0, st>>>(a);
    return launch_check("layernorm_fwd_wide_kernel");
  }
  // 128 registers a thread and 512 threads an SM; rows of 4097 to 5120 in two CTAs of up to 320 threads, of 96 registers
  Shape s = shape_of(a.rows, a.H, g, 32, 512, 2, 1);
  if (s.threads > 256 && s.threads <= 320) s = shape_of(a.rows, a.H, g, 32, 640, 1, 1);
  a.W = s.W;
  a.stride = static_cast<int64_t>(s.ctas) * s.groups;
  a.hop_x = a.stride * a.ld_x;
  a.hop_y = a.stride * a.ld_y;
  return g.shifted() || a.H % 8 ? fwd_shape_go<true>(a, s, st) : fwd_shape_go<false>(a, s, st);
}

// Partial rows at most: of the register pass (rows of any alignment), or of the column pass.
int bwd_parts(int64_t rows, int H) {
  const int wide = static_cast<int>(std::min<int64_t>(2 * SMS, (rows + 63) / 64));
  if (H > MAX_H_REG) return wide;
  int parts = wide;
  for (uintptr_t base : {uintptr_t(0), uintptr_t(2)})
    for (int ld : {0, 1, 2, 4})
      parts = std::max(parts, bwd_shape(rows, H, Granules(reinterpret_cast<const void*>(base), ld), false).ctas);
  return parts;
}

uint64_t bwd_ws_bytes(int64_t rows, int H) {
  return static_cast<uint64_t>(align_up(static_cast<int64_t>(std::max(1, bwd_parts(rows, H))) * 2 * H * 4, 256));
}

// The sums after the rows fit the rings: 8 H bytes a group, against 8 T NV >= H columns of 2 bytes in two operands and
// two rows at least.
template <typename Kernel>
mt_status bwd_launch(Kernel* kernel, SmemOptIn& opt, const LnBwd& a, const Shape& s, int64_t smem, cudaStream_t st) {
  if (smem > 40 * 1024) MT_TRY(opt.raise(reinterpret_cast<const void*>(kernel)));
  kernel<<<s.ctas, s.threads, smem, st>>>(a);
  return launch_check("layernorm_bwd_kernel");
}

template <int NV, bool RES, int THREADS, int CTAS>
mt_status bwd_go(const LnBwd& a, const Shape& s, cudaStream_t st) {
  static SmemOptIn opt;
  return bwd_launch(layernorm_bwd_kernel<NV, RES, THREADS, CTAS>, opt, a, s, s.smem, st);
}

template <bool RES>
mt_status bwd_edge_go(const LnBwd& a, const Shape& s, cudaStream_t st) {
  if (s.nv == 1) return s.threads <= 320 ? bwd_go<1, RES, 320, 2>(a, s, st) : bwd_go<1, RES, 640, 1>(a, s, st);
  return s.threads <= 256 ? bwd_go<2, RES, 256, 2>(a, s, st) : bwd_go<2, RES, 512, 1>(a, s, st);
}

template <int NV, int R, bool RES, int THREADS, int CTAS>
mt_status bwd_bulk_rows_go(const LnBwd& a, const Shape& s, int64_t slot, cudaStream_t st) {
  static SmemOptIn opt;
  return bwd_launch(layernorm_bwd_bulk_kernel<NV, R, RES, THREADS, CTAS>, opt, a, s, slot * a.slots, st);
}

// The ring holds as many rows as the SM's shared memory has for its CTAs: two at a time need four (the slots of the
// two before are filled while two are worked on), one at a time two.
template <int NV, bool RES, int THREADS, int CTAS>
mt_status bwd_bulk_go(LnBwd a, const Shape& s, cudaStream_t st) {
  const int64_t slot = static_cast<int64_t>(s.threads) * NV * 16 * (RES ? 3 : 2);
  const int resident = std::max(1, std::min(CTAS * THREADS / s.threads, 8));
  const int fit = static_cast<int>(std::min<int64_t>(MAX_SLOTS, (220 * 1024 / resident - 2048) / slot));
  if constexpr (NV == 2 && THREADS == 320) {  // two rows' values do not fit its registers: 177 us one at a time, 198 two
    a.slots = std::max(2, fit);
    return bwd_bulk_rows_go<NV, 1, RES, THREADS, CTAS>(a, s, slot, st);
  } else {
    a.slots = std::max(4, fit & ~1);
    return bwd_bulk_rows_go<NV, 2, RES, THREADS, CTAS>(a, s, slot, st);
  }
}

template <bool RES>
mt_status bwd_whole_go(const LnBwd& a, const Shape& s, cudaStream_t st) {
  if (s.nv == 1) return bwd_bulk_go<1, RES, 320, 2>(a, s, st);
  if (s.threads <= 256) return bwd_bulk_go<2, RES, 256, 2>(a, s, st);
  return s.threads <= 320 ? bwd_bulk_go<2, RES, 320, 2>(a, s, st) : bwd_bulk_go<2, RES, 512, 1>(a, s, st);
}

mt_status layernorm_bwd_launch(LnBwd a, cudaStream_t st) {
  if (a.rows == 0) {
    if (a.dg) MT_CUDA(cudaMemsetAsync(a.dg, 0, static_cast<size_t>(a.H) * 4, st));
    if (a.db) MT_CUDA(cudaMemsetAsync(a.db, 0, static_cast<size_t>(a.H) * 4, st));
    return MT_OK;
  }
  Granules g(a.x, a.ld_x);
  g.add(a.dy, a.ld_dy);
  g.add(a.dres, a.ld_dres);
  g.add(a.dx, a.ld_dx);
  int parts;
  if (!g.alike || a.H > MAX_H_REG) {
    parts = static_cast<int>(std::min<int64_t>(2 * SMS, (a.rows + 63) / 64));
    if (a.dg || a.db) {
      layernorm_bwd_wide_cols_kernel<<<dim3((a.H + 255) / 256, parts), 256, 0, st>>>(a);
      MT_TRY(launch_check("layernorm_bwd_wide_cols_kernel"));
    }
    const int64_t grid = std::min<int64_t>(a.rows, static_cast<int64_t>(num_sms()) * 2048 / wide_threads(a.H));
    layernorm_bwd_wide_dx_kernel<<<static_cast<unsigned>(grid), wide_threads(a.H), 0, st>>>(a);
    MT_TRY(launch_check("layernorm_bwd_wide_dx_kernel"));
  } else {
    const Shape s = bwd_shape(a.rows, a.H, g, a.dres != nullptr);
    a.W = s.W;
    a.stride = static_cast<int64_t>(s.ctas) * s.groups;
    a.hop_dy = a.stride * a.ld_dy;
    a.hop_x = a.stride * a.ld_x;
    a.hop_dres = a.stride * a.ld_dres;
    a.hop_dx = a.stride * a.ld_dx;
    parts = s.ctas;
    a.err = device_error_word();
    if (!a.err) return fail(MT_ERR_CUDA, "device error word unavailable");
    if (g.shifted() || a.H % 8)
      MT_TRY((a.dres ? bwd_edge_go<true>(a, s, st) : bwd_edge_go<false>(a, s, st)));
    else
      MT_TRY((a.dres ? bwd_whole_go<true>(a, s, st) : bwd_whole_go<false>(a, s, st)));
    if (parts == 1) return MT_OK;
  }
  if (!a.dg && !a.db) return MT_OK;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((2 * a.H + 31) / 32, 1, 1);
  cfg.blockDim = dim3(32 * REDUCE_Y, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  MT_CUDA(cudaLaunchKernelEx(&cfg, layernorm_bwd_reduce_kernel, static_cast<const float*>(a.part), parts, a.H, a.dg, a.db));
  return launch_check("layernorm_bwd_reduce_kernel");
}

bool aligned_to(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace
}  // namespace mt

using namespace mt;

extern "C" {

mt_status mt_layernorm_fwd(const mt_bf16* x, int64_t ld_x, const mt_bf16* g, const mt_bf16* b, mt_bf16* y, int64_t ld_y,
                           float* mean, float* rstd, int64_t rows, int32_t H, float eps, void* stream) {
  if (rows != 0 && (!x || !y)) return fail(MT_ERR_INVALID_ARG, "layernorm_fwd: NULL pointer");
  if (rows < 0 || H <= 0 || !(eps >= 0.f)) return fail(MT_ERR_INVALID_ARG, "layernorm_fwd: need rows >= 0, H > 0, eps >= 0");
  if (ld_x < H || ld_y < H) return fail(MT_ERR_INVALID_ARG, "layernorm_fwd: row stride smaller than H");
  if (x && y == x && ld_y != ld_x) return fail(MT_ERR_INVALID_ARG, "layernorm_fwd: in place needs ld_x == ld_y");
  if (H > MAX_H) return fail(MT_ERR_UNSUPPORTED, "layernorm_fwd: H above 2^28");
  if (!aligned_to(x, 2) || !aligned_to(y, 2) || !aligned_to(g, 2) || !aligned_to(b, 2) || !aligned_to(mean, 4) ||
      !aligned_to(rstd, 4))
    return fail(MT_ERR_ALIGNMENT, "layernorm_fwd: pointers must be aligned to their elements");
  if (rows == 0) return MT_OK;
  LnFwd a;
  a.x = reinterpret_cast<const __nv_bfloat16*>(x);
  a.g = reinterpret_cast<const __nv_bfloat16*>(g);
  a.b = reinterpret_cast<const __nv_bfloat16*>(b);
  a.y = reinterpret_cast<__nv_bfloat16*>(y);
  a.mean = mean;
  a.rstd = rstd;
  a.ld_x = ld_x;
  a.ld_y = ld_y;
  a.rows = rows;
  a.H = H;
  a.W = 0;
  a.eps = eps;
  a.stride = 0;
  a.inv_h = 1.0f / static_cast<float>(H);
  a.h = static_cast<float>(H);
  return layernorm_fwd_launch(a, as_stream(stream));
}

uint64_t mt_layernorm_bwd_workspace_bytes(int64_t rows, int32_t H) {
  if (rows < 0 || H <= 0 || H > MAX_H) return 0;
  return bwd_ws_bytes(rows, H);
}

mt_status mt_layernorm_bwd(const mt_bf16* dy, int64_t ld_dy, const mt_bf16* x, int64_t ld_x, const mt_bf16* g,
                           const float* mean, const float* rstd, const mt_bf16* dres, int64_t ld_dres, mt_bf16* dx,
                           int64_t ld_dx, float* dg, float* db, int64_t rows, int32_t H, void* ws, uint64_t ws_bytes,
                           void* stream) {
  if (rows != 0 && (!dy || !x || !mean || !rstd || !dx || !ws)) return fail(MT_ERR_INVALID_ARG, "layernorm_bwd: NULL pointer");
  if (rows < 0 || H <= 0) return fail(MT_ERR_INVALID_ARG, "layernorm_bwd: need rows >= 0, H > 0");
  if (ld_dy < H || ld_x < H || ld_dx < H || (dres && ld_dres < H))
    return fail(MT_ERR_INVALID_ARG, "layernorm_bwd: row stride smaller than H");
  if (H > MAX_H) return fail(MT_ERR_UNSUPPORTED, "layernorm_bwd: H above 2^28");
  if (rows != 0 && ((dx == dy && ld_dx != ld_dy) || (dres && dx == dres && ld_dx != ld_dres) || dx == x))
    return fail(MT_ERR_INVALID_ARG, "layernorm_bwd: dx may only be dy or dres itself, with the same row stride");
  if (!aligned_to(dy, 2) || !aligned_to(x, 2) || !aligned_to(g, 2) || !aligned_to(dres, 2) || !aligned_to(dx, 2) ||
      !aligned_to(mean, 4) || !aligned_to(rstd, 4) || !aligned_to(dg, 4) || !aligned_to(db, 4) || !aligned16(ws))
    return fail(MT_ERR_ALIGNMENT, "layernorm_bwd: pointers must be aligned to their elements, ws to 16 bytes");
  if (rows != 0 && ws_bytes < bwd_ws_bytes(rows, H)) return fail(MT_ERR_WORKSPACE, "layernorm_bwd: workspace too small");
  LnBwd a;
  a.dy = reinterpret_cast<const __nv_bfloat16*>(dy);
  a.x = reinterpret_cast<const __nv_bfloat16*>(x);
  a.g = reinterpret_cast<const __nv_bfloat16*>(g);
  a.mean = mean;
  a.rstd = rstd;
  a.dres = reinterpret_cast<const __nv_bfloat16*>(dres);
  a.dx = reinterpret_cast<__nv_bfloat16*>(dx);
  a.part = static_cast<float*>(ws);
  a.dg = dg;
  a.db = db;
  a.ld_dy = ld_dy;
  a.ld_x = ld_x;
  a.ld_dres = ld_dres;
  a.ld_dx = ld_dx;
  a.rows = rows;
  a.H = H;
  a.W = 0;
  a.stride = 0;
  a.inv_h = 1.0f / static_cast<float>(H);
  a.slots = 0;
  a.err = nullptr;
  return layernorm_bwd_launch(a, as_stream(stream));
}

}  // extern "C"
