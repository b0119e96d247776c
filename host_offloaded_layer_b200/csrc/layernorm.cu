// LayerNorm forward and backward over bf16 rows.
//
//   mean = sum_j x_j / H, rstd = 1 / sqrt(sum_j (x_j - mean)^2 / H + eps), xh = (x - mean) rstd, y = xh g + b
//   w = dy g, dx = rstd (w - mean_j(w) - xh mean_j(w xh)) + dres, dg = sum_rows dy xh, db = sum_rows dy
//
// Both are bound by HBM: the forward has to move 4 bytes an element, the backward 6 (8 with dres). So every
// element is read once: a group of W warps holds a whole row in registers (EPT elements a thread), which
// also lets the variance be taken of x - mean (a second sum over registers, exact for rows whose mean is
// large against their spread). The backward's column sums dg and db come from the same pass: a thread owns
// the same columns of every row its group visits and keeps their sums in registers; a group adds its sums
// to the CTA's in shared memory, a CTA leaves one partial row, and a second small kernel adds the partial
// rows in a fixed order. No atomics: the result depends on the sizes alone.
#include <algorithm>

#include "mt_internal.h"
#include "vec.cuh"

namespace mt {
namespace {

using namespace vec;

constexpr int SMS = 148;            // the partial rows of dg and db are counted for a whole B200, so that sums do not depend on the device
constexpr int GROUP_THREADS = 256;  // groups of few warps share a CTA of about this size
constexpr int MAX_H_REG = 8192;     // the widest row that 16 warps of 16 elements a thread hold (32 warps in the forward: 16384)

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

struct LnFwd {
  const __nv_bfloat16* x;
  const __nv_bfloat16 *g, *b;
  __nv_bfloat16* y;
  float *mean, *rstd;
  int64_t ld_x, ld_y, rows;
  int H, W;
  float eps;
};

// Groups of W warps, each a row at a time; the next row's loads are issued before this row's sums.
template <int VEC, int EPT>
__global__ void __launch_bounds__(1024, 1) layernorm_fwd_kernel(LnFwd a) {
  using V = typename Raw<VEC>::type;
  constexpr int NV = EPT / VEC;
  __shared__ float red[2][32];
  const int warp = threadIdx.x >> 5, W = a.W, T = W * 32;
  const int group = warp / W, wig = warp - group * W, groups = blockDim.x / T;
  const int t = threadIdx.x - group * T;
  const int nvec = a.H / VEC;
  const float inv_h = 1.0f / static_cast<float>(a.H);
  V xv[NV], nx[NV];
  int64_t row = static_cast<int64_t>(blockIdx.x) * groups + group;
  const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
  auto load = [&](V(&d)[NV], int64_t r) {
    const V* p = reinterpret_cast<const V*>(a.x + r * a.ld_x);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if (t + k * T < nvec)
        d[k] = p[t + k * T];
      else
        zero(d[k]);
    }
  };
  if (row < a.rows) load(xv, row);
  for (; row < a.rows; row += step) {
    const bool more = row + step < a.rows;
    if (more) load(nx, row + step);
    float f[EPT];
#pragma unroll
    for (int k = 0; k < NV; ++k) unpack(xv[k], f + k * VEC);
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < EPT; ++i) s[0] += f[i];
    group_sums<1>(s, W, wig, 1 + group, red[0] + group * W);
    const float mean = s[0] * inv_h;
    float q[1] = {0.f};
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const bool in = t + k * T < nvec;
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const float c = f[k * VEC + i] - mean;
        f[k * VEC + i] = c;
        if (in) q[0] = fmaf(c, c, q[0]);
      }
    }
    group_sums<1>(q, W, wig, 1 + group, red[1] + group * W);
    const float rstd = 1.0f / sqrtf(q[0] * inv_h + a.eps);
    if (t == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
    V* yp = reinterpret_cast<V*>(a.y + row * a.ld_y);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = t + k * T;
      if (c < nvec) {
        float o[VEC], w[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) o[i] = f[k * VEC + i] * rstd;
        if (a.g) {
          unpack(__ldg(reinterpret_cast<const V*>(a.g) + c), w);
#pragma unroll
          for (int i = 0; i < VEC; ++i) o[i] *= w[i];
        }
        if (a.b) {
          unpack(__ldg(reinterpret_cast<const V*>(a.b) + c), w);
#pragma unroll
          for (int i = 0; i < VEC; ++i) o[i] += w[i];
        }
        V out;
        pack(out, o);
        yp[c] = out;
      }
    }
    if (more) {
#pragma unroll
      for (int k = 0; k < NV; ++k) xv[k] = nx[k];
    }
  }
}

// Rows wider than the registers of a CTA hold: one CTA a row, three passes over it (the second and third
// from L2), an element at a time.
__global__ void __launch_bounds__(1024, 1) layernorm_fwd_wide_kernel(LnFwd a) {
  __shared__ float red[2][32];
  const int wig = threadIdx.x >> 5;
  const float inv_h = 1.0f / static_cast<float>(a.H);
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const __nv_bfloat16* x = a.x + row * a.ld_x;
    float s[1] = {0.f}, q[1] = {0.f};
    for (int j = threadIdx.x; j < a.H; j += 1024) s[0] += __bfloat162float(x[j]);
    group_sums<1>(s, 32, wig, 1, red[0]);
    const float mean = s[0] * inv_h;
    for (int j = threadIdx.x; j < a.H; j += 1024) {
      const float c = __bfloat162float(x[j]) - mean;
      q[0] = fmaf(c, c, q[0]);
    }
    group_sums<1>(q, 32, wig, 1, red[1]);
    const float rstd = 1.0f / sqrtf(q[0] * inv_h + a.eps);
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
    for (int j = threadIdx.x; j < a.H; j += 1024) {
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
  float* part;  // [gridDim.x][2][H]: partial dg and db; the final dg and db themselves with one CTA
  float *dg, *db;
  int64_t ld_dy, ld_x, ld_dres, ld_dx, rows;
  int H, W, depth;
};

// 16 or 4 bytes from global to shared memory, zeros where `live` is false (p is then any valid address).
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* p, bool live) {
  const int n = live ? BYTES : 0;
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(p), "r"(n) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(p), "r"(n) : "memory");
}

// Groups of W warps, R rows at a time (one exchange of 2R sums serves them). Rows arrive through a ring of
// `depth` stages that cp.async fills, `depth` - 1 ahead; a thread copies exactly the vectors that it reads,
// so the ring needs no barrier. Rows of single elements (VEC = 1: odd H or row stride), for which there is no
// such copy, come through registers, and more CTAs to an SM hide their latency.
template <int VEC, int EPT, int R>
__global__ void __launch_bounds__(512, 1) layernorm_bwd_kernel(LnBwd a) {
  using V = typename Raw<VEC>::type;
  constexpr int NV = EPT / VEC;
  constexpr bool RING = VEC > 1;
  extern __shared__ __align__(16) uint8_t smem[];  // the groups' rings; [2][H] sums after the rows
  __shared__ float red[2][32 * 4];
  const int warp = threadIdx.x >> 5, W = a.W, T = W * 32;
  const int group = warp / W, wig = warp - group * W, groups = blockDim.x / T;
  const int t = threadIdx.x - group * T;
  const int nvec = a.H / VEC;
  const float inv_h = 1.0f / static_cast<float>(a.H);
  const bool has_res = a.dres != nullptr;
  const int tensors = has_res ? 3 : 2;
  const uint32_t slice = static_cast<uint32_t>(T) * EPT * 2;  // one row of one tensor
  const uint32_t stage = slice * R * tensors;
  uint8_t* ring = smem + static_cast<size_t>(group) * a.depth * stage;
  const uint32_t ring_addr = static_cast<uint32_t>(__cvta_generic_to_shared(ring));

  float dg[EPT], db[EPT];
  V gain[NV];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    zero(gain[k]);
    if (a.g && t + k * T < nvec) gain[k] = __ldg(reinterpret_cast<const V*>(a.g) + t + k * T);
  }
#pragma unroll
  for (int i = 0; i < EPT; ++i) dg[i] = db[i] = 0.f;

  const int64_t step = static_cast<int64_t>(gridDim.x) * groups * R;
  const int64_t first = (static_cast<int64_t>(blockIdx.x) * groups + group) * R;
  auto fill = [&](int slot, int64_t row0) {
    if constexpr (RING) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const bool row_live = row0 + r < a.rows;
        const int64_t row = row_live ? row0 + r : 0;
        uint32_t dst = ring_addr + slot * stage + r * tensors * slice + t * VEC * 2;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
          const bool live = row_live && t + k * T < nvec;
          const int c = live ? (t + k * T) * VEC : 0;
          const uint32_t o = dst + k * T * VEC * 2;
          copy_async<VEC * 2>(o, a.dy + row * a.ld_dy + c, live);
          copy_async<VEC * 2>(o + slice, a.x + row * a.ld_x + c, live);
          if (has_res) copy_async<VEC * 2>(o + 2 * slice, a.dres + row * a.ld_dres + c, live);
        }
      }
    }
  };
  auto stats = [&](int64_t row0, float(&m)[R], float(&s)[R]) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const bool live = row0 + r < a.rows;
      m[r] = live ? a.mean[row0 + r] : 0.f;
      s[r] = live ? a.rstd[row0 + r] : 0.f;
    }
  };
  if constexpr (RING) {
    for (int s = 0; s < a.depth - 1; ++s) {
      fill(s, first + s * step);
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
  }
  float mean[R], rstd[R], next_mean[R], next_rstd[R];
  stats(first, next_mean, next_rstd);
  int buf = 0, slot = 0;
  for (int64_t row0 = first; row0 < a.rows; row0 += step) {
    V vdy[R][NV], vx[R][NV], vr[R][NV];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      mean[r] = next_mean[r];
      rstd[r] = next_rstd[r];
    }
    stats(row0 + step, next_mean, next_rstd);
    if constexpr (RING) {
      fill(slot == 0 ? a.depth - 1 : slot - 1, row0 + (a.depth - 1) * step);
      asm volatile("cp.async.commit_group;" ::: "memory");
      if (a.depth == 2)
        asm volatile("cp.async.wait_group 1;" ::: "memory");
      else if (a.depth == 3)
        asm volatile("cp.async.wait_group 2;" ::: "memory");
      else
        asm volatile("cp.async.wait_group 3;" ::: "memory");
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t row = row0 + r;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        if constexpr (RING) {
          const uint8_t* p = ring + slot * stage + r * tensors * slice + (t + k * T) * VEC * 2;
          vdy[r][k] = *reinterpret_cast<const V*>(p);
          vx[r][k] = *reinterpret_cast<const V*>(p + slice);
          if (has_res)
            vr[r][k] = *reinterpret_cast<const V*>(p + 2 * slice);
          else
            zero(vr[r][k]);
        } else {
          const bool live = row < a.rows && t + k * T < nvec;
          const int c = t + k * T;
          zero(vdy[r][k]);
          zero(vx[r][k]);
          zero(vr[r][k]);
          if (live) {
            vdy[r][k] = reinterpret_cast<const V*>(a.dy + row * a.ld_dy)[c];
            vx[r][k] = reinterpret_cast<const V*>(a.x + row * a.ld_x)[c];
            if (has_res) vr[r][k] = reinterpret_cast<const V*>(a.dres + row * a.ld_dres)[c];
          }
        }
      }
    }
    if (RING && ++slot == a.depth) slot = 0;
    float s[2 * R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      s[2 * r] = s[2 * r + 1] = 0.f;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        // columns past H and rows past the last hold dy = 0: they add nothing to any sum
        float d[VEC], x[VEC], g[VEC];
        unpack(vdy[r][k], d);
        unpack(vx[r][k], x);
        unpack(gain[k], g);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float xh = (x[i] - mean[r]) * rstd[r];
          const float w = a.g ? d[i] * g[i] : d[i];
          s[2 * r] += w;
          s[2 * r + 1] = fmaf(w, xh, s[2 * r + 1]);
          dg[k * VEC + i] = fmaf(d[i], xh, dg[k * VEC + i]);
          db[k * VEC + i] += d[i];
        }
      }
    }
    group_sums<2 * R>(s, W, wig, 1 + group, red[buf] + group * W * 2 * R);
    buf ^= 1;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int64_t row = row0 + r;
      if (row >= a.rows) continue;
      const float c1 = s[2 * r] * inv_h, c2 = s[2 * r + 1] * inv_h;
      V* po = reinterpret_cast<V*>(a.dx + row * a.ld_dx);
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        if (t + k * T < nvec) {
          float d[VEC], x[VEC], g[VEC], o[VEC];
          unpack(vdy[r][k], d);
          unpack(vx[r][k], x);
          unpack(vr[r][k], o);
          unpack(gain[k], g);
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            const float xh = (x[i] - mean[r]) * rstd[r];
            const float w = a.g ? d[i] * g[i] : d[i];
            o[i] = fmaf(rstd[r], w - c1 - xh * c2, o[i]);
          }
          V out;
          pack(out, o);
          po[t + k * T] = out;
        }
      }
    }
  }
  if constexpr (RING) asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
  // the groups' sums, added in group order
  float* sums = reinterpret_cast<float*>(smem);
  float* pg = gridDim.x == 1 ? a.dg : a.part + static_cast<int64_t>(blockIdx.x) * 2 * a.H;
  float* pb = gridDim.x == 1 ? a.db : pg + a.H;
  for (int gi = 0; gi < groups; ++gi) {
    if (gi > 0) __syncthreads();
    if (group == gi) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int c = t + k * T;
        if (c < nvec) {
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            float vg = dg[k * VEC + i], vb = db[k * VEC + i];
            const int j = c * VEC + i;
            if (gi > 0) {
              vg += sums[j];
              vb += sums[a.H + j];
            }
            if (gi + 1 < groups) {
              sums[j] = vg;
              sums[a.H + j] = vb;
            } else {
              if (pg) pg[j] = vg;
              if (pb) pb[j] = vb;
            }
          }
        }
      }
    }
  }
}

// dg and db from `parts` partial rows of 2H floats: 32 columns a block, 8 threads a column, each the sum of
// every eighth row, added in order.
__global__ void __launch_bounds__(256) layernorm_bwd_reduce_kernel(const float* __restrict__ part, int parts, int H,
                                                                   float* __restrict__ dg, float* __restrict__ db) {
  __shared__ float red[8][32];
  const int lane = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int64_t j = static_cast<int64_t>(blockIdx.x) * 32 + lane, cols = 2 * static_cast<int64_t>(H);
  float v = 0.f;
  if (j < cols) {
#pragma unroll 8
    for (int p = y; p < parts; p += 8) v += part[p * cols + j];
  }
  red[y][lane] = v;
  __syncthreads();
  if (y == 0 && j < cols) {
    for (int k = 1; k < 8; ++k) v += red[k][lane];
    if (j < H) {
      if (dg) dg[j] = v;
    } else if (db) {
      db[j - H] = v;
    }
  }
}

// Rows wider than the registers of a CTA hold: dx a row at a time (the second pass from L2), then the column
// sums in a kernel of their own (before dx, which may overwrite dy).
__global__ void __launch_bounds__(1024, 1) layernorm_bwd_wide_dx_kernel(LnBwd a) {
  __shared__ float red[2][64];
  const int wig = threadIdx.x >> 5;
  const float inv_h = 1.0f / static_cast<float>(a.H);
  int buf = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const __nv_bfloat16 *dy = a.dy + row * a.ld_dy, *x = a.x + row * a.ld_x;
    const float mean = a.mean[row], rstd = a.rstd[row];
    float s[2] = {0.f, 0.f};
    for (int j = threadIdx.x; j < a.H; j += 1024) {
      const float w = __bfloat162float(dy[j]) * (a.g ? __bfloat162float(a.g[j]) : 1.f);
      s[0] += w;
      s[1] = fmaf(w, (__bfloat162float(x[j]) - mean) * rstd, s[1]);
    }
    group_sums<2>(s, 32, wig, 1, red[buf]);
    buf ^= 1;
    for (int j = threadIdx.x; j < a.H; j += 1024) {
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

// The widest vector that divides H and keeps every row of every operand aligned.
struct RowsAlign {
  uintptr_t bits = 0;
  void add(const void* p, int64_t ld) {
    if (p) bits |= reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(ld) * 2;
  }
  int vec(int H) const {
    if (H % 8 == 0 && (bits & 15) == 0) return 8;
    if (H % 2 == 0 && (bits & 3) == 0) return 2;
    return 1;
  }
};

// Warps of a group that hold H elements at EPT a thread, and groups of a CTA.
struct Shape {
  int W, groups;
};
Shape group_shape(int H, int ept) {
  Shape s;
  s.W = (H + 32 * ept - 1) / (32 * ept);
  s.groups = std::max(1, GROUP_THREADS / (32 * s.W));
  return s;
}

template <int VEC, int EPT>
mt_status fwd_go(LnFwd a, cudaStream_t st) {
  const Shape s = group_shape(a.H, EPT);
  a.W = s.W;
  const int threads = s.groups * s.W * 32;
  const int resident = std::max(1, 2048 / (threads * 2));  // about half the SM's threads at the kernel's registers
  const int64_t want = (a.rows + s.groups - 1) / s.groups;
  const int64_t grid = std::min<int64_t>(want, static_cast<int64_t>(num_sms()) * resident);
  layernorm_fwd_kernel<VEC, EPT><<<static_cast<unsigned>(grid), threads, 0, st>>>(a);
  return launch_check("layernorm_fwd_kernel");
}

template <int EPT>
mt_status fwd_vec(const LnFwd& a, int vec, cudaStream_t st) {
  return vec == 8 ? fwd_go<8, EPT>(a, st) : vec == 2 ? fwd_go<2, EPT>(a, st) : fwd_go<1, EPT>(a, st);
}

// Elements a thread and rows a step of the backward: two rows of 8 up to 4096 columns, one of 16 above.
int bwd_ept(int H) { return H <= 4096 ? 8 : 16; }
int bwd_rows(int H) { return H <= 4096 ? 2 : 1; }

// CTAs of the backward, each of which leaves one partial row: as many threads to an SM as its registers allow.
int bwd_parts(int64_t rows, int H) {
  if (H > MAX_H_REG) return static_cast<int>(std::min<int64_t>(2 * SMS, (rows + 63) / 64));
  const Shape s = group_shape(H, bwd_ept(H));
  const int resident = std::max(2, std::min(4, 1024 / (s.groups * s.W * 32)));
  const int64_t step = bwd_rows(H) * s.groups;
  return static_cast<int>(std::min<int64_t>(SMS * resident, (rows + step - 1) / step));
}

uint64_t bwd_ws_bytes(int64_t rows, int H) {
  return static_cast<uint64_t>(align_up(static_cast<int64_t>(std::max(1, bwd_parts(rows, H))) * 2 * H * 4, 256));
}

template <int VEC, int EPT, int R>
mt_status bwd_go(LnBwd a, int parts, cudaStream_t st) {
  const Shape s = group_shape(a.H, EPT);
  const int threads = s.groups * s.W * 32;
  a.W = s.W;
  a.depth = 0;
  int64_t smem = s.groups > 1 ? 2ll * a.H * 4 : 0;  // groups > 1: H <= 1024
  if (VEC > 1) {
    // the deepest ring of 4 stages at most that leaves room for the other CTAs of the SM
    const int64_t stage = static_cast<int64_t>(threads) * EPT * 2 * R * (a.dres ? 3 : 2);
    const int64_t budget = 200 * 1024 / std::max(2, std::min(4, 1024 / threads));
    a.depth = static_cast<int>(std::max<int64_t>(2, std::min<int64_t>(4, budget / stage)));
    smem = std::max(smem, stage * a.depth);
  }
  static SmemOptIn opt;
  if (smem > 40 * 1024) MT_TRY(opt.raise(reinterpret_cast<const void*>(layernorm_bwd_kernel<VEC, EPT, R>)));
  layernorm_bwd_kernel<VEC, EPT, R><<<parts, threads, smem, st>>>(a);
  return launch_check("layernorm_bwd_kernel");
}

template <int EPT, int R>
mt_status bwd_vec(const LnBwd& a, int vec, int parts, cudaStream_t st) {
  return vec == 8 ? bwd_go<8, EPT, R>(a, parts, st) : vec == 2 ? bwd_go<2, EPT, R>(a, parts, st) : bwd_go<1, EPT, R>(a, parts, st);
}

mt_status layernorm_bwd_launch(LnBwd a, cudaStream_t st) {
  if (a.rows == 0) {
    if (a.dg) MT_CUDA(cudaMemsetAsync(a.dg, 0, static_cast<size_t>(a.H) * 4, st));
    if (a.db) MT_CUDA(cudaMemsetAsync(a.db, 0, static_cast<size_t>(a.H) * 4, st));
    return MT_OK;
  }
  const int parts = bwd_parts(a.rows, a.H);
  if (a.H > MAX_H_REG) {
    if (a.dg || a.db) {
      layernorm_bwd_wide_cols_kernel<<<dim3((a.H + 255) / 256, parts), 256, 0, st>>>(a);
      MT_TRY(launch_check("layernorm_bwd_wide_cols_kernel"));
    }
    layernorm_bwd_wide_dx_kernel<<<static_cast<unsigned>(std::min<int64_t>(a.rows, 2 * num_sms())), 1024, 0, st>>>(a);
    MT_TRY(launch_check("layernorm_bwd_wide_dx_kernel"));
  } else {
    RowsAlign al;
    al.add(a.dy, a.ld_dy);
    al.add(a.x, a.ld_x);
    al.add(a.dres, a.ld_dres);
    al.add(a.dx, a.ld_dx);
    al.add(a.g, 0);
    const int v = al.vec(a.H);
    if (a.H <= 4096)
      MT_TRY((bwd_vec<8, 2>(a, v, parts, st)));
    else
      MT_TRY((bwd_vec<16, 1>(a, v, parts, st)));
    if (parts == 1) return MT_OK;
  }
  if (!a.dg && !a.db) return MT_OK;
  layernorm_bwd_reduce_kernel<<<(2 * a.H + 31) / 32, 256, 0, st>>>(a.part, parts, a.H, a.dg, a.db);
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
  if (H > (1 << 28)) return fail(MT_ERR_UNSUPPORTED, "layernorm_fwd: H above 2^28");
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
  if (H > 2 * MAX_H_REG) {
    layernorm_fwd_wide_kernel<<<static_cast<unsigned>(std::min<int64_t>(rows, 2 * num_sms())), 1024, 0,
                                as_stream(stream)>>>(a);
    return launch_check("layernorm_fwd_wide_kernel");
  }
  RowsAlign al;
  al.add(x, ld_x);
  al.add(y, ld_y);
  al.add(g, 0);
  al.add(b, 0);
  const int v = al.vec(H);
  return H <= 256 ? fwd_vec<8>(a, v, as_stream(stream)) : fwd_vec<16>(a, v, as_stream(stream));
}

uint64_t mt_layernorm_bwd_workspace_bytes(int64_t rows, int32_t H) {
  if (rows < 0 || H <= 0) return 0;
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
  if (H > (1 << 28)) return fail(MT_ERR_UNSUPPORTED, "layernorm_bwd: H above 2^28");
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
  a.W = a.depth = 0;
  return layernorm_bwd_launch(a, as_stream(stream));
}

}  // extern "C"
