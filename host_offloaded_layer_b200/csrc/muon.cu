// Muon: momentum and orthogonalisation of a weight matrix's gradient by Newton-Schulz products.
//
//   m' = mu m + g, u = g + mu m' (Nesterov) or m', X = u / (|u|_F + eps)
//   steps times: A = X X^T, X <- a X + (b A + c A^2) X; out = bf16(scale * X)
//
// with (a, b, c) = (3.4445, -4.7750, 2.0315), X on its short side (A = X^T X and X <- a X + X (b A + c A^2)
// where the matrix is taller than wide: the tensor cores read either operand in either order, so nothing is
// transposed). Written m <= n for the two sides, a step is m^2 n + m^3 + 2 m^2 n operations when the two
// symmetric products compute only the tiles on and below the diagonal and store each twice.
//
// Number formats. The operands of the products are fp16, the sums fp32. bf16 operands, 8 bits, leave the
// result 1-10% off. fp16 has 11 bits, and its range is enough because the singular values of X stay below
// 1.2023 (the polynomial's maximum on [0, 1], which it maps into itself): X is held times 2^14, A (< 1.45)
// times 2^14, b A + c A^2 (> -2.81) and the whole polynomial (<= 3.4445) times 2^13. What fp16 operands
// would lose is the weak directions: their singular values grow by a factor of a each step, and so does the
// rounding noise that the strong directions leave in their place. In the early steps a X is therefore added
// from a two-term X (fp16 head + fp16 rest, 22 bits), while the products take the head alone: a rounding of
// b A + c A^2 moves strong directions only, where nothing is amplified. In the last two steps, which amplify
// little, the polynomial takes a on its diagonal and X its head only. Against the same steps in fp64 the
// result is 1e-3 to 1.5e-3 (root of the squares' sum) off before its rounding to bf16, which alone is 1.7e-3, for
// Gaussian matrices, and up to 3e-3 for one or a few strong directions with or without noise (emulated for short sides
// of 65..1500); fp16 throughout is up to 1.4e-2 off. Where one direction has elements of equal size, all roundings of
// an operand fall the same way: 4e-3 at most of those tried.
// |u|_F is summed in fp64, so that no magnitude of g that fp32 holds over- or underflows.
//
// Matrices whose short side is at most 64 take no tensor cores: their Gram matrix (in fp64) is all that the
// steps need, one cluster runs them on it (up to five in fp32, more in fp64), and the result is one product with u: four
// launches.
#include <cuda.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>

#include "mt_internal.h"
#include "tcgen05.cuh"

namespace mt {
namespace {

using namespace tc;

constexpr float NS_A = 3.4445f, NS_B = -4.7750f, NS_C = 2.0315f;
constexpr double NS64_A = 3.4445, NS64_B = -4.7750, NS64_C = 2.0315;
constexpr float S_X = 16384.f, S_A = 16384.f, S_P = 8192.f;
constexpr int64_t MAX_ELEMENTS = 1ll << 36;  // no device holds more; sizes and tile numbers stay in range
constexpr int TINY = 64;  // the widest short side of the Gram path
// Paths, splits of K and workspaces are chosen for a whole B200's SMs whatever the device: a workspace's size and a
// result's order of sums depend on the matrix alone.
constexpr int SMS = 148;

// ------------------------------------------------------------------ momentum, norm, head and rest of X
struct Grad {
  const float* g;
  const float* m_in;  // NULL: u = g
  float* m_out;
  int64_t ld_g, ld_m, rows, cols;
  float mu;
  int nesterov;
};

// m' and u of one element from g and m (two roundings of fp32 each, as written).
__device__ __forceinline__ float momentum_step(const Grad& p, float g, float m, float& mo) {
  mo = fmaf(p.mu, m, g);
  return p.nesterov ? fmaf(p.mu, mo, g) : mo;
}

constexpr int NORM_PARTS = 592;  // CTAs of the norm pass, each of which leaves one partial sum

__device__ __forceinline__ double block_sum(double v) {
  __shared__ double red[32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.0;
  for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) s += red[w];
  __syncthreads();
  return s;
}

// The passes over the matrix walk tiles of (256 / tx) * REPS rows and tx * VEC columns, tx a power of two that
// fits narrow matrices, VEC = 4 where rows are 16-byte aligned. A thread's REPS rows are in flight together.
constexpr int REPS = 8;
struct Walk {
  int tx_log2;
  int64_t col_tiles, tiles;
};

// load(k, row, col) for the thread's rows, then use(k, row, col).
template <int VEC, class L, class F>
__device__ __forceinline__ void walk(const Walk& w, int64_t rows, int64_t cols, L&& load, F&& use) {
  const int tx = 1 << w.tx_log2, ty = 256 >> w.tx_log2;
  const int x = threadIdx.x & (tx - 1), y = threadIdx.x >> w.tx_log2;
  for (int64_t tl = blockIdx.x; tl < w.tiles; tl += gridDim.x) {
    const int64_t rt = tl / w.col_tiles, ct = tl - rt * w.col_tiles;
    const int64_t col = (ct * tx + x) * VEC, row0 = rt * (REPS * ty) + y;
    if (col >= cols) continue;
#pragma unroll
    for (int k = 0; k < REPS; ++k)
      if (row0 + k * ty < rows) load(k, row0 + k * ty, col);
#pragma unroll
    for (int k = 0; k < REPS; ++k)
      if (row0 + k * ty < rows) use(k, row0 + k * ty, col);
  }
}

template <int VEC>
struct F32;
template <>
struct F32<4> {
  using type = float4;
};
template <>
struct F32<1> {
  using type = float;
};

template <int VEC>
__device__ __forceinline__ void ldv(float (&d)[VEC], const float* p) {
  *reinterpret_cast<typename F32<VEC>::type*>(d) = *reinterpret_cast<const typename F32<VEC>::type*>(p);
}

// The kernels of an update are launched one ahead: each starts when the one before it has started everywhere, sets
// itself up, and waits here until that one has completed before it touches what it works on. (What
// that one writes is no const __restrict__ here therefore, whose loads may go by the non-coherent path and ahead of the wait.)
__device__ __forceinline__ void release_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_last() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <class... Params, class... Args>
mt_status launch_ahead(void (*kernel)(Params...), const char* name, int grid, int threads, int64_t smem, int cluster,
                       cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 0 ? 2 : 1;
  MT_CUDA(cudaLaunchKernelEx(&cfg, kernel, Params(args)...));
  return launch_check(name);
}

// Writes m' and a partial |u|^2 (fp64) a CTA; the start of an update, so it also sets the grid barrier back.
template <int VEC>
__global__ void __launch_bounds__(256) muon_norm_kernel(Grad p, Walk w, double* __restrict__ parts, unsigned* counter) {
  release_next();
  if (blockIdx.x == 0 && threadIdx.x == 0) *counter = 0;  // the fused kernel's grid barrier
  double s = 0.0;
  float g[REPS][VEC], m[REPS][VEC];
  walk<VEC>(
      w, p.rows, p.cols,
      [&](int k, int64_t row, int64_t col) {
        ldv<VEC>(g[k], p.g + row * p.ld_g + col);
        if (p.m_in) ldv<VEC>(m[k], p.m_in + row * p.ld_m + col);
      },
      [&](int k, int64_t row, int64_t col) {
        if (p.m_in) {
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            float mo;
            g[k][i] = momentum_step(p, g[k][i], m[k][i], mo);
            m[k][i] = mo;
          }
          *reinterpret_cast<typename F32<VEC>::type*>(p.m_out + row * p.ld_m + col) =
              *reinterpret_cast<typename F32<VEC>::type*>(m[k]);
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i) s = fma(static_cast<double>(g[k][i]), static_cast<double>(g[k][i]), s);
      });
  s = block_sum(s);
  if (threadIdx.x == 0) parts[blockIdx.x] = s;
}

// X = S_X u / (|u| + eps) as fp16 head and rest, from g and the m' that the norm pass left. Threads from 256 on
// only join the sum.
template <int VEC>
__device__ __forceinline__ void scale_pass(const Grad& p, const Walk& w, const double* parts, int n_parts, double eps,
                                           __half* __restrict__ hi, __half* __restrict__ lo, int64_t ld_x) {
  double s = 0.0;
  for (int i = threadIdx.x; i < n_parts; i += blockDim.x) s += parts[i];
  s = block_sum(s);
  // the factor as a mantissa and two powers of two: u times it stays in fp32's range for any |u|
  int e;
  const float mant = static_cast<float>(frexp(static_cast<double>(S_X) / (sqrt(s) + eps), &e));
  const float p1 = ldexpf(1.f, e / 2), p2 = ldexpf(1.f, e - e / 2);
  if (threadIdx.x >= 256) return;
  float g[REPS][VEC], m[REPS][VEC];
  walk<VEC>(
      w, p.rows, p.cols,
      [&](int k, int64_t row, int64_t col) {
        if (!p.m_in || p.nesterov) ldv<VEC>(g[k], p.g + row * p.ld_g + col);
        if (p.m_in) ldv<VEC>(m[k], p.m_out + row * p.ld_m + col);
      },
      [&](int k, int64_t row, int64_t col) {
        __half h[VEC], l[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float u = !p.m_in ? g[k][i] : p.nesterov ? fmaf(p.mu, m[k][i], g[k][i]) : m[k][i];
          const float v = u * p1 * mant * p2;  // a subnormal u is lifted before the factor that rounds
          h[i] = __float2half_rn(v);
          l[i] = __float2half_rn(v - __half2float(h[i]));
        }
        const int64_t at = row * ld_x + col;
        if constexpr (VEC == 4) {
          *reinterpret_cast<uint2*>(hi + at) = *reinterpret_cast<uint2*>(h);
          if (lo) *reinterpret_cast<uint2*>(lo + at) = *reinterpret_cast<uint2*>(l);
        } else {
          hi[at] = h[0];
          if (lo) lo[at] = l[0];
        }
      });
}

template <int VEC>
__global__ void __launch_bounds__(256) muon_scale_kernel(Grad p, Walk w, const double* parts, int n_parts, double eps,
                                                         __half* __restrict__ hi, __half* __restrict__ lo, int64_t ld_x) {
  release_next();
  wait_for_last();
  scale_pass<VEC>(p, w, parts, n_parts, eps, hi, lo, ld_x);
}

// ------------------------------------------------------------------ products
// v = alpha * (A B^T)[r, c] + beta * add_hi[r, c] + beta_lo * add_lo[r, c] + diag (r == c), stored as fp16 (head, and rest
// where out_lo is set) or, where out_bf is set, as bf16. Internal matrices have rows of whole 64-element
// groups, so 16-column chunks are always stored whole there.
struct NsArgs {
  int M, N, K;
  int sym;     // square and symmetric: tiles on and below the diagonal only, each stored twice
  int raster;  // 1: row blocks outer; 2: column blocks outer (the polynomial's matrix stays in L2)
  int full_tiles;  // 256 x 256 tiles; the ones behind them are done in two halves of 128 columns
  float alpha, beta, beta_lo, diag;
  const __half *add_hi, *add_lo;
  __half *out_hi, *out_lo;
  int64_t ld_add, ld_out;
  __nv_bfloat16* out_bf;
  int64_t ld_bf;
  int bf_v16;  // out_bf rows hold 16-byte aligned chunks
};

// A = X X^T, times S_A.
__host__ __device__ __forceinline__ NsArgs gram_args(int m, int n, __half* A, int64_t ld_a) {
  NsArgs e = {};
  e.M = e.N = m;
  e.K = n;
  e.sym = 1;
  e.alpha = S_A / (S_X * S_X);
  e.out_hi = A;
  e.ld_out = ld_a;
  return e;
}

// A product of two m x m matrices that commute with each other (polynomials of A): symmetric.
__host__ __device__ __forceinline__ NsArgs square_args(int m, int64_t ld_a, __half* out, float alpha) {
  NsArgs e = {};
  e.M = e.N = e.K = m;
  e.sym = 1;
  e.alpha = alpha;
  e.out_hi = out;
  e.ld_add = e.ld_out = ld_a;
  return e;
}

// P = b A + c A^2 (fold: + a I), times S_P.
__host__ __device__ __forceinline__ NsArgs poly_args(int m, const __half* A, __half* P, int64_t ld_a, bool fold) {
  NsArgs e = square_args(m, ld_a, P, NS_C * S_P / (S_A * S_A));
  e.beta = NS_B * S_P / S_A;
  e.diag = fold ? NS_A * S_P : 0.f;
  e.add_hi = A;
  return e;
}

// X' = P X (X P in a tall matrix), P held times s_p, + lead * X where P lacks that multiple of I (lead = 0: it does
// not); the last one is the result.
__host__ __device__ __forceinline__ NsArgs apply_args(int m, int n, bool tall, float lead, float s_p, bool last, float scale,
                                                      const __half* x, const __half* lo, __half* out_hi, __half* out_lo, int64_t ld_x,
                                                      __nv_bfloat16* o, int64_t ld_o, int bf_v16) {
  NsArgs e = {};
  e.M = tall ? n : m;
  e.N = tall ? m : n;
  e.K = m;
  e.raster = tall ? 1 : 2;
  e.alpha = (last ? scale / S_X : 1.f) / s_p;
  if (lead != 0.f) {
    e.beta = e.beta_lo = lead;
    e.add_hi = x;
    e.add_lo = lo;
    e.ld_add = ld_x;
  }
  if (last) {
    e.out_bf = o;
    e.ld_bf = ld_o;
    e.bf_v16 = bf_v16;
  } else {
    e.out_hi = out_hi;
    e.out_lo = out_lo;
    e.ld_out = ld_x;
  }
  return e;
}

__device__ __forceinline__ void ld32B(const void* p, uint32_t (&r)[8]) {
  asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "l"(p)
               : "memory");
}
__device__ __forceinline__ void st32B(void* p, const uint32_t (&r)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ float2 h2f(uint32_t w) { return __half22float2(*reinterpret_cast<__half2*>(&w)); }
__device__ __forceinline__ uint32_t f2h(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The addend of 16 columns of a row (zeros where there is none): issued before the products are waited for.
struct Addend {
  uint32_t hi[8], lo[8];
};
__device__ __forceinline__ void load_addend(const NsArgs& e, int row, int col0, Addend& a) {
#pragma unroll
  for (int i = 0; i < 8; ++i) a.hi[i] = a.lo[i] = 0u;
  if (e.add_hi && row < e.M && col0 < e.N) {
    const int64_t at = static_cast<int64_t>(row) * e.ld_add + col0;
    ld32B(e.add_hi + at, a.hi);
    if (e.add_lo) ld32B(e.add_lo + at, a.lo);
  }
}

// Epilogue of 16 columns of the 32 rows that a warp holds, one row a lane (all lanes call it). stage: 32 x STAGE_LD
// bf16 of shared memory of the warp's own, for results whose rows have no 16-byte alignment: from there they are
// written two rows at a time, neighbouring lanes to neighbouring elements.
constexpr int STAGE_LD = 18;
constexpr int STAGE_BYTES = 32 * STAGE_LD * 2;
__device__ __forceinline__ void finish16(const NsArgs& e, int row, int col0, float (&v)[16], const Addend& a, bool mirror,
                                         uint16_t* stage) {
  const bool live = row < e.M;
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] *= e.alpha;
  if (e.add_hi) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 h = h2f(a.hi[i]);
      v[2 * i] = fmaf(e.beta, h.x, v[2 * i]);
      v[2 * i + 1] = fmaf(e.beta, h.y, v[2 * i + 1]);
    }
  }
  if (e.add_lo) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 l = h2f(a.lo[i]);
      v[2 * i] = fmaf(e.beta_lo, l.x, v[2 * i]);
      v[2 * i + 1] = fmaf(e.beta_lo, l.y, v[2 * i + 1]);
    }
  }
  if (e.diag != 0.f) {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (row == col0 + i) v[i] += e.diag;
  }
  if (e.out_bf) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    if (e.bf_v16 && col0 + 16 <= e.N) {
      uint4* o = reinterpret_cast<uint4*>(e.out_bf + static_cast<int64_t>(row) * e.ld_bf + col0);
      if (live) {
        o[0] = make_uint4(w[0], w[1], w[2], w[3]);
        o[1] = make_uint4(w[4], w[5], w[6], w[7]);
      }
    } else {
      const int lane = threadIdx.x & 31;
      uint32_t* mine = reinterpret_cast<uint32_t*>(stage + lane * STAGE_LD);
#pragma unroll
      for (int i = 0; i < 8; ++i) mine[i] = w[i];
      __syncwarp();
      const int c = lane & 15, row0 = row - lane;
      for (int r = lane >> 4; r < 32; r += 2)
        if (row0 + r < e.M && col0 + c < e.N)
          reinterpret_cast<uint16_t*>(e.out_bf)[static_cast<int64_t>(row0 + r) * e.ld_bf + col0 + c] = stage[r * STAGE_LD + c];
      __syncwarp();
    }
    return;
  }
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = f2h(v[2 * i], v[2 * i + 1]);
  if (live) {
    st32B(e.out_hi + static_cast<int64_t>(row) * e.ld_out + col0, w);
    if (e.out_lo) {
      uint32_t l[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 f = h2f(w[i]);
        l[i] = f2h(v[2 * i] - f.x, v[2 * i + 1] - f.y);
      }
      st32B(e.out_lo + static_cast<int64_t>(row) * e.ld_out + col0, l);
    }
  }
  if (mirror) {
    // transposed: lanes exchange their neighbour's pair of columns, so that each stores two rows of one column
    // (a pair (row, row + 1) that ends on the last row writes one element into the row's padding)
    const bool odd = threadIdx.x & 1;
    const int r2 = row & ~1;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t o = __shfl_xor_sync(0xffffffffu, w[i], 1);
      const uint32_t t = odd ? __byte_perm(o, w[i], 0x7632) : __byte_perm(w[i], o, 0x5410);
      const int c = col0 + 2 * i + (odd ? 1 : 0);
      if (r2 < e.M && c < e.N) *reinterpret_cast<uint32_t*>(e.out_hi + static_cast<int64_t>(c) * e.ld_out + r2) = t;
    }
  }
}

// Tile t of the walk: of a symmetric matrix the t-th on or below the diagonal, row by row.
__device__ __forceinline__ void ns_tile(const NsArgs& e, int t, int num_m, int num_n, int& mb, int& nb) {
  if (e.sym) {
    mb = static_cast<int>((sqrtf(8.f * static_cast<float>(t) + 1.f) - 1.f) * 0.5f);
    while ((mb + 1) * (mb + 2) / 2 <= t) ++mb;
    while (mb * (mb + 1) / 2 > t) --mb;
    nb = t - mb * (mb + 1) / 2;
  } else if (e.raster == 1) {
    mb = t / num_n;
    nb = t - mb * num_n;
  } else {
    nb = t / num_m;
    mb = t - nb * num_m;
  }
}

int ns_tiles(const NsArgs& e, int bm) {
  const int num_m = (e.M + bm - 1) / bm, num_n = (e.N + bm - 1) / bm;
  return e.sym ? num_m * (num_m + 1) / 2 : num_m * num_n;
}

constexpr int HALF = 128 * 64 * 2;    // 16 KiB: 128 rows of one operand, one 64-wide K atom
constexpr int MN_BOX = 64 * 64 * 2;   // one 64 x 64 MN-major box
constexpr int ATOMS = 6;              // K atoms of both operands that a CTA's ring holds: 192 KiB
constexpr int RING = ATOMS * 2 * HALF;
constexpr int SMEM_BYTES = RING + 256 + 4 * STAGE_BYTES + 1024;
constexpr int NS_THREADS = 192;       // TMA warp, MMA warp, four epilogue warps

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t map_to_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}

// One thread's bounded wait, the usual case inline (a role that is one thread needs no warp-wide agreement).
__device__ __forceinline__ bool wait_one(uint32_t bar, uint32_t parity, volatile int* abort_flag, int32_t* err, int code) {
  if (mbar_try(bar, parity)) return true;
  return mbar_wait(bar, parity, abort_flag, err, code);
}

// Instruction descriptor of kind::f16 with fp16 operands and fp32 sums.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool a_mn, bool b_mn) {
  return (1u << 4) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

// Bytes that loading 128 rows of an operand from r0 brings for one K atom (boxes past its R rows are not loaded).
__device__ __forceinline__ uint32_t rows_bytes(bool mn, int r0, int R) {
  if (!mn) return r0 < R ? HALF : 0;
  return (r0 < R ? MN_BOX : 0) + (r0 + 64 < R ? MN_BOX : 0);
}

// One K atom of 128 rows of an operand. K-major: a box of 64 (K) x 128 rows. MN-major: two boxes of 64 rows x
// 64 (K), `mn_stride` bytes apart.
template <bool MN, class Load>
__device__ __forceinline__ void load_atom(uint32_t dst, int mn_stride, int r0, int R, int k, Load&& load) {
  if (!MN) {
    if (r0 < R) load(dst, k, r0);
  } else {
#pragma unroll
    for (int j = 0; j < 2; ++j)
      if (r0 + 64 * j < R) load(dst + j * mn_stride, r0 + 64 * j, k);
  }
}

// Descriptor of a stage of KA atoms at `base`, and how far K step kk (16 wide) lies into it, in the descriptor's
// 16-byte units (added to its low word: one add a product, where building each would hold up the issuing thread).
// K-major: atom kk / 4 and 32 bytes a step inside the swizzled rows; MN-major: 16 rows of K (2 KiB) a step, the two
// 64-row halves KA boxes apart.
template <bool MN, int KA>
__device__ __forceinline__ uint64_t stage_desc(uint32_t base) {
  return MN ? smem_desc(base, KA * MN_BOX, 1024) : smem_desc(base, 16, 1024);
}
template <bool MN>
__device__ __forceinline__ constexpr uint64_t step_off(int kk) {
  return static_cast<uint64_t>(MN ? kk * 2048 : (kk >> 2) * HALF + (kk & 3) * 32) >> 4;
}

// ---------------------------------------------------------------- 256 x 256 tiles on two SMs
// A persistent cluster of two CTAs: each stages its 128 rows of A and 128 columns of B, the even one issues
// cta_group::2 products for both into one of two 256-column accumulators, and both drain theirs while the
// next tile runs. A last wave that would leave half of the clusters idle or more is done in half tiles (256 x 128):
// the 105 tiles of a symmetric 3584 x 3584 product take 74 clusters for 1.6 tiles' time instead of two.
template <bool A_MN, bool B_MN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(NS_THREADS, 1)
    ns_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const __grid_constant__ CUtensorMap tmB64, const __grid_constant__ NsArgs ep, int32_t* err) {
  constexpr int KA = 2, STAGES = ATOMS / KA, OP_STAGE = HALF * KA, BK = 64 * KA;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = smem + STAGES * OP_STAGE;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + RING);  // TMA (both CTAs) -> MMA, in the even CTA
  uint64_t* empty = full + STAGES;                            // MMA -> TMA, in each CTA
  uint64_t* tfull = empty + STAGES;                           // MMA -> epilogue, in each CTA
  uint64_t* tempty = tfull + 2;                               // epilogue warps of both CTAs -> MMA, in the even CTA
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tempty + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int cluster = blockIdx.x >> 1, n_clusters = gridDim.x >> 1;
  const int num_m = (ep.M + 255) / 256, num_n = (ep.N + 255) / 256;
  const int all_tiles = ep.sym ? num_m * (num_m + 1) / 2 : num_m * num_n;
  const int num_tiles = ep.full_tiles + 2 * (all_tiles - ep.full_tiles);
  const int num_kb = (ep.K + BK - 1) / BK;
  // tile t: its blocks, its first column, and whether it is half a tile
  auto locate = [&](int t, int& mb, int& nb, int& n0) {
    const int u = t - ep.full_tiles;
    ns_tile(ep, u < 0 ? t : ep.full_tiles + u / 2, num_m, num_n, mb, nb);
    n0 = nb * 256 + (u < 0 ? 0 : (u & 1) * 128);
    return u >= 0;
  };

  release_next();
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&tfull[b]), 1);
      mbar_init(smem_u32(&tempty[b]), 8);  // four epilogue warps of each CTA
    }
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  cluster_sync();
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_slot)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem_base = *tmem_slot;
  wait_for_last();

  uint32_t issued = 0;  // K stages that the producer has loaded
  if (warp == 0) {
    if (lane == 0) {
      uint32_t it = 0;
      bool ok = true;
      for (int t = cluster; t < num_tiles && ok; t += n_clusters) {
        int mb, nb, n0;
        const bool halved = locate(t, mb, nb, n0);
        const int m_own = mb * 256 + static_cast<int>(rank) * 128, n_own = n0 + static_cast<int>(rank) * (halved ? 64 : 128);
        const uint32_t bytes = rows_bytes(A_MN, mb * 256, ep.M) + rows_bytes(A_MN, mb * 256 + 128, ep.M) +
                               (halved ? (n0 < ep.N ? MN_BOX : 0) + (n0 + 64 < ep.N ? MN_BOX : 0)
                                       : rows_bytes(B_MN, n0, ep.N) + rows_bytes(B_MN, n0 + 128, ep.N));
        for (int kb = 0; kb < num_kb; ++kb, ++it) {
          const int s = it % STAGES;
          if (!wait_one(smem_u32(&empty[s]), ((it / STAGES) & 1u) ^ 1u, abort_flag, err, DEV_ERR_TIMEOUT_PRODUCER)) {
            ok = false;
            break;
          }
          const uint32_t fb = map_to_rank(smem_u32(&full[s]), 0);
          const int k0 = kb * BK, atoms = min(KA, (ep.K - k0 + 63) / 64);
          ++issued;
          if (rank == 0) mbar_expect_tx(smem_u32(&full[s]), bytes * static_cast<uint32_t>(atoms));
          auto load = [&](const CUtensorMap* map) {
            return [=](uint32_t dst, int c0, int c1) {
              asm volatile(
                  "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, "
                  "{%3, %4}], [%2];" ::"r"(dst),
                  "l"(reinterpret_cast<uint64_t>(map)), "r"(fb), "r"(c0), "r"(c1)
                  : "memory");
            };
          };
          const uint32_t a_dst = smem_u32(sA + s * OP_STAGE), b_dst = smem_u32(sB + s * OP_STAGE);
          for (int at = 0; at < atoms; ++at) {
            load_atom<A_MN>(a_dst + at * (A_MN ? MN_BOX : HALF), KA * MN_BOX, m_own, ep.M, k0 + 64 * at, load(&tmA));
            if (!halved) {
              load_atom<B_MN>(b_dst + at * (B_MN ? MN_BOX : HALF), KA * MN_BOX, n_own, ep.N, k0 + 64 * at, load(&tmB));
            } else if (n_own < ep.N) {  // 64 rows: one box in either order
              if (B_MN)
                load(&tmB64)(b_dst + at * MN_BOX, n_own, k0 + 64 * at);
              else
                load(&tmB64)(b_dst + at * HALF, k0 + 64 * at, n_own);
            }
          }
        }
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (rank == 0 && lane == 0) {
      constexpr uint16_t both = 0x3;
      auto commit = [&](uint64_t* bar) {
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                smem_u32(bar)),
            "h"(both)
            : "memory");
      };
      const uint64_t a_desc = stage_desc<A_MN, KA>(smem_u32(sA)), b_desc = stage_desc<B_MN, KA>(smem_u32(sB));
      uint32_t it = 0;
      int tl = 0;
      bool ok = true;
      for (int t = cluster; t < num_tiles && ok; t += n_clusters, ++tl) {
        const int ab = tl & 1;
        const uint32_t idesc = t < ep.full_tiles ? idesc_f16(256, 256, A_MN, B_MN) : idesc_f16(256, 128, A_MN, B_MN);
        if (!wait_one(smem_u32(&tempty[ab]), ((tl >> 1) & 1u) ^ 1u, abort_flag, err, DEV_ERR_TIMEOUT_MMA)) break;
        fence_after();
        const uint32_t d = tmem_base + static_cast<uint32_t>(ab * 256);
        for (int kb = 0; kb < num_kb; ++kb, ++it) {
          const int s = it % STAGES;
          if (!wait_one(smem_u32(&full[s]), (it / STAGES) & 1u, abort_flag, err, DEV_ERR_TIMEOUT_MMA)) {
            ok = false;
            break;
          }
          fence_after();
          const uint64_t ad = a_desc + s * (OP_STAGE >> 4), bd = b_desc + s * (OP_STAGE >> 4);
          const int atoms = min(KA, (ep.K - kb * BK + 63) / 64);
#pragma unroll
          for (int kk = 0; kk < 4 * KA; ++kk)
            if (kk < 4 * atoms)
              asm volatile(
                  "{\n\t.reg .pred p;\n\t"
                  "setp.ne.b32 p, %4, 0;\n\t"
                  "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                  "l"(ad + step_off<A_MN>(kk)), "l"(bd + step_off<B_MN>(kk)), "r"(idesc), "r"((kb > 0 || kk > 0) ? 1u : 0u));
          commit(&empty[s]);
        }
        if (ok) commit(&tfull[ab]);
      }
    }
    __syncwarp();
  } else {
    const int q = warp & 3;  // TMEM lanes [32 q, 32 q + 32)
    uint16_t* stage = reinterpret_cast<uint16_t*>(smem + RING + 256 + q * STAGE_BYTES);
    int tl = 0;
    for (int t = cluster; t < num_tiles; t += n_clusters, ++tl) {
      const int ab = tl & 1;
      int mb, nb, n0;
      const bool halved = locate(t, mb, nb, n0);
      if (!warp_wait(smem_u32(&tfull[ab]), (tl >> 1) & 1u, abort_flag, err, DEV_ERR_TIMEOUT_EPILOGUE)) break;
      fence_after();
      const int row = mb * 256 + static_cast<int>(rank) * 128 + q * 32 + lane;
      const uint32_t tbase = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(ab * 256);
      for (int c = 0; c < (halved ? 4 : 8); ++c) {
        const int col0 = n0 + c * 32;
        if (col0 >= ep.N) break;
        Addend add[2];
        load_addend(ep, row, col0, add[0]);
        load_addend(ep, row, col0 + 16, add[1]);
        uint32_t r[32];
        tmem_ld32(tbase + static_cast<uint32_t>(c * 32), r);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (col0 + 16 * h >= ep.N) break;
          float v[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[16 * h + i]);
          finish16(ep, row, col0 + 16 * h, v, add[h], ep.sym && mb != nb, stage);
        }
      }
      fence_before();
      __syncwarp();
      if (lane == 0)
        asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(
                         map_to_rank(smem_u32(&tempty[ab]), 0))
                     : "memory");
    }
  }

  fence_before();
  __syncthreads();
  if (*abort_flag && rank == 0) drain_ring(smem_u32(full), issued, STAGES);  // its barriers count both CTAs' loads
  cluster_sync();  // neither CTA leaves while its peer may still signal it
  fence_after();
  if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem_base) : "memory");
}

// ---------------------------------------------------------------- 128 x 128 tiles on one SM, K split over a cluster
// For matrices with too few 256 x 256 tiles to fill the GPU, where a product takes microseconds and latencies are
// what counts: one tile a cluster of 1 to 8 CTAs, each of which sums its share of K in its own TMEM. With more than
// one, the shares meet in shared memory: every CTA leaves its fp32 tile there and each finishes 128 / size columns,
// adding the peers' tiles in rank order. Eight epilogue warps, two to a TMEM lane quarter, fetch the addend while
// the products run.
constexpr int RED_LD = 132;  // floats of a row of the shared tile: 16-byte accesses of 8 rows hit 32 banks
static_assert(128 * RED_LD * 4 <= RING, "the tile overlays the ring");
constexpr int TILE_THREADS = 64 + 256;
constexpr int FUSED_SMEM = RING + 256 + 8 * STAGE_BYTES + 1024;

template <bool A_MN, bool B_MN>
__global__ void __launch_bounds__(TILE_THREADS, 1)
    ns_tile_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, const __grid_constant__ NsArgs ep,
                   int32_t* err) {
  constexpr int STAGES = ATOMS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = smem + STAGES * HALF;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + RING);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tfull + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_rank()), size = static_cast<int>(cluster_size());
  const int num_m = (ep.M + 127) / 128, num_n = (ep.N + 127) / 128;
  int mb, nb;
  ns_tile(ep, static_cast<int>(blockIdx.x) / size, num_m, num_n, mb, nb);
  const int atoms = (ep.K + 63) / 64;
  const int kb0 = static_cast<int>(static_cast<int64_t>(atoms) * rank / size);
  const int kb1 = static_cast<int>(static_cast<int64_t>(atoms) * (rank + 1) / size);  // size <= atoms: never empty

  release_next();
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    mbar_init(smem_u32(tfull), 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmA)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmB)) : "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 128;" ::"r"(smem_u32(tmem_slot)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem_base = *tmem_slot;
  wait_for_last();

  // What an epilogue thread finishes: `count` groups of 16 columns from first_col of row in_tile (its lane quarter's
  // row; the two warps of a quarter take the columns by halves).
  const int in_tile = (warp & 3) * 32 + lane, half = (warp - 2) >> 2;
  const int share16 = 8 / size, count = share16 >= 2 ? share16 / 2 : (half == 0 ? share16 : 0);
  const int first_col = nb * 128 + rank * (128 / size) + half * count * 16;
  const int row = mb * 128 + in_tile;
  const bool mirror = ep.sym && mb != nb;
  uint16_t* stage = reinterpret_cast<uint16_t*>(smem + 128 * RED_LD * 4 + max(warp - 2, 0) * STAGE_BYTES);  // the ring is read by then
  Addend add[4];
  bool done = true;     // this warp's waits all ended
  uint32_t issued = 0;  // K atoms that the producer has loaded
  if (warp == 0) {
    if (lane == 0) {
      const uint32_t bytes = rows_bytes(A_MN, mb * 128, ep.M) + rows_bytes(B_MN, nb * 128, ep.N);
      for (int kb = kb0; kb < kb1; ++kb) {
        const int it = kb - kb0, s = it % STAGES;
        if (!wait_one(smem_u32(&empty[s]), ((it / STAGES) & 1u) ^ 1u, abort_flag, err, DEV_ERR_TIMEOUT_PRODUCER)) break;
        const uint32_t fb = smem_u32(&full[s]);
        ++issued;
        mbar_expect_tx(fb, bytes);
        load_atom<A_MN>(smem_u32(sA + s * HALF), MN_BOX, mb * 128, ep.M, kb * 64,
                        [&](uint32_t dst, int c0, int c1) { tma_load_2d(dst, &tmA, fb, c0, c1); });
        load_atom<B_MN>(smem_u32(sB + s * HALF), MN_BOX, nb * 128, ep.N, kb * 64,
                        [&](uint32_t dst, int c0, int c1) { tma_load_2d(dst, &tmB, fb, c0, c1); });
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_f16(128, 128, A_MN, B_MN);
      const uint64_t a_desc = stage_desc<A_MN, 1>(smem_u32(sA)), b_desc = stage_desc<B_MN, 1>(smem_u32(sB));
      bool ok = true;
      for (int kb = kb0; kb < kb1; ++kb) {
        const int it = kb - kb0, s = it % STAGES;
        if (!wait_one(smem_u32(&full[s]), (it / STAGES) & 1u, abort_flag, err, DEV_ERR_TIMEOUT_MMA)) {
          ok = false;
          break;
        }
        fence_after();
        const uint64_t ad = a_desc + s * (HALF >> 4), bd = b_desc + s * (HALF >> 4);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          umma_bf16(tmem_base, ad + step_off<A_MN>(kk), bd + step_off<B_MN>(kk), idesc, (it > 0 || kk > 0) ? 1u : 0u);
        umma_commit(smem_u32(&empty[s]));
      }
      if (ok) umma_commit(smem_u32(tfull));
    }
    __syncwarp();
  } else {
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (c < count) load_addend(ep, row, first_col + 16 * c, add[c]);
    done = warp_wait(smem_u32(tfull), 0, abort_flag, err, DEV_ERR_TIMEOUT_EPILOGUE);
    fence_after();
    if (done) {
      const uint32_t tbase = tmem_base + (static_cast<uint32_t>((warp & 3) * 32) << 16) + static_cast<uint32_t>(half * 64);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t r[32];
        tmem_ld32(tbase + static_cast<uint32_t>(c * 32), r);
        if (size == 1) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int col0 = first_col + c * 32 + 16 * h;
            float v[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[16 * h + i]);
            if (col0 < ep.N) finish16(ep, row, col0, v, add[2 * c + h], mirror, stage);
          }
        } else {
          // every product that read the ring has completed: the tile may overlay it
          float4* p = reinterpret_cast<float4*>(reinterpret_cast<float*>(smem) + in_tile * RED_LD + half * 64 + c * 32);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            p[i] = make_float4(__uint_as_float(r[4 * i]), __uint_as_float(r[4 * i + 1]), __uint_as_float(r[4 * i + 2]),
                               __uint_as_float(r[4 * i + 3]));
        }
      }
    }
  }
  fence_before();
  __syncthreads();
  if (*abort_flag) drain_ring(smem_u32(full), issued, STAGES);
  if (size > 1) {
    cluster_sync();
    if (warp >= 2 && done) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int col0 = first_col + 16 * c;
        if (c < count && col0 < ep.N) {
          float v[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = 0.f;
          const uint32_t at = smem_u32(smem) + (in_tile * RED_LD + (col0 - nb * 128)) * 4;
          for (int p = 0; p < size; p += 2) {  // two peers' reads in flight
            float4 f[2][4];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const uint32_t from = map_to_rank(at, static_cast<uint32_t>(p + q));
#pragma unroll
              for (int i = 0; i < 4; ++i)
                asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                             : "=f"(f[q][i].x), "=f"(f[q][i].y), "=f"(f[q][i].z), "=f"(f[q][i].w)
                             : "r"(from + 16 * i)
                             : "memory");
            }
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                v[4 * i] += f[q][i].x;
                v[4 * i + 1] += f[q][i].y;
                v[4 * i + 2] += f[q][i].z;
                v[4 * i + 3] += f[q][i].w;
              }
          }
          finish16(ep, row, col0, v, add[c], mirror, stage);
        }
      }
    }
    cluster_sync();  // no CTA leaves while a peer reads its tile
  }
  fence_after();
  if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 128;" ::"r"(tmem_base) : "memory");
}

// ---------------------------------------------------------------- all steps in one kernel
// Small matrices spend their time between kernels, not in them: 15 products of a few microseconds. Where each
// product has no more 128 x 128 tiles than about the GPU has SMs, one cooperative kernel (every CTA resident) runs
// the scaling and all steps, a grid barrier after each. Tiles as in ns_tile_kernel; K of the Gram products, the long
// side, is split over CTAs that would have no tile, and a pass over the partial tiles (from L2) finishes them.
struct FusedArgs {
  Grad grad;
  Walk walk;
  const double* part;
  int parts, vec4;
  double eps;
  int m, n, tall, steps, two_term, split;  // split: parts of K of a Gram product
  float* partial;
  __half *hi[2], *lo, *A, *P;
  int64_t ld_x, ld_a;
  float scale;
  __nv_bfloat16* o;
  int64_t ld_o;
  int bf_v16;
  unsigned* counter;  // zeroed by the norm pass
};

struct FusedMaps {
  CUtensorMap x_short[2], x_long[2], A, P;
};

struct TileSmem {
  uint8_t *sA, *sB, *stages;
  uint64_t *full, *empty, *tfull;
  volatile int* abort_flag;
  uint32_t tmem;
};

// Everything that the grid's threads wrote is there for its threads' reads and tensor copies afterwards. Bounded
// like every wait; false: it ran out somewhere, and the kernel ends.
__device__ __forceinline__ bool grid_barrier(unsigned* counter, unsigned target, volatile int* abort_flag, int32_t* err) {
  asm volatile("fence.proxy.async.global;" ::: "memory");
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();  // cumulative: releases what the CTA's threads wrote before the barrier above
    asm volatile("red.relaxed.gpu.global.add.u32 [%0], 1;" ::"l"(counter) : "memory");
    const unsigned long long t0 = globaltimer();
    for (uint32_t i = 1;; ++i) {
      unsigned v;
      asm volatile("ld.relaxed.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(counter) : "memory");
      if (v >= target || *abort_flag) break;
      if ((i & 1023u) == 0 && globaltimer() - t0 > WAIT_NS) {
        *abort_flag = 1;
        atomicCAS(err, 0, DEV_ERR_TIMEOUT_PRODUCER);
        break;
      }
    }
    __threadfence();  // acquires what the other CTAs released
  }
  __syncthreads();
  asm volatile("fence.proxy.async.global;" ::: "memory");
  return *abort_flag == 0;
}

// A partial tile in the workspace: eight chunks of 16 columns, each [128 rows][16].
constexpr int PARTIAL = 128 * 128;

// One product's tiles over the grid. K of each is split into `split` parts: 1, and the tile is finished here; more,
// and each part's fp32 sums go to `partial`, in (tile, part) order, for finish_parts behind a grid barrier.
// it: K atoms that this CTA's ring has carried; tiles: tiles or parts that it has summed (the parity of tfull);
// issued: atoms that the calling thread has loaded.
template <bool A_MN, bool B_MN>
__device__ __forceinline__ void fused_product(const CUtensorMap* tmA, const CUtensorMap* tmB, const NsArgs& ep, int split,
                                              float* partial, const TileSmem& sm, uint32_t& it, uint32_t& tiles, uint32_t& issued, int32_t* err) {
  constexpr int STAGES = ATOMS;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int num_m = (ep.M + 127) / 128, num_n = (ep.N + 127) / 128;
  const int num_tiles = ep.sym ? num_m * (num_m + 1) / 2 : num_m * num_n;
  const int atoms = (ep.K + 63) / 64;
  const int in_tile = (warp & 3) * 32 + lane, half = (warp - 2) >> 2;
  for (int u = static_cast<int>(blockIdx.x); u < num_tiles * split; u += static_cast<int>(gridDim.x)) {
    const int t = u / split, part = u - t * split;
    const int kb0 = static_cast<int>(static_cast<int64_t>(atoms) * part / split);
    const int nk = static_cast<int>(static_cast<int64_t>(atoms) * (part + 1) / split) - kb0;  // split <= atoms: never none
    int mb, nb;
    ns_tile(ep, t, num_m, num_n, mb, nb);
    const int first_col = nb * 128 + half * 64, row = mb * 128 + in_tile;
    const bool mirror = ep.sym && mb != nb, diag = ep.sym && mb == nb;  // on the diagonal both operands are the same rows
    if (warp == 0) {
      if (lane == 0) {
        const uint32_t bytes = rows_bytes(A_MN, mb * 128, ep.M) + (diag ? 0 : rows_bytes(B_MN, nb * 128, ep.N));
        for (int i = 0; i < nk; ++i) {
          const uint32_t g = it + i, s = g % STAGES;
          if (!wait_one(smem_u32(&sm.empty[s]), ((g / STAGES) & 1u) ^ 1u, sm.abort_flag, err, DEV_ERR_TIMEOUT_PRODUCER)) break;
          const uint32_t fb = smem_u32(&sm.full[s]);
          ++issued;
          mbar_expect_tx(fb, bytes);
          load_atom<A_MN>(smem_u32(sm.sA + s * HALF), MN_BOX, mb * 128, ep.M, (kb0 + i) * 64,
                          [&](uint32_t dst, int c0, int c1) { tma_load_2d(dst, tmA, fb, c0, c1); });
          if (!diag)
            load_atom<B_MN>(smem_u32(sm.sB + s * HALF), MN_BOX, nb * 128, ep.N, (kb0 + i) * 64,
                            [&](uint32_t dst, int c0, int c1) { tma_load_2d(dst, tmB, fb, c0, c1); });
        }
      }
      __syncwarp();
    } else if (warp == 1) {
      if (lane == 0) {
        constexpr uint32_t idesc = idesc_f16(128, 128, A_MN, B_MN);
        const uint64_t a_desc = stage_desc<A_MN, 1>(smem_u32(sm.sA)), b_desc = stage_desc<B_MN, 1>(smem_u32(diag ? sm.sA : sm.sB));
        bool ok = true;
        for (int i = 0; i < nk; ++i) {
          const uint32_t g = it + i, s = g % STAGES;
          if (!wait_one(smem_u32(&sm.full[s]), (g / STAGES) & 1u, sm.abort_flag, err, DEV_ERR_TIMEOUT_MMA)) {
            ok = false;
            break;
          }
          fence_after();
          const uint64_t ad = a_desc + s * (HALF >> 4), bd = b_desc + s * (HALF >> 4);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            umma_bf16(sm.tmem, ad + step_off<A_MN>(kk), bd + step_off<B_MN>(kk), idesc, (i > 0 || kk > 0) ? 1u : 0u);
          umma_commit(smem_u32(&sm.empty[s]));
        }
        if (ok) umma_commit(smem_u32(sm.tfull));
      }
      __syncwarp();
    } else {
      uint16_t* stage = reinterpret_cast<uint16_t*>(sm.stages + (warp - 2) * STAGE_BYTES);
      Addend add[4];
      if (split == 1) {
#pragma unroll
        for (int c = 0; c < 4; ++c) load_addend(ep, row, first_col + 16 * c, add[c]);
      }
      if (warp_wait(smem_u32(sm.tfull), tiles & 1u, sm.abort_flag, err, DEV_ERR_TIMEOUT_EPILOGUE)) {
        fence_after();
        const uint32_t tbase = sm.tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + static_cast<uint32_t>(half * 64);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t r[32];
          tmem_ld32(tbase + static_cast<uint32_t>(c * 32), r);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (split == 1) {
              const int col0 = first_col + c * 32 + 16 * h;
              float v[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[16 * h + i]);
              if (col0 < ep.N) finish16(ep, row, col0, v, add[2 * c + h], mirror, stage);
            } else {
              float4* p = reinterpret_cast<float4*>(partial + static_cast<int64_t>(u) * PARTIAL +
                                                    ((half * 4 + 2 * c + h) * 128 + in_tile) * 16);
#pragma unroll
              for (int i = 0; i < 4; ++i)
                p[i] = make_float4(__uint_as_float(r[16 * h + 4 * i]), __uint_as_float(r[16 * h + 4 * i + 1]),
                                   __uint_as_float(r[16 * h + 4 * i + 2]), __uint_as_float(r[16 * h + 4 * i + 3]));
            }
          }
        }
      }
    }
    it += static_cast<uint32_t>(nk);
    ++tiles;
    fence_before();
    __syncthreads();  // the accumulator is read
    fence_after();
  }
}

// The tiles of a split symmetric product (no addend) from their parts, added in order: a warp 32 rows of a chunk.
__device__ __forceinline__ void finish_parts(const NsArgs& ep, int split, const float* partial, const TileSmem& sm) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp < 2) return;
  const int num_m = (ep.M + 127) / 128, num_tiles = num_m * (num_m + 1) / 2;
  Addend none;
#pragma unroll
  for (int i = 0; i < 8; ++i) none.hi[i] = none.lo[i] = 0u;
  for (int w = static_cast<int>(blockIdx.x) * 8 + warp - 2; w < num_tiles * 32; w += static_cast<int>(gridDim.x) * 8) {
    const int t = w >> 5, quarter = w & 3, chunk = (w >> 2) & 7;
    int mb, nb;
    ns_tile(ep, t, num_m, num_m, mb, nb);
    const int in_tile = quarter * 32 + lane, col0 = nb * 128 + chunk * 16;
    if (col0 >= ep.N || mb * 128 + quarter * 32 >= ep.M) continue;
    const float4* p = reinterpret_cast<const float4*>(partial + static_cast<int64_t>(t) * split * PARTIAL + (chunk * 128 + in_tile) * 16);
    float v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = 0.f;
    for (int s = 0; s < split; s += 4) {  // four parts' loads in flight
      float4 f[4][4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          f[q][i] = s + q < split ? p[static_cast<int64_t>(s + q) * (PARTIAL / 4) + i] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[4 * i] += f[q][i].x;
          v[4 * i + 1] += f[q][i].y;
          v[4 * i + 2] += f[q][i].z;
          v[4 * i + 3] += f[q][i].w;
        }
    }
    finish16(ep, mb * 128 + in_tile, col0, v, none, mb != nb, reinterpret_cast<uint16_t*>(sm.stages));
  }
}

template <bool TALL>
__global__ void __launch_bounds__(TILE_THREADS, 1)
    ns_fused_kernel(const __grid_constant__ FusedMaps maps, const __grid_constant__ FusedArgs a, int32_t* err) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  TileSmem sm;
  sm.sA = smem;
  sm.sB = smem + ATOMS * HALF;
  sm.full = reinterpret_cast<uint64_t*>(smem + RING);
  sm.empty = sm.full + ATOMS;
  sm.tfull = sm.empty + ATOMS;
  sm.stages = smem + RING + 256;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm.tfull + 1);
  sm.abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int s = 0; s < ATOMS; ++s) {
      mbar_init(smem_u32(&sm.full[s]), 1);
      mbar_init(smem_u32(&sm.empty[s]), 1);
    }
    mbar_init(smem_u32(sm.tfull), 1);
    *sm.abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 128;" ::"r"(smem_u32(tmem_slot)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  sm.tmem = *tmem_slot;
  if (a.vec4)
    scale_pass<4>(a.grad, a.walk, a.part, a.parts, a.eps, a.hi[0], a.two_term > 0 ? a.lo : nullptr, a.ld_x);
  else
    scale_pass<1>(a.grad, a.walk, a.part, a.parts, a.eps, a.hi[0], a.two_term > 0 ? a.lo : nullptr, a.ld_x);
  uint32_t it = 0, tiles = 0, issued = 0;
  unsigned target = gridDim.x;
  bool ok = grid_barrier(a.counter, target, sm.abort_flag, err);
  for (int s = 0; s < a.steps && ok; ++s) {
    const __half* x = a.hi[s & 1];
    const bool fold = s >= a.two_term, last = s + 1 == a.steps;
    NsArgs e = gram_args(a.m, a.n, a.A, a.ld_a);
    fused_product<TALL, TALL>(&maps.x_short[s & 1], &maps.x_short[s & 1], e, a.split, a.partial, sm, it, tiles, issued, err);
    if (a.split > 1) {
      ok = grid_barrier(a.counter, target += gridDim.x, sm.abort_flag, err);
      if (!ok) break;
      finish_parts(e, a.split, a.partial, sm);
    }
    ok = grid_barrier(a.counter, target += gridDim.x, sm.abort_flag, err);
    if (!ok) break;
    e = poly_args(a.m, a.A, a.P, a.ld_a, fold);
    fused_product<false, false>(&maps.A, &maps.A, e, 1, nullptr, sm, it, tiles, issued, err);
    ok = grid_barrier(a.counter, target += gridDim.x, sm.abort_flag, err);
    if (!ok) break;
    e = apply_args(a.m, a.n, TALL, fold ? 0.f : NS_A, S_P, last, a.scale, x, a.lo, a.hi[(s + 1) & 1], s + 1 < a.two_term ? a.lo : nullptr, a.ld_x,
                   a.o, a.ld_o, a.bf_v16);
    if (TALL)
      fused_product<false, false>(&maps.x_long[s & 1], &maps.P, e, 1, nullptr, sm, it, tiles, issued, err);
    else
      fused_product<false, true>(&maps.P, &maps.x_long[s & 1], e, 1, nullptr, sm, it, tiles, issued, err);
    if (!last) ok = grid_barrier(a.counter, target += gridDim.x, sm.abort_flag, err);
  }
  fence_before();
  __syncthreads();
  if (*sm.abort_flag) drain_ring(smem_u32(sm.full), issued, ATOMS);
  fence_after();
  if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 128;" ::"r"(sm.tmem) : "memory");
}

// An fp16 operand: element (r, k) at p[r * ld + k] (K-major) or p[k * ld + r] (MN-major).
struct Operand {
  const __half* p;
  int64_t ld;
  bool mn;
  int64_t rows;
};

// Its tensor maps: boxes of 128 rows (MN-major: 64), and of 64.
struct OperandMaps {
  CUtensorMap rows128, rows64;
  bool mn;
};
mt_status operand_maps(OperandMaps* m, const Operand& o, int64_t K) {
  m->mn = o.mn;
  if (o.mn) {
    MT_TRY(tma_map_2d(&m->rows128, o.p, o.rows, K, o.ld, 64, 64));
    m->rows64 = m->rows128;
    return MT_OK;
  }
  MT_TRY(tma_map_2d(&m->rows128, o.p, K, o.rows, o.ld, 64, 128));
  return tma_map_2d(&m->rows64, o.p, K, o.rows, o.ld, 64, 64);
}

// Clusters of two that run at once: one CTA an SM.
int pair_clusters() { return std::max(1, num_sms() / 2); }

template <bool A_MN, bool B_MN>
mt_status ns_launch(const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& tb64, NsArgs e, int split, cudaStream_t st) {
  int32_t* err = device_error_word();
  if (!err) return fail(MT_ERR_CUDA, "device error word unavailable");
  if (split == 0) {
    static SmemOptIn opt;
    MT_TRY(opt.raise(reinterpret_cast<const void*>(ns_pair_kernel<A_MN, B_MN>)));
    const int tiles = ns_tiles(e, 256), most = pair_clusters(), over = tiles % most;
    e.full_tiles = 2 * over <= most ? tiles - over : tiles;
    const int clusters = std::min(e.full_tiles + 2 * (tiles - e.full_tiles), most);
    return launch_ahead(ns_pair_kernel<A_MN, B_MN>, "ns_pair_kernel", 2 * clusters, NS_THREADS, SMEM_BYTES, 0, st, ta, tb, tb64, e,
                        err);
  }
  static SmemOptIn opt;
  MT_TRY(opt.raise(reinterpret_cast<const void*>(ns_tile_kernel<A_MN, B_MN>)));
  return launch_ahead(ns_tile_kernel<A_MN, B_MN>, "ns_tile_kernel", ns_tiles(e, 128) * split, TILE_THREADS, SMEM_BYTES, split, st,
                      ta, tb, e, err);
}

// 0: 256 x 256 tiles on SM pairs; else 128 x 128 tiles with K split over that many CTAs.
int pick_split(const NsArgs& e) {
  if (ns_tiles(e, 256) * 2 >= SMS / 2) return 0;
  const int tiles = ns_tiles(e, 128), atoms = (e.K + 63) / 64;
  int split = 1;
  // a split costs the meeting of the shares, about 2 us: taken while each CTA keeps 16 atoms (2 us)
  while (split < 8 && tiles * split * 2 <= SMS && atoms >= split * 32) split *= 2;
  return split;
}

mt_status ns_product(const OperandMaps& a, const OperandMaps& b, const NsArgs& e, cudaStream_t st) {
  const int split = pick_split(e);
  if (!a.mn && !b.mn) return ns_launch<false, false>(a.rows128, b.rows128, b.rows64, e, split, st);
  if (!a.mn) return ns_launch<false, true>(a.rows128, b.rows128, b.rows64, e, split, st);
  return ns_launch<true, true>(a.rows128, b.rows128, b.rows64, e, split, st);
}

// ------------------------------------------------------------------ short side of at most 64
// u of the element k on the long side, i on the short one.
struct TinyArgs {
  Grad p;
  int64_t n;   // long side
  int m;       // short side
  int tall;    // rows are the long side
  int steps;
  float scale;
  double eps, floor;  // floor: added to the diagonal of X X^T in fp64, relative to its trace
  double* gram;   // [parts][m * m]; the first becomes their sum, and then r
  int parts;
  __nv_bfloat16* o;
  int64_t ld_o;
};

constexpr int CHUNK = 64;  // long-side elements a CTA holds at a time

// u[k][i] p1 p2 of a chunk from k0 into shared memory; first: also writes m'. A thread's 16 elements are in flight
// together.
template <class T, int LD>
__device__ __forceinline__ void tiny_chunk(const TinyArgs& a, int64_t k0, T (*u)[LD], bool first, float p1 = 1.f, float p2 = 1.f) {
  constexpr int N = CHUNK * TINY / 256;
  const int kn = static_cast<int>(min(static_cast<int64_t>(CHUNK), a.n - k0));
  const bool want_g = !a.p.m_in || first || a.p.nesterov;
  const float* m = first ? a.p.m_in : a.p.m_out;
  float vg[N], vm[N];
#pragma unroll
  for (int q = 0; q < N; ++q) {
    const int e = threadIdx.x + q * 256;  // global memory's order: along a row of the matrix
    const int k = a.tall ? e / TINY : e % CHUNK, i = a.tall ? e % TINY : e / CHUNK;
    const int64_t row = a.tall ? k0 + k : i, col = a.tall ? i : k0 + k;
    const bool in = k < kn && i < a.m;
    vg[q] = in && want_g ? a.p.g[row * a.p.ld_g + col] : 0.f;
    vm[q] = in && a.p.m_in ? m[row * a.p.ld_m + col] : 0.f;
  }
#pragma unroll
  for (int q = 0; q < N; ++q) {
    const int e = threadIdx.x + q * 256;
    const int k = a.tall ? e / TINY : e % CHUNK, i = a.tall ? e % TINY : e / CHUNK;
    float v = vg[q];
    if (a.p.m_in) {
      if (first) {
        float mo;
        v = momentum_step(a.p, v, vm[q], mo);
        if (k < kn && i < a.m) a.p.m_out[(a.tall ? k0 + k : i) * a.p.ld_m + (a.tall ? i : k0 + k)] = mo;
      } else {
        v = a.p.nesterov ? fmaf(a.p.mu, vm[q], v) : vm[q];
      }
    }
    u[k][i] = static_cast<T>(first ? v : v * p1 * p2);
  }
}

// Partial Gram matrices u u^T in fp64, 4 x 4 of them a thread.
__global__ void __launch_bounds__(256) muon_tiny_gram_kernel(TinyArgs a) {
  __shared__ __align__(16) double u[CHUNK][TINY + 2];
  release_next();
  double acc[4][4] = {};
  // a thread's columns: pairs 32 apart, so that a warp reads whole rows without bank conflicts
  const int ti = threadIdx.x & 15, tj = threadIdx.x >> 4;
  auto at = [](int t, int q) { return (q >> 1) * 32 + 2 * t + (q & 1); };
  const int64_t chunks = (a.n + CHUNK - 1) / CHUNK;
  for (int64_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    __syncthreads();
    tiny_chunk<double, TINY + 2>(a, c * CHUNK, u, true);
    __syncthreads();
    if (2 * ti < a.m && 2 * tj < a.m) {
#pragma unroll 4
      for (int k = 0; k < CHUNK; ++k) {
        const double2 x0 = *reinterpret_cast<const double2*>(&u[k][2 * ti]), x1 = *reinterpret_cast<const double2*>(&u[k][2 * ti + 32]);
        const double2 y0 = *reinterpret_cast<const double2*>(&u[k][2 * tj]), y1 = *reinterpret_cast<const double2*>(&u[k][2 * tj + 32]);
        const double x[4] = {x0.x, x0.y, x1.x, x1.y}, y[4] = {y0.x, y0.y, y1.x, y1.y};
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] = fma(x[i], y[j], acc[i][j]);
      }
    }
  }
  double* out = a.gram + static_cast<int64_t>(blockIdx.x) * a.m * a.m;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int r = at(ti, i), s = at(tj, j);
      if (r < a.m && s < a.m) out[r * a.m + s] = acc[i][j];
    }
}

// Their sum, into the first: 32 elements a block, 8 threads an element, each every eighth part.
__global__ void __launch_bounds__(256) muon_tiny_reduce_kernel(TinyArgs a) {
  __shared__ double red[8][32];
  release_next();
  wait_for_last();
  const int mm = a.m * a.m, lane = threadIdx.x & 31, y = threadIdx.x >> 5, e = blockIdx.x * 32 + lane;
  double v = 0.0;
  if (e < mm) {
#pragma unroll 10
    for (int p = y; p < a.parts; p += 8) v += a.gram[static_cast<int64_t>(p) * mm + e];
  }
  red[y][lane] = v;
  __syncthreads();
  if (y == 0 && e < mm) {
    for (int k = 1; k < 8; ++k) v += red[k][lane];
    a.gram[e] = v;  // the element's own part is read only by this block
  }
}

// What the steps and the product behind them compute in: T = float or double, 16 bytes of either, and two of them.
template <class T>
struct TinyNum;
template <>
struct TinyNum<float> {
  using pair = float2;
  static constexpr float A = NS_A, B = NS_B, C = NS_C;
};
template <>
struct TinyNum<double> {
  using pair = double2;
  static constexpr double A = NS64_A, B = NS64_B, C = NS64_C;
};
template <class T>
struct __align__(16) Vec16 {
  static constexpr int N = 16 / sizeof(T);
  T v[N];
};
template <class T>
__device__ __forceinline__ Vec16<T> ld16(const T* p) {
  return *reinterpret_cast<const Vec16<T>*>(p);
}
__device__ __forceinline__ void st_pair(uint32_t at, float2 v) {
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(at), "f"(v.x), "f"(v.y) : "memory");
}
__device__ __forceinline__ void st_pair(uint32_t at, double2 v) {
  asm volatile("st.shared::cluster.v2.f64 [%0], {%1, %2};" ::"r"(at), "d"(v.x), "d"(v.y) : "memory");
}

template <class T>
using Mat64 = T (*)[TINY];
constexpr int TINY_CTAS = 8, TINY_ROWS = TINY / TINY_CTAS;  // the steps' cluster, and the rows of each product that a CTA computes

// This CTA's rows of s * a b, 64 x 64 matrices that every CTA of the cluster holds whole: thread (q, r, c) sums a
// quarter of k for 2 rows x 4 columns (one vector of 16 bytes, or two half a row apart: neighbouring threads read
// neighbouring vectors), the quarters meet in `part`, and thread t gets elements 2t, 2t + 1 of the CTA's 8 x 64.
// (Operands are symmetric but for rounding; reading a by columns would let that difference grow from step to step.)
template <class T>
__device__ __forceinline__ typename TinyNum<T>::pair mul64(Mat64<T> a, Mat64<T> b, int rank, T (*part)[TINY_ROWS * TINY]) {
  constexpr int E = Vec16<T>::N, H = 4 / E;
  const int c = threadIdx.x & 15, r = (threadIdx.x >> 4) & 3, q = threadIdx.x >> 6, row = rank * TINY_ROWS + 2 * r;
  T acc[2][4] = {};
#pragma unroll
  for (int k = q * 16; k < q * 16 + 16; k += E) {
    Vec16<T> x[2], y[E][H];
#pragma unroll
    for (int i = 0; i < 2; ++i) x[i] = ld16<T>(&a[row + i][k]);
#pragma unroll
    for (int l = 0; l < E; ++l)
#pragma unroll
      for (int h = 0; h < H; ++h) y[l][h] = ld16<T>(&b[k + l][32 * h + E * c]);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int l = 0; l < E; ++l)
#pragma unroll
        for (int h = 0; h < H; ++h)
#pragma unroll
          for (int j = 0; j < E; ++j) acc[i][E * h + j] = fma(x[i].v[l], y[l][h].v[j], acc[i][E * h + j]);
  }
  __syncthreads();  // `part` of the product before is read
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int h = 0; h < H; ++h) {
      Vec16<T> w;
#pragma unroll
      for (int j = 0; j < E; ++j) w.v[j] = acc[i][E * h + j];
      *reinterpret_cast<Vec16<T>*>(&part[q][(2 * r + i) * TINY + 32 * h + E * c]) = w;
    }
  __syncthreads();
  typename TinyNum<T>::pair v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<const typename TinyNum<T>::pair*>(&part[i][2 * threadIdx.x]);
  v[0].x = v[0].x + v[1].x + (v[2].x + v[3].x);
  v[0].y = v[0].y + v[1].y + (v[2].y + v[3].y);
  return v[0];
}

// Elements 2t, 2t + 1 of this CTA's rows of c, to every CTA of the cluster.
template <class T>
__device__ __forceinline__ void share64(Mat64<T> c, int rank, typename TinyNum<T>::pair v) {
  const uint32_t at = smem_u32(&c[rank * TINY_ROWS][0]) + threadIdx.x * sizeof(v);
#pragma unroll
  for (int p = 0; p < TINY_CTAS; ++p) st_pair(map_to_rank(at, static_cast<uint32_t>(p)), v);
}

template <class T>
constexpr int TINY_SMEM = (6 * TINY * TINY + 4 * TINY_ROWS * TINY) * sizeof(T);

// The steps on the Gram matrix, eight CTAs of a cluster with eight rows each: with P = a I + b A + c A^2,
// Q <- P Q, A <- A P^2. A product writes no matrix that it reads, and a cluster barrier stands behind each.
// r = Q / (|u| + eps) in fp64 (its elements leave fp32 for norms below 1e-36 with an eps as small), over the Gram
// matrix, which every CTA has read by then.
//
// A is never formed anew from X: what rounding leaves in directions that u lacks, of either sign, grows by a^2 = 11.9 a
// step, and the polynomial of a negative eigenvalue that has grown to about one only grows. In fp32 five steps stay
// within 7e-4 of exact ones (48 equal rows; 2e-4 for rank one over noise of 1e-3), six within 3e-3, eight are off by
// the result itself. More than five are therefore taken in fp64, and A starts with `floor` of its trace added to its
// diagonal, more than what the roundings of the Gram sums and of a step can take off (a sum's chain of additions, and 512,
// times 2^-53: the rows' absolute products have a 2-norm of at most the trace). No eigenvalue turns negative then, for any number of
// steps: the result is q(A) u, the exact steps but in directions weaker than sqrt(floor), some 2^-22 of |u|, which
// come out weaker than exact steps have them after a dozen. 60 x 20000, ten steps: 127 us, 84 in fp32.
template <class T>
__global__ void __cluster_dims__(TINY_CTAS, 1, 1) __launch_bounds__(256) muon_tiny_steps_kernel(TinyArgs a) {
  using Num = TinyNum<T>;
  extern __shared__ __align__(16) uint8_t tiny_smem[];
  Mat64<T> A = reinterpret_cast<Mat64<T>>(tiny_smem), A_next = A + TINY, P = A + 2 * TINY, P2 = A + 3 * TINY, Q = A + 4 * TINY,
           Q_next = A + 5 * TINY;
  T(*part)[TINY_ROWS * TINY] = reinterpret_cast<T(*)[TINY_ROWS * TINY]>(A + 6 * TINY);
  __shared__ double trace[TINY];
  const int rank = static_cast<int>(cluster_rank());
  release_next();
  wait_for_last();
  if (threadIdx.x < TINY) trace[threadIdx.x] = static_cast<int>(threadIdx.x) < a.m ? a.gram[threadIdx.x * (a.m + 1)] : 0.0;
  double own[TINY * TINY / 256];
#pragma unroll
  for (int q = 0; q < TINY * TINY / 256; ++q) {
    const int e = threadIdx.x + q * 256, i = e / TINY, j = e % TINY;
    own[q] = i < a.m && j < a.m ? a.gram[i * a.m + j] : 0.0;
  }
  __syncthreads();
  double sum = 0.0;
  for (int i = 0; i < a.m; ++i) sum += trace[i];
  const double norm = sqrt(sum) + a.eps, inv = 1.0 / norm;
#pragma unroll
  for (int q = 0; q < TINY * TINY / 256; ++q) {
    const int e = threadIdx.x + q * 256;
    const bool diag = e / TINY == e % TINY;
    A[e / TINY][e % TINY] = static_cast<T>((own[q] + (sizeof(T) == 8 && diag ? a.floor * sum : 0.0)) * inv * inv);
    Q[e / TINY][e % TINY] = diag ? T(1) : T(0);
  }
  cluster_sync();  // every CTA has started, and holds A
  const int own_row = rank * TINY_ROWS + (threadIdx.x >> 5), own_col = 2 * (threadIdx.x & 31);
  for (int st = 0; st < a.steps; ++st) {
    typename Num::pair v = mul64<T>(A, A, rank, part);
    v.x = fma(Num::C, v.x, fma(Num::B, A[own_row][own_col], own_row == own_col ? Num::A : T(0)));
    v.y = fma(Num::C, v.y, fma(Num::B, A[own_row][own_col + 1], own_row == own_col + 1 ? Num::A : T(0)));
    share64<T>(P, rank, v);
    cluster_sync();
    share64<T>(Q_next, rank, mul64<T>(P, Q, rank, part));
    if (st + 1 < a.steps) {
      share64<T>(P2, rank, mul64<T>(P, P, rank, part));
      cluster_sync();
      share64<T>(A_next, rank, mul64<T>(A, P2, rank, part));
    }
    cluster_sync();
    Mat64<T> t = Q;
    Q = Q_next;
    Q_next = t;
    t = A;
    A = A_next;
    A_next = t;
  }
#pragma unroll
  for (int q = 0; q < 2; ++q)
    if (own_row < a.m && own_col + q < a.m) a.gram[own_row * a.m + own_col + q] = Q[own_row][own_col + q] * inv;
}

// o = scale r u, a chunk of the long side a CTA. In fp32, (r 2^-e) (u 2^e) with 2^e about an element of r's diagonal,
// which is positive and within a factor of a^steps of the others, so that both stay in range for any norm and eps. After
// more than five steps in fp64, as r's elements grow by a with each and cancel in strong directions (60 x 20000: 7 us
// more). Rows of 16 bytes more than 64 elements in shared memory: a vector of j a read, no bank conflicts.
template <class T>
constexpr int APPLY_LD = TINY + Vec16<T>::N;
template <class T>
constexpr int APPLY_SMEM = (CHUNK + TINY) * APPLY_LD<T> * sizeof(T);
template <class T>
__global__ void __launch_bounds__(256) muon_tiny_apply_kernel(TinyArgs a) {
  constexpr int LD = APPLY_LD<T>, E = Vec16<T>::N;
  extern __shared__ __align__(16) uint8_t apply_smem[];
  T(*u)[LD] = reinterpret_cast<T(*)[LD]>(apply_smem), (*r)[LD] = u + CHUNK;
  wait_for_last();
  const double lead = a.gram[0];
  const int e = sizeof(T) == 4 && lead > 0.0 && isfinite(lead) ? ilogb(lead) : 0;
  const float p1 = ldexpf(1.f, e / 2), p2 = ldexpf(1.f, e - e / 2);  // 2^e may leave fp32 itself
  {
    double v[TINY * TINY / 256];
#pragma unroll
    for (int q = 0; q < TINY * TINY / 256; ++q) {
      const int i = (threadIdx.x + q * 256) / TINY, j = threadIdx.x % TINY;
      v[q] = i < a.m && j < a.m ? a.gram[i * a.m + j] : 0.0;
    }
    const double down = ldexp(1.0, -e);
#pragma unroll
    for (int q = 0; q < TINY * TINY / 256; ++q)
      r[(threadIdx.x + q * 256) / TINY][threadIdx.x % TINY] = static_cast<T>(v[q] * down);
  }
  const int64_t chunks = (a.n + CHUNK - 1) / CHUNK;
  // neighbouring threads write neighbouring elements of a row of o: along the short side of a tall matrix, the long
  // side of a wide one; 16 elements a thread, every fourth of the other side
  const int fast = threadIdx.x & 63, slow = threadIdx.x >> 6;
  for (int64_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    __syncthreads();
    tiny_chunk<T, LD>(a, c * CHUNK, u, false, p1, p2);
    __syncthreads();
    T s[16] = {};
    const T(*mine)[LD] = a.tall ? r : u, (*other)[LD] = a.tall ? u : r;
    for (int j = 0; j < a.m; j += E) {  // zeros behind a.m
      const Vec16<T> x = ld16<T>(&mine[fast][j]);
#pragma unroll
      for (int q = 0; q < 16; ++q) {
        const Vec16<T> y = ld16<T>(&other[slow + 4 * q][j]);
#pragma unroll
        for (int l = 0; l < E; ++l) s[q] = fma(x.v[l], y.v[l], s[q]);
      }
    }
#pragma unroll
    for (int q = 0; q < 16; ++q) {
      const int k = a.tall ? slow + 4 * q : fast, i = a.tall ? fast : slow + 4 * q;
      const int64_t lk = c * CHUNK + k;
      if (lk < a.n && i < a.m)
        a.o[a.tall ? lk * a.ld_o + i : static_cast<int64_t>(i) * a.ld_o + lk] = __float2bfloat16_rn(static_cast<float>(s[q] * a.scale));
    }
  }
}

// ------------------------------------------------------------------ workspace
struct Plan {
  int64_t m, n, ld_x, ld_a;
  int parts;
  double* part;
  unsigned* counter;
  int split;       // of the fused kernel's Gram products
  float* partial;  // and their parts
  __half *hi[2], *lo, *A, *P, *C;  // C: only where the first two steps share a Gram matrix
  double* gram;
  uint64_t bytes;
};

// Whether all steps run as one kernel: each product's tiles fit a B200 about once, so that whole SM pairs on
// 256 x 256 tiles would not be faster.
bool pick_fused(int64_t m, int64_t n) {
  const int64_t tm = (m + 127) / 128, tn = (n + 127) / 128;
  return tm * tn <= SMS && tm * (tm + 1) / 2 <= SMS;
}

// Parts of K of a Gram product in the fused kernel: CTAs without a tile take some, with at least six K atoms a part
// (a part costs a grid barrier and a pass over the partial tiles, about 4 us in all; an atom 0.2 us).
int fused_split(int64_t m, int64_t n) {
  const int64_t tm = (m + 127) / 128, atoms = (n + 63) / 64;
  const int64_t split = std::min<int64_t>(std::min<int64_t>(SMS / (tm * (tm + 1) / 2), atoms / 6), 16);
  return atoms - atoms / std::max<int64_t>(1, split) >= 16 ? static_cast<int>(split) : 1;
}

// Whether the first two steps of a matrix this wide share a Gram matrix: 3 m^2 n operations saved for 3 m^3 more.
bool pair_first_steps(int64_t m, int64_t n) { return n >= 2 * m; }

Plan plan(int64_t rows, int64_t cols, void* ws) {
  Plan p = {};
  p.m = std::min(rows, cols);
  p.n = std::max(rows, cols);
  Bump b(ws, ~0ull);
  if (p.m <= TINY) {
    p.parts = static_cast<int>(std::min<int64_t>(SMS, (p.n + CHUNK - 1) / CHUNK));
    p.gram = b.take<double>(static_cast<int64_t>(p.parts) * p.m * p.m);
  } else {
    p.parts = NORM_PARTS;
    p.ld_x = align_up(cols, 64);
    p.ld_a = align_up(p.m, 64);
    p.part = b.take<double>(NORM_PARTS);
    p.counter = b.take<unsigned>(1);
    for (auto& h : p.hi) h = b.take<__half>(rows * p.ld_x);
    p.lo = b.take<__half>(rows * p.ld_x);
    p.A = b.take<__half>(p.m * p.ld_a);
    p.P = b.take<__half>(p.m * p.ld_a);
    p.split = 1;
    if (pick_fused(p.m, p.n)) {
      p.split = fused_split(p.m, p.n);
      const int64_t tm = (p.m + 127) / 128;
      if (p.split > 1) p.partial = b.take<float>(tm * (tm + 1) / 2 * p.split * PARTIAL);
    }
    p.C = !pick_fused(p.m, p.n) && pair_first_steps(p.m, p.n) ? b.take<__half>(p.m * p.ld_a) : nullptr;
  }
  p.bytes = b.used;
  return p;
}

Walk make_walk(int64_t rows, int64_t cols, int vec) {
  Walk w;
  w.tx_log2 = 8;
  while (w.tx_log2 > 0 && (int64_t(1) << (w.tx_log2 - 1)) * vec >= cols) --w.tx_log2;
  const int64_t width = (int64_t(1) << w.tx_log2) * vec, ty = 256 >> w.tx_log2;
  w.col_tiles = (cols + width - 1) / width;
  w.tiles = w.col_tiles * ((rows + ty * REPS - 1) / (ty * REPS));
  return w;
}

// The steps on the Gram matrix, and the product behind them.
template <class T>
mt_status muon_tiny_rest(const TinyArgs& a, cudaStream_t st) {
  static SmemOptIn opt_steps, opt_apply;
  MT_TRY(opt_steps.raise(reinterpret_cast<const void*>(muon_tiny_steps_kernel<T>), TINY_SMEM<T>));
  MT_TRY(opt_apply.raise(reinterpret_cast<const void*>(muon_tiny_apply_kernel<T>), APPLY_SMEM<T>));
  MT_TRY(launch_ahead(muon_tiny_steps_kernel<T>, "muon_tiny_steps_kernel", TINY_CTAS, 256, TINY_SMEM<T>, 0, st, a));
  const int64_t chunks = (a.n + CHUNK - 1) / CHUNK;
  return launch_ahead(muon_tiny_apply_kernel<T>, "muon_tiny_apply_kernel", static_cast<int>(std::min<int64_t>(chunks, 4 * num_sms())),
                      256, APPLY_SMEM<T>, 0, st, a);
}

mt_status muon_tiny(const Grad& g, const mt_muon_cfg& c, mt_bf16* o, int64_t ld_o, const Plan& p, cudaStream_t st) {
  TinyArgs a;
  a.p = g;
  a.n = p.n;
  a.m = static_cast<int>(p.m);
  a.tall = g.rows > g.cols;
  a.steps = c.steps;
  a.scale = c.scale;
  a.eps = c.eps;
  // a Gram sum's chain of additions: the elements of a CTA's chunks, then the parts
  const int64_t chunks = (p.n + CHUNK - 1) / CHUNK;
  const int64_t chain = (chunks + p.parts - 1) / p.parts * CHUNK + (p.parts + 7) / 8 + 8;
  a.floor = std::ldexp(static_cast<double>(chain + 512), -53);
  a.gram = p.gram;
  a.parts = p.parts;
  a.o = reinterpret_cast<__nv_bfloat16*>(o);
  a.ld_o = ld_o;
  muon_tiny_gram_kernel<<<p.parts, 256, 0, st>>>(a);
  MT_TRY(launch_check("muon_tiny_gram_kernel"));
  MT_TRY(launch_ahead(muon_tiny_reduce_kernel, "muon_tiny_reduce_kernel", (a.m * a.m + 31) / 32, 256, 0, 0, st, a));
  return c.steps <= 5 ? muon_tiny_rest<float>(a, st) : muon_tiny_rest<double>(a, st);
}

template <bool TALL>
mt_status fused_launch(const FusedMaps& maps, const FusedArgs& a, cudaStream_t st) {
  int32_t* err = device_error_word();
  if (!err) return fail(MT_ERR_CUDA, "device error word unavailable");
  static SmemOptIn opt;
  MT_TRY(opt.raise(reinterpret_cast<const void*>(ns_fused_kernel<TALL>), FUSED_SMEM));
  // every CTA resident: one an SM, and no more of them than the largest product, or the scaling, has work for
  const int tm = (a.m + 127) / 128, tn = (a.n + 127) / 128;
  const int64_t want = std::max<int64_t>(std::max<int64_t>(tm * tn, tm * (tm + 1) / 2 * a.split), a.walk.tiles);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(std::min<int64_t>(want, num_sms())), 1, 1);
  cfg.blockDim = dim3(TILE_THREADS, 1, 1);
  cfg.dynamicSmemBytes = FUSED_SMEM;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  MT_CUDA(cudaLaunchKernelEx(&cfg, ns_fused_kernel<TALL>, maps, a, err));
  return launch_check("ns_fused_kernel");
}

mt_status muon_general(const Grad& g, const mt_muon_cfg& c, mt_bf16* o, int64_t ld_o, const Plan& p, cudaStream_t st) {
  const bool tall = g.rows > g.cols;
  auto a16 = [](const void* q) { return (reinterpret_cast<uintptr_t>(q) & 15) == 0; };
  const bool v4 = g.cols % 4 == 0 && g.ld_g % 4 == 0 && a16(g.g) &&
                  (!g.m_in || (g.ld_m % 4 == 0 && a16(g.m_in) && a16(g.m_out)));
  const Walk w = make_walk(g.rows, g.cols, v4 ? 4 : 1);
  const int parts = static_cast<int>(std::min<int64_t>(w.tiles, NORM_PARTS));
  // a two-term X for all steps but the last two
  const int two_term = c.steps - 2, m = static_cast<int>(p.m), n = static_cast<int>(p.n);
  __half* lo = two_term > 0 ? p.lo : nullptr;
  __nv_bfloat16* out = reinterpret_cast<__nv_bfloat16*>(o);
  const int bf_v16 = a16(o) && ld_o % 8 == 0;
  // X with the short or the long side as rows: K-major or MN-major by the matrix's orientation
  OperandMaps x_short[2], x_long[2], sq_a, sq_p, sq_c;
  for (int i = 0; i < 2; ++i) {
    MT_TRY(operand_maps(&x_short[i], Operand{p.hi[i], p.ld_x, tall, p.m}, n));
    MT_TRY(operand_maps(&x_long[i], Operand{p.hi[i], p.ld_x, !tall, p.n}, m));
  }
  MT_TRY(operand_maps(&sq_a, Operand{p.A, p.ld_a, false, p.m}, m));
  MT_TRY(operand_maps(&sq_p, Operand{p.P, p.ld_a, false, p.m}, m));
  if (v4)
    muon_norm_kernel<4><<<parts, 256, 0, st>>>(g, w, p.part, p.counter);
  else
    muon_norm_kernel<1><<<parts, 256, 0, st>>>(g, w, p.part, p.counter);
  MT_TRY(launch_check("muon_norm_kernel"));
  if (pick_fused(m, n)) {
    FusedMaps maps;
    for (int i = 0; i < 2; ++i) {
      maps.x_short[i] = x_short[i].rows128;
      maps.x_long[i] = x_long[i].rows128;
    }
    maps.A = sq_a.rows128;
    maps.P = sq_p.rows128;
    FusedArgs a;
    a.grad = g;
    a.walk = w;
    a.part = p.part;
    a.parts = parts;
    a.vec4 = v4;
    a.eps = c.eps;
    a.m = m;
    a.n = n;
    a.tall = tall;
    a.steps = c.steps;
    a.two_term = two_term;
    a.split = p.split;
    a.partial = p.partial;
    a.hi[0] = p.hi[0];
    a.hi[1] = p.hi[1];
    a.lo = p.lo;
    a.A = p.A;
    a.P = p.P;
    a.ld_x = p.ld_x;
    a.ld_a = p.ld_a;
    a.scale = c.scale;
    a.o = out;
    a.ld_o = ld_o;
    a.bf_v16 = bf_v16;
    a.counter = p.counter;
    return tall ? fused_launch<true>(maps, a, st) : fused_launch<false>(maps, a, st);
  }
  if (v4)
    MT_TRY(launch_ahead(muon_scale_kernel<4>, "muon_scale_kernel", parts, 256, 0, 0, st, g, w, p.part, parts, c.eps, p.hi[0], lo,
                        p.ld_x));
  else
    MT_TRY(launch_ahead(muon_scale_kernel<1>, "muon_scale_kernel", parts, 256, 0, 0, st, g, w, p.part, parts, c.eps, p.hi[0], lo,
                        p.ld_x));
  int s = 0;
  if (p.C && two_term >= 2) {
    // The first two steps on one Gram matrix: with P = b A + c A^2 the second step's is
    // A' = (a I + P) A (a I + P) = a^2 A + 2 a M + P M, M = P A, and X'' = (a I + P') (a I + P) X =
    // a^2 X + Q X, Q = a (P + P') + P' P. All of them commute, so each of the five products takes half its tiles:
    // 3 m^2 n + 5 m^3 operations where two steps take 6 m^2 n + 2 m^3. As accurate as two steps (the noise of
    // A's rounding has one step to grow), but for one direction with elements of equal size: a^2 + Q = 1.1 there, with Q
    // = -10.8 and X's head rounded the same way all over, where two steps have a + P = 0.7 with P = -2.7 (1200 x 2600 of
    // equal elements: 1.8e-2 off, 1200 x 1300: 1.2e-3). Three steps on one Gram matrix lose a factor of three.
    constexpr float S_Q = 4096.f;  // |Q| <= a^2 = 11.9
    MT_TRY(operand_maps(&sq_c, Operand{p.C, p.ld_a, false, p.m}, m));
    MT_TRY(ns_product(x_short[0], x_short[0], gram_args(m, n, p.A, p.ld_a), st));
    MT_TRY(ns_product(sq_a, sq_a, poly_args(m, p.A, p.P, p.ld_a, false), st));
    MT_TRY(ns_product(sq_p, sq_a, square_args(m, p.ld_a, p.C, S_P / (S_P * S_A)), st));  // M
    NsArgs e = square_args(m, p.ld_a, p.A, S_A / (S_P * S_P));                           // A', over A: a tile adds its own elements
    e.beta = NS_A * NS_A;
    e.add_hi = p.A;
    e.beta_lo = 2.f * NS_A * S_A / S_P;
    e.add_lo = p.C;
    MT_TRY(ns_product(sq_p, sq_c, e, st));
    MT_TRY(ns_product(sq_a, sq_a, poly_args(m, p.A, p.C, p.ld_a, false), st));  // P'
    e = square_args(m, p.ld_a, p.A, S_Q / (S_P * S_P));                         // Q
    e.beta = e.beta_lo = NS_A * S_Q / S_P;
    e.add_hi = p.P;
    e.add_lo = p.C;
    MT_TRY(ns_product(sq_c, sq_p, e, st));
    e = apply_args(m, n, tall, NS_A * NS_A, S_Q, false, c.scale, p.hi[0], p.lo, p.hi[1], two_term > 2 ? p.lo : nullptr, p.ld_x, out,
                   ld_o, bf_v16);
    MT_TRY(tall ? ns_product(x_long[0], sq_a, e, st) : ns_product(sq_a, x_long[0], e, st));
    s = 2;
  }
  for (int from = s == 2 ? 1 : 0; s < c.steps; ++s, from ^= 1) {
    const bool fold = s >= two_term, last = s + 1 == c.steps;
    MT_TRY(ns_product(x_short[from], x_short[from], gram_args(m, n, p.A, p.ld_a), st));
    MT_TRY(ns_product(sq_a, sq_a, poly_args(m, p.A, p.P, p.ld_a, fold), st));
    const NsArgs e = apply_args(m, n, tall, fold ? 0.f : NS_A, S_P, last, c.scale, p.hi[from], p.lo, p.hi[from ^ 1],
                                s + 1 < two_term ? p.lo : nullptr, p.ld_x, out, ld_o, bf_v16);
    MT_TRY(tall ? ns_product(x_long[from], sq_p, e, st) : ns_product(sq_p, x_long[from], e, st));
  }
  return MT_OK;
}

}  // namespace
}  // namespace mt

using namespace mt;

extern "C" {

uint64_t mt_muon_workspace_bytes(int64_t rows, int64_t cols) {
  if (rows <= 0 || cols <= 0 || rows >= (1ll << 31) || cols >= (1ll << 31) || rows > MAX_ELEMENTS / cols) return 0;
  return plan(rows, cols, nullptr).bytes;
}

mt_status mt_muon_update(const float* g, int64_t ld_g, const float* m_in, float* m_out, int64_t ld_m, mt_bf16* o,
                         int64_t ld_o, int64_t rows, int64_t cols, const mt_muon_cfg* cfg, void* ws, uint64_t ws_bytes,
                         void* stream) {
  const bool empty = rows == 0 || cols == 0;
  if (!cfg || (!empty && (!g || !o))) return fail(MT_ERR_INVALID_ARG, "muon_update: NULL pointer");
  if (!m_in != !m_out) return fail(MT_ERR_INVALID_ARG, "muon_update: m_in and m_out go together");
  if (rows < 0 || cols < 0 || rows >= (1ll << 31) || cols >= (1ll << 31))
    return fail(MT_ERR_INVALID_ARG, "muon_update: need 0 <= rows, cols < 2^31");
  if (cols > 0 && rows > MAX_ELEMENTS / cols) return fail(MT_ERR_UNSUPPORTED, "muon_update: more than 2^36 elements");
  if (ld_g < cols || ld_o < cols || (m_in && ld_m < cols))
    return fail(MT_ERR_INVALID_ARG, "muon_update: row stride smaller than cols");
  if (cfg->steps < 1 || cfg->steps > 100) return fail(MT_ERR_INVALID_ARG, "muon_update: 1 to 100 steps, got %d", cfg->steps);
  if (!std::isfinite(cfg->momentum) || !std::isfinite(cfg->scale) || !(cfg->eps > 0.f) || !std::isfinite(cfg->eps))
    return fail(MT_ERR_INVALID_ARG, "muon_update: momentum and scale must be finite, eps positive and finite");
  const uintptr_t f32 = reinterpret_cast<uintptr_t>(g) | reinterpret_cast<uintptr_t>(m_in) | reinterpret_cast<uintptr_t>(m_out);
  if ((f32 & 3) || (reinterpret_cast<uintptr_t>(o) & 1))
    return fail(MT_ERR_ALIGNMENT, "muon_update: pointers must be aligned to their elements");
  if (empty) return MT_OK;
  if (!ws) return fail(MT_ERR_INVALID_ARG, "muon_update: NULL workspace");
  if (reinterpret_cast<uintptr_t>(ws) & 255) return fail(MT_ERR_ALIGNMENT, "muon_update: workspace must be 256-byte aligned");
  const Plan p = plan(rows, cols, ws);
  if (ws_bytes < p.bytes) return fail(MT_ERR_WORKSPACE, "muon_update: workspace too small");
  Grad gr;
  gr.g = g;
  gr.m_in = m_in;
  gr.m_out = m_out;
  gr.ld_g = ld_g;
  gr.ld_m = ld_m;
  gr.rows = rows;
  gr.cols = cols;
  gr.mu = cfg->momentum;
  gr.nesterov = cfg->nesterov != 0;
  return p.m <= TINY ? muon_tiny(gr, *cfg, o, ld_o, p, as_stream(stream))
                     : muon_general(gr, *cfg, o, ld_o, p, as_stream(stream));
}

}  // extern "C"
