// Rotary positions with several axes (time, height, width of image and video tokens): rotate-half RoPE in
// which every rotated pair of a head takes its position from one of the axes.
//
//   R = 2 * sum(sections) columns of each head rotate, pair i = (i, i + R/2) by angle pos[axis(i)][row] * omega_i:
//   (a, b) -> (a cos - b sin, b cos + a sin); the columns behind R are copied.
//
// Bound by HBM: 4 bytes an element, against 3 flops. What could cost more than that is the angles, and they
// are one per token and pair, shared by all heads: a CTA forms the (cos, sin) of a tile of tokens in shared
// memory first and then rotates the tile's heads from it. omega is taken in turns (omega / 2 pi) in fp64 on
// the host; position * turns is rounded to its fraction of a turn in fp64, so that a position of 2^31 keeps
// an angle error below 5e-7, and only the fraction goes through the fp32 sincospi: two fp64 operations an
// angle instead of an fp64 sincos.
#include <algorithm>
#include <cmath>

#include "mt_internal.h"
#include "vec.cuh"

namespace mt {
namespace {

using namespace vec;

constexpr int MAX_PAIRS = 128, MAX_AXES = 8;
constexpr int THREADS = 256;
constexpr int TABLE = 2048;  // (cos, sin) pairs of a tile: 16 KiB
// Heads that share a thread's reads of the table, and CTAs of an SM: two heads of 16-byte vectors leave registers for
// four CTAs (98304 tokens, 32 heads of 128: 276 us against 283 with four heads and three CTAs; 80000 tokens, 5 heads
// of 80: 40 against 54), narrower vectors want four heads' loads in flight (60000 tokens, 20 heads of 72 in rows of odd
// stride: 118 us against 178).
__host__ __device__ constexpr int heads_a_thread(int vec) { return vec == 8 ? 2 : 4; }
constexpr int ctas_an_sm(int vec) { return vec == 8 ? 4 : 3; }

struct Mrope {
  const __nv_bfloat16* x;
  __nv_bfloat16* y;
  const int32_t* pos;
  int64_t ld_x, ld_y, ld_pos, rows;
  int heads, d, pairs, tile;  // tile: tokens of a tile, tile * pairs <= TABLE
  float sign;
  uint8_t axis[MAX_PAIRS];
  double turns[MAX_PAIRS];
};

// Turns the pair (lo, hi) of VEC features by their (cos, sin).
template <int VEC>
__device__ __forceinline__ void turn(typename Raw<VEC>::type& lo, typename Raw<VEC>::type& hi, const float (&c)[VEC],
                                     const float (&s)[VEC]) {
  float l[VEC], h[VEC];
  unpack(lo, l);
  unpack(hi, h);
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    const float p = l[i], q = h[i];
    l[i] = p * c[i] - q * s[i];
    h[i] = q * c[i] + p * s[i];
  }
  pack(lo, l);
  pack(hi, h);
}

// A thread takes one vector of features of two or four heads of a token at a time: their loads are in flight together, and
// the features' cos and sin are read from the table once for all of them. The first ones' loads are issued before
// the tile's angles are formed.
template <int VEC>
struct Item {
  using V = typename Raw<VEC>::type;
  static constexpr int HG = heads_a_thread(VEC);
  V lo[HG], hi[HG];
  uint32_t tok, v;
  int n;           // heads
  int64_t x, y;    // elements from the tile's start
  __device__ __forceinline__ void load(const Mrope& a, uint32_t it, uint32_t per_token, int rot, int64_t row0) {
    tok = it / per_token;
    const uint32_t in_token = it - tok * per_token, hg = in_token / rot;
    v = in_token - hg * rot;
    const int64_t at = static_cast<int64_t>(hg) * HG * a.d + v * VEC;
    x = (row0 + tok) * a.ld_x + at;
    y = (row0 + tok) * a.ld_y + at;
    n = min(HG, a.heads - static_cast<int>(hg) * HG);
#pragma unroll
    for (int h = 0; h < HG; ++h) {
      if (h < n) {
        lo[h] = *reinterpret_cast<const V*>(a.x + x + h * a.d);
        hi[h] = *reinterpret_cast<const V*>(a.x + x + h * a.d + a.pairs);
      }
    }
  }
};

template <int VEC>
__global__ void __launch_bounds__(THREADS, ctas_an_sm(VEC)) mrope_kernel(const __grid_constant__ Mrope a) {
  using V = typename Raw<VEC>::type;
  constexpr int HG = heads_a_thread(VEC);
  // cos and sin, [token][feature within a vector][vector]: threads of neighbouring vectors read neighbouring words
  __shared__ float cos_tab[TABLE], sin_tab[TABLE];
  const int rot = a.pairs / VEC;                                // rotated vectors of a head half
  const int tail = a.x == a.y ? 0 : (a.d - 2 * a.pairs) / VEC;  // vectors to copy behind them
  const int head_groups = (a.heads + HG - 1) / HG;
  const int64_t tiles = (a.rows + a.tile - 1) / a.tile;
  // each lane reads another pair's: from the parameters' constant bank they would come one at a time
  __shared__ double turns_s[MAX_PAIRS];
  __shared__ int axis_s[MAX_PAIRS];
  __shared__ int32_t pos_s[TABLE];  // each place is one thread's own
  for (int i = threadIdx.x; i < a.pairs; i += THREADS) {
    turns_s[i] = a.turns[i];
    axis_s[i] = a.axis[i];
  }
  const int tok0 = threadIdx.x / a.pairs, pair0 = threadIdx.x - tok0 * a.pairs, hop = THREADS / a.pairs, leap = THREADS - hop * a.pairs;
  for (int64_t tl = blockIdx.x; tl < tiles; tl += gridDim.x) {
    const int64_t row0 = tl * a.tile;
    const int tokens = static_cast<int>(min(static_cast<int64_t>(a.tile), a.rows - row0));
    const uint32_t per_token = rot * head_groups, items = tokens * per_token;
    Item<VEC> item;
    uint32_t it = threadIdx.x;
    if (it < items) item.load(a, it, per_token, rot, row0);
    __syncthreads();  // the last tile's table is read
    // the angles' positions are in flight together; pair i of token tok, `leap` pairs and `hop` tokens on for each
    constexpr int N = TABLE / THREADS;
    int tok = tok0, i = pair0;
#pragma unroll
    for (int u = 0; u < N; ++u) {
      if (tok < tokens) pos_s[threadIdx.x + u * THREADS] = a.pos[axis_s[i] * a.ld_pos + row0 + tok];
      tok += hop;
      i += leap;
      if (i >= a.pairs) {
        i -= a.pairs;
        ++tok;
      }
    }
    tok = tok0;
    i = pair0;
    for (int e = threadIdx.x; tok < tokens; e += THREADS) {  // e = tok * pairs + i
      const double p = static_cast<double>(pos_s[e]) * turns_s[i];
      float s, c;
      sincospif(2.0f * static_cast<float>(p - rint(p)), &s, &c);
      const int at = tok * a.pairs + (i % VEC) * rot + i / VEC;
      cos_tab[at] = c;
      sin_tab[at] = a.sign * s;
      tok += hop;
      i += leap;
      if (i >= a.pairs) {
        i -= a.pairs;
        ++tok;
      }
    }
    __syncthreads();
    while (it < items) {
      float c[VEC], s[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        c[i] = cos_tab[item.tok * a.pairs + i * rot + item.v];
        s[i] = sin_tab[item.tok * a.pairs + i * rot + item.v];
      }
#pragma unroll
      for (int h = 0; h < HG; ++h) {
        if (h < item.n) {
          turn<VEC>(item.lo[h], item.hi[h], c, s);
          *reinterpret_cast<V*>(a.y + item.y + h * a.d) = item.lo[h];
          *reinterpret_cast<V*>(a.y + item.y + h * a.d + a.pairs) = item.hi[h];
        }
      }
      it += THREADS;
      if (it < items) item.load(a, it, per_token, rot, row0);
    }
    if (tail > 0) {
      const int64_t copies = static_cast<int64_t>(tokens) * a.heads * tail;
      for (int64_t k = threadIdx.x; k < copies; k += THREADS) {
        const int64_t th = k / tail, tok = th / a.heads;
        const int64_t at = (th - tok * a.heads) * a.d + 2 * a.pairs + (k - th * tail) * VEC;
        *reinterpret_cast<V*>(a.y + (row0 + tok) * a.ld_y + at) =
            *reinterpret_cast<const V*>(a.x + (row0 + tok) * a.ld_x + at);
      }
    }
  }
}

template <int VEC>
mt_status go(Mrope a, cudaStream_t st) {
  // as many CTAs as the registers keep resident, tiles of even size: the least number of rounds that the table allows
  const int64_t ctas = static_cast<int64_t>(num_sms()) * ctas_an_sm(VEC), most = TABLE / a.pairs;
  const int64_t rounds = (a.rows + ctas * most - 1) / (ctas * most);
  const int64_t per_token = static_cast<int64_t>(a.pairs / VEC) * ((a.heads + heads_a_thread(VEC) - 1) / heads_a_thread(VEC));
  // (a tile's items are counted in 32 bits)
  a.tile = static_cast<int>(std::min<int64_t>((a.rows + ctas * rounds - 1) / (ctas * rounds), std::max<int64_t>(1, (1 << 30) / per_token)));
  const int64_t tiles = (a.rows + a.tile - 1) / a.tile;
  mrope_kernel<VEC><<<static_cast<unsigned>(std::min(tiles, ctas)), THREADS, 0, st>>>(a);
  return launch_check("mrope_kernel");
}

}  // namespace
}  // namespace mt

using namespace mt;

extern "C" mt_status mt_mrope(const mt_bf16* x, int64_t ld_x, mt_bf16* y, int64_t ld_y, const int32_t* pos, int64_t ld_pos,
                              const int32_t* sections, int32_t n_axes, int64_t rows, int32_t n_heads, int32_t head_dim,
                              float theta, int32_t interleaved, int32_t per_axis, int32_t inverse, void* stream) {
  if (!sections || (rows != 0 && n_heads != 0 && (!x || !y || !pos))) return fail(MT_ERR_INVALID_ARG, "mrope: NULL pointer");
  if (rows < 0 || n_heads < 0 || head_dim <= 0 || !(theta > 0.f) || !std::isfinite(theta))
    return fail(MT_ERR_INVALID_ARG, "mrope: bad sizes or theta");
  if (n_axes < 1 || n_axes > MAX_AXES) return fail(MT_ERR_INVALID_ARG, "mrope: 1 to %d axes, got %d", MAX_AXES, n_axes);
  int64_t pairs = 0;
  for (int i = 0; i < n_axes; ++i) {
    if (sections[i] < 0) return fail(MT_ERR_INVALID_ARG, "mrope: section %d is negative", i);
    pairs += sections[i];
  }
  if (pairs < 1 || 2 * pairs > head_dim)
    return fail(MT_ERR_INVALID_ARG, "mrope: the sections hold %lld pairs, need 1 to head_dim / 2 = %d", (long long)pairs,
                head_dim / 2);
  if (pairs > MAX_PAIRS) return fail(MT_ERR_UNSUPPORTED, "mrope: at most %d rotated pairs a head", MAX_PAIRS);
  const int64_t width = static_cast<int64_t>(n_heads) * head_dim;
  if (width >= (1ll << 27)) return fail(MT_ERR_UNSUPPORTED, "mrope: heads of 2^27 columns and more");
  if (ld_x < width || ld_y < width || ld_pos < rows) return fail(MT_ERR_INVALID_ARG, "mrope: ld too small");
  if (x && x == y && ld_x != ld_y) return fail(MT_ERR_INVALID_ARG, "mrope: in place needs ld_x == ld_y");
  const uintptr_t bits = reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(y);
  if ((bits & 1) || (reinterpret_cast<uintptr_t>(pos) & 3))
    return fail(MT_ERR_ALIGNMENT, "mrope: pointers must be aligned to their elements");
  if (rows == 0 || n_heads == 0) return MT_OK;
  Mrope a;
  a.x = reinterpret_cast<const __nv_bfloat16*>(x);
  a.y = reinterpret_cast<__nv_bfloat16*>(y);
  a.pos = pos;
  a.ld_x = ld_x;
  a.ld_y = ld_y;
  a.ld_pos = ld_pos;
  a.rows = rows;
  a.heads = n_heads;
  a.d = head_dim;
  a.pairs = static_cast<int>(pairs);
  a.tile = 1;
  a.sign = inverse ? -1.f : 1.f;
  // axis and frequency of each pair: the axes' pairs in runs, or dealt out to the axes in turn
  int used[MAX_AXES] = {0}, next = 0;
  const double log_theta = std::log(static_cast<double>(theta)), turn = 6.283185307179586476925286766559;
  for (int i = 0; i < a.pairs; ++i) {
    while (used[next] == sections[next]) next = (next + 1) % n_axes;
    const double expo = per_axis ? static_cast<double>(used[next]) / sections[next] : static_cast<double>(i) / a.pairs;
    a.axis[i] = static_cast<uint8_t>(next);
    a.turns[i] = std::exp(-expo * log_theta) / turn;
    ++used[next];
    if (interleaved) next = (next + 1) % n_axes;
  }
  for (int i = a.pairs; i < MAX_PAIRS; ++i) {
    a.axis[i] = 0;
    a.turns[i] = 0.0;
  }
  // the widest vector that divides the pairs and the head and keeps rows aligned
  const uintptr_t all = bits | static_cast<uintptr_t>(ld_x) * 2 | static_cast<uintptr_t>(ld_y) * 2 |
                        static_cast<uintptr_t>(a.pairs) * 2 | static_cast<uintptr_t>(head_dim) * 2;
  const cudaStream_t st = as_stream(stream);
  if (all % 16 == 0) return go<8>(a, st);
  if (all % 8 == 0) return go<4>(a, st);
  if (all % 4 == 0) return go<2>(a, st);
  return go<1>(a, st);
}
