// bf16 rows in vectors of 8, 4, 2 or 1 elements (the widest that a row's alignment allows), and warp sums of a
// few values at once.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace mt {
namespace vec {

template <int VEC>
struct Raw;
template <>
struct Raw<8> {
  using type = uint4;
};
template <>
struct Raw<4> {
  using type = uint2;
};
template <>
struct Raw<2> {
  using type = uint32_t;
};
template <>
struct Raw<1> {
  using type = uint16_t;
};

__device__ __forceinline__ float2 bf2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ void unpack(const uint4& u, float* f) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = bf2(w[i]);
    f[2 * i] = t.x;
    f[2 * i + 1] = t.y;
  }
}
__device__ __forceinline__ void unpack(const uint2& u, float* f) {
  const float2 t = bf2(u.x), v = bf2(u.y);
  f[0] = t.x;
  f[1] = t.y;
  f[2] = v.x;
  f[3] = v.y;
}
__device__ __forceinline__ void unpack(const uint32_t& u, float* f) {
  const float2 t = bf2(u);
  f[0] = t.x;
  f[1] = t.y;
}
__device__ __forceinline__ void unpack(const uint16_t& u, float* f) { f[0] = __uint_as_float(uint32_t(u) << 16); }

__device__ __forceinline__ void pack(uint4& u, const float* f) {
  u = make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}
__device__ __forceinline__ void pack(uint2& u, const float* f) { u = make_uint2(pack2(f[0], f[1]), pack2(f[2], f[3])); }
__device__ __forceinline__ void pack(uint32_t& u, const float* f) { u = pack2(f[0], f[1]); }
__device__ __forceinline__ void pack(uint16_t& u, const float* f) { u = __bfloat16_as_ushort(__float2bfloat16_rn(f[0])); }

__device__ __forceinline__ void zero(uint4& u) { u = make_uint4(0u, 0u, 0u, 0u); }
__device__ __forceinline__ void zero(uint32_t& u) { u = 0u; }
__device__ __forceinline__ void zero(uint16_t& u) { u = 0; }

// Two fp32 values in a register pair: sm_100's packed arithmetic does both in one instruction.
using f2 = unsigned long long;
__device__ __forceinline__ f2 f2_make(float lo, float hi) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ f2 f2_both(float v) { return f2_make(v, v); }
__device__ __forceinline__ void f2_split(f2 v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ float f2_sum(f2 v) {
  float a, b;
  f2_split(v, a, b);
  return a + b;
}
__device__ __forceinline__ f2 f2_add(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 f2_mul(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 f2_fma(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f2 f2_of(uint32_t w) { return f2_make(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)); }
__device__ __forceinline__ uint32_t f2_pack(f2 v) {
  float a, b;
  f2_split(v, a, b);
  return pack2(a, b);
}
__device__ __forceinline__ void words(const uint4& u, uint32_t (&w)[4]) {
  w[0] = u.x;
  w[1] = u.y;
  w[2] = u.z;
  w[3] = u.w;
}

// Sums of N values (N = 1, 2, 4 or 8) over the warp, left in every lane. The first log2(N) exchanges halve the
// number of values a lane carries, so N = 4 takes 10 shuffles instead of 20; the order of additions is fixed.
template <int N>
__device__ __forceinline__ void warp_sums(float (&v)[N]) {
  static_assert(N == 1 || N == 2 || N == 4 || N == 8, "");
  constexpr unsigned ALL = 0xffffffffu;
  const int lane = threadIdx.x & 31;
  int o = 16;
#pragma unroll
  for (int n = N / 2; n > 0; n /= 2, o /= 2) {
    const bool hi = lane & o;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float keep = hi ? v[n + i] : v[i], give = hi ? v[i] : v[n + i];
      v[i] = keep + __shfl_xor_sync(ALL, give, o);
    }
  }
  float s = v[0];
#pragma unroll
  for (int p = 16 / N; p > 0; p /= 2) s += __shfl_xor_sync(ALL, s, p);
  if constexpr (N == 1) {
    v[0] = s;
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __shfl_sync(ALL, s, i * (32 / N));
  }
}

}  // namespace vec
}  // namespace mt
