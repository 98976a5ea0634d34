// Element types of inputs that are not 8-bit codes, and the lane exchanges
// that the reductions over them share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "internal.h"

namespace fp8g {
namespace elem {

typedef __bf16 bf16_t;
typedef _Float16 f16_t;

// (conversions round to nearest even; bf16 and fp16 widen exactly)
template <typename T>
__device__ __forceinline__ float to_f32(T x) { return (float)x; }
template <typename T>
__device__ __forceinline__ T from_f32(float x) { return (T)x; }

// N consecutive elements moved as one access (N * sizeof(T) up to 16 bytes;
// the address is aligned to that) or one by one.
template <typename T, int N>
struct alignas(N * sizeof(T)) Pack {
  T v[N];
};

// Value of the lane `d` places on in a ring of 16 lanes (DPP row rotate: no
// LDS traffic, no address register).
template <int D>
__device__ __forceinline__ uint32_t ring16(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x120 + D, 0xF, 0xF, false);
}
template <int D>
__device__ __forceinline__ float ring16f(float x) {
  return __uint_as_float(ring16<D>(__float_as_uint(x)));
}

// All-lanes reductions over groups of LPR lanes (16 or 64). Above 16 lanes
// gfx950 exchanges whole rows of lanes between two registers: of two copies
// of x, each lane then holds its own row's value and the other row's.
template <int LPR, class F>
__device__ __forceinline__ uint32_t reduce_u32(uint32_t x, F f) {
  x = f(x, ring16<8>(x));
  x = f(x, ring16<4>(x));
  x = f(x, ring16<2>(x));
  x = f(x, ring16<1>(x));
  if constexpr (LPR == 64) {
    const auto p = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    x = f(p[0], p[1]);
    const auto q = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    x = f(q[0], q[1]);
  }
  return x;
}
template <int LPR, class F>
__device__ __forceinline__ float reduce_f32(float x, F f) {
  return __uint_as_float(reduce_u32<LPR>(__float_as_uint(x), [&](uint32_t a, uint32_t b) {
    return __float_as_uint(f(__uint_as_float(a), __uint_as_float(b)));
  }));
}
template <int LPR>
__device__ __forceinline__ float sum_lanes(float x) {
  return reduce_f32<LPR>(x, [](float a, float b) { return a + b; });
}
template <int LPR>
__device__ __forceinline__ float max_lanes(float x) {
  return reduce_f32<LPR>(x, [](float a, float b) { return __builtin_fmaxf(a, b); });
}

// Sum over the wave's 64 lanes, in fp64.
__device__ __forceinline__ double sum_wave(double x) {
  const auto other = [](double v, auto get) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    return __builtin_bit_cast(double, (uint64_t)get((uint32_t)u) | (uint64_t)get((uint32_t)(u >> 32)) << 32);
  };
  x += other(x, [](uint32_t w) { return ring16<8>(w); });
  x += other(x, [](uint32_t w) { return ring16<4>(w); });
  x += other(x, [](uint32_t w) { return ring16<2>(w); });
  x += other(x, [](uint32_t w) { return ring16<1>(w); });
  x += other(x, [](uint32_t w) { return (uint32_t)__shfl_xor((int)w, 16); });
  x += other(x, [](uint32_t w) { return (uint32_t)__shfl_xor((int)w, 32); });
  return x;
}

// exp(x) for x <= 0 (or NaN) within 2 ulp: 2^(x log2 e), with the product's rounding
// error and the constant's put back to first order. (Where the product is infinite that
// error is NaN or +inf and the power 0: the minimum, which drops a NaN, makes their
// product 0. It is below 2^-16 wherever the power is not 0.) The power alone is off by up to
// 1.2 |x| 2^-24, which bf16 and fp16 logits, whose differences are exact, do not excuse; it
// saves 0.9 us of 22.2 (T 32768, E 256, fp32; bf16 0.9 of 18.1) and 0.7 of 13.1 in the
// backward pass (T 30011, E 160, fp32).
__device__ __forceinline__ float exp_neg(float x) {
  constexpr float L2E = 0x1.715476p+0f, L2E_LO = 0x1.4ae0cp-26f, LN2 = 0x1.62e43p-1f;
  const float t = x * L2E;
  const float lo = __builtin_fminf(__builtin_fmaf(x, L2E_LO, __builtin_fmaf(x, L2E, -t)), 1.0f);
  const float y = __builtin_amdgcn_exp2f(t);
  return __builtin_fmaf(y, lo * LN2, y);
}

}  // namespace elem
}  // namespace fp8g
