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

// All-lanes reductions over groups of LPR lanes (16 or 64).
template <int LPR, class F>
__device__ __forceinline__ uint32_t reduce_u32(uint32_t x, F f) {
  x = f(x, ring16<8>(x));
  x = f(x, ring16<4>(x));
  x = f(x, ring16<2>(x));
  x = f(x, ring16<1>(x));
  if constexpr (LPR == 64) {
    x = f(x, (uint32_t)__shfl_xor((int)x, 16));
    x = f(x, (uint32_t)__shfl_xor((int)x, 32));
  }
  return x;
}
template <int LPR, class F>
__device__ __forceinline__ float reduce_f32(float x, F f) {
  x = f(x, ring16f<8>(x));
  x = f(x, ring16f<4>(x));
  x = f(x, ring16f<2>(x));
  x = f(x, ring16f<1>(x));
  if constexpr (LPR == 64) {
    x = f(x, __shfl_xor(x, 16));
    x = f(x, __shfl_xor(x, 32));
  }
  return x;
}
template <int LPR>
__device__ __forceinline__ float sum_lanes(float x) {
  return reduce_f32<LPR>(x, [](float a, float b) { return a + b; });
}
template <int LPR>
__device__ __forceinline__ float max_lanes(float x) {
  return reduce_f32<LPR>(x, [](float a, float b) { return __builtin_fmaxf(a, b); });
}

}  // namespace elem
}  // namespace fp8g
