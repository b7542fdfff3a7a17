// Exchanges over 16, 32 or 64 neighbouring lanes: every lane ends with the result.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

namespace moegg {
namespace {

typedef uint32_t v2u __attribute__((ext_vector_type(2)));

// (the bound control lets the compiler put the exchange into the instruction that
// uses it; every source lane exists)
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u(uint32_t x) {
  return static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(x), CTRL, 0xF, 0xF, true));
}

// STEP 0..3 pair lanes inside a 16-lane row (1, 2 apart, mirrored halves,
// mirrored row), 4 and 5 exchange rows and half waves.
template <int STEP>
__device__ __forceinline__ uint32_t partner(uint32_t x) {
  if constexpr (STEP == 0) return dpp_u<0xB1>(x);
  else if constexpr (STEP == 1) return dpp_u<0x4E>(x);
  else if constexpr (STEP == 2) return dpp_u<0x141>(x);
  else if constexpr (STEP == 3) return dpp_u<0x140>(x);
  else if constexpr (STEP == 4) {
    const v2u s = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    return (threadIdx.x & 16) ? s.x : s.y;
  } else {
    const v2u s = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    return (threadIdx.x & 32) ? s.x : s.y;
  }
}
template <int STEP>
__device__ __forceinline__ float partner(float x) {
  return __uint_as_float(partner<STEP>(__float_as_uint(x)));
}
template <int STEP>
__device__ __forceinline__ int32_t partner(int32_t x) {
  return static_cast<int32_t>(partner<STEP>(static_cast<uint32_t>(x)));
}
template <int STEP>
__device__ __forceinline__ double partner(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint64_t lo = partner<STEP>(static_cast<uint32_t>(u)), hi = partner<STEP>(static_cast<uint32_t>(u >> 32));
  return __builtin_bit_cast(double, lo | hi << 32);
}

template <int LPT, int STEP = 0, typename F>
__device__ __forceinline__ void steps(F&& f) {
  if constexpr ((1 << STEP) < LPT) {
    f(std::integral_constant<int, STEP>{});
    steps<LPT, STEP + 1>(f);
  }
}
template <int LPT, typename T>
__device__ __forceinline__ T lanes_sum(T v) {
  steps<LPT>([&](auto c) { v += partner<decltype(c)::value>(v); });
  return v;
}
template <int LPT>
__device__ __forceinline__ float lanes_max(float v) {
  steps<LPT>([&](auto c) { v = fmaxf(v, partner<decltype(c)::value>(v)); });
  return v;
}

}  // namespace
}  // namespace moegg
