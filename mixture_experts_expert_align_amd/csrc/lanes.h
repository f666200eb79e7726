// Sums and maxima over a row of 16 lanes or a whole wave, the same bits in every
// lane.
#pragma once

#include "device_common.h"

namespace moe {

template <int CTRL, class T>
__device__ __forceinline__ T dpp_of(T v) {
  static_assert(sizeof(T) == 4, "one register");
  return __builtin_bit_cast(T, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, false));
}

// f over LANES lanes: each step combines two values that two lanes hold in
// either order.  Rotations within the row (DPP), then swaps across the rows (rows
// 1 and 3 of one register with 0 and 2 of the other: (r0, r0, r2, r2) and (r1, r1,
// r3, r3); then the halves), without LDS.
template <int LANES, class T, class F>
__device__ __forceinline__ T lanes_all(T v, F f) {
  static_assert(LANES == 16 || LANES == 64, "a row of 16 lanes, or the wave");
  v = f(v, dpp_of<0x128>(v));
  v = f(v, dpp_of<0x124>(v));
  v = f(v, dpp_of<0x122>(v));
  v = f(v, dpp_of<0x121>(v));
  if (LANES == 64) {
    const uint32_t u = __builtin_bit_cast(uint32_t, v);
    const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    v = f(__builtin_bit_cast(T, (uint32_t)a[0]), __builtin_bit_cast(T, (uint32_t)a[1]));
    const uint32_t w = __builtin_bit_cast(uint32_t, v);
    const auto b = __builtin_amdgcn_permlane32_swap(w, w, false, false);
    v = f(__builtin_bit_cast(T, (uint32_t)b[0]), __builtin_bit_cast(T, (uint32_t)b[1]));
  }
  return v;
}
template <int LANES>
__device__ __forceinline__ float lanes_max(float v) {
  return lanes_all<LANES>(v, [](float a, float b) { return fmaxf(a, b); });
}
template <int LANES>
__device__ __forceinline__ int lanes_max(int v) {
  return lanes_all<LANES>(v, [](int a, int b) { return max(a, b); });
}
template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
  return lanes_all<LANES>(v, [](float a, float b) { return a + b; });
}

}  // namespace moe
