// wq_wave.hpp -- sums and maxima over groups of a wave's lanes, every lane ending with the same bits.  LANES: a
// power of two, the lanes of a group.
#pragma once
#include "wq_device.hpp"

namespace wq {

// The lane that a lane meets in step STEP of a reduction over 16 lanes.
template <int STEP>
__device__ __forceinline__ uint32_t wave_partner(uint32_t v) {
  constexpr int ctrl = STEP == 0   ? 0xB1    // lane ^ 1
                       : STEP == 1 ? 0x4E    // lane ^ 2
                       : STEP == 2 ? 0x141   // mirrored in 8: quads hold one value by now
                                   : 0x140;  // mirrored in 16
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, ctrl, 0xF, 0xF, true);
}

// join(v, the partner's v) over the group; join must not depend on the order of its arguments.
template <int LANES, class Join>
__device__ __forceinline__ uint32_t wave_join(uint32_t v, Join join) {
  if constexpr (LANES > 1) v = join(v, wave_partner<0>(v));
  if constexpr (LANES > 2) v = join(v, wave_partner<1>(v));
  if constexpr (LANES > 4) v = join(v, wave_partner<2>(v));
  if constexpr (LANES > 8) v = join(v, wave_partner<3>(v));
  if constexpr (LANES > 16) {  // the two of a swap are this lane's value and its partner's, in some order
    const auto p = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = join((uint32_t)p[0], (uint32_t)p[1]);
  }
  if constexpr (LANES > 32) {
    const auto p = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = join((uint32_t)p[0], (uint32_t)p[1]);
  }
  return v;
}
template <int LANES = 64>
__device__ __forceinline__ float wave_sum(float v) {
  return __uint_as_float(wave_join<LANES>(__float_as_uint(v), [](uint32_t a, uint32_t b) __attribute__((always_inline)) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}
// A NaN is passed over.
template <int LANES = 64>
__device__ __forceinline__ float wave_max(float v) {
  return __uint_as_float(wave_join<LANES>(__float_as_uint(v), [](uint32_t a, uint32_t b) __attribute__((always_inline)) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }));
}

__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint64_t larger(uint64_t a, uint64_t b) { return a > b ? a : b; }

template <int LANES = 64>
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  return wave_join<LANES>(v, [](uint32_t a, uint32_t b) __attribute__((always_inline)) { return larger(a, b); });
}
template <int LANES = 64>
__device__ __forceinline__ uint64_t wave_max(uint64_t v) {
  const uint32_t hi = (uint32_t)(v >> 32), top = wave_max<LANES>(hi);
  // among the lanes with the largest upper half the largest lower one
  return (uint64_t)top << 32 | wave_max<LANES>(hi == top ? (uint32_t)v : 0u);
}

}  // namespace wq
