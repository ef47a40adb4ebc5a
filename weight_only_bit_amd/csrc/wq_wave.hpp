// wq_wave.hpp -- sums and maxima over the lanes of a wave, every lane ending with the same bits.
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

__device__ __forceinline__ float wave_sum(float v) {
  v += __uint_as_float(wave_partner<0>(__float_as_uint(v)));
  v += __uint_as_float(wave_partner<1>(__float_as_uint(v)));
  v += __uint_as_float(wave_partner<2>(__float_as_uint(v)));
  v += __uint_as_float(wave_partner<3>(__float_as_uint(v)));
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint64_t larger(uint64_t a, uint64_t b) { return a > b ? a : b; }

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = larger(v, wave_partner<0>(v));
  v = larger(v, wave_partner<1>(v));
  v = larger(v, wave_partner<2>(v));
  v = larger(v, wave_partner<3>(v));
  const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = larger((uint32_t)a[0], (uint32_t)a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return larger((uint32_t)b[0], (uint32_t)b[1]);
}
template <int STEP>
__device__ __forceinline__ uint64_t wave_partner64(uint64_t v) {
  return (uint64_t)wave_partner<STEP>((uint32_t)(v >> 32)) << 32 | wave_partner<STEP>((uint32_t)v);
}
__device__ __forceinline__ uint64_t wave_max(uint64_t v) {
  v = larger(v, wave_partner64<0>(v));
  v = larger(v, wave_partner64<1>(v));
  v = larger(v, wave_partner64<2>(v));
  v = larger(v, wave_partner64<3>(v));
  const auto al = __builtin_amdgcn_permlane16_swap((uint32_t)v, (uint32_t)v, false, false);
  const auto ah = __builtin_amdgcn_permlane16_swap((uint32_t)(v >> 32), (uint32_t)(v >> 32), false, false);
  v = larger((uint64_t)ah[0] << 32 | (uint32_t)al[0], (uint64_t)ah[1] << 32 | (uint32_t)al[1]);
  const auto bl = __builtin_amdgcn_permlane32_swap((uint32_t)v, (uint32_t)v, false, false);
  const auto bh = __builtin_amdgcn_permlane32_swap((uint32_t)(v >> 32), (uint32_t)(v >> 32), false, false);
  return larger((uint64_t)bh[0] << 32 | (uint32_t)bl[0], (uint64_t)bh[1] << 32 | (uint32_t)bl[1]);
}

}  // namespace wq
