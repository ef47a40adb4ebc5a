// wq_rows.hpp -- rows of bf16 or fp32 values in 16-byte pieces, shared by the kernels that read and write
// whole rows.
#pragma once
#include "wq_device.hpp"

namespace wq {

// 16 bytes at any element's address.
struct __attribute__((packed, aligned(2))) Piece {
  u32x4 v;
};

template <typename T>
__device__ __forceinline__ u32x4 load_piece(const T* p) {
  return reinterpret_cast<const Piece*>(p)->v;
}
template <typename T>
__device__ __forceinline__ void store_piece(T* p, const u32x4& v) {
  reinterpret_cast<Piece*>(p)->v = v;
}

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(uint16_t v) { return bf16_bits_to_f32(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ uint16_t from_f32<uint16_t>(float v) { return (uint16_t)f32_to_bf16_bits(v); }

// The E = 16 / sizeof(T) values of a piece in fp32, and back with one rounding.
__device__ __forceinline__ void unpack(const u32x4& v, float (&f)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(v[i]);
}
__device__ __forceinline__ void unpack(const u32x4& v, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(v[i] << 16);
    f[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ u32x4 pack(const float (&f)[4]) {
  return (u32x4){__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])};
}
__device__ __forceinline__ u32x4 pack(const float (&f)[8]) {
  return (u32x4){pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                 pack_bf16x2(f[6], f[7])};
}

}  // namespace wq
