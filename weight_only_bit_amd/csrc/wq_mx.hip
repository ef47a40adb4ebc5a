// wq_mx.hip -- microscaled 4-bit floating point (MXFP4): quantisation, and the products whose
// operands are both MXFP4.
//
// A block of 32 values along k shares one power-of-two scale X = 2^(byte - 127); a value is
// X times one of the e2m1 magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6 with a sign.  The scaled
// matrix instructions take the codes as they are stored (32 codes, 16 bytes, per lane) and the
// block's scale byte beside them, so nothing is decoded on the way: a product of two MXFP4
// operands runs at four times the bf16 rate and reads 17/32 of a byte per value.
#include <hip/hip_runtime.h>

#include "wq_kernels.hpp"

namespace wq {
namespace {

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

// ---------------------------------------------------------------------------------------------
// Quantisation.  Rows are contiguous and k is a multiple of 64, so blocks of 32 tile the flat
// array and the kernel needs no row structure.  Four neighbouring lanes hold one block, 8 values
// each; the largest magnitude's bit pattern (an integer maximum: magnitudes order as their
// patterns, and a NaN or infinity is at least 0x7F800000) gives the scale byte
//   E - 2 for a maximum with exponent field E (never below 0): floor(log2 max) - 2 + 127,
// and v_cvt_scalef32_pk_fp4_* divides by the scale, rounds half to even and saturates at 6.
// ---------------------------------------------------------------------------------------------

// Maximum over the quad of lanes 4 i .. 4 i + 3.
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  const uint32_t a = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true);  // 1,0,3,2
  v = v > a ? v : a;
  const uint32_t b = (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true);  // 2,3,0,1
  return v > b ? v : b;
}

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

template <typename T>
__global__ __launch_bounds__(256) void mx_quantize_kernel(const T* __restrict__ x, int64_t octets,
                                                          uint8_t* __restrict__ codes,
                                                          uint8_t* __restrict__ scales) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;  // 8 values
  if (i >= octets) return;  // octets is a multiple of 8: quads stay whole
  uint32_t top = 0, c = 0;
  if constexpr (sizeof(T) == 2) {
    const u32x4 v = reinterpret_cast<const u32x4*>(x)[i];
#pragma unroll
    for (int d = 0; d < 4; ++d) top = umax(top, umax((v[d] << 16) & 0x7FFF0000u, v[d] & 0x7FFF0000u));
    top = quad_max(top);
    const uint32_t byte = umax(top >> 23, 2u) - 2u;
    const float s = __uint_as_float(byte << 23);
    // (scalars first: a bit cast of a vector's element would read element 0)
    const uint32_t v0 = v[0], v1 = v[1], v2 = v[2], v3 = v[3];
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, v0), s, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, v1), s, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, v2), s, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2_t, v3), s, 3);
  } else {
    const f32x4 a = reinterpret_cast<const f32x4*>(x)[2 * i];
    const f32x4 b = reinterpret_cast<const f32x4*>(x)[2 * i + 1];
#pragma unroll
    for (int d = 0; d < 4; ++d)
      top = umax(top, umax(__float_as_uint(a[d]) & 0x7FFFFFFFu, __float_as_uint(b[d]) & 0x7FFFFFFFu));
    top = quad_max(top);
    const uint32_t byte = umax(top >> 23, 2u) - 2u;
    const float s = __uint_as_float(byte << 23);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, a[0], a[1], s, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, a[2], a[3], s, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, b[0], b[1], s, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, b[2], b[3], s, 3);
  }
  const bool finite = top < 0x7F800000u;
  reinterpret_cast<uint32_t*>(codes)[i] = finite ? c : 0u;
  if ((threadIdx.x & 3) == 0) scales[i >> 2] = finite ? (uint8_t)(umax(top >> 23, 2u) - 2u) : (uint8_t)255;
}

// ---------------------------------------------------------------------------------------------
// Products of two MXFP4 operands.  v_mfma_scale_f32_16x16x128_f8f6f4: lane l supplies row l % 16
// of A (column of B), block l / 16 of the step's four blocks of 32, and that block's scale byte;
// it receives D[4 (l / 16) + i][l % 16].  Every product of two codes is exact, the blocks' scales
// are applied to the blocks' sums, and the accumulation is fp32.
// ---------------------------------------------------------------------------------------------
__device__ __forceinline__ f32x4 mfma_mx16(const u32x4& a, uint32_t sa, const u32x4& b, uint32_t sb,
                                           const f32x4& c) {
  const i32x8 av = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i32x8 bv = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, c, 4, 4, 0, (int)sa, 0, (int)sb);
}

__device__ __forceinline__ void store_out(void* out, int f32, int64_t at, float v) {
  if (f32) reinterpret_cast<float*>(out)[at] = v;
  else reinterpret_cast<uint16_t*>(out)[at] = (uint16_t)f32_to_bf16_bits(v);
}

// One workgroup of KS waves computes 16 MT rows by 16 columns (gate+up: of both matrices); its
// waves split the steps of 128 along k and their sums meet in LDS, in order.  Lanes whose block
// lies past k multiply zero codes with scale 1.
template <int MODE, int MT, int KS>
__global__ __launch_bounds__(64 * KS) void mx_stream_kernel(const MxArgs a) {
  constexpr int NM = MODE == MODE_GATEUP ? 2 : 1;
  __shared__ f32x4 red[KS][NM * MT][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nl = lane & 15, q = lane >> 4;
  const int64_t N = a.N;
  const int32_t nb = (int32_t)(a.K / 32);
  const int32_t steps = (nb + 3) / 4;
  const int32_t s_begin = (int32_t)((int64_t)steps * wave / KS);
  const int32_t s_end = (int32_t)((int64_t)steps * (wave + 1) / KS);

  int64_t e = 0, m_base = 0, m_total = a.M;
  if constexpr (MODE == MODE_DENSE) {
    m_base = (int64_t)blockIdx.z * (16 * MT);
    m_total = a.M - m_base < 16 * MT ? a.M - m_base : 16 * MT;
  } else {
    e = blockIdx.y;
    m_base = a.offsets[e];
    m_total = a.offsets[e + 1] - m_base;
    if (m_total <= 0) return;
  }
  const int64_t nrow = (int64_t)blockIdx.x * 16 + nl;
  const bool nvalid = nrow < N;
  const int64_t wr = e * N + (nvalid ? nrow : N - 1);
  const uint8_t* wc[NM];
  const uint8_t* ws[NM];
  wc[0] = a.w0_codes + wr * (a.K / 2);
  ws[0] = a.w0_scales + wr * nb;
  if constexpr (NM == 2) {
    wc[1] = a.w1_codes + wr * (a.K / 2);
    ws[1] = a.w1_scales + wr * nb;
  }

  for (int64_t ms = 0; ms < m_total; ms += 16 * MT) {
    const int64_t left = m_total - ms;
    const uint8_t* xc[MT];
    const uint8_t* xs[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const int64_t r = m_base + ms + (16 * t + nl < left ? 16 * t + nl : 0);
      int64_t src = r;
      if constexpr (MODE == MODE_GATEUP) src = a.sorted_pairs[r] / a.topk;
      xc[t] = a.x_codes + src * (a.K / 2);
      xs[t] = a.x_scales + src * nb;
    }
    f32x4 acc[NM][MT];
#pragma unroll
    for (int j = 0; j < NM; ++j)
#pragma unroll
      for (int t = 0; t < MT; ++t) acc[j][t] = (f32x4){0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int32_t s = s_begin; s < s_end; ++s) {
      const int32_t blk = 4 * s + q;
      const bool in = blk < nb;
      const int32_t b = in ? blk : 0;
      u32x4 w[NM], x[MT];
      uint32_t wsc[NM], xsc[MT];
#pragma unroll
      for (int j = 0; j < NM; ++j) {
        w[j] = *reinterpret_cast<const u32x4*>(wc[j] + (int64_t)b * 16);
        wsc[j] = ws[j][b];
      }
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        x[t] = *reinterpret_cast<const u32x4*>(xc[t] + (int64_t)b * 16);
        xsc[t] = xs[t][b];
      }
      if (!in) {
#pragma unroll
        for (int j = 0; j < NM; ++j) {
          w[j] = (u32x4){0, 0, 0, 0};
          wsc[j] = 127;
        }
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          x[t] = (u32x4){0, 0, 0, 0};
          xsc[t] = 127;
        }
      }
#pragma unroll
      for (int j = 0; j < NM; ++j)
#pragma unroll
        for (int t = 0; t < MT; ++t) acc[j][t] = mfma_mx16(x[t], xsc[t], w[j], wsc[j], acc[j][t]);
    }
    if (KS > 1) {
      if (ms > 0) __syncthreads();  // the previous pass's sums have been read
#pragma unroll
      for (int j = 0; j < NM; ++j)
#pragma unroll
        for (int t = 0; t < MT; ++t) red[wave][j * MT + t][lane] = acc[j][t];
      __syncthreads();
    }
    // row tile t is finished by wave t % KS
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      if (KS > 1 && wave != t % KS) continue;
      f32x4 g = acc[0][t], u = acc[NM - 1][t];
      if (KS > 1) {
        g = red[0][t][lane];
        u = red[0][(NM - 1) * MT + t][lane];
#pragma unroll
        for (int p = 1; p < KS; ++p) {
          g += red[p][t][lane];
          if constexpr (NM == 2) u += red[p][MT + t][lane];
        }
      }
      if (!nvalid) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t m = 16 * t + 4 * q + i;
        if (m >= left) continue;
        const int64_t at = (m_base + ms + m) * a.out_stride + nrow;
        if constexpr (MODE == MODE_GATEUP) store_out(a.out, 0, at, silu_f32(g[i]) * u[i]);
        else store_out(a.out, a.out_f32, at, g[i]);
      }
    }
  }
}

template <int MODE, int MT, int KS>
hipError_t launch_stream(const MxArgs& a, int64_t gy, int64_t gz, hipStream_t s) {
  hipLaunchKernelGGL((mx_stream_kernel<MODE, MT, KS>),
                     dim3((unsigned)((a.N + 15) / 16), (unsigned)gy, (unsigned)gz), dim3(64 * KS), 0,
                     s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_quantize(const void* x, int f32, int64_t n, int64_t k, uint8_t* codes,
                              uint8_t* scales, hipStream_t stream) {
  const int64_t octets = n * (k / 8);
  const int64_t wgs = (octets + 255) / 256;
  if (wgs > 0x7FFFFFFF) return hipErrorInvalidValue;
  if (f32)
    hipLaunchKernelGGL(mx_quantize_kernel<float>, dim3((unsigned)wgs), dim3(256), 0, stream,
                       static_cast<const float*>(x), octets, codes, scales);
  else
    hipLaunchKernelGGL(mx_quantize_kernel<uint16_t>, dim3((unsigned)wgs), dim3(256), 0, stream,
                       static_cast<const uint16_t*>(x), octets, codes, scales);
  return hipGetLastError();
}

hipError_t launch_mx_product(int mode, const MxArgs& a, int64_t experts, hipStream_t stream) {
  if (mode == MODE_GATEUP) return launch_stream<MODE_GATEUP, 1, 4>(a, experts, 1, stream);
  if (mode == MODE_DOWN) return launch_stream<MODE_DOWN, 1, 4>(a, experts, 1, stream);
  // the grid's z extent is 16 bits: more rows take further launches
  constexpr int64_t chunk = 65535ll * 32;
  for (int64_t r0 = 0; r0 < a.M; r0 += chunk) {
    MxArgs b = a;
    b.x_codes = a.x_codes + r0 * (a.K / 2);
    b.x_scales = a.x_scales + r0 * (a.K / 32);
    b.out = static_cast<uint8_t*>(a.out) + r0 * a.out_stride * (a.out_f32 ? 4 : 2);
    b.M = a.M - r0 < chunk ? a.M - r0 : chunk;
    const hipError_t e = b.M <= 16 ? launch_stream<MODE_DENSE, 1, 4>(b, 1, 1, stream)
                                   : launch_stream<MODE_DENSE, 2, 4>(b, 1, (b.M + 31) / 32, stream);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace wq
