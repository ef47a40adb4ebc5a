// wq_mx.hip -- microscaled 4-bit floating point (MXFP4): quantisation, and the products whose
// operands are both MXFP4.
//
// A block of 32 values along k shares one power-of-two scale X = 2^(byte - 127); a value is
// X times one of the e2m1 magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6 with a sign.  The scaled
// matrix instructions take the codes as they are stored (32 codes, 16 bytes, per lane) and the
// block's scale byte beside them, so nothing is decoded on the way: a product of two MXFP4
// operands runs at four times the bf16 rate and reads 17/32 of a byte per value.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "wq_kernels.hpp"
#include "wq_mx_select.hpp"
#include "wq_tiles.hpp"

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
// Bound by memory: 8192 x 8192 fp32 45 to 48 us (6.4 to 6.7 TB/s read and written; 61 right after another
// kernel has written 134 MB), bf16 25.5 us (6.6 TB/s); 17 x 4096 bf16 2.3 us, of which an empty kernel
// takes 1.6.
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
                                                          uint8_t* __restrict__ scales, int64_t first) {
  const int64_t i = (first + blockIdx.x) * 256 + threadIdx.x;  // 8 values
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
// Products of two MXFP4 operands.  Every product of two codes is exact, the blocks' scales are
// applied to the blocks' sums, and the accumulation is fp32.
//
// Few rows: the weights stream from memory straight into v_mfma_scale_f32_16x16x128_f8f6f4 operands.
// Lane l supplies row l % 16 of A (column of B) and one block of 32 with its scale byte; it receives
// D[4 (l / 16) + i][l % 16].  In a step of 512 along k lane group q = l / 16 takes the blocks
// 4 q .. 4 q + 3, one per instruction: 64 contiguous bytes of codes and one dword of scales, of which
// instruction s reads byte s.  Any order of the k sum is the same product.
// Bound by the weights' way from memory: 1 x 28672, k 4096 13 us (4.8 TB/s); experts' gate+up, 16 tokens
// top-8 of 64, 3584 x 8192 319 us (5.5 TB/s); a small layer by one round trip: 1 x 4096, k 4096 4.0 us.
// ---------------------------------------------------------------------------------------------
template <int S>
__device__ __forceinline__ f32x4 mfma_mx16(const u32x4& a, uint32_t sa, const u32x4& b, uint32_t sb,
                                           const f32x4& c) {
  const i32x8 av = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i32x8 bv = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, c, 4, 4, S, (int)sa, S, (int)sb);
}

__device__ __forceinline__ void store_out(void* out, int f32, int64_t at, float v) {
  if (f32) reinterpret_cast<float*>(out)[at] = v;
  else reinterpret_cast<uint16_t*>(out)[at] = (uint16_t)f32_to_bf16_bits(v);
}

struct __attribute__((packed, aligned(2))) Scales4 {
  uint32_t v;
};

// A lane's four blocks of a step: the row's codes and scales start at `codes` and `scales`.  A row
// holds an even number of blocks; of those behind its end the codes are the row's first (any codes
// do) and the scales 2^-127 on both sides: 2^-254 times 32 products of at most 36 is zero in fp32.
struct Part {
  u32x4 c[4];
  uint32_t s;
};
__device__ __forceinline__ void load_part(Part& p, const uint8_t* codes, const uint8_t* scales, int32_t block,
                                          int32_t nb) {
  if (block + 4 <= nb) {
#pragma unroll
    for (int i = 0; i < 4; ++i) p.c[i] = *reinterpret_cast<const u32x4*>(codes + ((int64_t)(block + i) << 4));
    p.s = reinterpret_cast<const Scales4*>(scales + block)->v;
  } else {
    const int64_t at = block < nb ? block : 0;
    p.c[0] = p.c[2] = *reinterpret_cast<const u32x4*>(codes + (at << 4));
    p.c[1] = p.c[3] = *reinterpret_cast<const u32x4*>(codes + (at << 4) + 16);
    p.s = block < nb ? *reinterpret_cast<const uint16_t*>(scales + block) : 0u;
  }
}

// One workgroup of KS waves computes 16 MT rows by 16 columns (gate+up: of both matrices); its
// waves split the steps along k and their sums meet in LDS, in order.  Four: with 2, 4, 8, 16 waves
// 1 x 28672, k 4096 takes 14.6, 13.0, 16.5, 21.3 us, 16 x 1024, k 8192 7.2, 6.9, 6.9, 7.0.
template <int MODE, int MT, int KS>
__global__ __launch_bounds__(64 * KS) void mx_stream_kernel(const MxArgs a) {
  constexpr int NM = MODE == MODE_GATEUP ? 2 : 1;
  __shared__ f32x4 red[KS][NM * MT][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nl = lane & 15, q = lane >> 4;
  const int64_t N = a.N;
  const int32_t nb = (int32_t)(a.K / 32);
  const int32_t steps = (nb + 15) / 16;
  const int32_t s_begin = steps * wave / KS, s_end = steps * (wave + 1) / KS;

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
    struct Step {
      Part w[NM], x[MT];
    };
    auto load = [&](Step& p, int32_t s) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < NM; ++j) load_part(p.w[j], wc[j], ws[j], 16 * s + 4 * q, nb);
#pragma unroll
      for (int t = 0; t < MT; ++t) load_part(p.x[t], xc[t], xs[t], 16 * s + 4 * q, nb);
    };
    auto multiply = [&](const Step& p) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < NM; ++j)
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          acc[j][t] = mfma_mx16<0>(p.x[t].c[0], p.x[t].s, p.w[j].c[0], p.w[j].s, acc[j][t]);
          acc[j][t] = mfma_mx16<1>(p.x[t].c[1], p.x[t].s, p.w[j].c[1], p.w[j].s, acc[j][t]);
          acc[j][t] = mfma_mx16<2>(p.x[t].c[2], p.x[t].s, p.w[j].c[2], p.w[j].s, acc[j][t]);
          acc[j][t] = mfma_mx16<3>(p.x[t].c[3], p.x[t].s, p.w[j].c[3], p.w[j].s, acc[j][t]);
        }
    };
    // two steps at hand, the next one's loads in flight under each product
    if (s_begin < s_end) {
      Step A, B;
      load(A, s_begin);
      int32_t s = s_begin;
      for (; s + 2 < s_end; s += 2) {
        load(B, s + 1);
        multiply(A);
        load(A, s + 2);
        multiply(B);
      }
      if (s + 1 < s_end) load(B, s + 1);
      multiply(A);
      if (s + 1 < s_end) multiply(B);
    }
    if (ms > 0) __syncthreads();  // the previous pass's sums have been read
#pragma unroll
    for (int j = 0; j < NM; ++j)
#pragma unroll
      for (int t = 0; t < MT; ++t) red[wave][j * MT + t][lane] = acc[j][t];
    __syncthreads();
    // row tile t is finished by wave t % KS
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      if (wave != t % KS) continue;
      f32x4 g = red[0][t][lane], u = red[0][(NM - 1) * MT + t][lane];
#pragma unroll
      for (int p = 1; p < KS; ++p) {
        g += red[p][t][lane];
        if constexpr (NM == 2) u += red[p][MT + t][lane];
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

// ---------------------------------------------------------------------------------------------
// Many rows: tiles staged in LDS.
//
// One workgroup of 4 waves, one per SIMD, computes 64 WM rows by 64 WN columns (256 x 256 for the
// large products); each wave 32 WM by 32 WN of them, as WM x WN blocks of 32 x 32 in registers.  k
// advances 256 per stage: 128 bytes of codes and 8 scale bytes per row.
//   * The weights are the A operand of v_mfma_scale_f32_32x32x64_f8f6f4 and the activations the B
//     operand, so a lane ends with four consecutive outputs of one row.  Lane (l, h) supplies row l
//     and a block of 32: slice s of a stage takes block 4 h + s, so a lane's four blocks are 64
//     contiguous bytes and their scales one dword, of which slice s reads byte s (the instruction's
//     byte select).  Any order of the k sum is the same product.
//   * Rows of a stage are 128 bytes in LDS, 16-byte piece p of row r in slot p ^ (r / 2 % 8), which
//     keeps the fragment reads free of bank conflicts; 8 lanes load a row.  Thread t carries the
//     scales of rows t through registers (rows of scale bytes are only 2-byte aligned).
//   * Two buffers, one workgroup per CU (256 x 256): codes pass through registers, which hold a third
//     stage on its way, so loads and LDS writes spread over the whole stage.  (Copies without
//     registers have to wait for the buffer that they fill, so all of a stage's are issued at once
//     and the MFMAs wait behind them: 1.75 us per stage of 256 CUs where the copies alone and the
//     rest alone take 0.95 each, with codes of zero; this way 1.2.)
//   * One buffer, two workgroups per CU (128 x 256): the next stage is copied without registers while
//     the other workgroup multiplies, which also covers a tile's first loads and its stores.  Through
//     registers: 176 us where this takes 165 (4096 x 8192, k 8192).
//   * A workgroup computes one tile.  One that went on to a next tile, whose first stages load under the
//     last ones, took 174 us against 146: loads and stores are counted together, in order, so the next
//     tile's second stage waits until the tile before has been written.
//   * Four more or twelve more waves for a 64 x 64 tile, each four a part of k, gain nothing (128 x 4096,
//     k 4096: 10.0, 10.3, 12.1 us): a CU takes in 30 KB/us of codes that its L2 does not hold, whoever
//     waits for them.
//   * The next slice's fragments are read under the current slice's MFMAs; the last slice of a
//     stage is multiplied after the barrier that ends the stage, over the next stage's first reads.
// Results of rows behind a ragged tile's end and of columns behind N are not stored.
// 256 x 256 (4096 x 8192, k 8192: 143 to 150 us, 3.7 to 3.8 PFLOP/s) is bound by power: a stage takes
// 2.04 us on random codes and 1.2 on codes of zero, with the clock at 1.6 GHz and the matrix units busy
// 0.57 of the time; matrix instructions alone, from registers, reach 6.6 and 8.9 PFLOP/s.  A tile's start
// and end take 6.9 us together.  64 x 64 is bound by the codes' way to a CU: 0.5 us a stage.
// ---------------------------------------------------------------------------------------------
constexpr int kStageBytes = 128;  // codes of one row of a stage

__device__ __forceinline__ f32x16 mfma_mx32(const u32x4& a, uint32_t sa, const u32x4& b, uint32_t sb,
                                            const f32x16& c, std::integral_constant<int, 0>) {
  const i32x8 av = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i32x8 bv = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, bv, c, 4, 4, 0, (int)sa, 0, (int)sb);
}
__device__ __forceinline__ f32x16 mfma_mx32(const u32x4& a, uint32_t sa, const u32x4& b, uint32_t sb,
                                            const f32x16& c, std::integral_constant<int, 1>) {
  const i32x8 av = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i32x8 bv = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, bv, c, 4, 4, 1, (int)sa, 1, (int)sb);
}
__device__ __forceinline__ f32x16 mfma_mx32(const u32x4& a, uint32_t sa, const u32x4& b, uint32_t sb,
                                            const f32x16& c, std::integral_constant<int, 2>) {
  const i32x8 av = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i32x8 bv = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, bv, c, 4, 4, 2, (int)sa, 2, (int)sb);
}
__device__ __forceinline__ f32x16 mfma_mx32(const u32x4& a, uint32_t sa, const u32x4& b, uint32_t sb,
                                            const f32x16& c, std::integral_constant<int, 3>) {
  const i32x8 av = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i32x8 bv = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, bv, c, 4, 4, 3, (int)sa, 3, (int)sb);
}

struct TileLds {
  uint8_t* x[2];
  uint8_t* w[2];
  uint8_t* s[2];  // 8 scale bytes per row: activation rows, then weight rows
};

struct __attribute__((packed, aligned(2))) Scales8 {
  uint64_t v;
};
struct __attribute__((packed, aligned(2))) Out16 {
  u32x4 v;
};

// Rows row0 .. row0 + rows - 1 (at most 64 WM) of expert e, columns of tile ctile.
template <int MODE, int WM, int WN, int BUFS>
__device__ __forceinline__ void mx_tile(const MxArgs& a, const TileLds& lds, int64_t e, int64_t row0,
                                        int64_t rows, int64_t ctile) {
  constexpr int XR = 64 * WM, WR = 64 * WN;                   // rows of a stage
  constexpr int NJ = MODE == MODE_GATEUP ? WN / 2 : WN;       // output blocks of a wave's columns
  static_assert(MODE != MODE_GATEUP || WN % 2 == 0, "gate and up blocks pair up");
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l32 = lane & 31, h = lane >> 5;
  const int wx = wave & 1, ww = wave >> 1;
  const int64_t N = a.N, half = a.K / 2;
  const int32_t nb = (int32_t)(a.K / 32);
  const int32_t steps = (nb + 7) / 8, last = steps - 1;
  const int64_t n0 = ctile * (64 * NJ);

  // Stage row r of the weights: wave column ww = r / (32 WN), block j = r / 32 % WN; gate+up:
  // blocks below WN / 2 are gate channels, the others the same channels of up.
  auto weight_row = [&](int r, bool& up) __attribute__((always_inline)) {
    const int c = r / (32 * WN), j = r / 32 % WN;
    up = MODE == MODE_GATEUP && j >= NJ;
    const int64_t n = n0 + 32 * (c * NJ + (up ? j - NJ : j)) + r % 32;
    return e * N + (n < N ? n : N - 1);
  };
  auto token_row = [&](int r) __attribute__((always_inline)) {
    const int64_t g = row0 + (r < rows ? r : 0);
    return MODE == MODE_GATEUP ? (int64_t)(a.sorted_pairs[g] / a.topk) : g;
  };

  // load role: load i of wave w brings stage rows 32 i + 8 w .. + 7, lane l the piece for its row's
  // slot l % 8.  Loads go through buffer resources: a uniform base for the 32 rows and the stage, and
  // a lane offset that is the same for every load (gate+up: one per row of tokens); rows behind the
  // tile's or the matrix's end lie out of range and read zeros.
  const int piece = (lane & 7) ^ ((4 * wave + (lane >> 4)) & 7);
  const uint32_t off = (uint32_t)((8 * wave + (lane >> 3)) * (uint32_t)half + piece * 16);
  uint32_t xoff[MODE == MODE_GATEUP ? 2 * WM : 1];
  if constexpr (MODE == MODE_GATEUP) {
#pragma unroll
    for (int i = 0; i < 2 * WM; ++i)
      xoff[i] = (uint32_t)(token_row(32 * i + 8 * wave + (lane >> 3)) * half) + piece * 16;
  }
  // scale role: thread t carries the scales of activation row t and of weight row t; with fewer rows
  // than threads several carry the same (a branch would cut the loop's code in two, and the compiler
  // moves MFMAs, whose results nothing waits for, from the first part into the second)
  const int xr = tid % XR, wrow = tid % WR;
  const uint8_t* xsc = a.x_scales + token_row(xr) * nb;
  const uint8_t* wsc;
  {
    bool up;
    const int64_t r = weight_row(wrow, up);
    wsc = (up ? a.w1_scales : a.w0_scales) + r * nb;
  }
  // In the last stage of a k that is no multiple of 256 the pieces behind k are filled with the
  // stage before's: any codes do, their blocks' scales are 2^-127 on both sides, and 2^-254 times
  // 32 products of at most 36 is zero in fp32.
  const int32_t behind = (int64_t)last * kStageBytes + piece * 16 >= half ? kStageBytes : 0;

  // Load i of stage g: do_load(i, resource, lane offset).
  constexpr int NX = 2 * WM, NC = 2 * WM + 2 * WN;
  auto load_codes = [&](int32_t g, int i, auto do_load) __attribute__((always_inline)) {
    const int32_t gc = g < last ? g : last;  // stages behind the last one load it again
    // a lane's offset is never below zero: what it does not go back it goes on from the stage before
    const uint32_t on = kStageBytes - (gc == last ? (uint32_t)behind : 0u);
    const int32_t at = (gc - 1) * kStageBytes;
    auto load = [&](const uint8_t* base, int32_t bytes, uint32_t lane_off) __attribute__((always_inline)) {
      const int32_t left = bytes - at;  // ranges are below 2^31 - 128 (checked on the host)
      do_load(__builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base + at), (short)0, left > 0 ? left : 0,
                                                0x00020000),
              (int)(lane_off + on));
    };
    if (i < NX) {
      if constexpr (MODE == MODE_GATEUP)
        load(a.x_codes, (int32_t)(a.M / a.topk * half), xoff[i < NX ? i : 0]);
      else
        load(a.x_codes + (row0 + 32 * i) * half, (int32_t)((rows - 32 * i) * half), off);
    } else {
      // rows 32 (i - NX) .. + 31 of the stage: block (i - NX) % WN of wave column (i - NX) / WN
      const int c = (i - NX) / WN, j = (i - NX) % WN;
      const bool up = MODE == MODE_GATEUP && j >= NJ;
      const int64_t n = n0 + 32 * (c * NJ + (up ? j - NJ : j));
      load((up ? a.w1_codes : a.w0_codes) + (e * N + n) * half, (int32_t)((N - n) * half), off);
    }
  };
  auto stage_rows = [&](int i, auto stc) __attribute__((always_inline)) {  // where load i's rows go
    constexpr int ST = decltype(stc)::value;
    return i < NX ? lds.x[ST] + (32 * i + 8 * wave) * kStageBytes
                  : lds.w[ST] + (32 * (i - NX) + 8 * wave) * kStageBytes;
  };
  // Two buffers: a stage's codes pass through NC registers of 16 bytes per lane, in four groups: fetch
  // loads group q of stage g, put writes it to a buffer.
  u32x4 held[BUFS == 2 ? NC : 1];
  auto fetch_to = [&](u32x4* to, int32_t g, auto qc) __attribute__((always_inline)) {
    constexpr int Q = decltype(qc)::value;
#pragma unroll
    for (int i = NC * Q / 4; i < NC * (Q + 1) / 4; ++i)
      load_codes(g, i, [&](__amdgpu_buffer_rsrc_t r, int at) __attribute__((always_inline)) {
        to[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0));
      });
  };
  auto put_from = [&](const u32x4* from, auto qc, auto stc) __attribute__((always_inline)) {
    constexpr int Q = decltype(qc)::value;
#pragma unroll
    for (int i = NC * Q / 4; i < NC * (Q + 1) / 4; ++i)
      *reinterpret_cast<u32x4*>(stage_rows(i, stc) + lane * 16) = from[i];
  };
  auto fetch = [&](int32_t g, auto qc) __attribute__((always_inline)) { fetch_to(held, g, qc); };
  auto put = [&](auto qc, auto stc) __attribute__((always_inline)) { put_from(held, qc, stc); };
  // One buffer: copied to LDS without registers.
  auto copy = [&](int32_t g) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NC; ++i)
      load_codes(g, i, [&](__amdgpu_buffer_rsrc_t r, int at) __attribute__((always_inline)) {
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            r, (__attribute__((address_space(3))) void*)stage_rows(i, std::integral_constant<int, 0>{}), 16, at, 0, 0, 0);
      });
  };
  // The stage's 8 scale bytes of a row.  The last, partial stage reads the row's last 8 bytes and
  // moves the ones it needs down (k >= 256: a row has 8); blocks behind k get byte 0, a finite scale.
  struct Scales {
    uint64_t x, w;
  };
  Scales scales;
  auto load_scales = [&](int32_t g) __attribute__((always_inline)) {
    const int32_t at = 8 * g < nb - 8 ? 8 * g : nb - 8;  // also behind the last stage
    return Scales{reinterpret_cast<const Scales8*>(xsc + at)->v, reinterpret_cast<const Scales8*>(wsc + at)->v};
  };
  auto put_scales = [&](const Scales& v, int32_t g, auto stc) __attribute__((always_inline)) {
    constexpr int ST = decltype(stc)::value;
    g = g < last ? g : last;
    const int32_t over = 8 * g > nb - 8 ? 8 * (8 * g - (nb - 8)) : 0;
    *reinterpret_cast<uint64_t*>(lds.s[ST] + xr * 8) = v.x >> over;
    *reinterpret_cast<uint64_t*>(lds.s[ST] + (XR + wrow) * 8) = v.w >> over;
  };

  f32x16 acc[WM][WN];
#pragma unroll
  for (int i = 0; i < WM; ++i)
#pragma unroll
    for (int j = 0; j < WN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

  struct Frag {
    u32x4 x[WM], w[WN];
  };
  uint32_t sx[2][WM], sw[2][WN];
  // Row r's piece 4 h + s lies at 128 r + 16 ((4 h + s) ^ (r / 2 % 8)); a lane's rows are 32 apart, so
  // its addresses of slice s are one base, its low bits exclusive-or 16 s, plus constants.
  const uint32_t fslot = (uint32_t)(((4 * h) ^ ((l32 >> 1) & 7)) << 4);
  const uint32_t fw = (uint32_t)((32 * WN * ww + l32) * kStageBytes) + fslot;
  const uint32_t fx = (uint32_t)((32 * WM * wx + l32) * kStageBytes) + fslot;
  const uint32_t fsw = (uint32_t)((XR + 32 * WN * ww + l32) * 8 + 4 * h);
  const uint32_t fsx = (uint32_t)((32 * WM * wx + l32) * 8 + 4 * h);
  auto read = [&](Frag& f, int s, auto stc) __attribute__((always_inline)) {
    constexpr int ST = decltype(stc)::value;
    const uint8_t* const w = lds.w[ST] + (fw ^ (uint32_t)(s << 4));
    const uint8_t* const x = lds.x[ST] + (fx ^ (uint32_t)(s << 4));
#pragma unroll
    for (int j = 0; j < WN; ++j) f.w[j] = *reinterpret_cast<const u32x4*>(w + 32 * kStageBytes * j);
#pragma unroll
    for (int i = 0; i < WM; ++i) f.x[i] = *reinterpret_cast<const u32x4*>(x + 32 * kStageBytes * i);
  };
  auto read_scales = [&](auto stc) __attribute__((always_inline)) {
    constexpr int ST = decltype(stc)::value;
#pragma unroll
    for (int j = 0; j < WN; ++j) sw[ST][j] = *reinterpret_cast<const uint32_t*>(lds.s[ST] + fsw + 256 * j);
#pragma unroll
    for (int i = 0; i < WM; ++i) sx[ST][i] = *reinterpret_cast<const uint32_t*>(lds.s[ST] + fsx + 256 * i);
  };
  auto mma = [&](const Frag& f, auto sc, auto stc) __attribute__((always_inline)) {
    constexpr int ST = decltype(stc)::value;
#pragma unroll
    for (int i = 0; i < WM; ++i)
#pragma unroll
      for (int j = 0; j < WN; ++j)
        acc[i][j] = mfma_mx32(f.w[j], sw[ST][j], f.x[i], sx[ST][i], acc[i][j], sc);
  };
  constexpr std::integral_constant<int, 0> c0{};
  constexpr std::integral_constant<int, 1> c1{};
  constexpr std::integral_constant<int, 2> c2{};
  constexpr std::integral_constant<int, 3> c3{};

  // ---- prologue: stage 0 written and the next on its way; with two buffers the first group of
  // stage 1 is written, too, and that of stage 2 on its way; stage 0's first slice read ----
  Frag X;
  if constexpr (BUFS == 2) {
    u32x4 early[NC];
    const Scales s0 = load_scales(0), s1 = load_scales(1);
    fetch_to(early, 0, c0);
    fetch_to(early, 0, c1);
    fetch_to(early, 0, c2);
    fetch_to(early, 0, c3);
    fetch(1, c0);
    fetch(1, c1);
    fetch(1, c2);
    fetch(1, c3);
    put_scales(s0, 0, c0);
    put_from(early, c0, c0);
    put_from(early, c1, c0);
    put_from(early, c2, c0);
    put_from(early, c3, c0);
    put_scales(s1, 1, c1);
    scales = load_scales(2);
    put(c0, c1);
    fetch(2, c0);
    __syncthreads();
    read_scales(c0);
    read(X, 0, c0);
  } else {
    scales = load_scales(0);
    copy(0);
    put_scales(scales, 0, c0);
    scales = load_scales(1);
    __builtin_amdgcn_s_waitcnt(0);
    __builtin_amdgcn_s_barrier();
  }

  // ---- stage g in buffers ST = g % 2 ----
  // Each slice's MFMAs cover the next slice's fragment reads, one group's writes to the other
  // buffers (a stage ahead) and, into the registers that frees, its loads (two stages ahead): a
  // load has a whole stage to arrive, and no wait but a write's own counts it.
  // Masks: 0x8 MFMA, 0x20 loads, 0x100 LDS reads, 0x200 LDS writes.
  auto stage = [&](int32_t g, auto stc) __attribute__((always_inline)) {
    constexpr int ST = decltype(stc)::value;
    constexpr std::integral_constant<int, ST ^ 1> other{};
    constexpr int NF = WM * WN, NR = WM + WN;  // MFMAs and fragment reads of a slice
    constexpr int NP = (NC + 3) / 4;           // pieces of a group
    auto interleave = [&](auto extra) __attribute__((always_inline)) {
      constexpr int XR2 = decltype(extra)::value;  // scale reads, a write and two loads
#pragma unroll
      for (int i = 0; i < (NF > 4 ? NF : 4); ++i) {
        constexpr int each = NF >= 8 ? 1 : 4;
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        if (i * each < NR + XR2) __builtin_amdgcn_sched_group_barrier(0x100, each + (XR2 ? 1 : 0), 0);
        if (NF >= 8 ? i >= NF / 2 && i < NF / 2 + NP : true) {
          __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    Frag Y;
    __builtin_amdgcn_sched_barrier(0);
    read(Y, 1, stc);
    put(c1, other);
    fetch(g + 2, c1);
    mma(X, c0, stc);
    interleave(c0);
    read(X, 2, stc);
    put(c2, other);
    fetch(g + 2, c2);
    mma(Y, c1, stc);
    interleave(c0);
    read(Y, 3, stc);
    put(c3, other);
    fetch(g + 2, c3);
    mma(X, c2, stc);
    interleave(c0);
    // This wave's writes of stage g + 1 are done and its reads of stage g returned; after the barrier
    // that holds for every wave, so g + 1 may be read and g's buffers written.
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    read_scales(other);
    read(X, 0, other);
    put_scales(scales, g + 2, stc);
    scales = load_scales(g + 3);
    put(c0, stc);
    fetch(g + 3, c0);
    mma(Y, c3, stc);
    interleave(std::integral_constant<int, NR>{});
  };
  // One buffer: once every wave's fragments of the last slice are in registers the next stage is
  // copied over it; the CU's second workgroup multiplies meanwhile.
  auto stage1 = [&](int32_t g) __attribute__((always_inline)) {
    constexpr int NF = WM * WN;
    constexpr int NR = WM + WN;
    Frag Y;
    auto reads = [&]() __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < NF; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        if (i < NR) __builtin_amdgcn_sched_group_barrier(0x100, NF >= NR ? 1 : NR, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    __builtin_amdgcn_sched_barrier(0);
    read_scales(c0);
    read(X, 0, c0);
    __builtin_amdgcn_sched_barrier(0);
    read(Y, 1, c0);
    mma(X, c0, c0);
    reads();
    read(X, 2, c0);
    mma(Y, c1, c0);
    reads();
    read(Y, 3, c0);
    mma(X, c2, c0);
    reads();
    __builtin_amdgcn_s_waitcnt(0xC07F);  // this wave's reads of the stage have returned
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    put_scales(scales, g + 1, c0);
    scales = load_scales(g + 2);
    copy(g + 1);
    __builtin_amdgcn_sched_barrier(0);
    mma(Y, c3, c0);
    __builtin_amdgcn_s_waitcnt(0);  // the next stage is written
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
  };
  int32_t g = 0;
  if constexpr (BUFS == 2) {
    for (; g + 1 < steps; g += 2) {
      stage(g, c0);
      stage(g + 1, c1);
    }
    if (g < steps) stage(g, c0);
  } else {
    for (; g < steps; ++g) stage1(g);
  }

  // ---- epilogue: lane (l, h) holds, of each block, row l and columns 8 q + 4 h + t (register
  // 4 q + t).  bf16: after packing, v_permlane32_swap gives the lower lanes the eight columns of an
  // even q and the upper ones those of the odd q behind it, so both types leave in 16-byte pieces,
  // 32 bytes of a row together, straight from registers. ----
  auto value = [&](int i, int j, int r) __attribute__((always_inline)) {
    if constexpr (MODE == MODE_GATEUP) return silu_f32(acc[i][j][r]) * acc[i][NJ + j][r];
    else return acc[i][j][r];
  };
  const int64_t nw = n0 + 32 * NJ * ww;  // the wave's first column
  const int mw = 32 * WM * wx;           // and row of the tile
  auto store = [&](auto eb) __attribute__((always_inline)) {
    constexpr int EB = decltype(eb)::value, PE = 16 / EB;  // elements of a piece
    constexpr int NP = 16 / PE;                            // pieces of a lane's row in a block
    const int64_t pitch = a.out_stride * EB;
    const int32_t cols = (int32_t)(N - nw < 32 * NJ ? N - nw : 32 * NJ) - PE * h;  // from the lane's first
    const uint32_t lane_off = (uint32_t)(l32 * pitch) + 16 * h;
#pragma unroll
    for (int i = 0; i < WM; ++i) {
      uint8_t* const base = static_cast<uint8_t*>(a.out) + ((row0 + mw + 32 * i) * a.out_stride + nw) * EB;
      const bool row = mw + 32 * i + l32 < rows;
      u32x4 last{};  // the piece that N cuts
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          u32x4 v;
          if constexpr (EB == 2) {
            uint32_t e[2], o[2];
#pragma unroll
            for (int d = 0; d < 2; ++d) {
              e[d] = cvt_pk_bf16(value(i, j, 8 * p + 2 * d), value(i, j, 8 * p + 2 * d + 1));
              o[d] = cvt_pk_bf16(value(i, j, 8 * p + 4 + 2 * d), value(i, j, 8 * p + 5 + 2 * d));
            }
            const auto r0 = __builtin_amdgcn_permlane32_swap(e[0], o[0], false, false);
            const auto r1 = __builtin_amdgcn_permlane32_swap(e[1], o[1], false, false);
            v = (u32x4){r0[0], r1[0], r0[1], r1[1]};
          } else {
#pragma unroll
            for (int d = 0; d < 4; ++d) v[d] = __float_as_uint(value(i, j, 4 * p + d));
          }
          const int at = 32 * j + 2 * PE * p;  // first column, from the lane's
          if (row && at + PE <= cols) reinterpret_cast<Out16*>(base + lane_off + at * EB)->v = v;
          if (at < cols) last = v;
        }
      const int cut = cols > 0 ? cols % (2 * PE) : 0;  // elements of the cut piece, if below PE
      if (row && cut > 0 && cut < PE) {
#pragma unroll
        for (int t = 0; t < PE - 1; ++t)
          if (t < cut) {
            uint8_t* const dst = base + lane_off + (cols - cut + t) * EB;
            if constexpr (EB == 2) *reinterpret_cast<uint16_t*>(dst) = (uint16_t)(last[t / 2] >> (16 * (t & 1)));
            else *reinterpret_cast<uint32_t*>(dst) = last[t];
          }
      }
    }
  };
  if (MODE == MODE_GATEUP || !a.out_f32) store(c2);
  else store(std::integral_constant<int, 4>{});
}

// WM: the largest tile's; a tile with few rows left takes a smaller one.
template <int MODE, int WM, int WN, int BUFS>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(BUFS == 1 ? 2 : 1, BUFS == 1 ? 2 : WM * WN >= 8 ? 1 : 2)))
void mx_tiled_kernel(const MxArgs a, int32_t experts) {
  constexpr int XR = 64 * WM, WR = 64 * WN;
  __shared__ __attribute__((aligned(16))) uint8_t codes0[(BUFS == 1 ? XR + WR : XR) * kStageBytes];
  __shared__ __attribute__((aligned(16))) uint8_t x1[BUFS == 1 ? 16 : XR * kStageBytes];
  __shared__ __attribute__((aligned(16))) uint8_t w0[BUFS == 1 ? 16 : WR * kStageBytes];
  __shared__ __attribute__((aligned(16))) uint8_t w1[BUFS == 1 ? 16 : WR * kStageBytes];
  __shared__ __attribute__((aligned(16))) uint8_t s0[(XR + WR) * 8];
  __shared__ __attribute__((aligned(16))) uint8_t s1[BUFS == 1 ? 16 : (XR + WR) * 8];
  // (two-buffer arrays apart: the compiler tells them apart, and waits for no write to the other)
  const TileLds lds{{codes0, x1}, {BUFS == 1 ? codes0 + XR * kStageBytes : w0, w1}, {s0, s1}};
  constexpr int64_t cols = MODE == MODE_GATEUP ? 32 * WN : 64 * WN;
  const int64_t col_tiles = (a.N + cols - 1) / cols;
  int64_t r, c, e = 0, row0, rows;
  if constexpr (MODE == MODE_DENSE) {
    if (!xcd_tile(blockIdx.x, (uint32_t)((a.M + XR - 1) / XR), (uint32_t)col_tiles, r, c)) return;
    row0 = r * XR;
    rows = a.M - row0 < XR ? a.M - row0 : XR;
  } else {
    ExpertTiles tiles{a.offsets, experts, XR};
    if (!xcd_tile(blockIdx.x, (uint32_t)tiles.total(), (uint32_t)col_tiles, r, c)) return;
    tiles.find((int32_t)r, e, row0, rows);
  }
  if constexpr (WM == 4) {
    if (rows > 128) mx_tile<MODE, 4, WN, BUFS>(a, lds, e, row0, rows, c);
    else if (rows > 64) mx_tile<MODE, 2, WN, BUFS>(a, lds, e, row0, rows, c);
    else mx_tile<MODE, 1, WN, BUFS>(a, lds, e, row0, rows, c);
  } else if constexpr (WM == 2) {
    if (rows > 64) mx_tile<MODE, 2, WN, BUFS>(a, lds, e, row0, rows, c);
    else mx_tile<MODE, 1, WN, BUFS>(a, lds, e, row0, rows, c);
  } else {
    mx_tile<MODE, 1, WN, BUFS>(a, lds, e, row0, rows, c);
  }
}

template <int MODE, int WM, int WN, int BUFS>
hipError_t launch_tiles(const MxArgs& a, int64_t experts, hipStream_t s) {
  constexpr int64_t cols = MODE == MODE_GATEUP ? 32 * WN : 64 * WN;
  constexpr int64_t size = 64 * WM;
  // an expert's last tile may be partial: at most one more row tile per expert
  const int64_t row_tiles = (a.M + size - 1) / size + (MODE == MODE_DENSE ? 0 : experts);
  const int64_t wgs = (row_tiles * ((a.N + cols - 1) / cols) + 7) / 8 * 8;
  if (wgs > 0x7FFFFFFF) return hipErrorInvalidValue;
  hipLaunchKernelGGL((mx_tiled_kernel<MODE, WM, WN, BUFS>), dim3((unsigned)wgs), dim3(256), 0, s, a, (int32_t)experts);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_quantize(const void* x, int f32, int64_t n, int64_t k, uint8_t* codes,
                              uint8_t* scales, hipStream_t stream) {
  const int64_t octets = n * (k / 8);
  return launch_in_parts((octets + 255) / 256, [&](int64_t first, dim3 grid) {
    if (f32)
      hipLaunchKernelGGL(mx_quantize_kernel<float>, grid, dim3(256), 0, stream,
                         static_cast<const float*>(x), octets, codes, scales, first);
    else
      hipLaunchKernelGGL(mx_quantize_kernel<uint16_t>, grid, dim3(256), 0, stream,
                         static_cast<const uint16_t*>(x), octets, codes, scales, first);
  });
}

namespace {

// Dense products: rows in passes of 16 MT; the grid's z extent is 16 bits, so more rows take further
// launches.
template <int MT>
hipError_t stream_dense(const MxArgs& a, hipStream_t stream) {
  constexpr int64_t chunk = 65535ll * 16 * MT;
  for (int64_t r0 = 0; r0 < a.M; r0 += chunk) {
    MxArgs b = a;
    b.x_codes = a.x_codes + r0 * (a.K / 2);
    b.x_scales = a.x_scales + r0 * (a.K / 32);
    b.out = static_cast<uint8_t*>(a.out) + r0 * a.out_stride * (a.out_f32 ? 4 : 2);
    b.M = a.M - r0 < chunk ? a.M - r0 : chunk;
    const hipError_t e = launch_stream<MODE_DENSE, MT, 4>(b, 1, mx_ceil_div(b.M, 16 * MT), stream);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t product_dense(const MxArgs& a, hipStream_t stream) {
  switch (mx_dense_kernel(a.M, a.N, a.K)) {
    case MX_TILES_256: return launch_tiles<MODE_DENSE, 4, 4, 2>(a, 1, stream);
    case MX_TILES_128x256_ONE: return launch_tiles<MODE_DENSE, 2, 4, 1>(a, 1, stream);
    case MX_TILES_128x256: return launch_tiles<MODE_DENSE, 2, 4, 2>(a, 1, stream);
    case MX_TILES_128: return launch_tiles<MODE_DENSE, 2, 2, 2>(a, 1, stream);
    case MX_TILES_64: return launch_tiles<MODE_DENSE, 1, 1, 2>(a, 1, stream);
    case MX_STREAM_32: return stream_dense<2>(a, stream);
    default: return stream_dense<1>(a, stream);
  }
}

template <int MODE>
hipError_t product_experts(const MxArgs& a, int64_t experts, hipStream_t stream) {
  switch (mx_experts_kernel(MODE == MODE_GATEUP ? a.M / a.topk : 0, a.M, a.N, a.K, experts)) {
    case MX_TILES_256: return launch_tiles<MODE, 4, 4, 2>(a, experts, stream);
    case MX_TILES_128x256_ONE: return launch_tiles<MODE, 2, 4, 1>(a, experts, stream);
    case MX_TILES_128x256: return launch_tiles<MODE, 2, 4, 2>(a, experts, stream);
    case MX_TILES_128: return launch_tiles<MODE, 2, 2, 2>(a, experts, stream);
    default: return launch_stream<MODE, 1, 4>(a, experts, 1, stream);
  }
}

}  // namespace

hipError_t launch_mx_product(int mode, const MxArgs& a, int64_t experts, hipStream_t stream) {
  if (mode == MODE_GATEUP) return product_experts<MODE_GATEUP>(a, experts, stream);
  if (mode == MODE_DOWN) return product_experts<MODE_DOWN>(a, experts, stream);
  return product_dense(a, stream);
}

}  // namespace wq
