// wq_i8.hip -- products whose operands are both int8: activations with an fp32 scale per row, weights with a
// bf16 scale per output channel,
//   y[m][n] = (f32(sum_k cx[m][k] cw[n][k]) * sx[m]) * sw[n].
// The sum is exact: products of codes are at most 2^14, and k stays below 2^17, so no partial sum leaves
// int32 and any order of the sum gives the same bits.  The scales leave the sum because they belong to a
// row and a channel, so the matrix instructions run on the codes as they are stored, at twice the bf16 rate.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "wq_i8_select.hpp"
#include "wq_kernels.hpp"
#include "wq_tiles.hpp"

namespace wq {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

__device__ __forceinline__ void store_out(void* out, int f32, int64_t at, float v) {
  if (f32) reinterpret_cast<float*>(out)[at] = v;
  else reinterpret_cast<uint16_t*>(out)[at] = (uint16_t)f32_to_bf16_bits(v);
}

// ---------------------------------------------------------------------------------------------
// Few rows: the weights stream from memory straight into v_mfma_i32_16x16x64_i8 operands.  Lane l supplies
// row l % 16 of A (column of B) and 16 codes; it receives D[4 (l / 16) + i][l % 16].  Instruction i
// of a step of 256 along k takes 64 of them, lane group q = l / 16 the codes 16 q .. 16 q + 15: a load touches
// one 64-byte line of every row.
// Bound by the operands' way: one round trip to memory and what a CU takes in, weights and (16 or 32 rows for every 16
// columns) as many or twice as many bytes of activations again, where the workgroups are few (1, 8, 32 x 4096, k 4096:
// 6.0, 6.9, 9.4 us; 32 rows: 64 KB + 128 KB a CU), memory where they are many (32 tokens, top-8 of 64 experts, 3584 x 8192:
// gate+up 600 us, 6.2 TB/s; 8192 x 3584: down 316).  More waves (8, 16) gain nothing.
// ---------------------------------------------------------------------------------------------
__device__ __forceinline__ i32x4 mfma16(const u32x4& a, const u32x4& b, const i32x4& c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
}

// A lane's four pieces of a step, zeros behind the row's end (k is a multiple of 64, a piece's 64 codes are all
// there or none).  codes: the row's first piece of this lane.
struct Part {
  u32x4 c[4];
};
__device__ __forceinline__ void load_part(Part& p, const int8_t* codes, int32_t at, int32_t k) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    p.c[i] = at + 64 * i < k ? *reinterpret_cast<const u32x4*>(codes + at + 64 * i) : (u32x4){0, 0, 0, 0};
}

// One workgroup of KS waves computes 16 MT rows by 16 columns (gate+up: of both matrices); its waves split
// the steps along k and their sums meet in LDS.
template <int MODE, int MT, int KS>
__global__ __launch_bounds__(64 * KS) void i8_stream_kernel(const I8Args a) {
  constexpr int NM = MODE == MODE_GATEUP ? 2 : 1;
  __shared__ i32x4 red[KS][NM * MT][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nl = lane & 15, q = lane >> 4;
  const int64_t N = a.N;
  const int32_t K = (int32_t)a.K;
  const int32_t steps = (K + 255) / 256;
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
  const int8_t* wc[NM];
  float sw[NM];
  wc[0] = a.w0_codes + wr * K + 16 * q;
  sw[0] = bf16_bits_to_f32(a.w0_scales[wr]);
  if constexpr (NM == 2) {
    wc[1] = a.w1_codes + wr * K + 16 * q;
    sw[1] = bf16_bits_to_f32(a.w1_scales[wr]);
  }

  for (int64_t ms = 0; ms < m_total; ms += 16 * MT) {
    const int64_t left = m_total - ms;
    const int8_t* xc[MT];
    float sx[MT];  // of row 16 t + nl
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const int64_t r = m_base + ms + (16 * t + nl < left ? 16 * t + nl : 0);
      int64_t src = r;
      if constexpr (MODE == MODE_GATEUP) src = a.sorted_pairs[r] / a.topk;
      xc[t] = a.x_codes + src * K + 16 * q;
      sx[t] = a.x_scales[src];
    }
    i32x4 acc[NM][MT];
#pragma unroll
    for (int j = 0; j < NM; ++j)
#pragma unroll
      for (int t = 0; t < MT; ++t) acc[j][t] = (i32x4){0, 0, 0, 0};
    struct Step {
      Part w[NM], x[MT];
    };
    auto load = [&](Step& p, int32_t s) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < NM; ++j) load_part(p.w[j], wc[j], 256 * s, K);
#pragma unroll
      for (int t = 0; t < MT; ++t) load_part(p.x[t], xc[t], 256 * s, K);
    };
    auto multiply = [&](const Step& p) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < NM; ++j)
#pragma unroll
          for (int t = 0; t < MT; ++t) acc[j][t] = mfma16(p.x[t].c[i], p.w[j].c[i], acc[j][t]);
    };
    if constexpr (MODE == MODE_DENSE) {
      // few workgroups: four steps on their way (2 / 3 / 4: 1 x 4096, k 4096 6.6 / 6.4 / 6.0; 20 x 4096, k 8192 14.2 /
      // 13.9 / 13.5)
      constexpr int AHEAD = 4;
      Step held[AHEAD];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i)
        if (s_begin + i < s_end) load(held[i], s_begin + i);
      for (int32_t s = s_begin; s < s_end; s += AHEAD) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
          if (s + i < s_end) {
            multiply(held[i]);
            if (s + i + AHEAD < s_end) load(held[i], s + i + AHEAD);
          }
      }
    } else if (s_begin < s_end) {
      // many: two, which leave room for more waves (2 / 3 / 4: 32 tokens, gate+up 598 / 602 / 690)
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
      i32x4 g = red[0][t][lane], u = red[0][(NM - 1) * MT + t][lane];
#pragma unroll
      for (int p = 1; p < KS; ++p) {
        g += red[p][t][lane];
        if constexpr (NM == 2) u += red[p][MT + t][lane];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t m = 16 * t + 4 * q + i;
        const float s = __shfl(sx[t], 4 * q + i);  // lane 4 q + i holds that row's scale
        if (!nvalid || m >= left) continue;
        const int64_t at = (m_base + ms + m) * N + nrow;
        const float v = (float)g[i] * s * sw[0];
        if constexpr (MODE == MODE_GATEUP) store_out(a.out, 0, at, silu_f32(v) * ((float)u[i] * s * sw[NM - 1]));
        else store_out(a.out, a.out_f32, at, v);
      }
    }
  }
}

template <int MODE, int MT, int KS>
hipError_t launch_stream(const I8Args& a, int64_t gy, int64_t gz, hipStream_t s) {
  hipLaunchKernelGGL((i8_stream_kernel<MODE, MT, KS>),
                     dim3((unsigned)((a.N + 15) / 16), (unsigned)gy, (unsigned)gz), dim3(64 * KS), 0,
                     s, a);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------------------------
// Tens to hundreds of rows and few outputs: 32 rows by 16 columns a workgroup, where 64 x 64 tiles would leave most
// CUs without one.  A CU takes in 26 to 45 KB/us, both operands counted, and each workgroup reads all of k for its rows
// and columns, so the columns are cut so finely that every CU takes in some, though the rows, which L2 holds, are read
// again by each: 64 x 2560, k 8192 19.7 us (22.1 with 64 x 64
// tiles, 24.5 streaming), 128 x 2048, k 4096 8.9 (9.9, 13.4).
//   * Stages of 256 bytes of a row, 16 lanes a row; two of them on their way in registers, two in LDS, 16-byte
//     piece p of row r in slot p ^ (r % 16): writes and fragment reads are free of bank conflicts.
//   * Wave v multiplies the codes 64 v .. 64 v + 63 of every stage, so each piece of LDS is read once; the waves'
//     sums meet in LDS at the end.
//   * The weights are the A operand: a lane ends with four consecutive outputs of one row.
// ---------------------------------------------------------------------------------------------
__global__ __launch_bounds__(256) void i8_narrow_kernel(const I8Args a) {
  constexpr int MT = 2, XR = 16 * MT, WR = 16, NC = MT + 1;  // rows of a stage, loads of a thread and stage
  constexpr int kRow = 256;                                  // bytes of a row of a stage
  __shared__ __attribute__((aligned(16))) uint8_t buf0[(XR + WR) * kRow], buf1[(XR + WR) * kRow];
  const int tid = threadIdx.x, lane = tid & 63, nl = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int32_t K = (int32_t)a.K, stages = (K + kRow - 1) / kRow, last = stages - 1;
  const int64_t n0 = (int64_t)blockIdx.x * WR, m0 = (int64_t)blockIdx.y * XR;
  const int rows = (int)(a.M - m0 < XR ? a.M - m0 : XR), cols = (int)(a.N - n0 < WR ? a.N - n0 : WR);

  // load role: row tid / 16 of 16 (load i: rows 16 i .. of the stage, activations and then weights), piece tid % 16.
  // Rows behind the matrices' ends and pieces behind k lie out of their resource's range and read zeros.
  const int r = tid >> 4, piece = tid & 15;
  const uint32_t off = (uint32_t)r * (uint32_t)K + piece * 16;
  const bool behind = last * kRow + piece * 16 >= K;
  const uint32_t to = (uint32_t)(r * kRow + ((piece ^ r) << 4));
  auto fetch = [&](u32x4 (&v)[NC], int32_t g) __attribute__((always_inline)) {
    const int at = (int)((off + (uint32_t)g * kRow) | (g == last && behind ? 0x7FFFFFF0u : 0u));
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int8_t* const base = i < MT ? a.x_codes + (m0 + 16 * i) * K : a.w0_codes + n0 * K;
      const int have = i < MT ? rows - 16 * i : cols;
      const auto rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t*>(base), (short)0,
                                                          have <= 0 ? 0 : (have < 16 ? have : 16) * K, 0x00020000);
      v[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rsrc, at, 0, 0));
    }
  };
  auto put = [&](const u32x4 (&v)[NC], uint8_t* buf) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NC; ++i) *reinterpret_cast<u32x4*>(buf + to + i * 16 * kRow) = v[i];
  };

  i32x4 acc[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) acc[t] = (i32x4){0, 0, 0, 0};
  const uint32_t from = (uint32_t)(nl * kRow + (((4 * wave + q) ^ nl) << 4));
  u32x4 even[NC], odd[NC];
  fetch(even, 0);
  if (1 < stages) fetch(odd, 1);
  put(even, buf0);
  if (2 < stages) fetch(even, 2);
  __syncthreads();
  // Stage g in `here`; the next one goes to `there` from the registers that hold it, which take stage g + 3.
  auto stage = [&](int32_t g, u32x4 (&next)[NC], const uint8_t* here, uint8_t* there) __attribute__((always_inline)) {
    u32x4 f[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) f[i] = *reinterpret_cast<const u32x4*>(here + from + i * 16 * kRow);
    if (g < last) put(next, there);
    if (g + 3 < stages) fetch(next, g + 3);
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[t] = mfma16(f[MT], f[t], acc[t]);
    __syncthreads();  // stage g has been read, stage g + 1 is written
  };
  for (int32_t g = 0; g < stages; g += 2) {
    stage(g, odd, buf0, buf1);
    if (g + 1 < stages) stage(g + 1, even, buf1, buf0);
  }

  i32x4* const red = reinterpret_cast<i32x4*>(buf0);  // [wave][row tile][lane]
#pragma unroll
  for (int t = 0; t < MT; ++t) red[(wave * MT + t) * 64 + lane] = acc[t];
  __syncthreads();
  const int row = 16 * wave + nl;  // row tile t is finished by wave t
  if (wave >= MT || row >= rows) return;
  i32x4 v = red[wave * 64 + lane];
#pragma unroll
  for (int w = 1; w < 4; ++w) v += red[(w * MT + wave) * 64 + lane];
  const float sx = a.x_scales[m0 + row];
  const int64_t n = n0 + 4 * q, at = (m0 + row) * a.N + n;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (n + i < a.N) store_out(a.out, a.out_f32, at + i, (float)v[i] * sx * bf16_bits_to_f32(a.w0_scales[n + i]));
}

hipError_t launch_narrow(const I8Args& a, hipStream_t s) {
  hipLaunchKernelGGL(i8_narrow_kernel, dim3((unsigned)i8_ceil_div(a.N, 16), (unsigned)i8_ceil_div(a.M, 32)), dim3(256), 0,
                     s, a);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------------------------
// Many rows: tiles staged in LDS.
//
// One workgroup of 4 waves, one per SIMD, computes 64 WM rows by 64 WN columns (256 x 256 for the
// large products); each wave 32 WM by 32 WN of them, as WM x WN blocks of 32 x 32 in registers.  k
// advances 128 per stage.
//   * The weights are the A operand of v_mfma_i32_32x32x32_i8 and the activations the B operand, so a lane
//     ends with four consecutive outputs of one row.  Lane (l, h) supplies row l and 16 codes: slice s of a
//     stage takes piece 4 h + s, so a lane's four pieces are 64 contiguous bytes.
//   * Rows of a stage are 128 bytes in LDS, 16-byte piece p of row r in slot p ^ (r / 2 % 8), which keeps
//     the fragment reads free of bank conflicts; 8 lanes load a row.
//   * Two buffers; codes pass through registers, which hold a third stage on its way (64 x 64 tiles: four more), so
//     loads and LDS writes spread over the whole stage.
//   * The next slice's fragments are read under the current slice's MFMAs; the last slice of a stage is
//     multiplied after the barrier that ends the stage, over the next stage's first reads.
//   * The scales of the tile's rows and channels go to LDS at its start and meet the sums at its end.
//   * 4096 x 8192, k 8192: 222 to 231 us, 2.38 to 2.48 PFLOP/s, bound by power: the matrix units are 0.76 busy at a
//     clock that falls to about 1.5 GHz.  8192 x 8192: 435 to 450 us, 2.44 to 2.53.
//   * Experts (64, top-8 of 4096 tokens): gate+up 3584 x 8192 1955 to 1993 us (0.66 busy), down 8192 x 3584 1050 to
//     1095 (0.56 busy): a tile's start and end, which do no matrix work, over its 64 or 28 stages, and the tiles that
//     routing cuts short (exactly 512 rows an expert: down 980 to 990; one expert: 863).  Such tiles take a height of 64, 128,
//     192 or 256 rows.
// Results of rows behind a ragged tile's end and of columns behind N are not stored.
// ---------------------------------------------------------------------------------------------
constexpr int kStageBytes = 128;  // codes of one row of a stage

__device__ __forceinline__ i32x16 mfma32(const u32x4& a, const u32x4& b, const i32x16& c) {
  return __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
}

struct TileLds {
  uint8_t* x[2];
  uint8_t* w[2];
  float* sx;  // scales of the activation rows
  float* sw;  // and of the weight rows
};

// A wave's WM x NJ blocks of 32 x 32 outputs, rows row0 .. row0 + rows - 1 (more than 32 WM: all of them)
// and columns n0 .. below N, to `out` in elements of EB bytes (2: bf16, 4: fp32).  value(i, j, r) is lane
// (l, h)'s value of block (i, j): row l, columns 8 q + 4 h + t in register r = 4 q + t.  bf16: after packing,
// v_permlane32_swap gives the lower lanes the eight columns of an even q and the upper ones those of the
// odd q behind it, so both types leave in 16-byte pieces, 32 bytes of a row together.
struct __attribute__((packed, aligned(2))) Out16 {
  u32x4 v;
};

template <int WM, int NJ, int EB, class Value>
__device__ __forceinline__ void store_blocks(void* out, int64_t stride, int64_t row0, int64_t rows, int64_t n0,
                                             int64_t N, Value value) {
  constexpr int PE = 16 / EB;  // elements of a piece
  constexpr int NP = 16 / PE;  // pieces of a lane's row in a block
  const int lane = threadIdx.x & 63, l32 = lane & 31, h = lane >> 5;
  const int64_t pitch = stride * EB;
  const int32_t cols = (int32_t)(N - n0 < 32 * NJ ? N - n0 : 32 * NJ) - PE * h;  // from the lane's first
  const uint32_t lane_off = (uint32_t)(l32 * pitch) + 16 * h;
#pragma unroll
  for (int i = 0; i < WM; ++i) {
    uint8_t* const base = static_cast<uint8_t*>(out) + ((row0 + 32 * i) * stride + n0) * EB;
    const bool row = 32 * i + l32 < rows;
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
}
// Rows row0 .. row0 + rows - 1 (at most 64 WM) of expert e, columns of tile ctile.
template <int MODE, int WM, int WN>
__device__ __forceinline__ void i8_tile(const I8Args& a, const TileLds& lds, int64_t e, int64_t row0,
                                        int64_t rows, int64_t ctile) {
  constexpr int XR = 64 * WM, WR = 64 * WN;                   // rows of a stage
  constexpr int NJ = MODE == MODE_GATEUP ? WN / 2 : WN;       // output blocks of a wave's columns
  static_assert(MODE != MODE_GATEUP || WN % 2 == 0, "gate and up blocks pair up");
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l32 = lane & 31, h = lane >> 5;
  const int wx = wave & 1, ww = wave >> 1;
  const int64_t N = a.N;
  const int32_t K = (int32_t)a.K;
  const int32_t steps = (K + kStageBytes - 1) / kStageBytes, last = steps - 1;
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
  // slot l % 8.  Loads go through buffer resources: a uniform base for the 32 rows, and a lane
  // offset that is the same for every load (gate+up: one per row of tokens) plus the stage's; rows behind the
  // tile's or the matrix's end lie out of range and read zeros.
  const int piece = (lane & 7) ^ ((4 * wave + (lane >> 4)) & 7);
  const uint32_t off = (uint32_t)((8 * wave + (lane >> 3)) * (uint32_t)K + piece * 16);
  uint32_t xoff[MODE == MODE_GATEUP ? 2 * WM : 1];
  if constexpr (MODE == MODE_GATEUP) {
#pragma unroll
    for (int i = 0; i < 2 * WM; ++i)
      xoff[i] = (uint32_t)(token_row(32 * i + 8 * wave + (lane >> 3)) * K) + piece * 16;
  }
  // In the last stage of a k that is no multiple of 128 the pieces behind k are out of range as well, on
  // both sides: their lanes' offsets are set to 2^31 - 16, which no resource holds.
  const bool behind = last * kStageBytes + piece * 16 >= K;

  // Load i of stage g: do_load(i, resource, lane offset).
  constexpr int NX = 2 * WM, NC = 2 * WM + 2 * WN;
  auto load_codes = [&](int32_t g, int i, auto do_load) __attribute__((always_inline)) {
    const int32_t gc = g < last ? g : last;  // stages behind the last one load it again
    const uint32_t at = (uint32_t)gc * kStageBytes, out = gc == last && behind ? 0x7FFFFFF0u : 0u;
    // the resources stay as they are from stage to stage; ranges are below 2^31 - 1024 (checked on the host)
    auto load = [&](const int8_t* base, int32_t bytes, uint32_t lane_off) __attribute__((always_inline)) {
      do_load(__builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t*>(base), (short)0, bytes > 0 ? bytes : 0, 0x00020000),
              (int)((lane_off + at) | out));
    };
    if (i < NX) {
      if constexpr (MODE == MODE_GATEUP)
        load(a.x_codes, (int32_t)(a.M / a.topk * K), xoff[i < NX ? i : 0]);
      else
        load(a.x_codes + (row0 + 32 * i) * K, (int32_t)((rows - 32 * i) * K), off);
    } else {
      // rows 32 (i - NX) .. + 31 of the stage: block (i - NX) % WN of wave column (i - NX) / WN
      const int c = (i - NX) / WN, j = (i - NX) % WN;
      const bool up = MODE == MODE_GATEUP && j >= NJ;
      const int64_t n = n0 + 32 * (c * NJ + (up ? j - NJ : j));
      load((up ? a.w1_codes : a.w0_codes) + (e * N + n) * K, (int32_t)((N - n) * K), off);
    }
  };
  auto stage_rows = [&](int i, auto stc) __attribute__((always_inline)) {  // where load i's rows go
    constexpr int ST = decltype(stc)::value;
    return i < NX ? lds.x[ST] + (32 * i + 8 * wave) * kStageBytes
                  : lds.w[ST] + (32 * (i - NX) + 8 * wave) * kStageBytes;
  };
  // A stage's codes pass through NC registers of 16 bytes per lane, in four groups: fetch loads group q of
  // stage g, put writes it to a buffer.  64 x 64 tiles, whose stages are short, have four sets of them, so that a
  // load has four stages to arrive (1, 2, 4, 8 sets: 128 x 4096, k 4096 19.4, 15.0, 13.0, 13.8 us; 64 x 8192, k 8192 38,
  // 28, 24.5, 25.2); larger ones gain nothing (128 x 128, 4 sets: 1024 x 4096 23.5 / 24.4, 256 x 256, 2: 224 / 226).
  constexpr int SETS = WM * WN == 1 ? 4 : 1;
  u32x4 held[SETS][NC];
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
  auto fetch = [&](int32_t g, auto qc, int set) __attribute__((always_inline)) { fetch_to(held[set], g, qc); };
  auto put = [&](auto qc, auto stc, int set) __attribute__((always_inline)) { put_from(held[set], qc, stc); };
  auto load_scales = [&]() __attribute__((always_inline)) {
    for (int r = tid; r < XR; r += 256) lds.sx[r] = a.x_scales[token_row(r)];
    for (int r = tid; r < WR; r += 256) {
      bool up;
      const int64_t n = weight_row(r, up);
      lds.sw[r] = bf16_bits_to_f32((up ? a.w1_scales : a.w0_scales)[n]);
    }
  };

  i32x16 acc[WM][WN];
#pragma unroll
  for (int i = 0; i < WM; ++i)
#pragma unroll
    for (int j = 0; j < WN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;

  struct Frag {
    u32x4 x[WM], w[WN];
  };
  // Row r's piece 4 h + s lies at 128 r + 16 ((4 h + s) ^ (r / 2 % 8)); a lane's rows are 32 apart, so
  // its addresses of slice s are one base, its low bits exclusive-or 16 s, plus constants.
  const uint32_t fslot = (uint32_t)(((4 * h) ^ ((l32 >> 1) & 7)) << 4);
  const uint32_t fw = (uint32_t)((32 * WN * ww + l32) * kStageBytes) + fslot;
  const uint32_t fx = (uint32_t)((32 * WM * wx + l32) * kStageBytes) + fslot;
  auto read = [&](Frag& f, int s, auto stc) __attribute__((always_inline)) {
    constexpr int ST = decltype(stc)::value;
    const uint8_t* const w = lds.w[ST] + (fw ^ (uint32_t)(s << 4));
    const uint8_t* const x = lds.x[ST] + (fx ^ (uint32_t)(s << 4));
#pragma unroll
    for (int j = 0; j < WN; ++j) f.w[j] = *reinterpret_cast<const u32x4*>(w + 32 * kStageBytes * j);
#pragma unroll
    for (int i = 0; i < WM; ++i) f.x[i] = *reinterpret_cast<const u32x4*>(x + 32 * kStageBytes * i);
  };
  auto mma = [&](const Frag& f) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < WM; ++i)
#pragma unroll
      for (int j = 0; j < WN; ++j) acc[i][j] = mfma32(f.w[j], f.x[i], acc[i][j]);
  };
  constexpr std::integral_constant<int, 0> c0{};
  constexpr std::integral_constant<int, 1> c1{};
  constexpr std::integral_constant<int, 2> c2{};
  constexpr std::integral_constant<int, 3> c3{};

  // ---- prologue: stage 0 and the first group of stage 1 written, the rest of stages 1 .. SETS and the first group
  // of the one behind on their way; stage 0's first slice read ----
  Frag X;
  {
    u32x4 early[NC];
    fetch_to(early, 0, c0);
    fetch_to(early, 0, c1);
    fetch_to(early, 0, c2);
    fetch_to(early, 0, c3);
#pragma unroll
    for (int i = 1; i <= SETS; ++i) {
      fetch(i, c0, i % SETS);
      fetch(i, c1, i % SETS);
      fetch(i, c2, i % SETS);
      fetch(i, c3, i % SETS);
    }
    load_scales();
    put_from(early, c0, c0);
    put_from(early, c1, c0);
    put_from(early, c2, c0);
    put_from(early, c3, c0);
    put(c0, c1, 1 % SETS);
    fetch(SETS + 1, c0, 1 % SETS);
    __syncthreads();
    read(X, 0, c0);
  }

  // ---- stage g, u = g % max(SETS, 2), in buffers ST = g % 2 ----
  // Each slice's MFMAs cover the next slice's fragment reads, one group's writes to the other
  // buffers (a stage ahead) and, into the registers that frees, its loads (1 + SETS stages ahead): a
  // load has SETS stages to arrive, and no wait but a write's own counts it.
  // Masks: 0x8 MFMA, 0x20 loads, 0x100 LDS reads, 0x200 LDS writes.
  auto stage = [&](int32_t g, auto uc) __attribute__((always_inline)) {
    constexpr int u = decltype(uc)::value, ST = u % 2, one = (u + 1) % SETS, two = (u + 2) % SETS;
    constexpr std::integral_constant<int, ST> stc{};
    constexpr std::integral_constant<int, ST ^ 1> other{};
    constexpr int NF = WM * WN, NR = WM + WN;  // MFMAs and fragment reads of a slice
    constexpr int NP = (NC + 3) / 4;           // pieces of a group
    auto interleave = [&]() __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < (NF > 4 ? NF : 4); ++i) {
        constexpr int each = NF >= 8 ? 1 : 4;
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        if (i * each < NR) __builtin_amdgcn_sched_group_barrier(0x100, each, 0);
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
    put(c1, other, one);
    fetch(g + 1 + SETS, c1, one);
    mma(X);
    interleave();
    read(X, 2, stc);
    put(c2, other, one);
    fetch(g + 1 + SETS, c2, one);
    mma(Y);
    interleave();
    read(Y, 3, stc);
    put(c3, other, one);
    fetch(g + 1 + SETS, c3, one);
    mma(X);
    interleave();
    // This wave's writes of stage g + 1 are done and its reads of stage g returned; after the barrier
    // that holds for every wave, so g + 1 may be read and g's buffers written.
    __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    read(X, 0, other);
    put(c0, stc, two);
    fetch(g + 2 + SETS, c0, two);
    mma(Y);
    interleave();
  };
  constexpr int U = SETS > 2 ? 4 : 2;
  int32_t g = 0;
  for (; g + U <= steps; g += U) {
    stage(g, c0);
    stage(g + 1, c1);
    if constexpr (U == 4) {
      stage(g + 2, c2);
      stage(g + 3, c3);
    }
  }
  if (g < steps) stage(g, c0);
  if constexpr (U == 4) {
    if (g + 1 < steps) stage(g + 1, c1);
    if (g + 2 < steps) stage(g + 2, c2);
  }

  // ---- epilogue, straight from registers ----
  float sx[WM];
  f32x4 sw[WN][4];
#pragma unroll
  for (int i = 0; i < WM; ++i) sx[i] = lds.sx[32 * (WM * wx + i) + l32];
#pragma unroll
  for (int j = 0; j < WN; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q) sw[j][q] = *reinterpret_cast<const f32x4*>(lds.sw + 32 * (WN * ww + j) + 8 * q + 4 * h);
  auto scaled = [&](int i, int j, int r) __attribute__((always_inline)) {
    return (float)acc[i][j][r] * sx[i] * sw[j][r / 4][r % 4];
  };
  auto value = [&](int i, int j, int r) __attribute__((always_inline)) {
    if constexpr (MODE == MODE_GATEUP) return silu_f32(scaled(i, j, r)) * scaled(i, NJ + j, r);
    else return scaled(i, j, r);
  };
  const int64_t nw = n0 + 32 * NJ * ww;  // the wave's first column
  const int mw = 32 * WM * wx;           // and row of the tile
  if (MODE == MODE_GATEUP || !a.out_f32) store_blocks<WM, NJ, 2>(a.out, N, row0 + mw, rows - mw, nw, N, value);
  else store_blocks<WM, NJ, 4>(a.out, N, row0 + mw, rows - mw, nw, N, value);
}

// WM: the largest tile's; a tile with few rows left takes a smaller one.
template <int MODE, int WM, int WN>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, WM * WN >= 8 ? 1 : 2)))
void i8_tiled_kernel(const I8Args a, int32_t experts) {
  constexpr int XR = 64 * WM, WR = 64 * WN;
  // (arrays apart: the compiler tells them apart, and waits for no write to the other buffer)
  __shared__ __attribute__((aligned(16))) uint8_t x0[XR * kStageBytes], x1[XR * kStageBytes];
  __shared__ __attribute__((aligned(16))) uint8_t w0[WR * kStageBytes], w1[WR * kStageBytes];
  __shared__ __attribute__((aligned(16))) float sx[XR], sw[WR];
  const TileLds lds{{x0, x1}, {w0, w1}, sx, sw};
  constexpr int64_t cols = MODE == MODE_GATEUP ? 32 * WN : 64 * WN;
  const int64_t col_tiles = (a.N + cols - 1) / cols;
  int64_t r, c, e = 0, row0, rows;
  if constexpr (MODE == MODE_DENSE) {
    if (!xcd_tile(blockIdx.x, (uint32_t)((a.M + XR - 1) / XR), (uint32_t)col_tiles, r, c)) return;
    row0 = r * XR;
    rows = a.M - row0 < XR ? a.M - row0 : XR;
  } else {
    ExpertTiles tiles{a.offsets, experts, XR};
    const uint32_t row_tiles = (uint32_t)tiles.total();
    if (WM == 4 ? !xcd_block_tile(blockIdx.x, row_tiles, (uint32_t)col_tiles, r, c)
                : !xcd_tile(blockIdx.x, row_tiles, (uint32_t)col_tiles, r, c))
      return;
    tiles.find((int32_t)r, e, row0, rows);
  }
  if constexpr (WM == 4) {
    if (rows > 192) i8_tile<MODE, 4, WN>(a, lds, e, row0, rows, c);
    else if (rows > 128) i8_tile<MODE, 3, WN>(a, lds, e, row0, rows, c);
    else if (rows > 64) i8_tile<MODE, 2, WN>(a, lds, e, row0, rows, c);
    else i8_tile<MODE, 1, WN>(a, lds, e, row0, rows, c);
  } else if constexpr (WM == 2) {
    if (rows > 64) i8_tile<MODE, 2, WN>(a, lds, e, row0, rows, c);
    else i8_tile<MODE, 1, WN>(a, lds, e, row0, rows, c);
  } else {
    i8_tile<MODE, 1, WN>(a, lds, e, row0, rows, c);
  }
}

template <int MODE, int WM, int WN>
hipError_t launch_tiles(const I8Args& a, int64_t experts, hipStream_t s) {
  constexpr int64_t cols = MODE == MODE_GATEUP ? 32 * WN : 64 * WN;
  constexpr int64_t size = 64 * WM;
  // an expert's last tile may be partial: at most one more row tile per expert
  const int64_t row_tiles = (a.M + size - 1) / size + (MODE == MODE_DENSE ? 0 : experts);
  const int64_t col_tiles = (a.N + cols - 1) / cols;
  const int64_t wgs = MODE != MODE_DENSE && WM == 4 ? block_grid(row_tiles, col_tiles) : (row_tiles * col_tiles + 7) / 8 * 8;
  if (wgs >= (1ll << 24)) return hipErrorInvalidValue;
  hipLaunchKernelGGL((i8_tiled_kernel<MODE, WM, WN>), dim3((unsigned)wgs), dim3(256), 0, s, a, (int32_t)experts);
  return hipGetLastError();
}

// Dense products: rows in passes of 16 MT; the grid's z extent is 16 bits, so more rows take further
// launches.
template <int MT>
hipError_t stream_dense(const I8Args& a, hipStream_t stream) {
  constexpr int64_t chunk = 65535ll * 16 * MT;
  for (int64_t r0 = 0; r0 < a.M; r0 += chunk) {
    I8Args b = a;
    b.x_codes = a.x_codes + r0 * a.K;
    b.x_scales = a.x_scales + r0;
    b.out = static_cast<uint8_t*>(a.out) + r0 * a.N * (a.out_f32 ? 4 : 2);
    b.M = a.M - r0 < chunk ? a.M - r0 : chunk;
    const hipError_t e = launch_stream<MODE_DENSE, MT, 4>(b, 1, i8_ceil_div(b.M, 16 * MT), stream);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t product_dense(const I8Args& a, hipStream_t stream) {
  switch (i8_dense_kernel(a.M, a.N, a.K)) {
    case I8_TILES_256: return launch_tiles<MODE_DENSE, 4, 4>(a, 1, stream);
    case I8_TILES_128x256: return launch_tiles<MODE_DENSE, 2, 4>(a, 1, stream);
    case I8_TILES_128: return launch_tiles<MODE_DENSE, 2, 2>(a, 1, stream);
    case I8_TILES_64: return launch_tiles<MODE_DENSE, 1, 1>(a, 1, stream);
    case I8_NARROW: return launch_narrow(a, stream);
    case I8_STREAM_32: return stream_dense<2>(a, stream);
    default: return stream_dense<1>(a, stream);
  }
}

template <int MODE>
hipError_t product_experts(const I8Args& a, int64_t experts, hipStream_t stream) {
  switch (i8_experts_kernel(MODE == MODE_GATEUP ? a.M / a.topk : 0, a.M, a.N, a.K, experts)) {
    case I8_TILES_256: return launch_tiles<MODE, 4, 4>(a, experts, stream);
    case I8_TILES_128x256: return launch_tiles<MODE, 2, 4>(a, experts, stream);
    case I8_TILES_128: return launch_tiles<MODE, 2, 2>(a, experts, stream);
    default: return launch_stream<MODE, 1, 4>(a, experts, 1, stream);
  }
}

}  // namespace

hipError_t launch_i8_product(int mode, const I8Args& a, int64_t experts, hipStream_t stream) {
  if (mode == MODE_GATEUP) return product_experts<MODE_GATEUP>(a, experts, stream);
  if (mode == MODE_DOWN) return product_experts<MODE_DOWN>(a, experts, stream);
  return product_dense(a, stream);
}

}  // namespace wq
