// wq_balance.hip -- the loss that keeps a router's experts evenly loaded, with its gradient.
//
//   p = softmax(logits);  c_e = the pairs of expert e;  T = the tokens that have a pair
//   share_e = E c_e / sum c;  loss = coefficient sum_e share_e (sum_t p_te / T)
//   d_logits_te = d_loss coefficient / T * p_te (share_e - sum_j share_j p_tj)
//
// Tokens whose ids all lie outside [0, E) are padding: they count nowhere, their logits are not used and
// get a gradient of zero.  Counts are integers (their order does not matter), the sums of p meet in a fixed
// order: the same bits every run.
//
// Both read the logits once, the gradient writes as many bytes, and e^z is computed again in the gradient rather than
// kept.  A lane holds 16 values, so a token of 64 experts is 4 lanes and a wave's sums and divisions serve 16 tokens.
// Large ones in fp32 are bound by memory: 65536 x 256 loss 22.5 to 23 us in a graph (15 us, 4.6 TB/s, and the parts'
// sums), gradient 30 us (27, 5.0 TB/s, and the launch); in bf16, where half the bytes bring as many values, by the vector
// operations of a value: 65536 x 512 34 and 44 us, of which four operations of the exponential take 4.  Small ones by
// launches: 4096 x 64 bf16 9.8 us (two of them) and 4.7; 256 x 8 fp32 5.8 to 6.1 (one workgroup, no parts) and 2.9.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "wq_kernels.hpp"
#include "wq_rows.hpp"
#include "wq_wave.hpp"

namespace wq {
namespace {

constexpr int kTopE = 512;
constexpr int kLossThreads = 1024, kLossWaves = kLossThreads / 64;  // few, large workgroups: each leaves a part
constexpr int kGradThreads = 256;

// e^x for x <= 0 as 2^hi e^lo: hi is x log2 e rounded, lo = x - hi ln 2 what its rounding and log2 e's own leave
// (below 1e-5, so e^lo = 1 + lo).  Off by at most 3 * 2^-24, also where x is far from 0; 2^hi alone would be off by
// |x| 2^-24 more.  The four operations cost 0 to 4 us at 65536 tokens (256 experts fp32: loss 22.1 to 23.0 us, gradient
// as before; 512 bf16: 30 to 34, 40 to 44).  x = -inf: lo is a NaN, which fmaxf passes over, and 2^hi zero; a NaN stays
// one through 2^hi.
__device__ __forceinline__ float exp_of(float x) {
  const float hi = x * 1.44269502f, y = __builtin_amdgcn_exp2f(hi);
  const float lo = __builtin_fmaf(hi, 1.9046543e-9f, __builtin_fmaf(hi, -0.693147182f, x));
  return __builtin_fmaf(y, fmaxf(lo, -1.f), y);
}

// A token's logits in a group of L lanes, each P pieces of 16 bytes: piece q of the row in lane q % L.  Values
// behind E are -inf.
template <typename T, int L, int P>
struct Row {
  static constexpr int PE = 16 / (int)sizeof(T), N = P * PE;
  float x[P][PE];  // logits, then e^(z - max)
  float inv;       // 1 / their sum
  __device__ __forceinline__ static int expert(int p, int i) { return ((int)(threadIdx.x & (L - 1)) + L * p) * PE + i; }
  __device__ __forceinline__ void load(const T* row, int32_t experts) {
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int e = expert(p, 0);
      if (e + PE <= experts) {
        unpack(load_piece(row + e), x[p]);
      } else {
#pragma unroll
        for (int i = 0; i < PE; ++i) x[p][i] = e + i < experts ? to_f32(row[e + i]) : -INFINITY;
      }
    }
  }
  // The probabilities' error is the rounding of z - max, |z - max| 2^-24 of them, and a few 2^-24 more.  A row of
  // -inf, as which padding counts, has no probability anywhere: zeros.
  __device__ __forceinline__ void softmax(bool real) {
    if (!real) {
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int i = 0; i < PE; ++i) x[p][i] = -INFINITY;
    }
    float top = x[0][0];
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int i = 0; i < PE; ++i) top = fmaxf(top, x[p][i]);
    top = wave_max<L>(top);  // (a NaN is no maximum, and its difference stays one)
    if (top == -INFINITY) top = 0.f;
    // sums and the gradient's dot in four chains: one of 16 made the gradient's error 1.4 times as large
    float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int i = 0; i < PE; ++i) {
        x[p][i] = exp_of(x[p][i] - top);
        s[i & 3] += x[p][i];
      }
    const float sum = wave_sum<L>((s[0] + s[1]) + (s[2] + s[3]));
    inv = sum == 0.f ? 0.f : 1.f / sum;
  }
};

// A token: its logits and this lane's first ids, on their way before the token in front of it is worked on.
template <typename T, int L, int P>
struct Token {
  static constexpr int Q = 4;  // ids of a lane
  Row<T, L, P> row;
  int32_t id[Q];
  __device__ __forceinline__ void load(const T* logits, const int32_t* ids, int64_t tok, int32_t topk, int32_t experts) {
    row.load(logits + tok * experts, experts);
    const int32_t in = threadIdx.x & (L - 1);
#pragma unroll
    for (int q = 0; q < Q; ++q) id[q] = in + q * L < topk ? ids[tok * topk + in + q * L] : -1;
  }
  // Whether it has a pair (every lane of its group knows); found(e) for each of this lane's.
  template <class Found>
  __device__ __forceinline__ bool pairs(const int32_t* ids, int64_t tok, int32_t topk, int32_t experts, Found found) const {
    bool any = false;
    const auto look = [&](int32_t e) __attribute__((always_inline)) {
      if ((uint32_t)e < (uint32_t)experts) {
        any = true;
        found(e);
      }
    };
#pragma unroll
    for (int q = 0; q < Q; ++q) look(id[q]);
    for (int32_t j = (threadIdx.x & (L - 1)) + Q * L; j < topk; j += L) look(ids[tok * topk + j]);
    return wave_join<L>(any ? 1u : 0u, [](uint32_t a, uint32_t b) __attribute__((always_inline)) { return a | b; }) != 0;
  }
};

// The sum over the lanes that hold the same place in the groups of L of a wave.
template <int L>
__device__ __forceinline__ float across(float v) {
  const auto turned = [](float f, auto c) __attribute__((always_inline)) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp((int)__float_as_uint(f), decltype(c)::value, 0xF, 0xF, true));
  };
  if constexpr (L <= 1) v += turned(v, std::integral_constant<int, 0xB1>{});   // lane ^ 1
  if constexpr (L <= 2) v += turned(v, std::integral_constant<int, 0x4E>{});   // lane ^ 2
  if constexpr (L <= 8) v += turned(v, std::integral_constant<int, 0x128>{});  // 8 lanes on, in the 16
  if constexpr (L <= 4) v += turned(v, std::integral_constant<int, 0x124>{});  // 4 lanes on
  if constexpr (L <= 16) {
    const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
  }
  if constexpr (L <= 32) {
    const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
  }
  return v;
}

// loss and counts[experts] from every thread's sum of c_e (its experts' sums of p) and of c_e.
__device__ __forceinline__ void conclude(double dot, int64_t all, int64_t tokens, int32_t experts, float coefficient,
                                         float* loss, double* meet, int64_t* meet_n) {
  for (int d = 32; d >= 1; d >>= 1) {
    dot += __shfl_xor(dot, d);
    all += __shfl_xor(all, d);
  }
  if ((threadIdx.x & 63) == 0) {
    meet[threadIdx.x >> 6] = dot;
    meet_n[threadIdx.x >> 6] = all;
  }
  __syncthreads();
  if (threadIdx.x >= 64) return;
  dot = threadIdx.x < kLossWaves ? meet[threadIdx.x] : 0.0;
  all = threadIdx.x < kLossWaves ? meet_n[threadIdx.x] : 0;
  for (int d = kLossWaves / 2; d >= 1; d >>= 1) {
    dot += __shfl_xor(dot, d);
    all += __shfl_xor(all, d);
  }
  if (threadIdx.x != 0) return;
  // no token with a pair: no loss
  *loss = tokens ? (float)((double)coefficient * experts * dot / ((double)all * (double)tokens)) : 0.f;
}

// Floats (and int32) of a part: experts + 1, the last count the tokens, in whole pieces of 16 bytes.
__host__ __device__ constexpr int32_t part_pitch(int32_t experts) { return (experts + 4) / 4 * 4; }

template <typename T, int L, int P>
__global__ __launch_bounds__(kLossThreads) void balance_kernel(const T* __restrict__ logits, const int32_t* __restrict__ ids,
                                                               int64_t t, int32_t topk, int32_t experts, float coefficient,
                                                               float* __restrict__ probs, int32_t* __restrict__ pairs,
                                                               float* __restrict__ loss, int32_t* __restrict__ counts) {
  typedef Row<T, L, P> R;
  __shared__ int32_t hist[kTopE + 1];
  __shared__ float sums[kLossWaves][L * R::N];
  __shared__ double meet[kLossWaves];
  __shared__ int64_t meet_n[kLossWaves];
  const int tid = threadIdx.x, lane = tid & 63;
  constexpr int each = kLossThreads / L;
  const int64_t stride = (int64_t)gridDim.x * each;
  int64_t tok = (int64_t)blockIdx.x * each + tid / L;
  Token<T, L, P> next;
  if (tok < t) next.load(logits, ids, tok, topk, experts);
  for (int i = tid; i <= experts; i += kLossThreads) hist[i] = 0;
  __syncthreads();
  float acc[P][R::PE];
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int i = 0; i < R::PE; ++i) acc[p][i] = 0.f;
  int32_t tokens = 0;
  for (; tok < t; tok += stride) {
    const Token<T, L, P> now = next;
    if (tok + stride < t) next.load(logits, ids, tok + stride, topk, experts);
    const bool real = now.pairs(ids, tok, topk, experts,
                                [&](int32_t e) __attribute__((always_inline)) { atomicAdd(&hist[e], 1); });
    R r = now.row;
    r.softmax(real);
    if (real && (tid & (L - 1)) == 0) ++tokens;
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int i = 0; i < R::PE; ++i) acc[p][i] = __builtin_fmaf(r.x[p][i], r.inv, acc[p][i]);
  }
  if (tokens) atomicAdd(&hist[experts], tokens);
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int i = 0; i < R::PE; ++i) {
      const float v = across<L>(acc[p][i]);
      if (lane < L) sums[tid >> 6][R::expert(p, i)] = v;
    }
  __syncthreads();
  const bool one = gridDim.x == 1;
  float* const prob = probs + (int64_t)blockIdx.x * part_pitch(experts);
  int32_t* const pair = pairs + (int64_t)blockIdx.x * part_pitch(experts);
  double dot = 0.0;
  int64_t all = 0;
  for (int e = tid; e <= experts; e += kLossThreads) {
    float s = 0.f;
    if (e < experts)
#pragma unroll
      for (int w = 0; w < kLossWaves; ++w) s += sums[w][e];
    const int32_t c = hist[e];
    if (one) {
      counts[e] = c;
      if (e < experts) {
        dot = (double)c * s;
        all = c;
      }
    } else {
      prob[e] = s;
      pair[e] = c;
    }
  }
  if (one) conclude(dot, all, hist[experts], experts, coefficient, loss, meet, meet_n);
}

// The parts' sums: a thread has four columns of a segment of eight parts (more where the workgroup has not that
// many threads), whose loads are all on their way together; segments in order, in fp64.  (As many segments as
// threads instead: 7 us where this takes 4, most of it adding them up.)
__global__ __launch_bounds__(kLossThreads) void balance_finish_kernel(const float* __restrict__ probs,
                                                                      const int32_t* __restrict__ pairs, int32_t wgs,
                                                                      int32_t experts, float coefficient,
                                                                      float* __restrict__ loss, int32_t* __restrict__ counts) {
  constexpr int U = 8;
  __shared__ double col_p[kLossThreads][4];
  __shared__ int32_t col_n[kLossThreads][4];
  __shared__ double meet[kLossWaves];
  __shared__ int64_t meet_n[kLossWaves];
  __shared__ int32_t tokens;
  const int32_t pitch = part_pitch(experts), cols = pitch / 4, most = kLossThreads / cols;
  const int32_t segs = (wgs + U - 1) / U < most ? (wgs + U - 1) / U : most;
  const int tid = threadIdx.x, seg = tid / cols, c = tid % cols;
  if (seg < segs) {
    const int32_t from = (int32_t)((int64_t)wgs * seg / segs), to = (int32_t)((int64_t)wgs * (seg + 1) / segs);
    double p[4] = {0.0, 0.0, 0.0, 0.0};
    int32_t n[4] = {0, 0, 0, 0};  // at most 2^30 pairs in all
    for (int32_t w = from; w < to; w += U) {
      f32x4 pv[U];
      u32x4 nv[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t at = (int64_t)(w + u < to ? w + u : w) * pitch + 4 * c;
        pv[u] = *reinterpret_cast<const f32x4*>(probs + at);
        nv[u] = *reinterpret_cast<const u32x4*>(pairs + at);
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (w + u < to)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            p[i] += (double)pv[u][i];
            n[i] += (int32_t)nv[u][i];
          }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      col_p[tid][i] = p[i];
      col_n[tid][i] = n[i];
    }
  }
  __syncthreads();
  double dot = 0.0;
  int64_t all = 0;
  if (tid <= experts) {
    double ps = 0.0;
    int32_t ns = 0;
#pragma unroll 4
    for (int s = 0; s < segs; ++s) {
      ps += col_p[s * cols + tid / 4][tid % 4];
      ns += col_n[s * cols + tid / 4][tid % 4];
    }
    counts[tid] = ns;
    if (tid < experts) {
      dot = (double)ns * ps;
      all = ns;
    } else {
      tokens = ns;
    }
  }
  __syncthreads();
  conclude(dot, all, tokens, experts, coefficient, loss, meet, meet_n);
}

// The same in two launches, where the parts are many bytes: one CU takes in 30 KB/us of what its L2 does not hold
// (256 parts of 256 experts 8 us, of 512 14 us).  16 columns a workgroup and a 64th of the parts a thread of four ...
constexpr int kColumns = 16;
__global__ __launch_bounds__(256) void balance_columns_kernel(const float* __restrict__ probs,
                                                              const int32_t* __restrict__ pairs, int32_t wgs,
                                                              int32_t pitch, double* __restrict__ col_p,
                                                              int32_t* __restrict__ col_n) {
  __shared__ double meet_p[64][kColumns];
  __shared__ int32_t meet_n[64][kColumns];
  const int tid = threadIdx.x, seg = tid / 4, c = blockIdx.x * kColumns + 4 * (tid % 4);
  double p[4] = {0.0, 0.0, 0.0, 0.0};
  int32_t n[4] = {0, 0, 0, 0};
  if (c < pitch) {
#pragma unroll 4
    for (int32_t w = seg; w < wgs; w += 64) {
      const f32x4 pv = *reinterpret_cast<const f32x4*>(probs + (int64_t)w * pitch + c);
      const u32x4 nv = *reinterpret_cast<const u32x4*>(pairs + (int64_t)w * pitch + c);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        p[i] += (double)pv[i];
        n[i] += (int32_t)nv[i];
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    meet_p[seg][4 * (tid % 4) + i] = p[i];
    meet_n[seg][4 * (tid % 4) + i] = n[i];
  }
  __syncthreads();
  const int at = blockIdx.x * kColumns + tid;
  if (tid >= kColumns || at >= pitch) return;
  double ps = 0.0;
  int32_t ns = 0;
#pragma unroll 8
  for (int s = 0; s < 64; ++s) {
    ps += meet_p[s][tid];
    ns += meet_n[s][tid];
  }
  col_p[at] = ps;
  col_n[at] = ns;
}

// ... and the loss from the columns' sums.
__global__ __launch_bounds__(kLossThreads) void balance_columns_finish_kernel(const double* __restrict__ col_p,
                                                                              const int32_t* __restrict__ col_n,
                                                                              int32_t experts, float coefficient,
                                                                              float* __restrict__ loss,
                                                                              int32_t* __restrict__ counts) {
  __shared__ double meet[kLossWaves];
  __shared__ int64_t meet_n[kLossWaves];
  const int tid = threadIdx.x;
  const int32_t tokens = col_n[experts], c = tid <= experts ? col_n[tid] : 0;
  if (tid <= experts) counts[tid] = c;
  const bool expert = tid < experts;
  conclude(expert ? (double)c * col_p[tid] : 0.0, expert ? c : 0, tokens, experts, coefficient, loss, meet, meet_n);
}

template <typename T, int L, int P>
__global__ __launch_bounds__(kGradThreads) void balance_grad_kernel(const T* __restrict__ logits,
                                                                    const int32_t* __restrict__ ids, int64_t t, int32_t topk,
                                                                    int32_t experts, float coefficient,
                                                                    const int32_t* __restrict__ counts,
                                                                    const float* __restrict__ d_loss,
                                                                    T* __restrict__ d_logits) {
  typedef Row<T, L, P> R;
  constexpr int each = kGradThreads / L;
  const int lane = threadIdx.x & 63;
  // every wave adds up the counts by itself
  int64_t all = 0;
  for (int e = lane; e < experts; e += 64) all += counts[e];
  for (int d = 32; d >= 1; d >>= 1) all += __shfl_xor(all, d);
  // share_e - 1 = (E c_e - sum c) / sum c: the p of a token sum to 1, so the formula holds as well with what a share
  // has over the mean, a whole number (below 2^53) and one rounding; shares near 1 would lose the digits that
  // differ (and experts that are used alike get a gradient of zero).
  const float scale = all > 0 ? 1.f / (float)all : 0.f;
  float share[P][R::PE];
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int i = 0; i < R::PE; ++i)
      share[p][i] = R::expert(p, i) < experts
                        ? (float)__builtin_fma((double)counts[R::expert(p, i)], (double)experts, -(double)all) * scale
                        : 0.f;
  const int32_t tokens = counts[experts];
  const float slope = tokens > 0 ? coefficient / (float)tokens * (d_loss ? *d_loss : 1.f) : 0.f;
  const int64_t stride = (int64_t)gridDim.x * each;
  int64_t tok = (int64_t)blockIdx.x * each + threadIdx.x / L;
  Token<T, L, P> next;
  if (tok < t) next.load(logits, ids, tok, topk, experts);
  for (; tok < t; tok += stride) {
    const Token<T, L, P> now = next;
    if (tok + stride < t) next.load(logits, ids, tok + stride, topk, experts);
    const bool real = now.pairs(ids, tok, topk, experts, [](int32_t) {});
    R r = now.row;
    r.softmax(real);
    float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int i = 0; i < R::PE; ++i) s[i & 3] = __builtin_fmaf(share[p][i], r.x[p][i], s[i & 3]);
    const float dot = wave_sum<L>((s[0] + s[1]) + (s[2] + s[3])) * r.inv;
    const float factor = real ? slope * r.inv : 0.f;  // (a slope that is not finite leaves padding's zeros)
    T* const out = d_logits + tok * experts;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int e = R::expert(p, 0);
      float d[R::PE];
#pragma unroll
      for (int i = 0; i < R::PE; ++i) d[i] = r.x[p][i] * factor * (share[p][i] - dot);
      if (e + R::PE <= experts) {
        store_piece(out + e, pack(d));
      } else {
#pragma unroll
        for (int i = 0; i < R::PE; ++i)
          if (e + i < experts) out[e + i] = from_f32<T>(d[i]);
      }
    }
  }
}

// run(L, P) for a number of experts: 16 values a lane, fewer lanes than a row's pieces, so that a wave holds
// several tokens and their sums and divisions are shared by more values.
template <typename T, class Run>
void with_lanes(int32_t experts, Run run) {
  constexpr int PE = 16 / (int)sizeof(T);
#define WQ_LANES(L, P) run(std::integral_constant<int, L>{}, std::integral_constant<int, P>{})
  if (experts <= PE) return WQ_LANES(1, 1);
  if constexpr (PE == 4) {
    if (experts <= 8) return WQ_LANES(1, 2);
  }
  constexpr int P = 16 / PE;
  if (experts <= 16) WQ_LANES(1, P);
  else if (experts <= 32) WQ_LANES(2, P);
  else if (experts <= 64) WQ_LANES(4, P);
  else if (experts <= 128) WQ_LANES(8, P);
  else if (experts <= 256) WQ_LANES(16, P);
  else WQ_LANES(32, P);
#undef WQ_LANES
}

// Rounds of a workgroup of `threads` over t tokens.
int64_t rounds(int64_t t, int32_t experts, int threads) {
  int lanes = 1;
  while (16 * lanes < experts) lanes *= 2;
  return (t * lanes + threads - 1) / threads;
}

}  // namespace

static int64_t balance_workgroups(int64_t t, int32_t experts) {
  const int64_t all = rounds(t, experts, kLossThreads);
  return all <= 2 ? 1 : all < 256 ? all : 256;
}

size_t balance_workspace_bytes(int64_t t, int32_t experts) {
  const int64_t wgs = balance_workgroups(t, experts);
  // the parts, and behind them the columns' sums
  return wgs > 1 ? (size_t)(8 * wgs + 12) * part_pitch(experts) : 0;
}

hipError_t launch_balance_loss(const void* logits, int f32, const int32_t* ids, int64_t t, int32_t topk, int32_t experts,
                               float coefficient, float* loss, int32_t* counts, void* ws, hipStream_t stream) {
  const int64_t wgs = balance_workgroups(t, experts);
  float* const probs = static_cast<float*>(ws);
  int32_t* const pairs = reinterpret_cast<int32_t*>(probs + wgs * part_pitch(experts));
  const auto run = [&](const auto* z) {
    typedef std::remove_const_t<std::remove_pointer_t<decltype(z)>> T;
    with_lanes<T>(experts, [&](auto l, auto p) {
      hipLaunchKernelGGL((balance_kernel<T, decltype(l)::value, decltype(p)::value>), dim3((unsigned)wgs),
                         dim3(kLossThreads), 0, stream, z, ids, t, topk, experts, coefficient, probs, pairs, loss, counts);
    });
  };
  if (f32) run(static_cast<const float*>(logits));
  else run(static_cast<const uint16_t*>(logits));
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || wgs == 1) return e;
  const int32_t pitch = part_pitch(experts);
  if (wgs * pitch > 16384) {
    double* const col_p = reinterpret_cast<double*>(pairs + wgs * pitch);  // (16-byte pieces up to here)
    int32_t* const col_n = reinterpret_cast<int32_t*>(col_p + pitch);
    hipLaunchKernelGGL(balance_columns_kernel, dim3((unsigned)((pitch + kColumns - 1) / kColumns)), dim3(256), 0, stream,
                       probs, pairs, (int32_t)wgs, pitch, col_p, col_n);
    const hipError_t e2 = hipGetLastError();
    if (e2 != hipSuccess) return e2;
    hipLaunchKernelGGL(balance_columns_finish_kernel, dim3(1), dim3(kLossThreads), 0, stream, col_p, col_n, experts,
                       coefficient, loss, counts);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(balance_finish_kernel, dim3(1), dim3(kLossThreads), 0, stream, probs, pairs, (int32_t)wgs, experts,
                     coefficient, loss, counts);
  return hipGetLastError();
}

hipError_t launch_balance_loss_grad(const void* logits, int f32, const int32_t* ids, int64_t t, int32_t topk,
                                    int32_t experts, float coefficient, const int32_t* counts, const float* d_loss,
                                    void* d_logits, hipStream_t stream) {
  const int64_t all = rounds(t, experts, kGradThreads), wgs = all < 1024 ? all : 1024;
  const auto run = [&](auto* d) {
    typedef std::remove_pointer_t<decltype(d)> T;
    with_lanes<T>(experts, [&](auto l, auto p) {
      hipLaunchKernelGGL((balance_grad_kernel<T, decltype(l)::value, decltype(p)::value>), dim3((unsigned)wgs),
                         dim3(kGradThreads), 0, stream, static_cast<const T*>(logits), ids, t, topk, experts, coefficient,
                         counts, d_loss, d);
    });
  };
  if (f32) run(static_cast<float*>(d_logits));
  else run(static_cast<uint16_t*>(d_logits));
  return hipGetLastError();
}

}  // namespace wq
