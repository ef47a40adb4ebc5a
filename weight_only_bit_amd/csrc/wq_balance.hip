// wq_balance.hip -- the loss that keeps a router's experts evenly loaded, with its gradient.
//
//   p = softmax(logits);  c_e = the pairs of expert e;  T = the tokens that have a pair
//   share_e = E c_e / sum c;  loss = coefficient sum_e share_e (sum_t p_te / T)
//   d_logits_te = d_loss coefficient / T * p_te (share_e - sum_j share_j p_tj)
//
// Tokens whose ids all lie outside [0, E) are padding: they count nowhere, their logits are not used and
// get a gradient of zero.  A token's E logits lie in a group of L lanes, the least power of two from E on, or in
// a wave with V logits a lane (expert e in lane e % 64); a group takes U tokens at a time, whose loads are all on
// their way before the first is used.  Counts are integers (their order does not matter), the sums of p meet in
// a fixed order: the same bits every run.
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

// e^x for x <= 0: 2^(x log2 e), the product's rounding and log2 e's own put right to first order.
__device__ __forceinline__ float exp_of(float x) {
  const float hi = x * 1.44269502f;
  const float lo = __builtin_fmaf(x, 1.44269502f, -hi) + x * 1.92596299e-8f;
  const float y = __builtin_amdgcn_exp2f(hi);
  // far below the range lo is no number (x = -inf): y is zero there
  return y > 0.f ? __builtin_fmaf(y, lo * 0.693147182f, y) : y;
}

constexpr int tokens_of(int V) { return V == 1 ? 4 : 2; }

// U tokens of a group: every G-th from `first` on.  Behind t the loads repeat the last token's.
template <typename T, int L, int V>
struct Tokens {
  static constexpr int U = tokens_of(V);
  float x[U][V];  // logits, then e^(z - max)
  float inv[U];   // 1 / sum of them
  int32_t id[U];  // this lane's first id
  __device__ __forceinline__ void load(const T* logits, const int32_t* ids, int64_t t, int32_t topk, int32_t experts,
                                       int64_t first, int64_t groups) {
    const int in = threadIdx.x & (L - 1);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t tok = first + u * groups < t ? first + u * groups : t - 1;
      id[u] = in < topk ? ids[tok * topk + in] : -1;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int e = in + 64 * v;
        x[u][v] = e < experts ? to_f32(logits[tok * experts + e]) : -INFINITY;
      }
    }
  }
  // Whether token u has a pair (every lane of the group knows); found(e) for each of this lane's.
  template <class Found>
  __device__ __forceinline__ bool pairs(int u, const int32_t* ids, int64_t t, int32_t topk, int32_t experts, int64_t first,
                                        int64_t groups, Found found) {
    bool any = (uint32_t)id[u] < (uint32_t)experts;
    if (any) found(id[u]);
    if (topk > L) {
      const int64_t tok = first + u * groups < t ? first + u * groups : t - 1;
      for (int32_t j = (threadIdx.x & (L - 1)) + L; j < topk; j += L) {
        const int32_t e = ids[tok * topk + j];
        if ((uint32_t)e < (uint32_t)experts) {
          any = true;
          found(e);
        }
      }
    }
    const uint64_t votes = __ballot(any);
    if constexpr (L == 64) return votes != 0;
    else return ((votes >> ((threadIdx.x & 63) & ~(L - 1))) & ((1ull << L) - 1)) != 0;
  }
  // A row of -inf has no probability anywhere: zeros.
  __device__ __forceinline__ void softmax() {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float top = x[u][0];
#pragma unroll
      for (int v = 1; v < V; ++v) top = fmaxf(top, x[u][v]);
      top = wave_max<L>(top);
      float sum = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        // (a NaN is no maximum: its difference stays one, also beside -inf)
        x[u][v] = top == -INFINITY && x[u][v] == top ? 0.f : exp_of(x[u][v] - top);
        sum += x[u][v];
      }
      sum = wave_sum<L>(sum);
      inv[u] = sum == 0.f ? 0.f : 1.f / sum;
    }
  }
};

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
  if (threadIdx.x != 0) return;
  dot = 0.0;
  all = 0;
  for (int w = 0; w < kLossWaves; ++w) {
    dot += meet[w];
    all += meet_n[w];
  }
  // no token with a pair: no loss
  *loss = tokens ? (float)((double)coefficient * experts * dot / ((double)all * (double)tokens)) : 0.f;
}

// Floats (and int32) of a part: experts + 1, the last count the tokens, in whole pieces of 16 bytes.
__host__ __device__ constexpr int32_t part_pitch(int32_t experts) { return (experts + 4) / 4 * 4; }

template <typename T, int L, int V>
__global__ __launch_bounds__(kLossThreads) void balance_kernel(const T* __restrict__ logits, const int32_t* __restrict__ ids,
                                                               int64_t t, int32_t topk, int32_t experts, float coefficient,
                                                               float* __restrict__ probs, int32_t* __restrict__ pairs,
                                                               float* __restrict__ loss, int32_t* __restrict__ counts) {
  __shared__ int32_t hist[kTopE + 1];
  __shared__ float sums[kLossWaves][L < 64 ? L : 64 * V];
  __shared__ double meet[kLossWaves];
  __shared__ int64_t meet_n[kLossWaves];
  constexpr int U = tokens_of(V);
  const int tid = threadIdx.x, lane = tid & 63;
  constexpr int each = kLossThreads / L;
  const int64_t group = (int64_t)blockIdx.x * each + tid / L, groups = (int64_t)gridDim.x * each;
  for (int i = tid; i <= experts; i += kLossThreads) hist[i] = 0;
  __syncthreads();
  float acc[V];
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = 0.f;
  int32_t tokens = 0;
  // whole waves go round together: the votes take every lane
  for (int64_t t0 = group; t0 - lane / L < t; t0 += groups * U) {
    Tokens<T, L, V> k;
    k.load(logits, ids, t, topk, experts, t0, groups);
    bool real[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool mine = t0 + u * groups < t;
      real[u] = k.pairs(u, ids, t, topk, experts, t0, groups, [&](int32_t e) __attribute__((always_inline)) {
        if (mine) atomicAdd(&hist[e], 1);
      }) && mine;
      if (real[u] && (tid & (L - 1)) == 0) ++tokens;
    }
    k.softmax();
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] += real[u] ? k.x[u][v] * k.inv[u] : 0.f;
  }
  if (tokens) atomicAdd(&hist[experts], tokens);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    for (int d = L; d < 64; d <<= 1) acc[v] += __shfl_xor(acc[v], d);  // the wave's groups
    if (lane < L) sums[tid >> 6][lane + 64 * v] = acc[v];
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

// The parts' sums: threads of four columns each, and as many of them as the workgroup holds beside each other
// for segments of the parts, eight loads in flight; segments and parts in order, in fp64.
__global__ __launch_bounds__(kLossThreads) void balance_finish_kernel(const float* __restrict__ probs,
                                                                      const int32_t* __restrict__ pairs, int32_t wgs,
                                                                      int32_t experts, float coefficient,
                                                                      float* __restrict__ loss, int32_t* __restrict__ counts) {
  __shared__ double col_p[kLossThreads][4];
  __shared__ int64_t col_n[kLossThreads][4];
  __shared__ double meet[kLossWaves];
  __shared__ int64_t meet_n[kLossWaves];
  __shared__ int64_t tokens;
  const int32_t pitch = part_pitch(experts), cols = pitch / 4, segs = kLossThreads / cols;
  const int tid = threadIdx.x, seg = tid / cols, c = tid % cols;
  double p[4] = {0.0, 0.0, 0.0, 0.0};
  int64_t n[4] = {0, 0, 0, 0};
  if (seg < segs) {
    const int32_t from = (int32_t)((int64_t)wgs * seg / segs), to = (int32_t)((int64_t)wgs * (seg + 1) / segs);
    constexpr int U = 8;
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
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    col_p[tid][i] = p[i];
    col_n[tid][i] = n[i];
  }
  __syncthreads();
  double dot = 0.0;
  int64_t all = 0;
  if (tid <= experts) {
    double ps = 0.0;
    int64_t ns = 0;
    for (int s = 0; s < segs; ++s) {
      ps += col_p[s * cols + tid / 4][tid % 4];
      ns += col_n[s * cols + tid / 4][tid % 4];
    }
    counts[tid] = (int32_t)ns;
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

template <typename T, int L, int V>
__global__ __launch_bounds__(kGradThreads) void balance_grad_kernel(const T* __restrict__ logits,
                                                                    const int32_t* __restrict__ ids, int64_t t, int32_t topk,
                                                                    int32_t experts, float coefficient,
                                                                    const int32_t* __restrict__ counts,
                                                                    const float* __restrict__ d_loss,
                                                                    T* __restrict__ d_logits) {
  constexpr int U = tokens_of(V);
  constexpr int each = kGradThreads / L;
  const int lane = threadIdx.x & 63, in = threadIdx.x & (L - 1);
  const int64_t group = (int64_t)blockIdx.x * each + threadIdx.x / L, groups = (int64_t)gridDim.x * each;
  float share[V];
  int64_t all = 0;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = in + 64 * v;
    const int32_t c = e < experts ? counts[e] : 0;
    share[v] = (float)c;
    all += c;
  }
  for (int d = L >> 1; d >= 1; d >>= 1) all += __shfl_xor(all, d);
  const int32_t tokens = counts[experts];
  const float scale = all > 0 ? (float)((double)experts / (double)all) : 0.f;
  const float slope = tokens > 0 ? coefficient / (float)tokens * (d_loss ? *d_loss : 1.f) : 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v) share[v] *= scale;
  for (int64_t t0 = group; t0 - lane / L < t; t0 += groups * U) {
    Tokens<T, L, V> k;
    k.load(logits, ids, t, topk, experts, t0, groups);
    bool real[U];
#pragma unroll
    for (int u = 0; u < U; ++u) real[u] = k.pairs(u, ids, t, topk, experts, t0, groups, [](int32_t) {});
    k.softmax();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float dot = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) dot = __builtin_fmaf(share[v], k.x[u][v], dot);
      dot = wave_sum<L>(dot) * k.inv[u];
      const int64_t tok = t0 + u * groups;
      if (tok >= t) continue;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int e = in + 64 * v;
        if (e < experts)
          d_logits[tok * experts + e] = from_f32<T>(real[u] ? slope * (k.x[u][v] * k.inv[u]) * (share[v] - dot) : 0.f);
      }
    }
  }
}

// run(L, V) for a number of experts.
template <class Run>
void with_lanes(int32_t experts, Run run) {
#define WQ_LANES(L, V) run(std::integral_constant<int, L>{}, std::integral_constant<int, V>{})
  if (experts <= 1) WQ_LANES(1, 1);
  else if (experts <= 2) WQ_LANES(2, 1);
  else if (experts <= 4) WQ_LANES(4, 1);
  else if (experts <= 8) WQ_LANES(8, 1);
  else if (experts <= 16) WQ_LANES(16, 1);
  else if (experts <= 32) WQ_LANES(32, 1);
  else if (experts <= 64) WQ_LANES(64, 1);
  else if (experts <= 128) WQ_LANES(64, 2);
  else if (experts <= 256) WQ_LANES(64, 4);
  else WQ_LANES(64, 8);
#undef WQ_LANES
}

// Rounds of a workgroup of `threads` over t tokens.
int64_t rounds(int64_t t, int32_t experts, int threads) {
  int64_t n = 0;
  with_lanes(experts, [&](auto l, auto v) {
    const int64_t each = threads / decltype(l)::value * tokens_of(decltype(v)::value);
    n = (t + each - 1) / each;
  });
  return n;
}

}  // namespace

static int64_t balance_workgroups(int64_t t, int32_t experts) {
  const int64_t all = rounds(t, experts, kLossThreads);
  return all <= 4 ? 1 : all < 256 ? all : 256;
}

size_t balance_workspace_bytes(int64_t t, int32_t experts) {
  const int64_t wgs = balance_workgroups(t, experts);
  return wgs > 1 ? (size_t)wgs * part_pitch(experts) * 8 : 0;
}

hipError_t launch_balance_loss(const void* logits, int f32, const int32_t* ids, int64_t t, int32_t topk, int32_t experts,
                               float coefficient, float* loss, int32_t* counts, void* ws, hipStream_t stream) {
  const int64_t wgs = balance_workgroups(t, experts);
  float* const probs = static_cast<float*>(ws);
  int32_t* const pairs = reinterpret_cast<int32_t*>(probs + wgs * part_pitch(experts));
  with_lanes(experts, [&](auto l, auto v) {
    constexpr int L = decltype(l)::value, V = decltype(v)::value;
    if (f32)
      hipLaunchKernelGGL((balance_kernel<float, L, V>), dim3((unsigned)wgs), dim3(kLossThreads), 0, stream,
                         static_cast<const float*>(logits), ids, t, topk, experts, coefficient, probs, pairs, loss, counts);
    else
      hipLaunchKernelGGL((balance_kernel<uint16_t, L, V>), dim3((unsigned)wgs), dim3(kLossThreads), 0, stream,
                         static_cast<const uint16_t*>(logits), ids, t, topk, experts, coefficient, probs, pairs, loss, counts);
  });
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || wgs == 1) return e;
  hipLaunchKernelGGL(balance_finish_kernel, dim3(1), dim3(kLossThreads), 0, stream, probs, pairs, (int32_t)wgs, experts,
                     coefficient, loss, counts);
  return hipGetLastError();
}

hipError_t launch_balance_loss_grad(const void* logits, int f32, const int32_t* ids, int64_t t, int32_t topk,
                                    int32_t experts, float coefficient, const int32_t* counts, const float* d_loss,
                                    void* d_logits, hipStream_t stream) {
  const int64_t all = rounds(t, experts, kGradThreads), wgs = all < 2048 ? all : 2048;
  with_lanes(experts, [&](auto l, auto v) {
    constexpr int L = decltype(l)::value, V = decltype(v)::value;
    if (f32)
      hipLaunchKernelGGL((balance_grad_kernel<float, L, V>), dim3((unsigned)wgs), dim3(kGradThreads), 0, stream,
                         static_cast<const float*>(logits), ids, t, topk, experts, coefficient, counts, d_loss,
                         static_cast<float*>(d_logits));
    else
      hipLaunchKernelGGL((balance_grad_kernel<uint16_t, L, V>), dim3((unsigned)wgs), dim3(kGradThreads), 0, stream,
                         static_cast<const uint16_t*>(logits), ids, t, topk, experts, coefficient, counts, d_loss,
                         static_cast<uint16_t*>(d_logits));
  });
  return hipGetLastError();
}

}  // namespace wq
