// wq_balance.hip -- the loss that keeps a router's experts evenly loaded, with its gradient.
//
//   p = softmax(logits);  c_e = the pairs of expert e;  T = the tokens that have a pair
//   share_e = E c_e / sum c;  loss = coefficient sum_e share_e (sum_t p_te / T)
//   d_logits_te = d_loss coefficient / T * p_te (share_e - sum_j share_j p_tj)
//
// Tokens whose ids all lie outside [0, E) are padding: they count nowhere, their logits are not used and
// get a gradient of zero.  A token's E logits lie in a group of lanes, the least power of two from E on, or
// a wave with V logits in each lane; a group takes every G-th token.  Counts are integers, the sums of p
// meet in a fixed order: the same bits every run.
#include <hip/hip_runtime.h>

#include "wq_kernels.hpp"
#include "wq_rows.hpp"
#include "wq_wave.hpp"

namespace wq {
namespace {

constexpr int kTopE = 512;

// e^x for x <= 0: 2^(x log2 e), the product's rounding and log2 e's own put right to first order.
__device__ __forceinline__ float exp_of(float x) {
  const float hi = x * 1.44269502f;
  const float lo = __builtin_fmaf(x, 1.44269502f, -hi) + x * 1.92596299e-8f;
  const float y = __builtin_amdgcn_exp2f(hi);
  // far below the range lo is no number (x = -inf): y is zero there
  return y > 0.f ? __builtin_fmaf(y, lo * 0.693147182f, y) : y;
}

// Sum and maximum over a group of `lanes` lanes, a power of two.
__device__ __forceinline__ float group_sum(float v, int lanes) {
  if (lanes == 64) return wave_sum(v);
  for (int d = lanes >> 1; d >= 1; d >>= 1) v += __shfl_xor(v, d);
  return v;
}
__device__ __forceinline__ float group_max(float v, int lanes) {
  for (int d = lanes >> 1; d >= 1; d >>= 1) v = fmaxf(v, __shfl_xor(v, d));
  return v;
}

// Where a thread's logits lie: lane `in` of group `group` of the launch holds the experts in, in + 64, ...
struct Place {
  int lanes, in;
  int64_t group, groups;
};
__device__ __forceinline__ Place place(int32_t experts) {
  Place p;
  p.lanes = 1;
  while (p.lanes < 64 && p.lanes < experts) p.lanes *= 2;
  p.in = threadIdx.x & (p.lanes - 1);
  const int each = 256 / p.lanes;
  p.group = (int64_t)blockIdx.x * each + threadIdx.x / p.lanes;
  p.groups = (int64_t)gridDim.x * each;
  return p;
}

// Whether token t has a pair (all lanes of its group agree); found(e) for every pair of it.
template <class Found>
__device__ __forceinline__ bool token_pairs(const int32_t* ids, int64_t t, int32_t topk, int32_t experts, const Place& at,
                                            Found found) {
  bool any = false;
  for (int32_t j = at.in; j < topk; j += at.lanes) {
    const int32_t e = ids[t * topk + j];
    if ((uint32_t)e < (uint32_t)experts) {
      any = true;
      found(e);
    }
  }
  const uint64_t votes = __ballot(any);
  if (at.lanes == 64) return votes != 0;
  const int first = (threadIdx.x & 63) & ~(at.lanes - 1);
  return ((votes >> first) & ((1ull << at.lanes) - 1)) != 0;
}

// The logits of token t, and e^(z - max) with the reciprocal of its sum.  A row of -inf has no probability
// anywhere: zeros.
template <typename T, int V>
__device__ __forceinline__ float softmax(const T* logits, int64_t t, int32_t experts, const Place& at, float (&x)[V]) {
  float top = -INFINITY;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = at.in + 64 * v;
    x[v] = e < experts ? to_f32(logits[t * experts + e]) : -INFINITY;
    top = fmaxf(top, x[v]);
  }
  top = group_max(top, at.lanes);
  float sum = 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    // (a NaN is no maximum: its difference stays one, also beside -inf)
    x[v] = top == -INFINITY && x[v] == top ? 0.f : exp_of(x[v] - top);
    sum += x[v];
  }
  sum = group_sum(sum, at.lanes);
  return sum == 0.f ? 0.f : 1.f / sum;
}

// The loss from `wgs` rows of probability sums [E] and counts [E + 1] (the last: tokens): threads
// segment x expert, segments of rows in order, in fp64.
__device__ __forceinline__ void finish(const float* probs, const int32_t* pairs, int32_t wgs, int32_t experts,
                                       float coefficient, float* loss, int32_t* counts, double* meet, int64_t* meet_n) {
  const int threads = blockDim.x, tid = threadIdx.x;
  // sums of every column: experts, and the tokens behind them
  for (int c0 = 0; c0 <= experts; c0 += threads) {
    const int cols = experts + 1 - c0 < threads ? experts + 1 - c0 : threads;
    const int segs = threads / cols, seg = tid / cols, c = c0 + tid % cols;
    double p = 0.0;
    int64_t n = 0;
    if (seg < segs) {
      const int32_t from = (int32_t)((int64_t)wgs * seg / segs), to = (int32_t)((int64_t)wgs * (seg + 1) / segs);
      for (int32_t w = from; w < to; ++w) {
        if (c < experts) p += (double)probs[(int64_t)w * experts + c];
        n += pairs[(int64_t)w * (experts + 1) + c];
      }
    }
    __syncthreads();
    meet[tid] = p;
    meet_n[tid] = n;
    __syncthreads();
    if (tid < cols) {
      for (int s = 1; s < segs; ++s) {
        p += meet[s * cols + tid];
        n += meet_n[s * cols + tid];
      }
      counts[c] = (int32_t)n;
    }
    // (256 threads and more than 255 experts: several rounds, so what the loss needs is kept below)
    __syncthreads();
    if (tid < cols) {
      meet[threads + c] = p;
      meet_n[threads + c] = n;
    }
  }
  __syncthreads();
  double dot = 0.0;
  int64_t all = 0;
  for (int e = tid; e < experts; e += threads) {
    dot += (double)meet_n[threads + e] * meet[threads + e];
    all += meet_n[threads + e];
  }
  meet[tid] = dot;
  meet_n[tid] = all;
  __syncthreads();
  for (int d = threads / 2; d >= 1; d /= 2) {
    if (tid < d) {
      meet[tid] += meet[tid + d];
      meet_n[tid] += meet_n[tid + d];
    }
    __syncthreads();
  }
  if (tid == 0) {
    const int64_t tokens = meet_n[threads + experts];
    // no token with a pair: no loss
    *loss = tokens ? (float)((double)coefficient * experts * meet[0] / ((double)meet_n[0] * (double)tokens)) : 0.f;
  }
}

template <typename T, int V>
__global__ __launch_bounds__(256) void balance_kernel(const T* __restrict__ logits, const int32_t* __restrict__ ids,
                                                      int64_t t, int32_t topk, int32_t experts, float coefficient,
                                                      float* __restrict__ probs, int32_t* __restrict__ pairs,
                                                      float* __restrict__ loss, int32_t* __restrict__ counts) {
  __shared__ int32_t hist[kTopE + 1];
  __shared__ float sums[256 * V];
  __shared__ float prob[kTopE];
  __shared__ double meet[256 + kTopE + 1];
  __shared__ int64_t meet_n[256 + kTopE + 1];
  const int tid = threadIdx.x;
  const Place at = place(experts);
  for (int i = tid; i <= experts; i += 256) hist[i] = 0;
  __syncthreads();
  float acc[V];
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = 0.f;
  int32_t tokens = 0;
  // whole waves go round together: the reductions take every lane
  const int64_t first = at.group - (threadIdx.x & 63) / at.lanes;
  for (int64_t t0 = 0; first + t0 < t; t0 += at.groups) {
    const int64_t tok = at.group + t0 < t ? at.group + t0 : t - 1;
    const bool mine = at.group + t0 < t;
    const bool real = token_pairs(ids, tok, topk, experts, at, [&](int32_t e) __attribute__((always_inline)) {
      if (mine) atomicAdd(&hist[e], 1);
    }) && mine;
    float x[V];
    const float inv = softmax<T, V>(logits, tok, experts, at, x);
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] += real ? x[v] * inv : 0.f;
    if (real && at.in == 0) ++tokens;
  }
  if (tokens) atomicAdd(&hist[experts], tokens);
#pragma unroll
  for (int v = 0; v < V; ++v) sums[v * 256 + tid] = acc[v];
  __syncthreads();
  // expert e: lane e % lanes of every group of the workgroup, in order
  const bool one = gridDim.x == 1;
  for (int e = tid; e < experts; e += 256) {
    float s = 0.f;
    for (int g = 0; g < 256; g += at.lanes) s += sums[(e >> 6) * 256 + g + (e & (at.lanes - 1))];
    if (one) prob[e] = s;
    else probs[(int64_t)blockIdx.x * experts + e] = s;
  }
  if (!one) {
    for (int e = tid; e <= experts; e += 256) pairs[(int64_t)blockIdx.x * (experts + 1) + e] = hist[e];
    return;
  }
  __syncthreads();
  finish(prob, hist, 1, experts, coefficient, loss, counts, meet, meet_n);
}

__global__ __launch_bounds__(1024) void balance_finish_kernel(const float* __restrict__ probs,
                                                              const int32_t* __restrict__ pairs, int32_t wgs,
                                                              int32_t experts, float coefficient,
                                                              float* __restrict__ loss, int32_t* __restrict__ counts) {
  __shared__ double meet[1024 + kTopE + 1];
  __shared__ int64_t meet_n[1024 + kTopE + 1];
  finish(probs, pairs, wgs, experts, coefficient, loss, counts, meet, meet_n);
}

template <typename T, int V>
__global__ __launch_bounds__(256) void balance_grad_kernel(const T* __restrict__ logits, const int32_t* __restrict__ ids,
                                                           int64_t t, int32_t topk, int32_t experts, float coefficient,
                                                           const int32_t* __restrict__ counts,
                                                           const float* __restrict__ d_loss, T* __restrict__ d_logits) {
  const Place at = place(experts);
  float share[V];
  int64_t all = 0;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int e = at.in + 64 * v;
    const int32_t c = e < experts ? counts[e] : 0;
    share[v] = (float)c;
    all += c;
  }
  for (int d = at.lanes >> 1; d >= 1; d >>= 1) all += __shfl_xor(all, d);
  const int32_t tokens = counts[experts];
  const float scale = all > 0 ? (float)((double)experts / (double)all) : 0.f;
  const float slope = tokens > 0 ? coefficient / (float)tokens * (d_loss ? *d_loss : 1.f) : 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v) share[v] *= scale;
  const int64_t first = at.group - (threadIdx.x & 63) / at.lanes;
  for (int64_t t0 = 0; first + t0 < t; t0 += at.groups) {
    const bool mine = at.group + t0 < t;
    const int64_t tok = mine ? at.group + t0 : t - 1;
    const bool real = token_pairs(ids, tok, topk, experts, at, [](int32_t) {});
    float x[V];
    const float inv = softmax<T, V>(logits, tok, experts, at, x);
    float dot = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) dot = __builtin_fmaf(share[v], x[v], dot);
    dot = group_sum(dot, at.lanes) * inv;
    if (!mine) continue;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = at.in + 64 * v;
      if (e < experts)
        d_logits[tok * experts + e] = from_f32<T>(real ? slope * (x[v] * inv) * (share[v] - dot) : 0.f);
    }
  }
}

// Tokens that a workgroup of 256 takes at a time.
int64_t tokens_at_a_time(int32_t experts) {
  int lanes = 1;
  while (lanes < 64 && lanes < experts) lanes *= 2;
  return 256 / lanes;
}

template <typename T, int V>
void loss_v(const T* logits, const int32_t* ids, int64_t t, int32_t topk, int32_t experts, float coefficient, float* probs,
            int32_t* pairs, int64_t wgs, float* loss, int32_t* counts, hipStream_t s) {
  hipLaunchKernelGGL((balance_kernel<T, V>), dim3((unsigned)wgs), dim3(256), 0, s, logits, ids, t, topk, experts,
                     coefficient, probs, pairs, loss, counts);
}
template <typename T, int V>
void grad_v(const T* logits, const int32_t* ids, int64_t t, int32_t topk, int32_t experts, float coefficient,
            const int32_t* counts, const float* d_loss, T* d_logits, hipStream_t s) {
  const int64_t all = (t + tokens_at_a_time(experts) - 1) / tokens_at_a_time(experts);
  hipLaunchKernelGGL((balance_grad_kernel<T, V>), dim3((unsigned)(all < 2048 ? all : 2048)), dim3(256), 0, s, logits, ids,
                     t, topk, experts, coefficient, counts, d_loss, d_logits);
}

}  // namespace

int64_t balance_workgroups(int64_t t, int32_t experts) {
  const int64_t each = 4 * tokens_at_a_time(experts);  // four rounds
  const int64_t all = (t + each - 1) / each;
  return all < 1 ? 1 : all < 512 ? all : 512;
}

hipError_t launch_balance_loss(const void* logits, int f32, const int32_t* ids, int64_t t, int32_t topk, int32_t experts,
                               float coefficient, float* loss, int32_t* counts, void* ws, hipStream_t stream) {
  const int64_t wgs = balance_workgroups(t, experts);
  float* const probs = static_cast<float*>(ws);
  int32_t* const pairs = wgs > 1 ? reinterpret_cast<int32_t*>(probs + wgs * experts) : nullptr;
  auto run = [&](auto vc) {
    constexpr int V = decltype(vc)::value;
    if (f32)
      loss_v<float, V>(static_cast<const float*>(logits), ids, t, topk, experts, coefficient, probs, pairs, wgs, loss,
                       counts, stream);
    else
      loss_v<uint16_t, V>(static_cast<const uint16_t*>(logits), ids, t, topk, experts, coefficient, probs, pairs, wgs,
                          loss, counts, stream);
  };
  if (experts <= 64) run(std::integral_constant<int, 1>{});
  else if (experts <= 128) run(std::integral_constant<int, 2>{});
  else if (experts <= 256) run(std::integral_constant<int, 4>{});
  else run(std::integral_constant<int, 8>{});
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || wgs == 1) return e;
  hipLaunchKernelGGL(balance_finish_kernel, dim3(1), dim3(1024), 0, stream, probs, pairs, (int32_t)wgs, experts,
                     coefficient, loss, counts);
  return hipGetLastError();
}

hipError_t launch_balance_loss_grad(const void* logits, int f32, const int32_t* ids, int64_t t, int32_t topk,
                                    int32_t experts, float coefficient, const int32_t* counts, const float* d_loss,
                                    void* d_logits, hipStream_t stream) {
  auto run = [&](auto vc) {
    constexpr int V = decltype(vc)::value;
    if (f32)
      grad_v<float, V>(static_cast<const float*>(logits), ids, t, topk, experts, coefficient, counts, d_loss,
                       static_cast<float*>(d_logits), stream);
    else
      grad_v<uint16_t, V>(static_cast<const uint16_t*>(logits), ids, t, topk, experts, coefficient, counts, d_loss,
                          static_cast<uint16_t*>(d_logits), stream);
  };
  if (experts <= 64) run(std::integral_constant<int, 1>{});
  else if (experts <= 128) run(std::integral_constant<int, 2>{});
  else if (experts <= 256) run(std::integral_constant<int, 4>{});
  else run(std::integral_constant<int, 8>{});
  return hipGetLastError();
}

}  // namespace wq
