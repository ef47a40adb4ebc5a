// wq_dispatch.hip -- token rows into expert order and back: positions of the (token, slot) pairs,
// the permutation, the weighted way back, and the gradients of both.
//
// Everything is driven per token through positions[p], the row of pair p = token * topk + slot in
// expert order (-1: dropped), so a thread adds all of an output element's contributions, in slot
// order: no atomics, the same bits every run.  All of it is bound by memory (a copy of 2 GiB: 4.8 to
// 5.3 TB/s); rows are read and written in 16-byte pieces, at any element's address, which a row of
// odd length starts at.  4096 tokens x 8 of 8192 bf16 (32 tokens): positions 2 to 5 us (1.4), permutation
// 102 to 121 us, 5.0 to 5.9 TB/s (4.2), way back 117 us, 5.2 TB/s (4.1), gradient 214 to 237 us, 4.8 to
// 5.3 TB/s (7.3).
#include <hip/hip_runtime.h>

#include "wq_kernels.hpp"
#include "wq_rows.hpp"

namespace wq {
namespace {

// positions[p] = the row of pair p, from the two directions that the routing sort leaves: a
// placed pair by its place, a pair whose id is no expert's by its id.
__global__ __launch_bounds__(256) void positions_kernel(const int32_t* __restrict__ ids, int32_t npairs,
                                                        int32_t experts,
                                                        const int32_t* __restrict__ offsets,
                                                        const int32_t* __restrict__ sorted_pairs,
                                                        int32_t* __restrict__ positions) {
  const int32_t i = (int32_t)(blockIdx.x * 256 + threadIdx.x);
  if (i >= npairs) return;
  if ((uint32_t)ids[i] >= (uint32_t)experts) positions[i] = -1;
  if (i < offsets[experts]) {
    const int32_t p = sorted_pairs[i];
    if ((uint32_t)p < (uint32_t)npairs) positions[p] = i;
  }
}

// One work item: a lane's piece of one token's row.  kLanes neighbouring lanes take consecutive pieces
// of a row.  More leave lanes idle behind short rows, fewer gain nothing on long ones (us for 65536
// tokens x 4, way back, with 8, 32, 64 lanes: 64 values 6.9, 16, 29; 128 values 15, 18, 30; 512 values
// 67, 68, 68; 4096 x 8, 8192 values: 122 each).  The last piece of a row ends with it, over some of the
// values of the one before, which get the same bits twice (32 tokens x 8, 1027 values: 3.7 us; 8.0 with
// a row's end value by value); a row shorter than a piece has a lane for each value.
constexpr int kLanes = 8;
struct Item {
  int64_t token;
  int64_t col;
};
template <int E>
__device__ __forceinline__ Item item(int64_t first, int64_t t, int64_t hidden) {
  const uint32_t slices = (uint32_t)((hidden + kLanes * E - 1) / (kLanes * E));
  const int64_t group = ((first + blockIdx.x) * 256 + threadIdx.x) / kLanes;
  Item r;
  r.token = group / slices;
  r.col = ((group % slices) * kLanes + (threadIdx.x & (kLanes - 1))) * (hidden < E ? 1 : E);
  if (r.col >= hidden) r.token = t;  // nothing to do
  else if (hidden >= E && r.col + E > hidden) r.col = hidden - E;
  return r;
}

// Rows that no pair has become zero: workgroup c of a launch's first W = 2^log2_wgs takes the rows c,
// c + W, c + 2 W, ... (dropped pairs leave the last ones, which so fall to all of them).  It reads all
// positions, marks its rows in LDS, and writes those without a mark: no scratch, no order among the
// workgroups, and where nothing was dropped only the reads, beside the other workgroups' copies.
constexpr int kClearRows = 65536;  // of one workgroup at most
struct Clear {
  int32_t wgs, log2_wgs;  // wgs 0: nothing to do
};
struct __attribute__((packed, aligned(4))) Positions4 {
  int32_t v[4];
};
template <typename T>
__device__ __forceinline__ void clear_rows(const int32_t* __restrict__ positions, int64_t npairs,
                                           int64_t hidden, T* __restrict__ out, uint32_t wg, Clear clear) {
  constexpr int E = 16 / (int)sizeof(T);
  __shared__ uint32_t used[kClearRows / 32];
  const int tid = threadIdx.x;
  const uint32_t n = ((uint32_t)npairs - wg + (uint32_t)clear.wgs - 1) >> clear.log2_wgs;  // rows, wg < npairs
  for (uint32_t i = tid; i < (n + 31) / 32; i += 256) used[i] = 0;
  __syncthreads();
  auto mark = [&](int32_t p) __attribute__((always_inline)) {
    const uint32_t i = (uint32_t)p >> clear.log2_wgs;
    if (((uint32_t)p & (uint32_t)(clear.wgs - 1)) == wg && i < n) atomicOr(&used[i >> 5], 1u << (i & 31));
  };
  const int64_t quads = npairs / 4;
  constexpr int U = 8;  // loads of a thread before the first use
  for (int64_t i0 = tid; i0 < quads; i0 += 256 * U) {
    Positions4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t i = i0 + 256 * u;
      v[u] = reinterpret_cast<const Positions4*>(positions)[i < quads ? i : i0];
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < 4; ++j) mark(v[u].v[j]);
  }
  if (tid < (int)(npairs & 3)) mark(positions[4 * quads + tid]);
  __syncthreads();
  const int lane = tid & 63;
  const uint32_t mine = 0x11111111u << __builtin_amdgcn_readfirstlane(tid >> 6);  // a wave's of 32 rows
  for (uint32_t b = 0; b < n; b += 32) {
    uint32_t free = ~used[b >> 5] & mine;
    if (n - b < 32) free &= (1u << (n - b)) - 1u;
    for (; free; free &= free - 1) {
      const int64_t r = ((int64_t)(b + __builtin_ctz(free)) << clear.log2_wgs) + wg;
      T* const row = out + r * hidden;
      for (int64_t c = (int64_t)lane * E; c + E <= hidden; c += 64 * E)
        store_piece(row + c, (u32x4){0, 0, 0, 0});
      const int64_t c = hidden / E * E + lane;
      if (c < hidden) row[c] = T(0);
    }
  }
}

// Zeros in `pieces` pieces of 16 bytes and then `rest` 2-byte units.
__global__ __launch_bounds__(256) void fill_kernel(u32x4* __restrict__ out, int64_t pieces, int32_t rest,
                                                   int64_t first) {
  const int64_t i = (first + blockIdx.x) * 256 + threadIdx.x;
  if (i < pieces) out[i] = (u32x4){0, 0, 0, 0};
  else if (i < pieces + rest) reinterpret_cast<uint16_t*>(out + pieces)[i - pieces] = 0;
}

template <typename T>
__global__ __launch_bounds__(256) void permute_kernel(const T* __restrict__ x, int64_t t, int32_t topk,
                                                      int64_t hidden, const int32_t* __restrict__ positions,
                                                      T* __restrict__ rows, Clear clear, int64_t first) {
  constexpr int E = 16 / (int)sizeof(T);
  if (first + blockIdx.x < clear.wgs) {  // all of them in the first launch
    clear_rows(positions, t * topk, hidden, rows, blockIdx.x, clear);
    return;
  }
  const Item it = item<E>(first - clear.wgs, t, hidden);
  if (it.token >= t) return;
  const int64_t npairs = t * topk;
  const int32_t* pos = positions + it.token * topk;
  const T* src = x + it.token * hidden + it.col;
  if (hidden >= E) {
    const u32x4 v = load_piece(src);
    for (int j = 0; j < topk; ++j) {
      const int64_t r = pos[j];
      if (r >= 0 && r < npairs) store_piece(rows + r * hidden + it.col, v);
    }
  } else {
    const T v = *src;
    for (int j = 0; j < topk; ++j) {
      const int64_t r = pos[j];
      if (r >= 0 && r < npairs) rows[r * hidden + it.col] = v;
    }
  }
}

// y[t] = sum_j w[t][j] rows[pos[t][j]] in fp32, j in order; w null: 1.
template <typename T>
__global__ __launch_bounds__(256) void unpermute_kernel(const T* __restrict__ rows,
                                                        const int32_t* __restrict__ positions,
                                                        const float* __restrict__ weights, int64_t t,
                                                        int32_t topk, int64_t hidden, T* __restrict__ y,
                                                        int64_t first) {
  constexpr int E = 16 / (int)sizeof(T);
  const Item it = item<E>(first, t, hidden);
  if (it.token >= t) return;
  const int64_t npairs = t * topk;
  const int64_t p0 = it.token * topk;
  T* dst = y + it.token * hidden + it.col;
  if (hidden >= E) {
    float acc[E];
#pragma unroll
    for (int i = 0; i < E; ++i) acc[i] = 0.f;
    for (int j0 = 0; j0 < topk; j0 += 8) {
      u32x4 v[8];
      float w[8];
#pragma unroll
      for (int jj = 0; jj < 8; ++jj) {
        w[jj] = 0.f;
        v[jj] = (u32x4){0, 0, 0, 0};
        if (j0 + jj < topk) {
          const int64_t r = positions[p0 + j0 + jj];
          if (r >= 0 && r < npairs) {
            v[jj] = load_piece(rows + r * hidden + it.col);
            w[jj] = weights ? weights[p0 + j0 + jj] : 1.f;
          }
        }
      }
#pragma unroll
      for (int jj = 0; jj < 8; ++jj) {
        float f[E];
        unpack(v[jj], f);
#pragma unroll
        for (int i = 0; i < E; ++i) acc[i] = __builtin_fmaf(w[jj], f[i], acc[i]);
      }
    }
    store_piece(dst, pack(acc));
  } else {
    float acc = 0.f;
    for (int j = 0; j < topk; ++j) {
      const int64_t r = positions[p0 + j];
      if (r >= 0 && r < npairs)
        acc = __builtin_fmaf(weights ? weights[p0 + j] : 1.f, to_f32(rows[r * hidden + it.col]), acc);
    }
    *dst = from_f32<T>(acc);
  }
}

// One wave per pair: d_rows[pos] = w dy[token], d_w = <dy[token], rows[pos]> in fp32 (each lane
// its pieces in order, then a tree over the lanes: a fixed order).
template <typename T>
__global__ __launch_bounds__(256) void unpermute_grad_kernel(const T* __restrict__ dy,
                                                             const T* __restrict__ rows,
                                                             const int32_t* __restrict__ positions,
                                                             const float* __restrict__ weights,
                                                             int64_t npairs, int32_t topk, int64_t hidden,
                                                             T* __restrict__ d_rows,
                                                             float* __restrict__ d_weights, Clear clear,
                                                             int64_t first) {
  constexpr int E = 16 / (int)sizeof(T);
  const int lane = threadIdx.x & 63;
  const int64_t wg = first + blockIdx.x - clear.wgs;
  if (wg < 0) {  // all of them in the first launch
    clear_rows(positions, npairs, hidden, d_rows, blockIdx.x, clear);
    return;
  }
  const int64_t p = wg * 4 + __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  if (p >= npairs) return;
  const int64_t r = positions[p];
  if (r < 0 || r >= npairs) {
    if (d_weights && lane == 0) d_weights[p] = 0.f;
    return;
  }
  const float w = weights ? weights[p] : 1.f;
  const T* const g = dy + p / topk * hidden;
  const T* const in = rows + (rows ? r * hidden : 0);
  T* const out = d_rows + (d_rows ? r * hidden : 0);
  float dot = 0.f;
  // U pieces a round, all loads before the first use (32 tokens x 8 of 8192 bf16: 7.9 us with one, 6.5
  // with four)
  constexpr int U = 4;
  const int64_t whole = hidden / E * E;
  for (int64_t c0 = (int64_t)lane * E; c0 < whole; c0 += 64 * E * U) {
    u32x4 gv[U], rv[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t c = c0 + 64 * E * u;
      if (c < whole) {
        gv[u] = load_piece(g + c);
        if (d_weights) rv[u] = load_piece(in + c);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t c = c0 + 64 * E * u;
      if (c >= whole) break;
      float f[E], o[E];
      unpack(gv[u], f);
      if (d_weights) {
        float v[E];
        unpack(rv[u], v);
#pragma unroll
        for (int i = 0; i < E; ++i) dot = __builtin_fmaf(f[i], v[i], dot);
      }
      if (d_rows) {
#pragma unroll
        for (int i = 0; i < E; ++i) o[i] = w * f[i];
        store_piece(out + c, pack(o));
      }
    }
  }
  const int64_t c = whole + lane;  // the row's last elements, fewer than E
  if (c < hidden) {
    const float f = to_f32(g[c]);
    if (d_weights) dot = __builtin_fmaf(f, to_f32(in[c]), dot);
    if (d_rows) out[c] = from_f32<T>(w * f);
  }
  if (d_weights) {
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) dot += __shfl_xor(dot, d);
    if (lane == 0) d_weights[p] = dot;
  }
}

// Workgroups for t rows of `hidden` elements, E per lane.
int64_t row_wgs(int64_t t, int64_t hidden, int E) {
  const int64_t slices = (hidden + (int64_t)kLanes * E - 1) / ((int64_t)kLanes * E);
  return (t * slices * kLanes + 255) / 256;
}

// How rows that no pair has become zero: by a launch's first workgroups, or by a fill before the launch
// (wgs 0).  8 rows a workgroup spread the writes of a small call; many pairs take fewer workgroups, for
// each reads all of the positions, 0.2 ns a pair beside the copies.  So the fill serves rows below `fill`
// bytes of 32768 pairs or more (us beyond the permutation's own, first workgroups and fill: 32768 pairs
// of 256 bytes 3.3 to 4.4 and 4.1 to 4.3, of 2 KiB 0.8 to 2.1 and 10.2; 262144 of 1 KiB 29 to 55 and 32
// to 38; 16384 of 128 bytes 1.2 to 1.5 and 1.9 to 2.0), and rows that are fewer bytes than all those
// reads once marks for 65536 rows ask for more workgroups.  The gradient takes longer a pair and hides
// the reads at every length (262144 pairs of 256 bytes: 2 to 7 and 10).
template <typename T>
hipError_t plan_clear(T* rows, int64_t npairs, int64_t hidden, int64_t fill, Clear* c, hipStream_t s) {
  int log2_wgs = 8;
  while (log2_wgs > 0 && npairs < (8ll << log2_wgs)) --log2_wgs;
  while (log2_wgs > 6 && npairs << log2_wgs > 1ll << 23) --log2_wgs;
  while ((int64_t)kClearRows << log2_wgs < npairs) {
    ++log2_wgs;
    if (fill < 4ll << log2_wgs) fill = 4ll << log2_wgs;
  }
  *c = Clear{1 << log2_wgs, log2_wgs};
  if (npairs < 32768 || hidden * (int64_t)sizeof(T) >= fill) return hipSuccess;
  *c = Clear{0, 0};
  const int64_t units = npairs * hidden * (int64_t)sizeof(T) / 2, pieces = units / 8;
  return launch_in_parts((pieces + units % 8 + 255) / 256, [&](int64_t first, dim3 grid) {
    hipLaunchKernelGGL(fill_kernel, grid, dim3(256), 0, s, reinterpret_cast<u32x4*>(rows), pieces,
                       (int32_t)(units % 8), first);
  });
}

}  // namespace

hipError_t launch_positions(const int32_t* ids, int64_t npairs, int32_t experts, const int32_t* offsets,
                            const int32_t* sorted_pairs, int32_t* positions, hipStream_t stream) {
  hipLaunchKernelGGL(positions_kernel, dim3((unsigned)((npairs + 255) / 256)), dim3(256), 0, stream, ids,
                     (int32_t)npairs, experts, offsets, sorted_pairs, positions);
  return hipGetLastError();
}

template <typename T>
static hipError_t permute_t(const T* x, int64_t t, int32_t topk, int64_t hidden, const int32_t* positions,
                            T* rows, int clear, hipStream_t s) {
  constexpr int E = 16 / (int)sizeof(T);
  Clear c{0, 0};
  if (clear) {
    const hipError_t e = plan_clear(rows, t * topk, hidden, 1024, &c, s);
    if (e != hipSuccess) return e;
  }
  return launch_in_parts(c.wgs + row_wgs(t, hidden, E), [&](int64_t first, dim3 grid) {
    hipLaunchKernelGGL(permute_kernel<T>, grid, dim3(256), 0, s, x, t, topk, hidden, positions, rows, c, first);
  });
}

hipError_t launch_permute(const void* x, int f32, int64_t t, int32_t topk, int64_t hidden,
                          const int32_t* positions, void* rows, int clear, hipStream_t stream) {
  return f32 ? permute_t(static_cast<const float*>(x), t, topk, hidden, positions, static_cast<float*>(rows),
                         clear, stream)
             : permute_t(static_cast<const uint16_t*>(x), t, topk, hidden, positions,
                         static_cast<uint16_t*>(rows), clear, stream);
}

template <typename T>
static hipError_t unpermute_t(const T* rows, const int32_t* positions, const float* weights, int64_t t,
                              int32_t topk, int64_t hidden, T* y, hipStream_t s) {
  constexpr int E = 16 / (int)sizeof(T);
  return launch_in_parts(row_wgs(t, hidden, E), [&](int64_t first, dim3 grid) {
    hipLaunchKernelGGL(unpermute_kernel<T>, grid, dim3(256), 0, s, rows, positions, weights, t, topk, hidden, y, first);
  });
}

hipError_t launch_unpermute(const void* rows, int f32, const int32_t* positions, const float* weights,
                            int64_t t, int32_t topk, int64_t hidden, void* y, hipStream_t stream) {
  return f32 ? unpermute_t(static_cast<const float*>(rows), positions, weights, t, topk, hidden,
                           static_cast<float*>(y), stream)
             : unpermute_t(static_cast<const uint16_t*>(rows), positions, weights, t, topk, hidden,
                           static_cast<uint16_t*>(y), stream);
}

template <typename T>
static hipError_t unpermute_grad_t(const T* dy, const T* rows, const int32_t* positions, const float* weights,
                                   int64_t t, int32_t topk, int64_t hidden, T* d_rows, float* d_weights,
                                   int clear, hipStream_t s) {
  const int64_t npairs = t * topk;
  Clear c{0, 0};
  if (clear && d_rows) {
    const hipError_t e = plan_clear(d_rows, npairs, hidden, 0, &c, s);
    if (e != hipSuccess) return e;
  }
  return launch_in_parts(c.wgs + (npairs + 3) / 4, [&](int64_t first, dim3 grid) {
    hipLaunchKernelGGL(unpermute_grad_kernel<T>, grid, dim3(256), 0, s, dy, rows, positions, weights, npairs,
                       topk, hidden, d_rows, d_weights, c, first);
  });
}

hipError_t launch_unpermute_grad(const void* dy, const void* rows, int f32, const int32_t* positions,
                                 const float* weights, int64_t t, int32_t topk, int64_t hidden,
                                 void* d_rows, float* d_weights, int clear, hipStream_t stream) {
  return f32 ? unpermute_grad_t(static_cast<const float*>(dy), static_cast<const float*>(rows), positions,
                                weights, t, topk, hidden, static_cast<float*>(d_rows), d_weights, clear, stream)
             : unpermute_grad_t(static_cast<const uint16_t*>(dy), static_cast<const uint16_t*>(rows), positions,
                                weights, t, topk, hidden, static_cast<uint16_t*>(d_rows), d_weights, clear,
                                stream);
}

}  // namespace wq
