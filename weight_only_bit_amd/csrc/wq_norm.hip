// wq_norm.hip -- rows in int8 with a scale each, and the root-mean-square norm of a sum of two rows, with its
// gradients.
//
//   quantise  a = max_j |x_j|;  scale = a / 127;  code_j = rint(127 x_j / a)
//   norm      r = T(x + residual);  inv = 1 / sqrt(mean_j r_j^2 + eps);  y_j = T(r_j inv w_j)
//   in int8   v_j = r_j w_j;  a = max_j |v_j|;  scale = a inv / 127;  code_j = rint(127 v_j / a)
//   gradient  g_j = dy_j w_j;  m = inv^2 mean_j g_j r_j;  dx_j = T(inv (g_j - r_j m) + d_sum_j)
//             d_weight_j = sum over rows of dy_j r_j inv
//
// All of them are bound by memory.  A row is held in registers between the pass that sums it and the pass
// that writes it, so it is read once; only rows beyond 65536 bf16 (32768 fp32) values, in the gradient 16384
// (8192), are read again.  4096 x 8192 bf16: norm 53 us (5.1 TB/s, copies of 2 GiB 4.8 to 5.6), in int8 50 us (4.7), the
// gradient 62 us (4.3, its parts included); 32 x 8192: 3.7, 4.1 and 6.5 us, of which a launch takes 1.6.  Short rows
// are bound by a chain of dependent steps a row, with no next row on its way and, below 16 pieces, idle lanes: 65536 x 64
// bf16 10.6, 12.3 and 17.3 us where their bytes take 6, 5 and 6.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "wq_kernels.hpp"
#include "wq_rows.hpp"
#include "wq_wave.hpp"

namespace wq {
namespace {

// ---------------------------------------------------------------------------------------------
// Magnitudes as integers: bit patterns without the sign order as magnitudes do, and an infinity or a NaN
// is at least the type's infinity.  The products v of two bf16 values are exact in fp32, those of two fp32
// values in fp64.
// ---------------------------------------------------------------------------------------------
template <typename T>
struct Wide;
template <>
struct Wide<uint16_t> {
  typedef float V;
  typedef uint32_t M;
};
template <>
struct Wide<float> {
  typedef double V;
  typedef uint64_t M;
};
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }
__device__ __forceinline__ uint64_t magnitude(double v) {
  return __builtin_bit_cast(uint64_t, v) & 0x7FFFFFFFFFFFFFFFull;
}
__device__ __forceinline__ double value_of(uint32_t m) { return (double)__uint_as_float(m); }
__device__ __forceinline__ double value_of(uint64_t m) { return __builtin_bit_cast(double, m); }
__device__ __forceinline__ bool is_finite(uint32_t m) { return m < 0x7F800000u; }
__device__ __forceinline__ bool is_finite(uint64_t m) { return m < 0x7FF0000000000000ull; }

// rint(v f), half way to the even integer, as the definition has it: the product in fp64 is first rounded to
// a multiple of 2^-34 (the sum with 1.5 * 2^18 has that unit), which brings a quotient that lies exactly half
// way back to it after the rounding of f; quotients of bf16 values, and of their products with bf16 weights,
// lie half way or at least 2^-25 from it.  The sum with 1.5 * 2^52 leaves the integer in the low bits.
__device__ __forceinline__ int32_t code_of(double v, double f) {
  double q = v * f;
  q = (q + 393216.0) - 393216.0;
  return (int32_t)(uint32_t)__builtin_bit_cast(uint64_t, q + 6755399441055744.0);
}
__device__ __forceinline__ uint32_t pack4(int32_t a, int32_t b, int32_t c, int32_t d) {
  return (uint32_t)(a & 255) | (uint32_t)(b & 255) << 8 | (uint32_t)(c & 255) << 16 | (uint32_t)d << 24;
}
struct __attribute__((packed)) Codes4 {
  uint32_t v;
};
struct __attribute__((packed)) Codes8 {
  uint32_t lo, hi;
};

// 1 / sqrt(mean + eps), and 0 where both are 0 (a row of zeros, or of values whose squares vanish in fp32).
__device__ __forceinline__ float inverse_root(float squares, int64_t k, float eps) {
  const float m = squares / (float)k + eps;
  return m == 0.f ? 0.f : 1.f / sqrtf(m);
}

enum { OUT_NORM = 0, OUT_NORM_I8 = 1, OUT_ROWS = 2, OUT_WEIGHT = 3 };

struct NormArgs {
  const void* x;
  const void* residual;  // null: r = x
  const void* weight;
  void* sum;             // r, where there is a residual
  void* y;               // OUT_NORM
  int8_t* codes;         // the others
  void* scales;          // fp32 (OUT_WEIGHT: bf16)
  float eps;
  int64_t n, k;
};

// What the elements of a row are held as between the passes: pieces of 16 bytes, and one of the last
// k % E elements in each of the first lanes.
template <typename T, int LANES, int P, int OUT>
__global__ __launch_bounds__(LANES < 256 ? 256 : LANES) void norm_kernel(const NormArgs a, int64_t first) {
  constexpr int E = 16 / (int)sizeof(T);
  constexpr bool I8 = OUT != OUT_NORM, NORM = OUT <= OUT_NORM_I8;
  constexpr int WAVES = LANES < 64 ? 1 : LANES / 64;
  typedef typename Wide<T>::V V;
  typedef typename Wide<T>::M M;
  const int tid = LANES < 256 ? (int)threadIdx.x % LANES : (int)threadIdx.x;
  const int64_t row = LANES < 256 ? (first + blockIdx.x) * (256 / LANES) + threadIdx.x / LANES : first + blockIdx.x;
  if (row >= a.n) return;  // whole groups of LANES, and of rows of several waves the whole workgroup
  const int64_t k = a.k, pieces = k / E, base = row * k;
  const int tail = (int)(k % E);
  const int64_t tcol = pieces * E + tid;  // of the lanes below `tail`
  const T* const x = static_cast<const T*>(a.x) + base;
  const T* const res = NORM && a.residual ? static_cast<const T*>(a.residual) + base : nullptr;
  const T* const weight = static_cast<const T*>(a.weight);
  T* const sum = NORM && a.sum ? static_cast<T*>(a.sum) + base : nullptr;

  float ss = 0.f;
  M top = 0;
  auto take = [&](const float (&f)[E], const float (&w)[E]) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < E; ++i) {
      if constexpr (NORM) ss = __builtin_fmaf(f[i], f[i], ss);
      if constexpr (I8) top = larger(top, magnitude(NORM ? (V)f[i] * (V)w[i] : (V)f[i]));
    }
  };
  auto add_piece = [&](u32x4 v, u32x4 other, int64_t p) __attribute__((always_inline)) {  // r's piece, stored
    float f[E], g[E];
    unpack(v, f);
    unpack(other, g);
#pragma unroll
    for (int i = 0; i < E; ++i) f[i] += g[i];
    v = pack(f);
    store_piece(sum + p * E, v);
    return v;
  };
  u32x4 r[P > 0 ? P : 1], wp[P > 0 ? P : 1], rp[P > 0 ? P : 1];
  T rt{}, wt{};
  if constexpr (P > 0) {
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int64_t j = p * LANES + tid;
      r[p] = wp[p] = (u32x4){0, 0, 0, 0};
      if (j < pieces) {
        r[p] = load_piece(x + j * E);
        if (NORM && res) rp[p] = load_piece(res + j * E);
        if constexpr (NORM) wp[p] = load_piece(weight + j * E);
      }
    }
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int64_t j = p * LANES + tid;
      if (NORM && res && j < pieces) r[p] = add_piece(r[p], rp[p], j);
      float f[E], w[E];
      unpack(r[p], f);
      if constexpr (NORM) unpack(wp[p], w);
      take(f, w);
    }
  } else {
    for (int64_t j = tid; j < pieces; j += LANES) {
      u32x4 v = load_piece(x + j * E);
      if (NORM && res) v = add_piece(v, load_piece(res + j * E), j);
      float f[E], w[E];
      unpack(v, f);
      if constexpr (NORM) unpack(load_piece(weight + j * E), w);
      take(f, w);
    }
  }
  if (tid < tail) {
    rt = x[tcol];
    if constexpr (NORM) {
      wt = weight[tcol];
      if (res) {
        rt = from_f32<T>(to_f32(rt) + to_f32(res[tcol]));
        sum[tcol] = rt;
      }
    }
    const float f = to_f32(rt);
    if constexpr (NORM) ss = __builtin_fmaf(f, f, ss);
    if constexpr (I8) top = larger(top, magnitude(NORM ? (V)f * (V)to_f32(wt) : (V)f));
  }

  if constexpr (NORM) ss = wave_sum<(LANES < 64 ? LANES : 64)>(ss);
  if constexpr (I8) top = wave_max<(LANES < 64 ? LANES : 64)>(top);
  if constexpr (WAVES > 1) {
    __shared__ float ss_all[WAVES];
    __shared__ M top_all[WAVES];
    if ((tid & 63) == 0) {
      ss_all[tid >> 6] = ss;
      top_all[tid >> 6] = top;
    }
    __syncthreads();
    ss = 0.f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      if constexpr (NORM) ss += ss_all[w];
      if constexpr (I8) top = larger(top, top_all[w]);
    }
  }
  float inv = 1.f;
  if constexpr (NORM) inv = inverse_root(ss, k, a.eps);

  // r of the long rows comes again from where this thread left it
  const T* const again = NORM && res ? sum : x;
  if constexpr (!I8) {
    T* const y = static_cast<T*>(a.y) + base;
    auto put = [&](u32x4 v, u32x4 wv, int64_t j) __attribute__((always_inline)) {
      float f[E], w[E];
      unpack(v, f);
      unpack(wv, w);
#pragma unroll
      for (int i = 0; i < E; ++i) f[i] = f[i] * inv * w[i];
      store_piece(y + j * E, pack(f));
    };
    if constexpr (P > 0) {
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const int64_t j = p * LANES + tid;
        if (j < pieces) put(r[p], wp[p], j);
      }
    } else {
      for (int64_t j = tid; j < pieces; j += LANES) put(load_piece(again + j * E), load_piece(weight + j * E), j);
    }
    if (tid < tail) y[tcol] = from_f32<T>(to_f32(rt) * inv * to_f32(wt));
  } else {
    const double most = value_of(top);
    const bool finite = is_finite(top);
    double f = 0.0;  // rows of zeros: codes and scale 0; rows that are not finite: codes 0, scale NaN
    if constexpr (OUT == OUT_WEIGHT) {
      const uint32_t sb = finite ? f32_to_bf16_bits((float)(most / 127.0)) : 0x7FC0u;
      const float s = bf16_bits_to_f32(sb);
      if (finite && s > 0.f) f = 1.0 / (double)s;
      if (tid == 0) static_cast<uint16_t*>(a.scales)[row] = (uint16_t)sb;
    } else {
      if (finite && most > 0.0) f = 127.0 / most;
      if (tid == 0)
        static_cast<float*>(a.scales)[row] = finite ? (float)(most * (double)inv / 127.0) : __uint_as_float(0x7FC00000u);
    }
    auto code = [&](float v, float w) __attribute__((always_inline)) {
      const V p = NORM ? (V)v * (V)w : (V)v;
      int32_t c = code_of((double)p, f);
      // a scale rounded down takes the largest values beyond the last code
      if constexpr (OUT == OUT_WEIGHT) c = c > 127 ? 127 : c < -127 ? -127 : c;
      return finite ? c : 0;
    };
    int8_t* const out = a.codes + base;
    auto put = [&](u32x4 v, u32x4 wv, int64_t j) __attribute__((always_inline)) {
      float x0[E], w[E];
      unpack(v, x0);
      if constexpr (NORM) unpack(wv, w);
      else {
#pragma unroll
        for (int i = 0; i < E; ++i) w[i] = 1.f;
      }
      int32_t c[E];
#pragma unroll
      for (int i = 0; i < E; ++i) c[i] = code(x0[i], w[i]);
      if constexpr (E == 8)
        *reinterpret_cast<Codes8*>(out + j * E) = Codes8{pack4(c[0], c[1], c[2], c[3]), pack4(c[4], c[5], c[6], c[7])};
      else
        *reinterpret_cast<Codes4*>(out + j * E) = Codes4{pack4(c[0], c[1], c[2], c[3])};
    };
    if constexpr (P > 0) {
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const int64_t j = p * LANES + tid;
        if (j < pieces) put(r[p], wp[p], j);
      }
    } else {
      for (int64_t j = tid; j < pieces; j += LANES)
        put(load_piece(again + j * E), NORM ? load_piece(weight + j * E) : (u32x4){0, 0, 0, 0}, j);
    }
    if (tid < tail) out[tcol] = (int8_t)code(to_f32(rt), to_f32(wt));
  }
}

// ---------------------------------------------------------------------------------------------
// Gradients.  A workgroup takes the rows wg, wg + W, ... and keeps its columns' sums of dy r inv in
// registers (rows of many pieces: in its row of the workspace); the sums of the W workgroups meet in a
// second launch, in order.
// ---------------------------------------------------------------------------------------------
struct NormGradArgs {
  const void* dy;
  const void* d_sum;  // null: none
  const void* sum;    // r
  const void* weight;
  void* dx;
  float* parts;       // [workgroups][k], null: no gradient of the weight
  float eps;
  int64_t n, k;
};

template <typename T, int LANES, int P>
__global__ __launch_bounds__(LANES < 256 ? 256 : LANES) void norm_grad_kernel(const NormGradArgs a) {
  constexpr int E = 16 / (int)sizeof(T);
  constexpr int WAVES = LANES < 64 ? 1 : LANES / 64, GROUPS = LANES < 256 ? 256 / LANES : 1;
  const int tid = LANES < 256 ? (int)threadIdx.x % LANES : (int)threadIdx.x;
  const int group = LANES < 256 ? (int)threadIdx.x / LANES : 0;
  const int64_t k = a.k, pieces = k / E;
  const int tail = (int)(k % E);
  const int64_t tcol = pieces * E + tid;
  const T* const weight = static_cast<const T*>(a.weight);
  float* const part = a.parts ? a.parts + (int64_t)blockIdx.x * k : nullptr;
  __shared__ float ss_all[2][WAVES], dot_all[2][WAVES];
  __shared__ float meet[GROUPS > 1 ? 256 * (P * E + 1) : 1];

  u32x4 wp[P > 0 ? P : 1];
  float dw[P > 0 ? P : 1][E], dwt = 0.f;
  float wt = 0.f;
  if constexpr (P > 0) {
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int64_t j = p * LANES + tid;
      wp[p] = (u32x4){0, 0, 0, 0};
      if (j < pieces) wp[p] = load_piece(weight + j * E);
#pragma unroll
      for (int i = 0; i < E; ++i) dw[p][i] = 0.f;
    }
  }
  if (tid < tail) wt = to_f32(weight[tcol]);

  int turn = 0;
  bool begun = false;
  const int64_t row0 = (int64_t)blockIdx.x * GROUPS + group, stride = (int64_t)gridDim.x * GROUPS;
  for (int64_t row = row0; row < a.n; row += stride) {
    const int64_t base = row * k;
    const T* const dy = static_cast<const T*>(a.dy) + base;
    const T* const r = static_cast<const T*>(a.sum) + base;
    const T* const ds = a.d_sum ? static_cast<const T*>(a.d_sum) + base : nullptr;
    T* const dx = static_cast<T*>(a.dx) + base;
    float ss = 0.f, dot = 0.f;
    auto take = [&](u32x4 rv, u32x4 gv, u32x4 wv) __attribute__((always_inline)) {
      float f[E], g[E], w[E];
      unpack(rv, f);
      unpack(gv, g);
      unpack(wv, w);
#pragma unroll
      for (int i = 0; i < E; ++i) {
        ss = __builtin_fmaf(f[i], f[i], ss);
        dot = __builtin_fmaf(g[i] * w[i], f[i], dot);
      }
    };
    u32x4 rv[P > 0 ? P : 1], gv[P > 0 ? P : 1], sv[P > 0 ? P : 1];
    float rt = 0.f, gt = 0.f;
    if constexpr (P > 0) {
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const int64_t j = p * LANES + tid;
        rv[p] = gv[p] = sv[p] = (u32x4){0, 0, 0, 0};
        if (j < pieces) {
          rv[p] = load_piece(r + j * E);
          gv[p] = load_piece(dy + j * E);
          if (ds) sv[p] = load_piece(ds + j * E);
        }
      }
#pragma unroll
      for (int p = 0; p < P; ++p) take(rv[p], gv[p], wp[p]);
    } else {
      for (int64_t j = tid; j < pieces; j += LANES)
        take(load_piece(r + j * E), load_piece(dy + j * E), load_piece(weight + j * E));
    }
    if (tid < tail) {
      rt = to_f32(r[tcol]);
      gt = to_f32(dy[tcol]);
      ss = __builtin_fmaf(rt, rt, ss);
      dot = __builtin_fmaf(gt * wt, rt, dot);
    }
    ss = wave_sum<(LANES < 64 ? LANES : 64)>(ss);
    dot = wave_sum<(LANES < 64 ? LANES : 64)>(dot);
    if constexpr (WAVES > 1) {
      if ((tid & 63) == 0) {
        ss_all[turn][tid >> 6] = ss;
        dot_all[turn][tid >> 6] = dot;
      }
      __syncthreads();  // one a row: the next row's sums go to the other half
      ss = dot = 0.f;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) {
        ss += ss_all[turn][w];
        dot += dot_all[turn][w];
      }
      turn ^= 1;
    }
    const float inv = inverse_root(ss, k, a.eps);
    const float m = dot / (float)k * inv * inv;
    auto put = [&](u32x4 rv1, u32x4 gv1, u32x4 wv, u32x4 sv1, int64_t j, float (&d)[E]) __attribute__((always_inline)) {
      float f[E], g[E], w[E], s[E];
      unpack(rv1, f);
      unpack(gv1, g);
      unpack(wv, w);
      unpack(sv1, s);
#pragma unroll
      for (int i = 0; i < E; ++i) {
        d[i] = __builtin_fmaf(g[i], f[i] * inv, d[i]);
        s[i] += inv * __builtin_fmaf(-f[i], m, g[i] * w[i]);
      }
      if (j < pieces) store_piece(dx + j * E, pack(s));
    };
    if constexpr (P > 0) {
#pragma unroll
      for (int p = 0; p < P; ++p) put(rv[p], gv[p], wp[p], sv[p], p * LANES + tid, dw[p]);
    } else {
      for (int64_t j = tid; j < pieces; j += LANES) {
        float d[E];
#pragma unroll
        for (int i = 0; i < E; ++i) d[i] = part && begun ? part[j * E + i] : 0.f;
        put(load_piece(r + j * E), load_piece(dy + j * E), load_piece(weight + j * E),
            ds ? load_piece(ds + j * E) : (u32x4){0, 0, 0, 0}, j, d);
        if (part)
#pragma unroll
          for (int i = 0; i < E; ++i) part[j * E + i] = d[i];
      }
    }
    if (tid < tail) {
      dwt = __builtin_fmaf(gt, rt * inv, dwt);
      const float s = ds ? to_f32(ds[tcol]) : 0.f;
      dx[tcol] = from_f32<T>(s + inv * __builtin_fmaf(-rt, m, gt * wt));
    }
    begun = true;
  }
  if (!part) return;
  if constexpr (GROUPS > 1) {  // the groups' sums, in order
    constexpr int S = P * E + 1;
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int i = 0; i < E; ++i) meet[(p * E + i) * 256 + threadIdx.x] = dw[p][i];
    meet[(S - 1) * 256 + threadIdx.x] = dwt;
    __syncthreads();
    if (group != 0) return;
#pragma unroll
    for (int g = 1; g < GROUPS; ++g) {
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int i = 0; i < E; ++i) dw[p][i] += meet[(p * E + i) * 256 + g * LANES + tid];
      dwt += meet[(S - 1) * 256 + g * LANES + tid];
    }
  }
  if constexpr (P > 0) {
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int64_t j = p * LANES + tid;
      if (j < pieces)
#pragma unroll
        for (int i = 0; i < E; ++i) part[j * E + i] = dw[p][i];
    }
  }
  if (tid < tail) part[tcol] = dwt;
}

// d_weight[c] = sum over the parts, in fp64 (up to 512 of them; chains of 32 and 16 in fp32 were off by 1.25e-7 of the
// gradient at 333 x 1111 fp32, this by 6.3e-8) and in a fixed order: 64 columns a workgroup, a sixteenth of the parts
// a wave, and then the sixteenths.  Eight loads of a lane in flight, none under a condition: the parts have just been
// written, and with one at a time (and four waves) their way back took longer than the kernel before (4096 x 8192:
// 35 us).
constexpr int kPartWaves = 16;
__global__ __launch_bounds__(64 * kPartWaves) void norm_parts_kernel(const float* __restrict__ parts, int32_t count,
                                                                     int64_t k, float* __restrict__ out, int64_t first) {
  __shared__ double meet[kPartWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t c = (first + blockIdx.x) * 64 + lane;
  const int32_t from = (int32_t)((int64_t)count * wave / kPartWaves), to = (int32_t)((int64_t)count * (wave + 1) / kPartWaves);
  double s = 0.0;
  if (c < k) {
    const float* p = parts + (int64_t)from * k + c;
    int32_t left = to - from;
    const auto add = [&](auto count) __attribute__((always_inline)) {
      constexpr int U = decltype(count)::value;
      float v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) v[u] = p[u * k];
      double t[2] = {0.0, 0.0};
#pragma unroll
      for (int u = 0; u < U; ++u) t[u & 1] += (double)v[u];
      s += t[0] + t[1];
      p += U * k;
      left -= U;
    };
    while (left >= 8) add(std::integral_constant<int, 8>{});
    if (left >= 4) add(std::integral_constant<int, 4>{});
    if (left >= 2) add(std::integral_constant<int, 2>{});
    if (left > 0) add(std::integral_constant<int, 1>{});
  }
  meet[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && c < k) {
    double all[2] = {0.0, 0.0};
#pragma unroll
    for (int w = 0; w < kPartWaves; ++w) all[w & 1] += meet[w][lane];
    out[c] = (float)(all[0] + all[1]);
  }
}

// Lanes of a row x pieces of a lane.
enum Shape { S16x1, S64x1, S64x2, S64x4, S256x1, S256x2, S1024x1, S1024x2, S1024x4, S1024x8, S_LOOP };
int64_t pieces_of(int64_t k, int f32) { return k / (f32 ? 4 : 8); }

// By what was measured on both sides (us, in a graph, rows from memory; norm, in int8, gradient):
//   16 lanes for rows of up to 16 pieces, a wave above (16 / 64): 65536 x 128 bf16 15.5 / 25.1, 16.8 / 33.6, 21 / 45
//   with at most a row for every CU the lanes that take a piece each (64x2 / 256x1: 1 x 1111 3.3 / 2.4;
//     256x2 / 1024x1: 32 x 4096 3.0 / 2.6, 3.3 / 3.0, 5.9 / 5.6)
//   with more rows few lanes, for a row of several waves waits for them all: 32768 x 1024 (64x2 / 256x1) 53.7 /
//     50.5, 50.0 / 54.8, 59 / 101;  8192 x 4096 (256x2 / 1024x1) 51.9 / 54.0, 48.7 / 55.4, 61 / 71;  but 4096 x
//     8192 (256x4 / 1024x1) 56.3 / 54.0, 52.5 / 51.2, 64 / 63
//   129 to 256 pieces, 16384 x 2048 (64x4 / 256x1): 57.0 / 51.4, 53.9 / 47.9, 61 / 65
//   long rows from registers as far as they hold them: 512 x 65536 (1024x8 / read again) 56 / 70, 60 / 64; the
//     gradient holds three arrays and its columns' sums, up to 2048 pieces (above 1024 of bf16 16 of its 128
//     registers spill: 1024 x 16384 42 us where the bytes take 24); longer rows are read twice and their columns'
//     sums go through the workspace for every row, 8 bytes more a value (512 x 65536 131, the bytes 48)
Shape shape_of(int64_t n, int64_t pieces, bool grad) {
  if (pieces <= 16) return S16x1;
  if (pieces <= 64) return S64x1;
  if (n <= 256) {
    if (pieces <= 256) return S256x1;
    if (pieces <= 1024) return S1024x1;
  }
  if (pieces <= 128) return S64x2;
  if (pieces <= 256) return grad ? S64x4 : S256x1;
  if (pieces <= 512) return S256x2;
  if (pieces <= 1024) return S1024x1;
  if (pieces <= 2048) return S1024x2;
  if (pieces <= 4096 && !grad) return S1024x4;
  if (pieces <= 8192 && !grad) return S1024x8;
  return S_LOOP;
}
Shape grad_shape_of(int64_t n, int64_t k, int f32) { return shape_of(n, pieces_of(k, f32), true); }

// run(lanes, pieces) with the shape's constants; the gradient has no shapes above 2048 pieces, the norm no 64x4.
template <bool GRAD, class Run>
hipError_t with_shape(Shape s, Run run) {
#define WQ_SHAPE(L, P) return run(std::integral_constant<int, L>{}, std::integral_constant<int, P>{})
  switch (s) {
    case S16x1: WQ_SHAPE(16, 1);
    case S64x1: WQ_SHAPE(64, 1);
    case S64x2: WQ_SHAPE(64, 2);
    case S256x1: WQ_SHAPE(256, 1);
    case S256x2: WQ_SHAPE(256, 2);
    case S1024x1: WQ_SHAPE(1024, 1);
    case S1024x2: WQ_SHAPE(1024, 2);
    default: break;
  }
  if constexpr (GRAD) {
    if (s == S64x4) WQ_SHAPE(64, 4);
  } else {
    if (s == S1024x4) WQ_SHAPE(1024, 4);
    if (s == S1024x8) WQ_SHAPE(1024, 8);
  }
  WQ_SHAPE(1024, 0);
#undef WQ_SHAPE
}

template <typename T, int OUT>
hipError_t norm_t(const NormArgs& a, hipStream_t s) {
  return with_shape<false>(shape_of(a.n, pieces_of(a.k, sizeof(T) == 4), false), [&](auto lanes, auto pieces) {
    constexpr int LANES = decltype(lanes)::value, P = decltype(pieces)::value;
    constexpr int threads = LANES < 256 ? 256 : LANES, rows = threads / LANES;
    return launch_in_parts((a.n + rows - 1) / rows, [&](int64_t first, dim3 grid) {
      hipLaunchKernelGGL((norm_kernel<T, LANES, P, OUT>), grid, dim3(threads), 0, s, a, first);
    }, threads);
  });
}
template <int OUT>
hipError_t norm_any(const NormArgs& a, int f32, hipStream_t s) {
  return f32 ? norm_t<float, OUT>(a, s) : norm_t<uint16_t, OUT>(a, s);
}

// Workgroups of the gradient: as many as a CU holds at a time, for each leaves a row of parts (256, 512, 1024:
// 4096 x 8192 63, 66, 72 us; 65536 x 512 85, 59, 64); fewer for few rows.
int64_t grad_workgroups(int64_t n, int64_t k, int f32) {
  const Shape s = grad_shape_of(n, k, f32);
  const int64_t rows = s == S16x1 ? 16 : s <= S64x4 ? 4 : 1, most = s >= S1024x1 ? 256 : 512;
  const int64_t all = (n + rows - 1) / rows;
  return all < most ? all : most;
}
template <typename T>
hipError_t grad_t(const NormGradArgs& a, int64_t wgs, hipStream_t s) {
  return with_shape<true>(grad_shape_of(a.n, a.k, sizeof(T) == 4), [&](auto lanes, auto pieces) {
    constexpr int LANES = decltype(lanes)::value, P = decltype(pieces)::value;
    hipLaunchKernelGGL((norm_grad_kernel<T, LANES, P>), dim3((unsigned)wgs), dim3(LANES < 256 ? 256 : LANES), 0, s, a);
    return hipGetLastError();
  });
}

}  // namespace

hipError_t launch_quantize_i8(const void* x, int f32, int64_t n, int64_t k, int8_t* codes, void* scales,
                              int scales_f32, hipStream_t stream) {
  NormArgs a{};
  a.x = x;
  a.codes = codes;
  a.scales = scales;
  a.n = n;
  a.k = k;
  return scales_f32 ? norm_any<OUT_ROWS>(a, f32, stream) : norm_any<OUT_WEIGHT>(a, f32, stream);
}

hipError_t launch_norm(const void* x, int f32, const void* residual, const void* weight, float eps, int64_t n,
                       int64_t k, void* sum, void* y, int8_t* codes, float* scales, hipStream_t stream) {
  const NormArgs a{x, residual, weight, sum, y, codes, scales, eps, n, k};
  return codes ? norm_any<OUT_NORM_I8>(a, f32, stream) : norm_any<OUT_NORM>(a, f32, stream);
}

int64_t norm_grad_parts(int64_t n, int64_t k, int f32) {
  const int64_t wgs = grad_workgroups(n, k, f32);
  return wgs > 1 ? wgs : 0;
}

hipError_t launch_norm_grad(const void* dy, int f32, const void* d_sum, const void* sum, const void* weight,
                            float eps, int64_t n, int64_t k, void* dx, float* d_weight, float* parts,
                            hipStream_t stream) {
  const int64_t wgs = grad_workgroups(n, k, f32);
  if (wgs > 0) {
    // one workgroup's sums are the gradient
    const NormGradArgs a{dy, d_sum, sum, weight, dx, !d_weight ? nullptr : wgs > 1 ? parts : d_weight, eps, n, k};
    const hipError_t e = f32 ? grad_t<float>(a, wgs, stream) : grad_t<uint16_t>(a, wgs, stream);
    if (e != hipSuccess) return e;
  }
  if (!d_weight || wgs == 1) return hipSuccess;  // (no workgroup: no parts, zeros)
  return launch_in_parts((k + 63) / 64, [&](int64_t first, dim3 grid) {
    hipLaunchKernelGGL(norm_parts_kernel, grid, dim3(64 * kPartWaves), 0, stream, parts, (int32_t)wgs, k, d_weight, first);
  }, 64 * kPartWaves);
}

}  // namespace wq
