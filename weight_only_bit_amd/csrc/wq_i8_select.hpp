// wq_i8_select.hpp -- which kernel of wq_i8.hip a product of two int8 operands takes.  Plain host C++: the
// rules hold no device code, so their borders can be looked at without a GPU.
#pragma once

#include <cstdint>

namespace wq {

// Rows x columns of a workgroup's outputs.
enum I8Kernel : int32_t {
  I8_STREAM_16 = 0,  // 16 x 16, weights straight from memory
  I8_STREAM_32,      // 32 x 16
  I8_TILES_64,       // 64 x 64, two buffers
  I8_TILES_128,      // 128 x 128, two buffers
  I8_TILES_128x256,  // two buffers
  I8_TILES_128x256_ONE,  // one buffer, two workgroups per CU
  I8_TILES_256       // 256 x 256, two buffers
};

// The sum of k products of two codes (at most 2^14 each) stays below 2^31.
constexpr int64_t kI8MaxK = 131008;

inline int64_t i8_ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The tiles' 32-bit ranges: one expert's codes and, gathered, the codes of `gathered` tokens (0: rows are
// not gathered), each below 2^31 less a stage's bytes: gathered rows lie anywhere, so one range covers them
// all, and from 262144 tokens of hidden 8192 on gate+up streams 16 rows at a time.
inline bool i8_tiles_fit(int64_t gathered, int64_t N, int64_t K) {
  constexpr int64_t most = (1ll << 31) - 1024;
  return N * K <= most && gathered * K <= most;
}

inline I8Kernel i8_dense_kernel(int64_t M, int64_t N, int64_t K) {
  const auto tiles = [&](int64_t bm, int64_t bn) { return i8_ceil_div(M, bm) * i8_ceil_div(N, bn); };
  if (M > 32 && i8_tiles_fit(0, N, K)) {
    if (tiles(256, 256) >= 192 && K > 1024) return I8_TILES_256;
    if (tiles(128, 256) >= 512) return I8_TILES_128x256_ONE;
    if (tiles(128, 256) >= 192) return I8_TILES_128x256;
    if (tiles(128, 128) >= 128) return I8_TILES_128;
    if (tiles(32, 16) >= 850) return I8_TILES_64;
  }
  return M > 16 && tiles(32, 16) >= 256 ? I8_STREAM_32 : I8_STREAM_16;
}

// The same for experts, `pairs` rows in all, gate+up of `gathered` tokens (down: 0), by the rows that an
// expert has on average.
inline I8Kernel i8_experts_kernel(int64_t gathered, int64_t pairs, int64_t N, int64_t K, int64_t experts) {
  const int64_t active = pairs < experts ? pairs : experts;  // at most
  const double rows = (double)pairs / (double)experts;
  const int64_t cols = i8_ceil_div(gathered ? 2 * N : N, 256);
  if (!i8_tiles_fit(gathered, N, K) || rows < 3.0) return I8_STREAM_16;
  if ((pairs / 128 + active) * cols < 128) return rows <= 32.0 ? I8_STREAM_16 : I8_TILES_128;
  if (rows < 128.0) return I8_TILES_128x256;
  if (K <= 1024 || (pairs / 256 + active) * cols < 512) return I8_TILES_128x256_ONE;
  return I8_TILES_256;
}

}  // namespace wq
