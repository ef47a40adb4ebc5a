// wq_mx_select.hpp -- which kernel of wq_mx.hip a product of two MXFP4 operands takes.  Plain host C++: the
// rules hold no device code, so their borders can be looked at without a GPU.
#pragma once

#include <cstdint>

namespace wq {

// Rows x columns of a workgroup's outputs.
enum MxKernel : int32_t {
  MX_STREAM_16 = 0,  // 16 x 16, weights straight from memory
  MX_STREAM_32,      // 32 x 16
  MX_TILES_64,       // 64 x 64, two buffers
  MX_TILES_128,      // 128 x 128, two buffers
  MX_TILES_128x256,  // two buffers
  MX_TILES_128x256_ONE,  // one buffer, two workgroups per CU
  MX_TILES_256       // 256 x 256, two buffers
};

inline int64_t mx_ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The tiles' 32-bit ranges: one expert's codes, a tile's rows (k below 2^23) and, gathered, the codes of
// `gathered` tokens (0: rows are not gathered), each below 2^31 less a stage's bytes: gathered rows lie
// anywhere, so one range covers them all, and from 524288 tokens of hidden 8192 on gate+up streams 16 rows
// at a time.  A stage needs 256 columns: k below that streams at every number of rows.
inline bool mx_tiles_fit(int64_t gathered, int64_t N, int64_t K) {
  constexpr int64_t most = (1ll << 31) - 1024;
  if (K < 256 || K >= (1ll << 23) || N * (K / 2) > most) return false;
  return gathered * (K / 2) <= most;
}

// By what was measured on both sides of each border (us, in a graph, weights from memory):
//   256 x 256 tiles, one workgroup per CU, for long k; 128 x 256 with one buffer, two per CU, whose
//   neighbour covers a tile's start and end, for short k (256 x 256 / 128 x 256):
//     8192 x 8192, k 1024: 74 / 63;  k 2048: 100 / 97;  k 4096: 168 / 175;  4096 x 8192, k 8192: 150 / 164
//   128 x 256 with one buffer from 512 tiles on, two buffers below (one / two): 4096 x 4096 (512), k 1024:
//     19 / 25;  3000 x 2048 (192), k 1024: 12.5 / 11.7, k 4096: 34 / 23.5
//   128 x 128 where 128 x 256 would leave CUs without a tile (128 x 128 / 128 x 256): 2048 x 2048 (128), k
//     4096: 18.1 / 21.3;  3000 x 2048 (192): 28 / 23.5
//   64 x 64 where 128 x 128 would (64 x 64 / 128 x 128): 256 x 4096 (64 tiles of 128 x 128), k 4096: 10.9 /
//     14.8;  512 x 4096 (128): 19.2 / 15.4
//   streaming where few workgroups of 32 x 16 suffice (streaming / 64 x 64, k 512, 2048, 4096, 8192):
//     64 x 4096 (512 of them): 4.2 / 4.0, 7.0 / 6.6, 10.4 / 11.0, 17.0 / 18.1
//     333 x 1111 (770): 5.4 / 4.4, 9.8 / 6.7, 15.0 / 11.0, 26.7 / 17.5 (the border lies late)
//     128 x 4096 (1024): 5.4 / 4.0, 11.0 / 6.7, 17.0 / 10.9, 30 / 18.0
inline MxKernel mx_dense_kernel(int64_t M, int64_t N, int64_t K) {
  const auto tiles = [&](int64_t bm, int64_t bn) { return mx_ceil_div(M, bm) * mx_ceil_div(N, bn); };
  if (M > 32 && mx_tiles_fit(0, N, K)) {
    if (tiles(256, 256) >= 192 && K > 2048) return MX_TILES_256;
    if (tiles(128, 256) >= 512) return MX_TILES_128x256_ONE;
    if (tiles(128, 256) >= 192) return MX_TILES_128x256;
    if (tiles(128, 128) >= 128) return MX_TILES_128;
    if (tiles(32, 16) >= 850) return MX_TILES_64;
  }
  // 16 rows a workgroup where 32 would leave CUs without one: 64 x 1024, k 8192: 7.3 against 9.8
  return M > 16 && tiles(32, 16) >= 256 ? MX_STREAM_32 : MX_STREAM_16;
}

// The same for experts, `pairs` rows in all, gate+up of `gathered` tokens (down: 0), by the rows that an
// expert has on average (gate+up, down; 64 experts, hidden 8192, inter 3584 unless said otherwise):
//   streaming for few, else 128 x 256 tiles (streaming / tiles): 2 rows 292 / 302, 186 / 179; 3 rows 342 /
//     338, 205 / 185; 4 rows 367 / 350, 219 / 188
//   with few tiles streaming up to 32 rows, then 128 x 128 (8 experts, 1024 x 1024): 8 rows 4.8 / 6.2, 4.1 /
//     5.7; 16 rows 6.4 / 6.2, 4.9 / 5.8; 32 rows 7.9 / 6.3, 6.6 / 5.9
//   128 x 256 tiles (64 rows where an expert has no more) below 128 rows, 256 x 256 from there (128 x 256 /
//     256 x 256): 64 rows 431 / 437, 249 / 246; 100 rows 430 / 434, 270 / 267; 128 rows 608 / 497, 342 / 310;
//     512 rows 1592 / 1229, 917 / 779
//   128 x 256 with one buffer for short k (one / two / 256 x 256; down, 16 experts, 4096 x 2048): 200 rows
//     27.9 / 35.9 / 29.3; 512 rows 67 / 80 / 74;  k 4096 (gate+up, 2048 x 4096), 512 rows 119 / 117 / 106
inline MxKernel mx_experts_kernel(int64_t gathered, int64_t pairs, int64_t N, int64_t K, int64_t experts) {
  const int64_t active = pairs < experts ? pairs : experts;  // at most
  const double rows = (double)pairs / (double)experts;
  const int64_t cols = mx_ceil_div(gathered ? 2 * N : N, 256);
  if (!mx_tiles_fit(gathered, N, K) || rows < 3.0) return MX_STREAM_16;
  if ((pairs / 128 + active) * cols < 128) return rows <= 32.0 ? MX_STREAM_16 : MX_TILES_128;
  if (rows < 128.0) return MX_TILES_128x256;
  if (K <= 2048 || (pairs / 256 + active) * cols < 512) return MX_TILES_128x256_ONE;
  return MX_TILES_256;
}

}  // namespace wq
