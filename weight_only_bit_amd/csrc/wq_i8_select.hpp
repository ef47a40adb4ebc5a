// wq_i8_select.hpp -- which kernel of wq_i8.hip a product of two int8 operands takes.  Plain host C++: the
// rules hold no device code, so their borders can be looked at without a GPU.
#pragma once

#include <cstdint>

namespace wq {

// Rows x columns of a workgroup's outputs.
enum I8Kernel : int32_t {
  I8_STREAM_16 = 0,  // 16 x 16, weights straight from memory
  I8_STREAM_32,      // 32 x 16
  I8_NARROW,         // 32 x 16, staged in LDS
  I8_TILES_64,       // 64 x 64
  I8_TILES_128,      // 128 x 128
  I8_TILES_128x256,
  I8_TILES_256       // 256 x 256
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

// By what was measured on both sides of each border (us, in a graph, weights from memory):
//   256 x 256 tiles where they fill the chip (256 x 256 / 128 x 256): 2048 x 8192 (256 tiles), k 8192: 113 / 133;
//     4096 x 4096, k 1024: 24 / 28, k 4096: 62 / 73;  1024 x 8192 (128), k 8192: 79 / 68
//   128 x 256 where those do (128 x 256 / 128 x 128): 1024 x 8192 (256), k 8192: 68 / 75;  2048 x 4096, k 4096: 37 /
//     41;  2048 x 2048 (128), k 4096: 30 / 24
//   128 x 128 above half the chip (128 x 128 / 64 x 64): 640 x 4096 (160), k 4096: 22.8 / 26.1;  320 x 8192 (192), k
//     8192: 41 / 54;  512 x 4096 (128): 22.9 / 19.1;  256 x 8192 (128), k 8192: 43.4 / 39.1
//   but 64 x 64 for up to 64 rows, of which a taller tile computes no more (64 x 64 / 128 x 128 / 256 x 256): 33 x 24576, k
//     8192: 47.4 / 55.6 / 62.9;  33 x 128256, k 4096: 126.6 / 144.4 / 136.5;  64 x 28672: 30.8 / 31.3 / 35.8;  64 x
//     128256: 130.7 / 140.6 / 137.3;  64 x 49152, k 1024: 16.7 / 15.1 / 15.5;  65 x 49152, k 4096: 60.3 / 49.2 / 50.0
//   64 x 64 from a third of the chip on (64 x 64 / 32 x 16 / streaming 32 x 16): 128 x 4096 (128 tiles), k 4096: 13.0 /
//     14.2 / 25;  333 x 1111 (108), k 4160: 10.9 / 11.8 / 16.9;  48 x 5120 (80), k 8192: 21.1 / 21.8 / 33;  256 x 1280
//     (80), k 4096: 10.1 / 9.6 / 18.8;  64 x 4608 (72): 13.8 / 13.3 / 19.5;  256 x 1024 (64), k 8192: 15.9 / 14.1 / 24;
//     17 to 32 rows 32 x 8192 (128), k 8192: 20.9 / 23.1 / 26.2;  32 x 4112 (65), k 4096: 11.7 / 12.1 / 14.2;  at 80
//     tiles either may be 5 % faster
//   streaming where its workgroups are at most one for every CU (streaming / 32 x 16): 32 x 4096 (256), k 4096: 9.5 /
//     11.7;  64 x 2048 (256): 8.6 / 8.6;  96 x 2048 (384): 13.5 / 8.9;  64 x 4096 (512): 14.3 / 12.2;  and 16 rows where
//     those are (16 x 16 / 32 x 16): 32 x 2048 (256) 6.7 / 8.5;  200 x 300 (247), k 8192: 10.4 / 13.8;  32 x 2560 (320), k
//     4096: 9.9 / 8.6;  64 x 1536 (384): 10.0 / 8.6
//   up to 16 rows 64 x 64 where the weights are many (64 x 64 / 16 x 16): 16 x 11264 (176), k 4096: 13.5 / 15.7;  16 x
//     8192 (128): 11.8 / 11.9, k 8192: 19.7 / 20.6;  16 x 6144 (96), k 4096: 11.2 / 11.3;  8 x 28672 (448): 27.5 / 30.7;  8 x
//     11264: 13.4 / 13.6;  1 x 28672: 26.8 / 27.8;  1 x 16384 (256): 18.2 / 16.0;  8 x 8192 (128), k 8192: 19.2 / 18.4
inline I8Kernel i8_dense_kernel(int64_t M, int64_t N, int64_t K) {
  const auto tiles = [&](int64_t bm, int64_t bn) { return i8_ceil_div(M, bm) * i8_ceil_div(N, bn); };
  const bool fit = i8_tiles_fit(0, N, K);
  if (M <= 16) return fit && tiles(64, 64) >= (M > 8 ? 128 : 384) ? I8_TILES_64 : I8_STREAM_16;
  if (tiles(16, 16) <= 256) return I8_STREAM_16;
  if (tiles(32, 16) <= 256 || !fit) return I8_STREAM_32;
  if (M <= 32) return I8_TILES_64;
  if (M > 64) {
    if (tiles(256, 256) >= 192) return I8_TILES_256;
    if (tiles(128, 256) >= 192) return I8_TILES_128x256;
    if (tiles(128, 128) >= 144) return I8_TILES_128;
  }
  return tiles(64, 64) >= 80 ? I8_TILES_64 : I8_NARROW;
}

// The same for experts, `pairs` rows in all, gate+up of `gathered` tokens (down: 0), by the rows that an
// expert has on average, measured with even routing (gate+up, down; 64 experts, hidden 8192, inter 3584 unless said
// otherwise).  Uneven routing costs the streaming kernel, whose workgroup takes an expert's rows 16 at a time, and not the
// tiles (8 experts, 1024 x 1024, 512 rows on average, skew 0 / 1.1: streaming 99 / 209, 128 x 128 tiles 21.2 / 21.3):
//   streaming for few, which reads the weights at memory's rate (streaming / 128 x 256): 3 rows 565 / 618, 302 /
//     312; 4 rows 600 / 642, 332 / 326; 8 rows 623 / 650, 389 / 330; 16 rows 874 / 658, 554 / 337.  Gate+up goes on to
//     10 rows, down, whose k is shorter, to 4; with few tiles to 16 (8 experts, 1024 x 1024; streaming / 128 x 128):
//     8 rows 5.5 / 6.9, 4.3 / 6.4; 16 rows 7.3 / 7.0, 5.2 / 6.4; 32 rows 10.5 / 6.9, 7.4 / 6.5
//   256 x 256 tiles from 128 rows on where they fill the chip, 128 x 256 below (256 x 256 / 128 x 256): 64 rows 691 /
//     690, 378 / 379; 100 rows 719 / 712, 410 / 408; 128 rows 818 / 902, 459 / 525; 512 rows 2019 / 2329, 1112 / 1330
//   128 x 128 where those would be few (128 x 128 / 256 x 256; 8 experts, 1024 x 1024): 128 rows (96 and 48 tiles) 9.3 /
//     18.8, 8.2 / 17.1; 1024 rows (320 and 160) 32.5 / 41.4, 20.4 / 20.2; 16 experts, 2048 x 4096: 200 rows (456) 81 /
//     66, 42.5 / 37.3; and (/ 128 x 256) 64 rows (384) 46.8 / 46.5, 24.8 / 26.7;
//     64 experts, 1024 x 2048: 8 rows (544) 43.8 / 46.4, 25.7 / 27.9, 64 rows (544) 50.4 / 52.2, 28.9 / 32.5; hidden
//     8192, inter 3584: 8 rows (1808) 635 / 632, 329 / 330
//   not told apart: 128 x 256 from 128 rows on, where 256 x 256 tiles are few (/ 128 x 128; 16 experts, 2048 x 4096, 128
//     rows: 75.4 / 87.3, 41.9 / 39.3);  not built: 64 x 64 tiles (/ 128 x 128; 8 experts, 1024 x 1024, 64 rows: 7.9 / 8.8,
//     6.1 / 7.8; 64 experts, 1024 x 2048, 16 rows: 42.8 / 44.6, 27.9 / 26.3, 64 rows: 59.8 / 50.4, 39.6 / 28.9)
inline I8Kernel i8_experts_kernel(int64_t gathered, int64_t pairs, int64_t N, int64_t K, int64_t experts) {
  const int64_t active = pairs < experts ? pairs : experts;  // at most
  const double rows = (double)pairs / (double)experts;
  const int64_t cols = i8_ceil_div(gathered ? 2 * N : N, 256);
  const int64_t tiles = (pairs / 128 + active) * cols;  // of 128 x 256, at most
  if (!i8_tiles_fit(gathered, N, K) || rows < (tiles < 512 ? 16.0 : gathered ? 10.0 : 4.0)) return I8_STREAM_16;
  if (rows < 128.0) return tiles < 700 ? I8_TILES_128 : I8_TILES_128x256;
  return (pairs / 256 + active) * cols < 400 ? I8_TILES_128 : I8_TILES_256;
}

}  // namespace wq
