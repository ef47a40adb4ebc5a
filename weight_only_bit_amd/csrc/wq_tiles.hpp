// wq_tiles.hpp -- what the tiled products with LDS-staged operands share: the order of a grid's tiles
// and the row tiles of an MoE product.
#pragma once
#include "wq_device.hpp"

namespace wq {

// The tile of workgroup wg among row_tiles x col_tiles, in an order for the 8 XCDs (workgroup w runs
// on XCD w % 8, each with an L2 of its own): an XCD takes a contiguous eighth of the list [groups of
// 4 row tiles][column tiles][row tiles of the group], so the tiles that it computes at a time share
// 4 row tiles' activations and a few column tiles' weights.  (Experts' tiles cost unequally; blocks
// of 4 x 8 tiles going round the XCDs even that out, 843 us against 860 for 4096 tokens, but cost
// the decode step of 32 tokens more: 372 against 332.)  false: no tile.
__device__ __forceinline__ bool xcd_tile(uint32_t wg, uint32_t row_tiles, uint32_t col_tiles, int64_t& r,
                                         int64_t& c) {
  const uint32_t total = row_tiles * col_tiles, share = (total + 7) / 8;  // a grid: below 2^31
  const uint32_t k = wg >> 3, t = (wg & 7) * share + k;
  if (k >= share || t >= total) return false;
  const uint32_t group = t / (4 * col_tiles), in = t % (4 * col_tiles);
  const uint32_t left = row_tiles - 4 * group, here = left < 4 ? left : 4;
  c = in / here;
  r = 4 * group + in % here;
  return true;
}

// The same in blocks of kBlockRows x kBlockCols tiles that go round the XCDs, for experts' tiles that cost
// unequally: an XCD's share of the list is then no run of them.  A grid of block_grid workgroups.  (int8, 4096 tokens
// of 64 experts: together with a height of 192 rows down 1127 to 1159 us became 1060 to 1095, gate+up 2034 to 2111 became
// 1955 to 1993; blocks of 2 x 8, 3 x 8, 4 x 4, 4 x 8 and 4 x 16 are slower.)
constexpr uint32_t kBlockRows = 8, kBlockCols = 4;
__host__ __device__ inline int64_t block_grid(int64_t row_tiles, int64_t col_tiles) {
  const int64_t blocks = (row_tiles + kBlockRows - 1) / kBlockRows * ((col_tiles + kBlockCols - 1) / kBlockCols);
  return (blocks + 7) / 8 * 8 * (kBlockRows * kBlockCols);
}
__device__ __forceinline__ bool xcd_block_tile(uint32_t wg, uint32_t row_tiles, uint32_t col_tiles, int64_t& r,
                                               int64_t& c) {
  constexpr uint32_t size = kBlockRows * kBlockCols;
  const uint32_t k = wg >> 3, block = k / size * 8 + (wg & 7), in = k % size;
  const uint32_t across = (col_tiles + kBlockCols - 1) / kBlockCols;
  r = block / across * kBlockRows + in % kBlockRows;
  c = block % across * kBlockCols + in / kBlockRows;
  return r < row_tiles && c < col_tiles;
}

// The row tiles of an MoE product: every expert's rows in tiles of `size`, experts in order.  Every
// wave counts and finds them by itself; lane l holds experts l, l + 64, ...
struct ExpertTiles {
  const int32_t* offsets;
  int32_t experts, size;
  int32_t from, count, incl, tiles;  // of the 64 experts from `base` on: first row, rows, tiles up to
  int32_t base = -1;                 // and with this lane's, this lane's
  __device__ __forceinline__ void load(int32_t eb) {
    if (base == eb) return;
    base = eb;
    const int lane = threadIdx.x & 63, ex = eb + lane;
    from = ex < experts ? offsets[ex] : 0;
    count = ex < experts ? offsets[ex + 1] - from : 0;
    tiles = count > 0 ? (count + size - 1) / size : 0;
    incl = tiles;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int32_t v = __shfl_up(incl, d);
      if (lane >= d) incl += v;
    }
  }
  __device__ __forceinline__ int32_t total() {
    int32_t sum = 0;
    for (int32_t eb = 0; eb < experts; eb += 64) {
      load(eb);
      sum += __builtin_amdgcn_readlane(incl, 63);
    }
    return sum;
  }
  __device__ __forceinline__ void find(int32_t tile, int64_t& e, int64_t& row0, int64_t& rows) {
    for (int32_t eb = 0; eb < experts; eb += 64) {
      load(eb);
      const int32_t all = __builtin_amdgcn_readlane(incl, 63);
      if (tile < all) {
        const uint64_t hit = __ballot(tile >= incl - tiles && tile < incl);
        const int at = __builtin_amdgcn_readfirstlane(__ffsll((unsigned long long)hit) - 1);
        const int32_t k = tile - __builtin_amdgcn_readlane(incl - tiles, at);
        e = eb + at;
        row0 = __builtin_amdgcn_readlane(from, at) + k * size;
        const int32_t left = __builtin_amdgcn_readlane(count, at) - k * size;
        rows = left < size ? left : size;
        return;
      }
      tile -= all;
    }
    rows = 0;
  }
};

}  // namespace wq
