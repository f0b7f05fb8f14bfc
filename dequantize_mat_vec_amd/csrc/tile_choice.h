// Which kernel of gemm_tile.h serves a shape, and how many workgroups it gets:
// arithmetic on sizes alone, without HIP, so that a host program can ask for
// the kernel that a call would take.
#pragma once

#include <algorithm>
#include <cstdint>

namespace pesti_host {

constexpr int64_t kCus = 256, kCuLds = 160 * 1024;   // compute units, bytes of LDS on each

struct TileShape {
  int64_t rows;
  int64_t n;
  int64_t experts;   // 0: one matrix, all rows
  int64_t kbytes;    // bytes of a row of X or W
  bool gated;        // gate and up projections joined
};

// kRows*: the rows kernel with that many rows of Y a workgroup.
enum class TileKernel { kRows16, kRows32, kRows64, kTile64x128, kTile128x128, kTile128x256, kTile256x256 };

// Wavefronts of the rows kernel, of 4 lines in flight each where there are 2
// and of 5 where there are 4.  Few lines are issued in vain past the end of
// short rows, more are in flight for long ones (us for 2 x 4 and 4 x 5): one
// row of 8-bit 896x896 3.2 / 3.6, 16x4864x896 4.5 / 5.2, eight experts of one row,
// 1024x2048, 6.6 / 6.8, gated 9.5 / 9.8; against these 8x896x2080 4.0 / 3.9, rows
// of 4864 bytes 6.3 / 6.3, four binary16 experts of one row, 896x2432,
// 7.4 / 6.9.  Not on the better side: eight gated binary16 ones, 1024x2048 (rows
// of 4096 bytes), 13.4 / 14.9.
constexpr int rows_wavefronts(int64_t kbytes) { return kbytes <= 2048 ? 2 : 4; }

// Dynamic LDS of the tile kernel: two steps of X and W, two sets of scales and
// bias, the next tile's rows of X, the tile table.
constexpr int64_t tile_lds(const TileShape& s, int64_t bm, int64_t bn) {
  return (bm + bn) * 128 * 2 + 2 * 4 * (bm + 2 * bn) + 4 * bm + 16 * s.experts;
}
// Its workgroups at most: they fill the chip once and take tiles in turn.
constexpr int64_t tile_workgroups(const TileShape& s, int64_t bm, int64_t bn) {
  return kCus * (kCuLds / tile_lds(s, bm, bn));
}

// Most row tiles of height bm there can be: each expert with rows ends in at
// most one partial tile.
inline int64_t most_row_tiles(const TileShape& s, int64_t bm) {
  if (!s.experts) return (s.rows + bm - 1) / bm;
  return s.rows / bm + std::min(s.experts, s.rows);
}

// Tiles of bm rows and cols columns that a launch comes to, in tenths: a half
// tile takes 6 tenths of a whole one's time, and an expert's last tile,
// anywhere from empty to full, on average 3 more than its rows' share.
inline int64_t tenths_of_tiles(const TileShape& s, int64_t bm, int64_t cols) {
  int64_t row_tiles;
  if (s.experts) {
    row_tiles = s.rows * 10 / bm + 3 * std::min(s.experts, s.rows);
  } else {
    const int64_t left = s.rows % bm;
    row_tiles = s.rows / bm * 10 + (left > bm / 2 ? 10 : left > 0 ? 6 : 0);
  }
  return row_tiles * ((s.n + cols - 1) / cols);
}

// The kernel for a shape.
//
// Fewer 64 x 128 tiles than compute units leave them idle: the rows kernel
// takes over as long as its workgroups fit the chip about once, with the
// fewest rows each that do it (us for 16, 32 and 64 rows and the 64 x 128
// tile: 8-bit 64x896x4864 7.2 / 9.4 / 13 / 16, 128x896x4864 12 / 9.7 / 14 / 17,
// 256x896x4864 21 / 16 / 14 / 17, 100x4864x896 10 / 9.3 / 9.4 / 7.3; 8 experts of one
// row, gated 1024x2048, 9.4 against 12; but 40x4864x896 6.1 / 6.9 / 6.3 / 6.9, whose
// workgroups of 16 rows fit the chip three and a half times).
// With more tiles, tiles win for one row as for many (8-bit 1x151936x896 27
// against 28 us, 16x151936x896 31 against 38), but for experts of up to four
// rows with long rows of W or with few tiles: two tokens of four experts,
// binary16 896x2432, 9.9 against 18 us, eight 21 against 25; 24 tokens of
// eight of 64 experts, gated 8-bit 1024x2048, 43 against 46; but 60 experts of
// two rows, 2944x896, 26 against 24, of 1024 and more tiles.
//
// Among the tiles, time goes by how many each compute unit gets.  The price
// of a tile, in tenths of a 64 x 128 one: 128 x 128 16, 128 x 256 30,
// 256 x 256 53 (a product costs (BM + BN) / (BM BN) bytes into LDS).  The least
// of tiles per unit times price is taken.  Measured (us at 64x128 / 128x128 /
// 128x256 / 256x256; the rule's choice in brackets): 8-bit 8192x4096x4096
// 167 / 144 / 130 / [110], 4096x4096x4096 80 / 65 / 64 / [57], 2048x4864x896
// 19 / [20] / 22 / 20, 4096x896x4864 28 / [26] / 34 / 52, 513x2304x768 [6.9] / 8.5 /
// 14 / 18; 64 experts, 512 rows each, 2048x1024 147 / 120 / 113 / [110]; 60
// experts, 173 rows, 1408x2048 77 / [63] / 67 / 60; binary16, 8 experts, 255
// rows, 2429x1056 28 / 28 / [25] / 34, gated, 32 experts, 256 rows, 1408x2048
// 194 / 155 / 151 / [149].
inline TileKernel tile_kernel(const TileShape& s) {
  const int64_t g = s.gated ? 2 : 1;
  const int64_t tiles = most_row_tiles(s, 64) * ((s.n + 128 / g - 1) / (128 / g));
  if (s.experts && s.rows <= 4 * s.experts && (tiles < 2 * kCus || s.kbytes >= 2048)) return TileKernel::kRows16;
  if (tiles < kCus) {
    const int64_t cols = (s.n + 15) / 16, limit = kCus * 3 / 2;
    const int64_t r1 = most_row_tiles(s, 16), r2 = most_row_tiles(s, 32), r4 = most_row_tiles(s, 64);
    if (r1 * cols <= limit || r1 == r4) return TileKernel::kRows16;
    if (r2 * cols <= limit || (s.gated && r2 == r4)) return TileKernel::kRows32;
    if (!s.gated && r4 * cols <= kCus) return TileKernel::kRows64;
  }
  auto cost = [&](int64_t bm, int64_t bn, int64_t unit) {
    return (tenths_of_tiles(s, bm, bn / g) + 10 * kCus - 1) / (10 * kCus) * unit;
  };
  const int64_t c0 = cost(64, 128, 10), c1 = cost(128, 128, 16), c2 = cost(128, 256, 30), c3 = cost(256, 256, 53);
  const int64_t low = std::min(std::min(c0, c1), std::min(c2, c3));
  if (c3 == low) return TileKernel::kTile256x256;
  if (c2 == low) return TileKernel::kTile128x256;
  if (c1 == low) return TileKernel::kTile128x128;
  return TileKernel::kTile64x128;
}

}  // namespace pesti_host
