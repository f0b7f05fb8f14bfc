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

// Wavefronts of the rows kernel.
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
// tile: 8-bit 64x896x4864 7.8 / 10 / 14 / 16, 128x896x4864 12 / 10 / 15 / 17,
// 256x896x4864 21 / 18 / 15 / 18, 40x4864x896 6.8 / 7.6 / 7.1 / 7.4, 100x4864x896
// 11 / 10 / 10 / 7.8; 8 experts of one row, gated 1024x2048, 9.9 against 13).
// With more tiles, tiles win for one row as for many (8-bit 1x151936x896 29
// against 30 us, 16x151936x896 32 against 39), but for experts of up to four
// rows with long rows of W or with few tiles: two tokens of four experts,
// binary16 896x2432, 11 against 19 us, eight 23 against 27; 24 tokens of
// eight of 64 experts, gated 8-bit 1024x2048, 44 against 48; but 60 experts of
// two rows, 2944x896, 29 against 25, of 1024 and more tiles.
//
// Among the tiles, time goes by how many each compute unit gets (a 128 x 128
// tile takes 1.6 times a 64 x 128 one, 128 x 256 3 times, 256 x 256 5.3
// times: a product costs (BM + BN) / (BM BN) bytes into LDS), so the
// least of tiles per unit times that is taken.  Measured (us at 64x128 /
// 128x128 / 128x256 / 256x256): 8-bit 8192x4096x4096 175 / 153 / 135 / 114,
// 4096x4096x4096 91 / 70 / 67 / 60, 2048x4864x896 19 / 19 / 22 / 20,
// 4096x896x4864 28 / 24 / 32 / 49, 513x2304x768 7.6 / 8.9 / 11 / 16; 64
// experts, 512 rows each, 2048x1024 147 / 129 / 118 / 114; 60 experts, 173
// rows, 1408x2048 78 / 66 / 68 / 69; binary16, 8 experts, 255 rows,
// 2429x1056 28 / 28 / 26 / 36, gated, 32 experts, 256 rows, 1408x2048 196 /
// 159 / 158 / 172.
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
