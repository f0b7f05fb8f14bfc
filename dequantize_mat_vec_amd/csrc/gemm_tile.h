// Products of rows of X with the rows of one weight matrix, or of one matrix
// per expert: Y = X W^T (+ b) on binary16 or on 8-bit integers with a scale
// per row of X and per row of W.  Shared by the dense 8-bit linear layer
// (csrc/gemm_i8.hip) and the expert-grouped products (csrc/gemm_experts.hip).
//
// Both element types feed the matrix cores the same way: a lane's operand of
// v_mfma_i32_16x16x64_i8 and of v_mfma_f32_16x16x32_f16 is 16 consecutive
// bytes of a row, the four lane groups of a wavefront taking the four
// 16-byte chunks of a 64-byte k-step.  The kernels here therefore count K in
// bytes and differ by type only in the instruction and the epilogue.
//
// The operands are W first and X second, so a lane ends with four
// consecutive output columns of one row of X and stores them at once.
#pragma once

#include <type_traits>

#include "common.h"
#include "tile_choice.h"

namespace pesti {

typedef int i32x4 __attribute__((ext_vector_type(4)));

struct TileArgs {
  const uint8_t* w;        // [experts][n][kbytes]
  const uint8_t* w2;       // gated: the up projection, as w
  const float* ws;         // 8-bit: [experts][n]
  const float* ws2;        // gated 8-bit
  const uint8_t* x;        // [x_tokens][kbytes]
  const float* xs;         // 8-bit: [x_tokens]
  const int32_t* x_rows;   // row of X for each row of Y, or null
  const int32_t* offsets;  // [experts + 1] first rows of Y, or null (one matrix, all rows)
  void* y;                 // [rows][n]
  const float* bias;       // [experts][n] or null
  int64_t rows;
  int64_t x_tokens;
  int64_t n;
  int32_t kbytes;
  int32_t experts;
  int32_t tiles_n;         // column tiles of the kernel's width
  int32_t y_f16;           // Y in binary16, else float32
};

struct ElemI8 {
  typedef i32x4 Acc;
  static constexpr bool kScaled = true;
  __device__ __forceinline__ static Acc zero() { return i32x4{0, 0, 0, 0}; }
  __device__ __forceinline__ static Acc mma(i32x4 a, i32x4 b, Acc c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
  }
};
struct ElemF16 {
  typedef f32x4 Acc;
  static constexpr bool kScaled = false;
  __device__ __forceinline__ static Acc zero() { return f32x4{0.f, 0.f, 0.f, 0.f}; }
  __device__ __forceinline__ static Acc mma(i32x4 a, i32x4 b, Acc c) {
    typedef _Float16 h8 __attribute__((ext_vector_type(8)));
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, a), __builtin_bit_cast(h8, b), c, 0, 0, 0);
  }
};

// One workgroup's tile: rows row0..row_end-1 of Y (at most the kernel's
// height of them are its own) times column tile nt of expert `expert`.
struct TileAt {
  int64_t row0, row_end;
  int expert;
  int nt;
  bool whole;   // more than half the kernel's height
};

// First and last row of expert e, kept inside 0..rows whatever the offsets hold.
__device__ __forceinline__ void expert_rows(const TileArgs& a, int e, int* first, int* last) {
  const int rows = static_cast<int>(a.rows);
  int f = a.offsets[e], l = a.offsets[e + 1];
  f = f < 0 ? 0 : (f > rows ? rows : f);
  l = l < f ? f : (l > rows ? rows : l);
  *first = f;
  *last = l;
}

// Inclusive sum over the lanes of a wavefront: within rows of 16 lanes, then
// each row's last lane into the rows after it.
__device__ __forceinline__ int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);   // row_shr:1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);   // row_shr:2
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);   // row_shr:4
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);   // row_shr:8
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);   // row_bcast:15 into rows 1 and 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);   // row_bcast:31 into rows 2 and 3
  return v;
}

// Row tiles of `rows` rows: those of more than BM / 2 rows, and the one of
// fewer that may be left (with HALVES; else that counts as whole).
template <int BM, bool HALVES>
__device__ __forceinline__ int whole_tiles(int rows) {
  return HALVES ? rows / BM + (rows % BM > BM / 2) : (rows + BM - 1) / BM;
}
template <int BM, bool HALVES>
__device__ __forceinline__ int half_tiles(int rows) {
  return HALVES && rows % BM > 0 && rows % BM <= BM / 2;
}

// Where the tiles are.  Their total is known only here, so the grid is
// launched for the most there can be and workgroups without a tile leave.
// Every wavefront looks tiles up by itself, in LDS: per expert the whole and
// the half row tiles up to its end and its first and last row.  A kernel that
// looks up one tile (ONE) keeps up to 64 experts in a register of its lanes
// instead, without a barrier; in the others these registers were spilled.
template <int BM, bool ONE>
struct TileMap {
  int f, l, incl;     // ONE: of expert `lane`
  int whole, halves;  // row tiles
  int* table;         // [4][experts]

  // Called by all threads of the workgroup.
  __device__ __forceinline__ void init(const TileArgs& a, int* table_lds) {
    table = table_lds;
    halves = 0;
    if (!a.offsets) {
      whole = whole_tiles<BM, !ONE>(static_cast<int>(a.rows));
      halves = half_tiles<BM, !ONE>(static_cast<int>(a.rows));
      return;
    }
    const int lane = threadIdx.x & 63;
    if (ONE && a.experts <= 64) {
      f = l = 0;
      if (lane < a.experts) expert_rows(a, lane, &f, &l);
      incl = wave_scan(whole_tiles<BM, !ONE>(l - f));
      whole = __builtin_amdgcn_readlane(incl, 63);
      return;
    }
    for (int e = threadIdx.x; e < a.experts; e += blockDim.x) {
      int first, last;
      expert_rows(a, e, &first, &last);
      table[e] = whole_tiles<BM, !ONE>(last - first);
      table[a.experts + e] = half_tiles<BM, !ONE>(last - first);
      table[2 * a.experts + e] = first;
      table[3 * a.experts + e] = last;
    }
    __syncthreads();
    whole = 0;
    for (int e0 = 0; e0 < a.experts; e0 += 64) {
      const int e = e0 + lane < a.experts ? e0 + lane : a.experts - 1;
      const bool in = e0 + lane < a.experts;
      const int w = whole + wave_scan(in ? table[e] : 0);
      const int h = halves + (ONE ? 0 : wave_scan(in ? table[a.experts + e] : 0));
      whole = __builtin_amdgcn_readlane(w, 63);
      halves = __builtin_amdgcn_readlane(h, 63);
      __syncthreads();   // all wavefronts have read these 64; the first replaces them
      if (in && threadIdx.x < 64) {
        table[e] = w;
        table[a.experts + e] = h;
      }
    }
    __syncthreads();
  }

  // Rows and expert of whole row tile mt, or of half tile mt.
  __device__ __forceinline__ void rows_of(const TileArgs& a, int mt, bool is_whole, TileAt* at) const {
    int e = 0, first = 0, last = static_cast<int>(a.rows), before = 0;
    if (ONE && a.offsets && a.experts <= 64) {
      e = __builtin_ctzll(__ballot(incl > mt));
      first = __builtin_amdgcn_readlane(f, e);
      last = __builtin_amdgcn_readlane(l, e);
      before = __builtin_amdgcn_readlane(incl, e) - whole_tiles<BM, !ONE>(last - first);
    } else if (a.offsets) {
      const int lane = threadIdx.x & 63;
      const int* t = is_whole ? table : table + a.experts;
      for (int e0 = 0; e0 < a.experts; e0 += 64)   // experts whose tiles all come before mt
        e += __builtin_popcountll(__ballot(e0 + lane < a.experts && t[e0 + lane] <= mt));
      first = __builtin_amdgcn_readfirstlane(table[2 * a.experts + e]);
      last = __builtin_amdgcn_readfirstlane(table[3 * a.experts + e]);
      before = e ? __builtin_amdgcn_readfirstlane(t[e - 1]) : 0;
    }
    at->expert = e;
    at->row0 = first + static_cast<int64_t>(is_whole ? mt - before : (last - first) / BM) * BM;
    at->row_end = last;
    at->whole = is_whole;
  }

  // The i-th tile of XCD `xcd`; false past its last.  Workgroups go to the 8
  // XCDs in turn, each with its own L2: an XCD takes a contiguous run of the
  // whole tiles, then one of the half tiles, and a run walks groups of 8 row
  // tiles column by column, so the workgroups that one XCD runs at a time
  // share rows of X and of W.
  __device__ __forceinline__ bool find(const TileArgs& a, uint32_t xcd, int64_t i, TileAt* at) const {
    for (int part = 0; part < 2; ++part) {
      const int row_tiles = part ? halves : whole;
      const int64_t total = static_cast<int64_t>(row_tiles) * a.tiles_n;
      const int64_t per = total / kXcds;
      const uint32_t rem = static_cast<uint32_t>(total % kXcds);
      const int64_t count = per + (xcd < rem ? 1 : 0);
      if (i >= count) {
        i -= count;
        continue;
      }
      const uint32_t lin = static_cast<uint32_t>(xcd * per + (xcd < rem ? xcd : rem) + i);   // below 2^31
      constexpr uint32_t kGroup = 8;
      const uint32_t width = kGroup * static_cast<uint32_t>(a.tiles_n);
      const uint32_t g = lin / width, in = lin % width;
      const uint32_t left = static_cast<uint32_t>(row_tiles) - g * kGroup;
      const uint32_t gm = left < kGroup ? left : kGroup;
      at->nt = static_cast<int>(in / gm);
      rows_of(a, static_cast<int>(g * kGroup + in % gm), part == 0, at);
      return true;
    }
    return false;
  }
};

__device__ __forceinline__ float silu_mul(float g, float u) { return g / (1.f + expf(-g)) * u; }

// Stores N consecutive columns n..n+N-1 of row r, rounding once to binary16
// where Y is that.  Rows of odd n start anywhere: the vectors ask for no more
// than their element's alignment, which global memory gives them.
template <int N>
__device__ __forceinline__ void store_f16(const TileArgs& a, int64_t r, int64_t n, const float* v) {
  typedef _Float16 hu __attribute__((ext_vector_type(N), aligned(2)));
  _Float16* y = static_cast<_Float16*>(a.y) + r * a.n + n;
  if (n + N <= a.n) {
    hu h;
#pragma unroll
    for (int q = 0; q < N; ++q) h[q] = static_cast<_Float16>(v[q]);
    *reinterpret_cast<hu*>(y) = h;
  } else {
#pragma unroll
    for (int q = 0; q < N - 1; ++q)
      if (n + q < a.n) y[q] = static_cast<_Float16>(v[q]);
  }
}
__device__ __forceinline__ void store_f32(const TileArgs& a, int64_t r, int64_t n, const float* v) {
  typedef float fu __attribute__((ext_vector_type(4), aligned(4)));
  float* y = static_cast<float*>(a.y) + r * a.n + n;
  if (n + 4 <= a.n) {
    *reinterpret_cast<fu*>(y) = fu{v[0], v[1], v[2], v[3]};
  } else {
#pragma unroll
    for (int q = 0; q < 3; ++q)
      if (n + q < a.n) y[q] = v[q];
  }
}
__device__ __forceinline__ void store4(const TileArgs& a, int64_t r, int64_t n, const float* v) {
  if (a.y_f16)
    store_f16<4>(a, r, n, v);
  else
    store_f32(a, r, n, v);
}

// Four per-column values (scales or bias) at columns n..n+3 of an [experts][n]
// array, 0 past the last.
__device__ __forceinline__ void load4(const float* p, int64_t n, int64_t count, float* v) {
  if (n + 3 < count) {
    typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));
    const f32x4u t = *reinterpret_cast<const f32x4u*>(p + n);
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = t[q];
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = n + q < count ? p[n + q] : 0.f;
  }
}

// The value of four sums for a row of X with scale xs (0: no row of X): for
// 8-bit operands acc * xs * ws, in this order so that small scales do not
// meet first and underflow; the integer sum is exact and rounded once to
// float32.
template <typename E, typename V>
__device__ __forceinline__ void scaled(const typename E::Acc& c, float xs, const V& ws, const V& b, float* v) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if constexpr (E::kScaled)
      v[q] = __builtin_fmaf(static_cast<float>(c[q]) * xs, ws[q], b[q]);
    else
      v[q] = (xs == 0.f ? 0.f : c[q]) + b[q];
  }
}

// ---------------------------------------------------------------------------
// Tiles staged through LDS.  A workgroup of WM * WN wavefronts owns BM rows
// of Y and BN rows of W (gated: BN / 2 columns, 16 rows of the gate and 16 of
// the up projection in turn); K advances 128 bytes a step through two
// buffers.  Loads go from memory straight into LDS, 1 KB (8 rows of 128
// bytes, whole cache lines) per wavefront instruction.
//
// What bounds it where there are enough rows is power first: 8192x4096x4096
// in 8 bits takes 85 us with operands of zeros and 110-118 with random ones,
// and the matrix cores by themselves reach 4400-4800 and 3570-3990 TOP/s
// (binary16 2260-2410 and 1730-1840), 69-77 us with random operands.  On a
// slower card, 126 us, the kernel took 103 with nothing loaded, read or
// stored: between that and the products by themselves lie the barriers, the
// epilogue's arithmetic and that card's clock, not told apart.  Short rows are
// bound by stores as well, experts of few rows by reading W.  A step of a 256 x 256
// tile is 2048 cycles of products per SIMD and 64 KB of loads, one step's
// worth in flight (three and four steps of 64-byte rows took as long): loads
// run all the time, and a buffer is refilled in two parts, each as soon as
// it has been read.  A wavefront takes a step in four phases,
//
//   phase  products           reads for the next       refills
//     0    rows half 0, k 0   half 0, k 1; W k 1
//     1    half 0, k 1        half 1, k 0              half 0 of X, W
//     2    half 1, k 0        half 1, k 1              half 0 of X, W
//     3    half 1, k 1        next step: half 0, W     half 1 of X
//
// with a barrier before 1 (half 0 and W are read by all; half 1 has landed)
// and before 3 (half 1 is read by all; the next step's half 0 and W have
// landed), and the reads and loads of a phase spread among its products: in
// a burst they hold up the products of both wavefronts of a SIMD.
//
// LDS holds 128-byte rows with their 16-byte chunks permuted, chunk c of row
// r at place c ^ (r & 7): a wavefront's operand read (16 rows, one chunk
// each per lane group) then spreads over all banks.  The permutation is made
// by the lanes' source addresses, the destination being linear.
//
// K past the row's end (kbytes is a multiple of 32, the step 128) reads
// zeros; rows past the tile's own read the last row in their place and
// are not stored.
//
// The grid fills the chip once and a workgroup takes tiles in turn, the loads
// of the next tile's first two steps running under the last steps and the
// epilogue of the one before: with a workgroup per tile, finding it, filling
// the buffers and storing took 59 of 127 us for 64 experts of 512 rows,
// 2048 x 1024 (this kernel: 108-110).
//
// 8192x4096x4096 in 8 bits, binary16 Y: 110 us (2.5 POP/s) in 256 x 256
// tiles.
// ---------------------------------------------------------------------------
#ifdef __HIP_DEVICE_COMPILE__   // the host compiler needs only the kernels' names
// A value that what is computed from it is computed from again: the compiler
// would take such sums of lane numbers out of the loop over tiles, at the
// price of registers that its 256 x 256 instance does not have (it reloaded
// them one by one, each time waiting for all loads in flight).
__device__ __forceinline__ int again(int v) {
  asm volatile("" : "+v"(v));
  return v;
}
#endif

// Steps of a tile at least: what is loaded for the next tile's turn (rows of
// X at a tile's start, scales two steps before its end) has then been waited
// for by the steps' own waits when it is read.
constexpr int kMinSteps = 4;

template <typename E, int BM, int BN, int WM, int WN, bool GATED>
__global__ __launch_bounds__(WM * WN * 64) void gemm_tile_kernel(TileArgs a) {
#ifdef __HIP_DEVICE_COMPILE__
  constexpr int kWaves = WM * WN;
  constexpr int kTM = BM / WM / 16, kTN = BN / WN / 16;
  constexpr int kHalf = kTM / 2;
  static_assert(kTM % 2 == 0, "a wavefront takes its rows of X in two halves");
  constexpr int kXh = BM / 16 / kWaves, kWn = BN / 8 / kWaves, kPer = 2 * kXh + kWn;
  static_assert(kXh * kWaves * 16 == BM && kWn * kWaves * 8 == BN, "loads divide evenly among the wavefronts");
  constexpr int kStage = (BM + BN) * 128;
  constexpr int kCols = GATED ? BN / 2 : BN;
  static_assert(kTN % (GATED ? 4 : 2) == 0, "a wavefront holds pairs of sub-tiles, gate and up of the same columns");
  extern __shared__ __align__(16) uint8_t lds[];
  typedef __attribute__((address_space(3))) uint8_t Lds;
  typedef __attribute__((address_space(3))) void LdsAny;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tid = threadIdx.x;

  // LDS: two steps of X and W; two sets of the scales and bias that epilogues
  // read; rows of X of the next tile; the tile table.
  constexpr int kSet = 4 * (BM + 2 * BN);
  const int sets = 2 * kStage, index = sets + 2 * kSet;
  int* const index_l = reinterpret_cast<int*>(lds + index);
  TileMap<BM, false> map;
  map.init(a, index_l + BM);
  const uint32_t xcd = blockIdx.x % kXcds;
  const int64_t slots = gridDim.x / kXcds;
  // The XCD's tiles, whole ones first, are dealt to its workgroups back and
  // forth, so that those with fewer whole tiles get more of the halves.
  const int64_t slot = blockIdx.x / kXcds;
  int64_t turn = 0;
  TileAt at, to;
  if (!map.find(a, xcd, slot, &at)) return;

  const int chunk = ((lane & 7) ^ (lane >> 3)) * 16;   // the same place in every row this lane loads
  const int last_step = (a.kbytes + 127) >> 7;
  const int steps = last_step < kMinSteps ? kMinSteps : last_step;

  // Columns of a pair of 16-row operands: sub-tile jj's four of lane group g.
  // In float32 a lane stores four columns at a time and four lanes 64 bytes
  // in a row; in binary16 the pair's rows of W are taken in an order that
  // gives a lane eight columns in a row, so that its store is as wide.
  auto pair_col = [&](int jj, int g) { return a.y_f16 ? 8 * g + 4 * jj : 16 * jj + 4 * g; };

  // The wavefront's load instructions of a step, 8 LDS rows each: first those
  // of the first half of the rows of X (kXh) and of W (kWn), then those of
  // the second half of X.  Addresses are 32-bit offsets from
  // bases that stay for a tile, the step in a scalar register: with 64-bit
  // addresses advanced per step the vector ALU work of the loads cost 5-8%
  // (8192x4096x4096 124 against 116 us).  An offset past the end loads zeros.
  uint32_t src[kPer];
  int dst[kPer];
  BufferRsrc rx, rw, rw2;
  uint32_t limit;   // bytes of a row that loads may reach: 0 where there is no tile
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    if (j < kXh || j >= kXh + kWn) {
      dst[j] = (j < kXh ? wave * kXh + j : BM / 16 + wave * kXh + j - kXh - kWn) * 1024;
    } else {
      dst[j] = (BM / 8 + wave * kWn + j - kXh) * 1024;
    }
  }
  // Rows of X that tile t picks, into LDS (a load, to be waited for).
  auto load_index = [&](const TileAt& t) {
    if (a.x_rows && wave < BM / 64) {
      const int64_t rows = t.row_end - t.row0 < BM ? t.row_end - t.row0 : BM;   // past them: row 0, not stored
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          buffer_of(reinterpret_cast<const uint8_t*>(a.x_rows + t.row0), rows * 4),
          (LdsAny*)((Lds*)lds + index + wave * 256), 4, tid * 4, 0, 0, 0);
    }
  };
  // Turns the loads to tile t (its rows of X in LDS), and starts the loads of
  // its scales and bias into set `set`: they are read by an epilogue at the
  // earliest kMinSteps steps later.  A row without a row of X has scale 0.
  auto turn_to = [&](const TileAt& t, int set) {
    const int tid = again(threadIdx.x), lane = tid & 63;
    const int64_t n0 = static_cast<int64_t>(t.nt) * kCols, first = t.expert * a.n + n0;
    const int cols = a.n - n0 < kCols ? static_cast<int>(a.n - n0) : kCols;
    const int rows = t.row_end - t.row0 < BM ? static_cast<int>(t.row_end - t.row0) : BM;
    const int64_t x0 = a.x_rows ? 0 : t.row0, x_left = a.x_tokens - x0;
    rx = buffer_of(a.x + x0 * a.kbytes, (a.x_rows ? a.x_tokens : x_left < BM ? (x_left < 0 ? 0 : x_left) : BM) * a.kbytes);
    rw = buffer_of(a.w + first * a.kbytes, static_cast<int64_t>(cols) * a.kbytes);
    if constexpr (GATED) rw2 = buffer_of(a.w2 + first * a.kbytes, static_cast<int64_t>(cols) * a.kbytes);
    limit = a.kbytes;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if (j < kXh || j >= kXh + kWn) {
        int r = dst[j] / 128 + (lane >> 3);
        r = r < rows ? r : rows - 1;
        const int i = a.x_rows ? index_l[r] : r;
        // a row that there is not loads zeros; its products are dropped below
        const bool ok = i >= 0 && i < (a.x_rows ? a.x_tokens : x_left) && (t.whole || j < kXh);
        src[j] = ok ? static_cast<uint32_t>(i) * a.kbytes + chunk : kNoOffset;
      } else {
        const int c = dst[j] / 128 - BM + (lane >> 3), sub = GATED ? c >> 5 : c >> 4;
        const int col = (sub >> 1) * 32 + pair_col(sub & 1, (c & 15) >> 2) + (c & 3);
        src[j] = static_cast<uint32_t>(col < cols ? col : cols - 1) * a.kbytes + chunk;
      }
    }
    Lds* to_l = (Lds*)lds + sets + set * kSet + wave * 256;
    if (wave < BM / 64) {
      const int i = a.x_rows ? index_l[tid < rows ? tid : 0] : tid;
      const bool ok = i >= 0 && i < (a.x_rows ? a.x_tokens : x_left);
      if constexpr (E::kScaled)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            buffer_of(reinterpret_cast<const uint8_t*>(a.xs + x0), (a.x_tokens - x0) * 4), (LdsAny*)to_l, 4,
            ok ? static_cast<uint32_t>(i) * 4 : kNoOffset, 0, 0, 0);
      else
        *reinterpret_cast<float*>(lds + sets + set * kSet + tid * 4) = ok ? 1.f : 0.f;
    }
    if (wave < kCols / 64) {
      const uint32_t o = tid * 4;
      if constexpr (E::kScaled)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(buffer_of(reinterpret_cast<const uint8_t*>(a.ws + first), cols * 4),
                                                 (LdsAny*)(to_l + 4 * BM), 4, o, 0, 0, 0);
      if constexpr (E::kScaled && GATED)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(buffer_of(reinterpret_cast<const uint8_t*>(a.ws2 + first), cols * 4),
                                                 (LdsAny*)(to_l + 4 * (BM + kCols)), 4, o, 0, 0, 0);
      if constexpr (!GATED)   // without a bias every offset is past the end: zeros
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            buffer_of(reinterpret_cast<const uint8_t*>(a.bias ? a.bias + first : nullptr), a.bias ? cols * 4 : 0),
            (LdsAny*)(to_l + 4 * (BM + kCols)), 4, o, 0, 0, 0);
    }
  };
  // Loads j0..j1-1 of step s of the tile turned to, into buffer `buf`; past
  // the row's end they read zeros, so that no phase of the loop has a branch.
  auto issue = [&](int s, int buf, int j0, int j1) {
    Lds* base = (Lds*)lds + buf * kStage;
    const bool in = static_cast<uint32_t>(s * 128 + chunk) < limit;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      if (j < j0 || j >= j1) continue;
      const bool is_x = j < kXh || j >= kXh + kWn;
      const bool up = GATED && ((wave * kWn + j - kXh) & 2);   // 16 rows of the gate, 16 of the up projection
      __builtin_amdgcn_raw_ptr_buffer_load_lds(is_x ? rx : (up ? rw2 : rw), (LdsAny*)(base + dst[j]), 16,
                                               in ? src[j] : kNoOffset, s * 128, 0, 0);
    }
  };

  typename E::Acc acc[kTM][kTN];
  const int wm = wave % WM, wn = wave / WM;
  const int place = ((lane >> 4) ^ (lane & 7)) * 16;
  const int xrow = (wm * kHalf * 16 + (lane & 15)) * 128;
  const int wrow = (BM + wn * kTN * 16 + (lane & 15)) * 128;
  i32x4 xa[kHalf], xb[kHalf], wa[kTN], wb[kTN];
  auto read_x = [&](const uint8_t* buf, int half, int ks, i32x4* f) {
#pragma unroll
    for (int i = 0; i < kHalf; ++i)
      f[i] = *reinterpret_cast<const i32x4*>(buf + xrow + half * (BM * 64) + i * 2048 + (place ^ (64 * ks)));
  };
  auto read_w = [&](const uint8_t* buf, int ks, i32x4* f) {
#pragma unroll
    for (int j = 0; j < kTN; ++j) f[j] = *reinterpret_cast<const i32x4*>(buf + wrow + j * 2048 + (place ^ (64 * ks)));
  };
  // One phase: the products of rows i0..i1-1 of a half and of half a step,
  // among them the READS of the next phase and LOADS of a later step.
  auto mma = [&](int half, auto i0, auto i1, const i32x4* x, const i32x4* w, auto reads, auto loads) {
    constexpr int kI0 = decltype(i0)::value, kI1 = decltype(i1)::value;
    constexpr int kReads = decltype(reads)::value, kLoads = decltype(loads)::value;
#pragma unroll
    for (int i = kI0; i < kI1; ++i)
#pragma unroll
      for (int j = 0; j < kTN; ++j) acc[half * kHalf + i][j] = E::mma(w[j], x[i], acc[half * kHalf + i][j]);
    constexpr int kEach = (kI1 - kI0) * kTN / (kReads + kLoads ? kReads + kLoads : 1), kRun = kEach < 1 ? 1 : kEach;
#pragma unroll
    for (int r = 0; r < kReads; ++r) {
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, kRun, 0);
    }
#pragma unroll
    for (int l = 0; l < kLoads; ++l) {
      __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, kRun, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  constexpr int kFirst = kXh + kWn, kMid = (kFirst + 1) / 2;
  constexpr std::integral_constant<int, 0> kNone{};
  constexpr std::integral_constant<int, kHalf> kX{};
  constexpr std::integral_constant<int, kHalf + kTN> kXW{};
  constexpr std::integral_constant<int, kMid> kL1{};
  constexpr std::integral_constant<int, kFirst - kMid> kL2{};
  constexpr std::integral_constant<int, kXh> kL3{};
  constexpr std::integral_constant<int, kPer> kAll{};
  constexpr std::integral_constant<int, (kHalf + 1) / 2> kMidRow{};   // of a half's sub-tiles
  // Waits for all but the newest N loads and for the reads; then for the
  // other wavefronts.
  auto sync = [&](bool loads, auto newest) {
    if (loads) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(decltype(newest)::value) : "memory");
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };

  if (a.x_rows) {
    load_index(at);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    sync(false, kAll);
  }
  turn_to(at, 0);
  issue(0, 0, 0, kPer);
  issue(1, 1, 0, kPer);
  sync(true, kAll);
  read_x(lds, 0, 0, xa);
  read_w(lds, 0, wa);
  int buf = 0, set = 0;
  for (;;) {
    ++turn;
    const bool more = map.find(a, xcd, turn * slots + (turn & 1 ? slots - 1 - slot : slot), &to);
    if (more) load_index(to);
#pragma unroll
    for (int i = 0; i < kTM; ++i)
#pragma unroll
      for (int j = 0; j < kTN; ++j) acc[i][j] = E::zero();
    __builtin_amdgcn_sched_barrier(0);
    // The loads run two steps ahead: in the last two steps of a tile they
    // are the first two of the next.  A tile's first step has been waited for
    // before the epilogue.
    auto turn_at = [&](int s) {
      if (s != steps - 2) return;
      if (more)
        turn_to(to, set ^ 1);
      else
        limit = 0;
    };
    auto step = [&](int s, auto whole) {
      const uint8_t* here = lds + buf * kStage;
      const uint8_t* next = lds + (buf ^ 1) * kStage;
      const int ahead = s + 2 < steps ? s + 2 : s + 2 - steps;
      read_x(here, 0, 1, xb);
      read_w(here, 1, wb);
      mma(0, kNone, kX, xa, wa, kXW, kNone);
      sync(s > 0, kAll);
      turn_at(s);
      if constexpr (decltype(whole)::value) {
        read_x(here, 1, 0, xa);
        issue(ahead, buf, 0, kMid);
        mma(0, kNone, kX, xb, wb, kX, kL1);
        read_x(here, 1, 1, xb);
        issue(ahead, buf, kMid, kFirst);
        mma(1, kNone, kX, xa, wa, kX, kL2);
        sync(true, kAll);
        read_x(next, 0, 0, xa);
        read_w(next, 0, wa);
        issue(ahead, buf, kFirst, kPer);
        mma(1, kNone, kX, xb, wb, kXW, kL3);
      } else {
        // half a tile: phases 0 and 1 alone, the barrier before the next
        // step's operands in the middle of phase 1
        issue(ahead, buf, 0, kPer);
        mma(0, kNone, kMidRow, xb, wb, kNone, kAll);
        sync(true, kAll);
        read_x(next, 0, 0, xa);
        read_w(next, 0, wa);
        mma(0, kMidRow, kX, xb, wb, kXW, kNone);
      }
      buf ^= 1;
    };
    if (at.whole)
      for (int s = 0; s < steps; ++s) step(s, std::true_type{});
    else
      for (int s = 0; s < steps; ++s) step(s, std::false_type{});
    // the next tile's first step, before this tile's stores count as the newest
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kPer) : "memory");
    const int64_t n0 = static_cast<int64_t>(at.nt) * kCols;
    const float* xs_l = reinterpret_cast<const float*>(lds + sets + set * kSet);
    const float* ws_l = xs_l + BM;
    const float* b_l = ws_l + kCols;   // gated: the up projection's scales
    // Columns in pairs of sub-tiles (gated: two gates and their two ups).
    const int lane = again(threadIdx.x & 63), g = lane >> 4;
    constexpr int kG = GATED ? 2 : 1;
#pragma unroll
    for (int i = 0; i < kTM; ++i) {
      if (i >= kHalf && !at.whole) break;
      const int r = i / kHalf * (BM / 2) + (wm * kHalf + i % kHalf) * 16 + (lane & 15);
      const int64_t row = at.row0 + r;
      const float xs = xs_l[r];
#pragma unroll
      for (int p = 0; p < kTN / (2 * kG); ++p) {
        const int c0 = (wn * kTN / (2 * kG) + p) * 32;
        float v[8];
#pragma unroll
        for (int jj = 0; jj < 2; ++jj) {
          const int c = c0 + pair_col(jj, g);
          const f32x4 s = E::kScaled ? *reinterpret_cast<const f32x4*>(ws_l + c) : f32x4{};
          const f32x4 b = GATED ? f32x4{0.f, 0.f, 0.f, 0.f} : *reinterpret_cast<const f32x4*>(b_l + c);
          scaled<E>(acc[i][kG * (2 * p + jj)], xs, s, b, v + 4 * jj);
          if constexpr (GATED) {
            const f32x4 s2 = E::kScaled ? *reinterpret_cast<const f32x4*>(b_l + c) : f32x4{};
            float u[4];
            scaled<E>(acc[i][kG * (2 * p + jj) + 1], xs, s2, b, u);
#pragma unroll
            for (int q = 0; q < 4; ++q) v[4 * jj + q] = silu_mul(v[4 * jj + q], u[q]);
          }
        }
        if (row >= at.row_end) continue;
        if (a.y_f16) {
          store_f16<8>(a, row, n0 + c0 + 8 * g, v);
        } else {
          store_f32(a, row, n0 + c0 + 4 * g, v);
          store_f32(a, row, n0 + c0 + 16 + 4 * g, v + 4);
        }
      }
    }
    if (!more) break;
    at = to;
    set ^= 1;
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // the last zeros are in before LDS is given up
#endif
}

// ---------------------------------------------------------------------------
// Few tiles: where 64 x 128 tiles would leave most compute units idle, a
// workgroup owns 16 columns and up to 16 * MT rows of Y, and its NW
// wavefronts split K into contiguous slices, each streaming its part of W and
// X from memory straight into operand registers, D lines of 128 bytes (two
// k-steps) per row in flight; the partial sums meet in LDS in wavefront order.
// What bounds it is latency: finding the expert, the picked rows, the trips
// for W, the sum.  NW * D lines of a row are in flight at once: 1 KB with 2 x 4
// and 2.5 KB with 4 x 5, so 896 bytes come in one trip, 2048 and 4864 in two.
// Four experts of one row, binary16 896x2432 (17.4 MB of W): 6.6 us, 2.6 TB/s;
// eight, gated 8-bit 1024x2048 (33.6 MB): 9.2 us, 3.7 TB/s; one token, 8-bit
// 896x896: 3.9-4.7 by itself, 3.2 after another launch of its kind.
// ---------------------------------------------------------------------------
template <typename E, int MT, int NW, int D, bool GATED>
__global__ __launch_bounds__(NW * 64) void gemm_rows_kernel(TileArgs a) {
#ifdef __HIP_DEVICE_COMPILE__
  constexpr int kG = GATED ? 2 : 1;
  constexpr int C = 2;
  __shared__ typename E::Acc part[NW][MT][kG][kWave];
  extern __shared__ __align__(16) uint8_t lds[];   // the tile table of more than 64 experts
  TileMap<16 * MT, true> map;
  map.init(a, reinterpret_cast<int*>(lds));
  TileAt at;
  if (!map.find(a, blockIdx.x % kXcds, blockIdx.x / kXcds, &at)) return;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int i = lane & 15, g = lane >> 4;
  const int64_t n0 = static_cast<int64_t>(at.nt) * 16, first = at.expert * a.n + n0;
  const int cols = a.n - n0 < 16 ? static_cast<int>(a.n - n0) : 16;
  const int steps = (a.kbytes + 63) >> 6, per = (steps + NW - 1) / NW;
  const uint32_t begin = wave * per * 64;
  const uint32_t end = begin + per * 64 < static_cast<uint32_t>(a.kbytes) ? begin + per * 64 : a.kbytes;

  const int64_t x0 = a.x_rows ? 0 : at.row0, x_left = a.x_tokens - x0;
  int xi[MT];
  bool ok[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int64_t row = at.row0 + 16 * t + i < at.row_end ? at.row0 + 16 * t + i : at.row_end - 1;
    xi[t] = a.x_rows ? a.x_rows[row] : static_cast<int>(row - x0);
    ok[t] = xi[t] >= 0 && xi[t] < (a.x_rows ? a.x_tokens : x_left);
  }
  const BufferRsrc rw = buffer_of(a.w + first * a.kbytes, static_cast<int64_t>(cols) * a.kbytes);
  const BufferRsrc rw2 = GATED ? buffer_of(a.w2 + first * a.kbytes, static_cast<int64_t>(cols) * a.kbytes) : rw;
  const BufferRsrc rx = buffer_of(
      a.x + x0 * a.kbytes, (a.x_rows ? a.x_tokens : x_left < 16 * MT ? (x_left < 0 ? 0 : x_left) : 16 * MT) * a.kbytes);
  const uint32_t wrow = static_cast<uint32_t>(i < cols ? i : cols - 1) * a.kbytes;
  struct Buf {
    i32x4 w[C][kG], x[C][MT];
  };
  // Past the slice, and in the half step past a row's end, both are zeros.
  auto load_w = [&](uint32_t o, Buf& b) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const uint32_t p = o + 64 * c + 16 * g, q = p < end ? wrow + p : kNoOffset;
      b.w[c][0] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(rw, q, 0, 0));
      if constexpr (GATED) b.w[c][1] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(rw2, q, 0, 0));
    }
  };
  auto load_x = [&](uint32_t o, Buf& b) {
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const uint32_t p = o + 64 * c + 16 * g;
        const uint32_t q = ok[t] && p < end ? static_cast<uint32_t>(xi[t]) * a.kbytes + p : kNoOffset;
        b.x[c][t] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(rx, q, 0, 0));
      }
  };
  typename E::Acc acc[MT][kG];
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int k = 0; k < kG; ++k) acc[t][k] = E::zero();
  auto mma = [&](const Buf& b) {
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int k = 0; k < kG; ++k) acc[t][k] = E::mma(b.w[c][k], b.x[c][t], acc[t][k]);
  };
  // W first: it does not wait for the rows of X to be known.
  Buf ring[D];
#pragma unroll
  for (int d = 0; d < D; ++d) load_w(begin + 128 * d, ring[d]);
#pragma unroll
  for (int d = 0; d < D; ++d) load_x(begin + 128 * d, ring[d]);
  // What the epilogue needs, before the products: lane l of the wavefront
  // that stores a row tile has its row l % 16 and four columns.
  float xs[MT], ws[kG][4], b4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int t = 0; t < MT; ++t) xs[t] = ok[t] ? (E::kScaled ? a.xs[x0 + xi[t]] : 1.f) : 0.f;
  if constexpr (E::kScaled) {
    load4(a.ws + at.expert * a.n, n0 + 4 * g, a.n, ws[0]);
    if constexpr (GATED) load4(a.ws2 + at.expert * a.n, n0 + 4 * g, a.n, ws[kG - 1]);
  }
  if (!GATED && a.bias) load4(a.bias + at.expert * a.n, n0 + 4 * g, a.n, b4);
  uint32_t o = begin;
  for (; o + 128 * D < end; o += 128 * D)
#pragma unroll
    for (int d = 0; d < D; ++d) {
      mma(ring[d]);
      load_w(o + 128 * (D + d), ring[d]);
      load_x(o + 128 * (D + d), ring[d]);
    }
#pragma unroll
  for (int d = 0; d < D; ++d) mma(ring[d]);   // the last: zeros past the slice
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int k = 0; k < kG; ++k) part[wave][t][k][lane] = acc[t][k];
  __syncthreads();
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    if (wave != t % NW) continue;
    float v[kG][4];
#pragma unroll
    for (int k = 0; k < kG; ++k) {
      typename E::Acc r = part[0][t][k][lane];
#pragma unroll
      for (int w = 1; w < NW; ++w) r += part[w][t][k][lane];
      scaled<E>(r, xs[t], ws[k], b4, v[k]);
    }
    if constexpr (GATED)
#pragma unroll
      for (int q = 0; q < 4; ++q) v[0][q] = silu_mul(v[0][q], v[1][q]);
    const int64_t row = at.row0 + 16 * t + i;
    if (row < at.row_end) store4(a, row, n0 + 4 * g, v[0]);
  }
#endif
}

}  // namespace pesti

namespace pesti_host {

// The launch behind the entry points: args with everything but the tile
// count set, `gated` for the joined gate and up products.
int gemm_tiles_i8(const pesti::TileArgs& a, bool gated, hipStream_t st);
int gemm_tiles_f16(const pesti::TileArgs& a, bool gated, hipStream_t st);

inline TileShape shape_of(const pesti::TileArgs& a, bool gated) {
  return TileShape{a.rows, a.n, a.offsets ? a.experts : 0, a.kbytes, gated};
}

// most: workgroups to launch at most (each then takes several tiles in turn), 0 for one tile each.
inline int launch_tiles(const void* fn, pesti::TileArgs a, int bm, int cols, int threads, size_t lds, int64_t most,
                        hipStream_t st) {
  const int64_t tn = (a.n + cols - 1) / cols;
  const int64_t total = most_row_tiles(shape_of(a, false), bm) * tn;
  // Tiles are numbered in 31 bits; the grid is rounded up to whole turns of the XCDs.
  if (total > INT32_MAX - pesti::kXcds) return PESTI_ERR_SHAPE;
  a.tiles_n = static_cast<int32_t>(tn);
  void* params[] = {&a};
  unsigned grid = static_cast<unsigned>((total + pesti::kXcds - 1) / pesti::kXcds * pesti::kXcds);
  if (most > 0 && grid > most) grid = static_cast<unsigned>(most);
  if (grid == 0) return PESTI_OK;
  return hipLaunchKernel(fn, dim3(grid), dim3(threads), params, lds, st) == hipSuccess ? PESTI_OK : PESTI_ERR_LAUNCH;
}

template <typename E, int BM, int BN, int WM, int WN, bool GATED>
int launch_tile(const pesti::TileArgs& a, hipStream_t st) {
  const TileShape s = shape_of(a, GATED);
  return launch_tiles(reinterpret_cast<const void*>(&pesti::gemm_tile_kernel<E, BM, BN, WM, WN, GATED>), a, BM,
                      GATED ? BN / 2 : BN, WM * WN * 64, tile_lds(s, BM, BN), tile_workgroups(s, BM, BN), st);
}

template <typename E, int MT, int NW, int D, bool GATED>
int launch_rows_w(const pesti::TileArgs& a, hipStream_t st) {
  return launch_tiles(reinterpret_cast<const void*>(&pesti::gemm_rows_kernel<E, MT, NW, D, GATED>), a, 16 * MT, 16,
                      NW * 64, a.offsets && a.experts > 64 ? 16 * a.experts : 0, 0, st);
}
template <typename E, int MT, bool GATED>
int launch_rows(const pesti::TileArgs& a, hipStream_t st) {
  return rows_wavefronts(a.kbytes) == 2 ? launch_rows_w<E, MT, 2, 4, GATED>(a, st)
                                        : launch_rows_w<E, MT, 4, 5, GATED>(a, st);
}

template <typename E, bool GATED>
int launch_any(const pesti::TileArgs& a, hipStream_t st) {
  switch (tile_kernel(shape_of(a, GATED))) {
    case TileKernel::kRows16: return launch_rows<E, 1, GATED>(a, st);
    case TileKernel::kRows32: return launch_rows<E, 2, GATED>(a, st);
    case TileKernel::kRows64:
      if constexpr (!GATED) return launch_rows<E, 4, GATED>(a, st);
      break;   // not chosen for gated products
    case TileKernel::kTile64x128: return launch_tile<E, 64, 128, 2, 2, GATED>(a, st);
    case TileKernel::kTile128x128: return launch_tile<E, 128, 128, 2, 2, GATED>(a, st);
    case TileKernel::kTile128x256: return launch_tile<E, 128, 256, 2, 4, GATED>(a, st);
    case TileKernel::kTile256x256: return launch_tile<E, 256, 256, 2, 4, GATED>(a, st);
  }
  return PESTI_ERR_SHAPE;
}

}  // namespace pesti_host
