// Attention of one new token per sequence over the paged key-value cache
// ("PESTI ..." README, "Conformance" and "Current Status": grouped-query
// attention, paged attention during generation), for the query heads h of one
// KV head:
//   y[h] = sum_t p_t v[t] / sum_t p_t,  p_t = 2^(s_t - max), s_t = scale log2(e) q[h] . k[t]
// in one pass over the cache with the running maximum and sum of the softmax.
//
// What bounds it is the cache's bytes: a step of one wavefront is 32 tokens of
// one KV head, and the matrix cores' time for it (D / 32 + D / 16 of
// v_mfma_f32_16x16x32_f16 per head tile and half of the tokens) is a small part
// of what its loads take.  So precision is free there and the layout is chosen
// for the loads:
//   * S = K Q^T: A is 16 tokens (rows) of K as they lie in a page, 16 bytes a
//     lane; B is Q.  The 16 columns are 8 heads, each twice: columns 0-7 hold
//     the first binary16 part of q, 8-15 what it leaves, 2^11 times as large.
//   * Column c of S is one head in all 64 lanes' registers, so the softmax's
//     maximum, weights and sums stay in the lanes of their column: one exchange
//     joins the parts, two the maximum of a column.
//   * y = V^T P: the weights of 32 tokens are B as S left them in the registers
//     (no exchange: lane group g holds tokens 4g..4g+3 of both halves, so those
//     are the k indices of its lanes), in two parts over the columns as q was.
//     A needs 8 tokens of one dimension per lane: each lane loads 8 token rows,
//     the same run of up to 8 dimensions of each, and the transposition is the
//     choice of which 16-bit halves form a register (v_perm), with the
//     dimensions of a run spread over as many matrix instructions.  No LDS.
// LDS is used once, to join the wavefronts of a workgroup, which take the
// tiles of its part of the sequence in turn.  Parts are joined by a second
// kernel (attn_paged.hip) where a sequence has more than one.  Measured, with that:
// 131071 tokens of 8 KV heads of 128 98 us in binary16 (5.5 TB/s), 57 in 8 bits; 97
// tokens of 2 heads of 64 5.2, of which the launch is 2.0 and the rest the way from
// one load to the next and some 700 vector instructions of a wavefront alone on its SIMD.
#pragma once

#include <type_traits>

#include "kv_cache.h"

namespace pesti {

typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2a __attribute__((ext_vector_type(2), aligned(8)));

struct AttnArgs {
  KvArgs kv;               // pools of the layer
  const int32_t* seq_ids;
  const void* q;
  int64_t q_stride;
  void* y;
  float* parts;            // [rows][heads][splits][head_dim], unnormalised
  float* stats;            // [rows][heads][splits][2]: maximum (base 2), sum (kNoPart: nothing else is written)
  float scale;             // scale * log2(e)
  int32_t heads;
  int32_t group;           // query heads per KV head
  int32_t head_blocks;     // workgroups per KV head
  int32_t splits;
  int32_t part_tiles;      // tiles of a part
  int32_t waves;           // wavefronts of a workgroup
  int32_t q_f32, y_f32;
};

// Wavefronts of a workgroup: four, or eight where a sequence is one part.
constexpr int attn_most_waves(int d, int nt) { return d * nt <= 128 ? 8 : 4; }
constexpr int kTile = 32;            // tokens of one step of a wavefront
constexpr float kNoPart = -1.f;      // the sum of a part without tokens

// Tiles per part, and parts, of a sequence of `length` tokens.  Parts of all
// sequences have one size, so that workgroups of a batch of uneven lengths
// finish together (48 sequences up to 8191 in 8 bits, the same number of parts
// each: 107 us); only a sequence past the caller's bound has larger ones.
__device__ __forceinline__ int32_t attn_part_tiles(int32_t length, int32_t splits, int32_t part_tiles) {
  const int32_t tiles = (length + kTile - 1) / kTile, per = (tiles + splits - 1) / splits;
  return per > part_tiles ? per : part_tiles;
}
__device__ __forceinline__ int32_t attn_parts(int32_t length, int32_t per) {
  return ((length + kTile - 1) / kTile + per - 1) / per;
}

// Four values of y, at a multiple of four.
__device__ __forceinline__ void store_y(const AttnArgs& p, int64_t at, const f32x4& y) {
  if (p.y_f32) {
    *reinterpret_cast<f32x4*>(static_cast<float*>(p.y) + at) = y;
  } else {
    typedef _Float16 h4 __attribute__((ext_vector_type(4)));
    *reinterpret_cast<h4*>(static_cast<_Float16*>(p.y) + at) =
        h4{static_cast<_Float16>(y[0]), static_cast<_Float16>(y[1]), static_cast<_Float16>(y[2]), static_cast<_Float16>(y[3])};
  }
}

#ifdef __HIP_DEVICE_COMPILE__

// Largest value of a column: over the four lane groups.
__device__ __forceinline__ float column_max(float v) {
  const uint32_t b = __builtin_bit_cast(uint32_t, v);
  const auto h = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  v = fmaxf(__builtin_bit_cast(float, static_cast<uint32_t>(h[0])), __builtin_bit_cast(float, static_cast<uint32_t>(h[1])));
  const uint32_t c = __builtin_bit_cast(uint32_t, v);
  const auto r = __builtin_amdgcn_permlane16_swap(c, c, false, false);
  return fmaxf(__builtin_bit_cast(float, static_cast<uint32_t>(r[0])), __builtin_bit_cast(float, static_cast<uint32_t>(r[1])));
}
__device__ __forceinline__ float column_sum(float v) {
  const uint32_t b = __builtin_bit_cast(uint32_t, v);
  const auto h = __builtin_amdgcn_permlane32_swap(b, b, false, false);
  v = __builtin_bit_cast(float, static_cast<uint32_t>(h[0])) + __builtin_bit_cast(float, static_cast<uint32_t>(h[1]));
  const uint32_t c = __builtin_bit_cast(uint32_t, v);
  const auto r = __builtin_amdgcn_permlane16_swap(c, c, false, false);
  return __builtin_bit_cast(float, static_cast<uint32_t>(r[0])) + __builtin_bit_cast(float, static_cast<uint32_t>(r[1]));
}
__device__ __forceinline__ float other_part(float v) { return dpp<0x128>(v); }   // row_ror:8, column c ^ 8

// Both to binary16, to nearest even (v_cvt_pk_f16_f32).
__device__ __forceinline__ h2 pair_of(float a, float b) {
  typedef float f2 __attribute__((ext_vector_type(2)));
  return __builtin_convertvector((f2{a, b}), h2);
}

constexpr float kPart = 0x1p-11f;   // the second part is held 2^11 times as large

// First and second binary16 part of x (|x| < 2^15); an infinity or NaN is all in the first.
__device__ __forceinline__ _Float16 part_of(float x, bool second) {
  const _Float16 hi = static_cast<_Float16>(x);
  const float lo = (x - static_cast<float>(hi)) * 0x1p11f;
  return second ? static_cast<_Float16>(lo - lo == 0.f ? lo : 0.f) : hi;
}

// Both parts of a sum of products: an infinity of the first stands, since the
// second's products with it are infinities or NaN of any kind.
__device__ __forceinline__ float both_parts(float hi, float lo) {
  return __builtin_fabsf(hi) == INFINITY ? hi : fmaf(lo, kPart, hi);
}

// A column's score from its own and the other part, `share` being what its own
// counts for.  Product, then sum, never one fma: both lanes have to get the same
// bits, since one keeps the first and the other the second part of its weight.
__device__ __forceinline__ float joined(float own, float share) {
#pragma clang fp contract(off)
  const float p = own * share;
  return p + other_part(p);
}

// Four signed bytes as binary16: xor 0x80 makes them 0..255 (code + 128), which
// over 0x6400 read as 1024 + u.
__device__ __forceinline__ h2 bytes_h2(uint32_t u, uint32_t sel) {
  const uint32_t v = __builtin_amdgcn_perm(0x64646464u, u, sel);   // bytes 4-7 of the pair are 0x64
  return __builtin_bit_cast(h2, v) - h2{static_cast<_Float16>(1152.f), static_cast<_Float16>(1152.f)};
}
__device__ __forceinline__ h8 codes_h8(uint32_t a, uint32_t b) {
  a ^= 0x80808080u;
  b ^= 0x80808080u;
  const h2 v0 = bytes_h2(a, 0x04010400u), v1 = bytes_h2(a, 0x04030402u), v2 = bytes_h2(b, 0x04010400u),
           v3 = bytes_h2(b, 0x04030402u);
  return h8{v0[0], v0[1], v1[0], v1[1], v2[0], v2[1], v3[0], v3[1]};
}

// One run of dimensions of V: 16 lanes hold E neighbouring ones each, of 8
// tokens; frag(n) is dimension n of the lanes' runs as a matrix operand.
template <bool I8, int E>
struct VRun {
  static constexpr int kWords = I8 ? (E + 3) / 4 : E / 2;
  uint32_t w[8][kWords];
  __device__ __forceinline__ void load(int j, const uint8_t* p) {
    if constexpr (I8 && E == 2) {
      w[j][0] = *reinterpret_cast<const uint16_t*>(p);
    } else if constexpr (kWords == 1) {
      w[j][0] = *reinterpret_cast<const uint32_t*>(p);
    } else if constexpr (kWords == 2) {
      const u32x2a v = *reinterpret_cast<const u32x2a*>(p);
      w[j][0] = v.x;
      w[j][1] = v.y;
    } else {
      const u32x4a v = *reinterpret_cast<const u32x4a*>(p);
#pragma unroll
      for (int i = 0; i < 4; ++i) w[j][i] = v[i];
    }
  }
  __device__ __forceinline__ void clear(int j) {   // codes of zero too
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[j][i] = 0;
  }
  __device__ __forceinline__ h8 frag(int n) const {
    typedef uint32_t u4 __attribute__((ext_vector_type(4)));
    u4 r;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (!I8) {
        r[j] = __builtin_amdgcn_perm(w[2 * j + 1][n / 2], w[2 * j][n / 2], n % 2 ? 0x07060302u : 0x05040100u);
      } else {
        const uint32_t b = n % 4;
        const uint32_t u = __builtin_amdgcn_perm(w[2 * j + 1][n / 4], w[2 * j][n / 4], 0x0C000C00u | b | ((b + 4) << 16));
        const h2 v = __builtin_bit_cast(h2, (u ^ 0x00800080u) | 0x64006400u) -
                     h2{static_cast<_Float16>(1152.f), static_cast<_Float16>(1152.f)};
        r[j] = __builtin_bit_cast(uint32_t, v);
      }
    }
    return __builtin_bit_cast(h8, r);
  }
};

// head_dim as runs of 128, 64 and 32 dimensions (8, 4 and 2 a lane).
template <bool I8, int D>
struct VTile {
  static constexpr int kA = D / 128, kB = D % 128 / 64, kC = D % 64 / 32;
  VRun<I8, 8> a[kA ? kA : 1];
  VRun<I8, 4> b[1];
  VRun<I8, 2> c[1];
  static constexpr int kSize = I8 ? 1 : 2;
  __device__ __forceinline__ void load(int j, const uint8_t* row, int col) {
#pragma unroll
    for (int r = 0; r < kA; ++r) a[r].load(j, row + (128 * r + 8 * col) * kSize);
    if constexpr (kB) b[0].load(j, row + (128 * kA + 4 * col) * kSize);
    if constexpr (kC) c[0].load(j, row + (128 * kA + 64 * kB + 2 * col) * kSize);
  }
  __device__ __forceinline__ void clear(int j) {
#pragma unroll
    for (int r = 0; r < kA; ++r) a[r].clear(j);
    if constexpr (kB) b[0].clear(j);
    if constexpr (kC) c[0].clear(j);
  }
  __device__ __forceinline__ h8 frag(int f) const {
    if (f < 8 * kA) return a[f / 8].frag(f % 8);
    if (f < 8 * kA + 4 * kB) return b[0].frag(f - 8 * kA);
    return c[0].frag(f - 8 * kA - 4 * kB);
  }
};

// The first of the 8 dimensions that lane group g holds in step s of the
// scores.  In 8 bits two steps share a 16-byte load.
template <bool I8>
__device__ __forceinline__ constexpr int k_dim(int s, int steps, int g) {
  return I8 && s < steps / 2 * 2 ? 64 * (s / 2) + 16 * g + 8 * (s % 2) : 32 * s + 8 * g;
}

#endif  // __HIP_DEVICE_COMPILE__

// Wavefronts per SIMD that the registers are to leave room for.  Stated, since
// the compiler left to itself adds accumulator registers up to two wavefronts'
// share where three fit (8 bits, D 128: 113 -> 107 us), or one's where two do (32
// rows up to 3000 of 4 heads of 256 in 8 bits 62 -> 41; in binary16 those have 76
// registers too many for two, which takes 90 instead of 76).
constexpr int attn_waves(bool i8, int d, int nt, bool small) {
  return d * nt <= 64 ? 4 : (d * nt <= (i8 || !small ? 128 : 96) ? 3 : (i8 || d * nt <= 192 ? 2 : 1));
}

// One workgroup: the NT * 8 query heads of block blockIdx.x of a KV head, a part
// of row blockIdx.z's sequence.  Workgroups go to the 8 XCDs in turn: heads, which
// have equal work, lie next to each other, and a row's parts, of which short
// sequences lack the last ones, start at another place in each row (48 sequences
// up to 8191 in 8 parts, the part first and unrotated: 136 us, the last parts'
// XCDs idle).  SMALL: pages of 8 or 16 tokens, up
// to four in a tile; else a tile lies in one page.
template <bool I8, int D, int NT, bool SMALL>
__global__ __launch_bounds__(64 * attn_most_waves(D, NT)) __attribute__((amdgpu_waves_per_eu(attn_waves(I8, D, NT, SMALL))))
void attn_kernel(AttnArgs p) {
#ifdef __HIP_DEVICE_COMPILE__
  constexpr int kSteps = D / 32, kFrags = D / 16, kSize = I8 ? 1 : 2, kPages = SMALL ? 4 : 1;
  constexpr int kMostWaves = attn_most_waves(D, NT), kRow = D + 4;   // (padded against bank conflicts)
  extern __shared__ __attribute__((aligned(16))) float lds[];   // per wavefront: y of 8 NT heads, their maxima, their sums
  const KvArgs& a = p.kv;
  const int waves = p.waves;
  float* joint = lds;
  float* wave_max = lds + waves * 8 * NT * kRow;
  float* wave_sum = wave_max + waves * 8 * NT;
  float* joint_max = wave_sum + waves * 8 * NT;   // and the workgroup's
  float* joint_sum = joint_max + 8 * NT;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 15, g = lane >> 4;
  const bool second = col >= 8;
  const int64_t row = blockIdx.z;
  const int kvh = blockIdx.x / p.head_blocks, hb = blockIdx.x % p.head_blocks;
  const int head0 = hb * 8 * NT, heads_here = p.group - head0 < 8 * NT ? p.group - head0 : 8 * NT;
  const int64_t first_head = static_cast<int64_t>(kvh) * p.group + head0;
  const int32_t part = static_cast<int32_t>((blockIdx.y + blockIdx.z) % static_cast<uint32_t>(p.splits));

  // A short sequence's time is the way from one load to the next: q, the length
  // and the pages of the first tiles, where they lie unless the sequence is
  // longer than the caller's bound, are asked for together.
  const int64_t seq = p.seq_ids ? p.seq_ids[row] : row;
  const bool known = seq >= 0 && seq < a.seqs && a.pages > 0 && a.width > 0;
  const int32_t* row_pages = a.table + (known ? seq : 0) * a.width;
  auto page_index = [&](int32_t tile, int j) {
    return ((static_cast<int64_t>(tile) + lane * waves) * kTile + 8 * j) >> a.page_shift;
  };
  int32_t ids[kPages];   // lane i: the pages of the wavefront's i-th tile from here
#pragma unroll
  for (int j = 0; j < kPages; ++j) {
    const int64_t idx = page_index(part * p.part_tiles + wave, j);
    ids[j] = known ? row_pages[idx < a.width ? idx : a.width - 1] : -1;
  }
  const int32_t length = known ? kv_length(a, static_cast<int32_t>(seq)) : 0;
  f32x4 q32[NT][kSteps][2];
  h8 q16[NT][kSteps];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int h = 8 * n + (col & 7);
    const int64_t q0 = row * p.q_stride + (first_head + (h < heads_here ? h : 0)) * D;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int64_t e0 = q0 + k_dim<I8>(s, kSteps, g);
      if (p.q_f32) {
        const f32x4* src = reinterpret_cast<const f32x4*>(static_cast<const float*>(p.q) + e0);
        q32[n][s][0] = src[0];
        q32[n][s][1] = src[1];
      } else {
        q16[n][s] = *reinterpret_cast<const h8*>(static_cast<const _Float16*>(p.q) + e0);
      }
    }
  }
  const int32_t per = attn_part_tiles(length, p.splits, p.part_tiles), parts = attn_parts(length, per);
  const int32_t tiles = (length + kTile - 1) / kTile;
  const int32_t end = part * per + per < tiles ? part * per + per : tiles;
  if (p.splits > 1 && part >= parts) {   // nothing there: the join is told so
    if (tid < heads_here) {
      float* stats = p.stats + 2 * ((row * p.heads + first_head + tid) * p.splits + part);
      stats[0] = -INFINITY;
      stats[1] = kNoPart;
    }
    return;
  }

  const int32_t held = kv_pages_of(a, length);
  const int32_t page_mask = (1 << a.page_shift) - 1;
  const int32_t first_tile = part * per + wave, last_tile = end - 1;

  // Where a tile lies: rows of the layer's pools that its token 0 would have in
  // the page of K's tokens (column col) and of V's (lane group g), by half.
  struct Place {
    int64_t k_row[2], v_row[2];
    uint32_t there;   // bit t: token t of the tile is in the cache
  };
  auto locate = [&](int32_t tile, int step) {   // step: of the wavefront
    step &= 63;
    if (step == 0 && (tile != first_tile || per != p.part_tiles)) {
#pragma unroll
      for (int j = 0; j < kPages; ++j) {
        const int64_t idx = page_index(tile, j);
        ids[j] = idx < held ? row_pages[idx] : -1;
      }
    }
    Place w;
    const int32_t t0 = tile * kTile, left = length - t0;
    w.there = left >= 32 ? 0xFFFFFFFFu : (1u << left) - 1;
    auto row_in = [&](int32_t page, int first) {
      return page * a.page_rows + (static_cast<int64_t>(kvh) << a.page_shift) + ((t0 + first) & page_mask) - first;
    };
    int32_t page[kPages];
#pragma unroll
    for (int j = 0; j < kPages; ++j) {
      page[j] = __builtin_amdgcn_readlane(ids[j], step);
      if (!kv_page_ok(a, page[j])) {
        w.there &= SMALL ? ~(0xFFu << (8 * j)) : 0u;
        page[j] = 0;   // read instead, and not used
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if constexpr (SMALL) {
        w.k_row[h] = row_in(second ? page[2 * h + 1] : page[2 * h], 16 * h + (second ? 8 : 0));
        w.v_row[h] = row_in(g >= 2 ? page[2 * h + 1] : page[2 * h], 16 * h + (g >= 2 ? 8 : 0));
      } else {
        w.k_row[h] = w.v_row[h] = row_in(page[0], 0);
      }
    }
    return w;
  };
  // K: token col of each half.
  u32x4a kw[2][I8 ? (kSteps + 1) / 2 : kSteps];
  f32x4 ks[2], vs[2];
  auto load_k = [&](const Place& w) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint8_t* r = a.k + w.k_row[h] * (D * kSize) + (16 * h + col) * (D * kSize);
      if constexpr (!I8) {
#pragma unroll
        for (int s = 0; s < kSteps; ++s) kw[h][s] = *reinterpret_cast<const u32x4a*>(r + (32 * s + 8 * g) * 2);
      } else {
#pragma unroll
        for (int s = 0; s < kSteps / 2; ++s) kw[h][s] = *reinterpret_cast<const u32x4a*>(r + 64 * s + 16 * g);
        if constexpr (kSteps % 2) {
          const u32x2a v = *reinterpret_cast<const u32x2a*>(r + 32 * (kSteps - 1) + 8 * g);
          kw[h][kSteps / 2] = u32x4a{v.x, v.y, 0u, 0u};
        }
      }
    }
  };
  // V: tokens 4g..4g+3 of each half, in the lane's runs of dimensions, and both
  // scales of those tokens.
  VTile<I8, D> vt;
  auto load_v = [&](const Place& w) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint8_t* r = a.v + w.v_row[h] * (D * kSize) + (16 * h + 4 * g) * (D * kSize);
#pragma unroll
      for (int i = 0; i < 4; ++i) vt.load(4 * h + i, r + i * (D * kSize), col);
      if constexpr (I8) {
        ks[h] = *reinterpret_cast<const f32x4*>(a.k_scales + w.v_row[h] + 16 * h + 4 * g);
        vs[h] = *reinterpret_cast<const f32x4*>(a.v_scales + w.v_row[h] + 16 * h + 4 * g);
      }
    }
  };

  // K of the next tile is asked for as soon as the scores have used this one's
  // registers, V after the weighted sums: each is in flight under the other's
  // half of a step, without a second set of registers.
  Place at{};
  if (first_tile <= last_tile) {
    at = locate(first_tile, 0);
    load_k(at);
    load_v(at);
  }
  __builtin_amdgcn_sched_barrier(0);

  // How the second part of a value is made, per lane.
  const float less = second ? -1.f : 0.f, times = second ? 0x1p11f : 1.f;

  // Q: columns 0-7 the first parts, 8-15 the second ones, of heads that exist;
  // scaled so that a head's largest finite value lies in [2^14, 2^15).
  h8 qf[NT][kSteps];
  float factor[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int h = 8 * n + (col & 7);
    const bool there = h < heads_here;
    float v[kSteps][8];
    uint32_t top = 0;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[s][e] = p.q_f32 ? q32[n][s][e / 4][e % 4] : static_cast<float>(q16[n][s][e]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t u = __builtin_bit_cast(uint32_t, v[s][e]) & 0x7FFFFFFFu;
        top = u > top ? u : top;
      }
    }
    const bool finite = !__any(top >= 0x7F800000u);
    if (!finite) {   // the largest finite value
      top = 0;
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t u = __builtin_bit_cast(uint32_t, v[s][e]) & 0x7FFFFFFFu;
          top = u < 0x7F800000u && u > top ? u : top;
        }
    }
    // magnitudes are ordered as floats too
    const uint32_t big = __builtin_bit_cast(uint32_t, column_max(__builtin_bit_cast(float, top)));
    int up = 14 + 127 - static_cast<int>(big >> 23);   // the exponent to add
    up = big == 0 ? 0 : (up > 126 ? 126 : up);
    const float lift = there ? __builtin_bit_cast(float, static_cast<uint32_t>(up + 127) << 23) : 0.f;
    factor[n] = p.scale * __builtin_bit_cast(float, static_cast<uint32_t>(127 - up) << 23);
    // first part: the value; second: what its rounding leaves
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const float x0 = v[s][e] * lift, x1 = v[s][e + 1] * lift;
        const h2 hi = pair_of(x0, x1);
        const h2 part = pair_of(fmaf(static_cast<float>(hi[0]), less, x0) * times, fmaf(static_cast<float>(hi[1]), less, x1) * times);
        qf[n][s][e] = part[0];
        qf[n][s][e + 1] = part[1];
      }
    if (!finite) {
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
#pragma unroll
        for (int e = 0; e < 8; ++e) qf[n][s][e] = there ? part_of(v[s][e] * lift, second) : static_cast<_Float16>(0.f);
    }
  }

  f32x4 acc[NT][kFrags];
  // Weights and their sum are 2^kLift times as large, so that the second part of a
  // weight reaches further down.  ref: y is held as acc * 2^ref (8 bits, whose
  // weights are scaled by their tokens' scales; else the maximum alone scales it).
  constexpr float kLift = I8 ? 0.f : 14.f;
  float most[NT], sum[NT], ref[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    most[n] = -INFINITY;
    sum[n] = 0.f;
    ref[n] = -126.f;
#pragma unroll
    for (int f = 0; f < kFrags; ++f) acc[n][f] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  // Per lane: what its part of a score counts for (softmax's scale in it).
  float share[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) share[n] = second ? factor[n] * kPart : factor[n];

  int step = 0;
  for (int32_t tile = first_tile; tile <= last_tile; tile += waves) {
    f32x4 s[NT][2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        s[n][h] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int t = 0; t < kSteps; ++t) {
          h8 kf;
          if constexpr (!I8) kf = __builtin_bit_cast(h8, kw[h][t]);
          else kf = t % 2 ? codes_h8(kw[h][t / 2].z, kw[h][t / 2].w) : codes_h8(kw[h][t / 2].x, kw[h][t / 2].y);
          s[n][h] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, qf[n][t], s[n][h], 0, 0, 0);
        }
      }
    const uint32_t there = at.there;
    const bool whole = there == 0xFFFFFFFFu;
    // bit 4h + i: the lane's token is there
    const uint32_t mine = (there >> (4 * g) & 15u) | (there >> (16 + 4 * g) & 15u) << 4;
    __builtin_amdgcn_sched_barrier(0);
    // (the last one's are loaded again)
    if (tile + waves <= last_tile) at = locate(tile + waves, ++step);
    load_k(at);
    __builtin_amdgcn_sched_barrier(0);
    h8 pf[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float x[8], e[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        x[j] = joined(s[n][j / 4][j % 4], share[n]);
        if constexpr (I8) x[j] *= ks[j / 4][j % 4];
      }
      float now, add;
      auto weigh = [&]() {
        if (!whole) {
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] = mine >> j & 1 ? x[j] : -INFINITY;
        }
        const float here = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
        now = fmaxf(most[n], column_max(here));
        const float top = now == -INFINITY ? 0.f : now, base = top - kLift;
        add = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          e[j] = __builtin_amdgcn_exp2f(x[j] - base);
          add += e[j];
        }
        if (!I8 && __any(__builtin_fabsf(base) >= 0x1p24f)) {   // no number may lie kLift below the maximum
          add = 0.f;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            e[j] = __builtin_amdgcn_exp2f(x[j] - top) * 0x1p14f;
            add += e[j];
          }
        }
      };
      weigh();
      if (__any(add != add)) {   // an infinity of K or q, whose second parts' products are of any kind, or a NaN
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float own = s[n][j / 4][j % 4], oth = other_part(own);
          x[j] = (second ? both_parts(oth, own) : both_parts(own, oth)) * factor[n];
          if constexpr (I8) x[j] *= ks[j / 4][j % 4];
        }
        weigh();
      }
      const bool higher = now > most[n];
      const float down = higher ? __builtin_amdgcn_exp2f(most[n] - now) : 1.f;
      sum[n] = fmaf(sum[n], down, add);
      float old = down;   // what y so far is to be scaled by
      float lift = 1.f;
      bool moved = higher;
      if constexpr (I8) {
        // The weights of the codes are p times the token's scale: y is held
        // relative to the largest of them, 2^ref, as p is to the maximum.
        float top = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          e[j] *= vs[j / 4][j % 4];
          if (!whole) e[j] = mine >> j & 1 ? e[j] : 0.f;
          top = fmaxf(top, __builtin_fabsf(e[j]));
        }
        top = column_max(top);
        const float r = higher && most[n] > -INFINITY ? ref[n] + (most[n] - now) : ref[n];
        const float need = static_cast<float>(static_cast<int>(__builtin_bit_cast(uint32_t, top) >> 23) - 127 - 13);
        const float to = fmaxf(fmaxf(need, r), -126.f);
        moved = to > r;
        old = moved ? __builtin_amdgcn_exp2f(r - to) : 1.f;
        ref[n] = to;
        lift = __builtin_amdgcn_exp2f(-to);
      }
      most[n] = now;
      if (__any(moved)) {
#pragma unroll
        for (int f = 0; f < kFrags; ++f)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[n][f][i] *= old;
      }
#pragma unroll
      for (int j = 0; j < 8; j += 2) {   // first part: the weight; second: what its rounding leaves
        const float v0 = I8 ? e[j] * lift : e[j], v1 = I8 ? e[j + 1] * lift : e[j + 1];
        const h2 hi = pair_of(v0, v1);
        const h2 part = pair_of(fmaf(static_cast<float>(hi[0]), less, v0) * times, fmaf(static_cast<float>(hi[1]), less, v1) * times);
        pf[n][j] = part[0];
        pf[n][j + 1] = part[1];
      }
    }
    if (!whole) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (!(mine >> j & 1)) vt.clear(j);
    }
    // V's operands are formed again for a second head tile rather than held
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int f = 0; f < kFrags; ++f)
        acc[n][f] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vt.frag(f), pf[n], acc[n][f], 0, 0, 0);
    __builtin_amdgcn_sched_barrier(0);
    load_v(at);
    __builtin_amdgcn_sched_barrier(0);
  }

  // Join the wavefronts: y relative to the workgroup's maximum.
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const float all = column_sum(sum[n]);
    if (lane < 8) {
      wave_max[wave * 8 * NT + 8 * n + lane] = most[n];
      wave_sum[wave * 8 * NT + 8 * n + lane] = all;
    }
  }
  __syncthreads();
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int h = 8 * n + (col & 7);
    float top = -INFINITY, total = 0.f, m[kMostWaves], l[kMostWaves];
#pragma unroll
    for (int w = 0; w < kMostWaves; ++w) {
      m[w] = wave_max[(w < waves ? w : 0) * 8 * NT + h];
      l[w] = wave_sum[(w < waves ? w : 0) * 8 * NT + h];
      top = fmaxf(top, m[w]);
    }
    if (wave == 0) {
#pragma unroll
      for (int w = 0; w < kMostWaves; ++w)
        total += w < waves ? (m[w] == -INFINITY ? l[w] : l[w] * __builtin_amdgcn_exp2f(m[w] - top)) : 0.f;   // l is 0 there, or NaN
      if (lane < 8) {
        joint_max[h] = top;
        joint_sum[h] = total;
      }
    }
    float scale = most[n] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(most[n] - top + (I8 ? ref[n] : 0.f));
    if (sum[n] != sum[n]) scale = 1.f;   // NaN without a maximum: y is NaN already
    // Both columns of a head have its sums: the first writes rows 4g and 4g + 1 of each
    // operand, the second the other two, a run of E neighbouring dimensions at once.
    float* to = joint + (wave * 8 * NT + h) * kRow;
    auto put = [&](auto run, int f0, int dim0) {
      constexpr int E = decltype(run)::value;
      typedef float fE __attribute__((ext_vector_type(E < 4 ? 2 : 4)));
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float y[E];
#pragma unroll
        for (int k = 0; k < E; ++k) {
          const float a0 = acc[n][f0 + k][i], a1 = acc[n][f0 + k][i + 2], o0 = other_part(a0), o1 = other_part(a1);
          y[k] = both_parts(second ? o1 : a0, second ? a1 : o0) * scale;
        }
        float* at = to + dim0 + E * (4 * g + i + (second ? 2 : 0));
        if constexpr (E == 2) {
          *reinterpret_cast<fE*>(at) = fE{y[0], y[1]};
        } else {
#pragma unroll
          for (int k = 0; k < E; k += 4) *reinterpret_cast<fE*>(at + k) = fE{y[k], y[k + 1], y[k + 2], y[k + 3]};
        }
      }
    };
    constexpr int kA = VTile<I8, D>::kA, kB = VTile<I8, D>::kB, kC = VTile<I8, D>::kC;
#pragma unroll
    for (int f = 0; f < kA; ++f) put(std::integral_constant<int, 8>{}, 8 * f, 128 * f);
    if constexpr (kB) put(std::integral_constant<int, 4>{}, 8 * kA, 128 * kA);
    if constexpr (kC) put(std::integral_constant<int, 2>{}, 8 * kA + 4 * kB, 128 * kA + 64 * kB);
  }
  __syncthreads();
  for (int e = tid; e < heads_here * (D / 4); e += 64 * waves) {
    const int h = e / (D / 4), d = e % (D / 4) * 4;
    f32x4 y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < kMostWaves; ++w) {
      if (w >= waves) break;
      const f32x4 v = *reinterpret_cast<const f32x4*>(joint + (w * 8 * NT + h) * kRow + d);
#pragma unroll
      for (int j = 0; j < 4; ++j) y[j] += v[j];
    }
    const float total = joint_sum[h];
    const int64_t at = row * p.heads + first_head + h;
    if (p.splits <= 1) {
#pragma unroll
      for (int j = 0; j < 4; ++j) y[j] = total == 0.f ? 0.f : y[j] / total;
      store_y(p, at * D + d, y);
    } else {
      const int64_t slot = at * p.splits + part;
      *reinterpret_cast<f32x4*>(p.parts + slot * D + d) = y;
      if (d == 0) {
        p.stats[2 * slot] = joint_max[h];
        p.stats[2 * slot + 1] = total;
      }
    }
  }
#endif
}

}  // namespace pesti

namespace pesti_attn {

// Head tiles of 8 that a workgroup takes: two where a KV head has more than 8
// query heads and the registers leave three wavefronts on a SIMD (16 rows up to
// 2000, 16 query heads to a KV head of 128, where they leave one: 22.6 us with
// one tile, 24.7 with two).  Blocks of more heads read K and V each for themselves:
// 131071 tokens of 8 KV heads of 128 with 8, 16 and 32 query heads to each 102, 153
// and 299 us (538, 1075 and 2149 MB from memory).
inline int head_tiles(int64_t group, int64_t head_dim) { return group > 8 && head_dim <= 64 ? 2 : 1; }

template <bool I8, int D, int NT, bool SMALL>
int launch(const pesti::AttnArgs& p, int64_t rows, hipStream_t st) {
  pesti::AttnArgs args = p;
  void* params[] = {&args};
  return pesti_kv::launch(reinterpret_cast<const void*>(&pesti::attn_kernel<I8, D, NT, SMALL>),
                          dim3(static_cast<unsigned>(p.kv.kv_heads * p.head_blocks), static_cast<unsigned>(p.splits),
                               static_cast<unsigned>(rows)),
                          dim3(64 * p.waves), params, static_cast<size_t>(p.waves * (D + 6) + 2) * 8 * NT * 4, st);
}

template <bool I8, int D>
int launch_d(const pesti::AttnArgs& p, int64_t rows, hipStream_t st) {
  const bool small = p.kv.page_shift < 5;
  if constexpr (D <= 64) {
    if (head_tiles(p.group, D) == 2) return small ? launch<I8, D, 2, true>(p, rows, st) : launch<I8, D, 2, false>(p, rows, st);
  }
  return small ? launch<I8, D, 1, true>(p, rows, st) : launch<I8, D, 1, false>(p, rows, st);
}

template <bool I8>
int launch_format(const pesti::AttnArgs& p, int64_t rows, hipStream_t st) {
  switch (p.kv.head_dim) {
    case 32: return launch_d<I8, 32>(p, rows, st);
    case 64: return launch_d<I8, 64>(p, rows, st);
    case 96: return launch_d<I8, 96>(p, rows, st);
    case 128: return launch_d<I8, 128>(p, rows, st);
    case 160: return launch_d<I8, 160>(p, rows, st);
    case 192: return launch_d<I8, 192>(p, rows, st);
    case 224: return launch_d<I8, 224>(p, rows, st);
    case 256: return launch_d<I8, 256>(p, rows, st);
    default: return PESTI_ERR_SHAPE;
  }
}

int launch_f16(const pesti::AttnArgs& p, int64_t rows, hipStream_t st);
int launch_i8(const pesti::AttnArgs& p, int64_t rows, hipStream_t st);

}  // namespace pesti_attn
