// Mat-vec of 4-bit weights with a scale and a zero point per group:
//   y[b][o] = sum_i s[o][i / G] (q[o][i] - z[o][i / G]) x[b][i] + bias[o]
//
// Codes become binary16 integers in pairs: two 4-bit codes of a register under
// the exponent of 1024 (or of 16 codes higher, and a sixteenth of it), and one
// packed addition of -(1024 + z): q - z exactly, 9 vector instructions for 8
// weights.  Two kernels multiply them:
//
//   few products (one column, or a small matrix)   on the vector ALUs, with one
//     fma of a binary16 and a float32 factor per weight and column.  x stays in
//     registers as it is: a lane holds the same 32 (or 64) elements of one or two
//     columns for every row it serves, so nothing is staged and a short launch is
//     one memory round trip.
//   more   on the matrix cores, v_mfma_f32_16x16x32_f16, with x as the 16-row
//     operand and 16 rows of W as the columns.  Rows 0-7 of x are the first
//     binary16 parts of up to eight columns, rows 8-15 what these leave, 2^11 times
//     as large.  A column of the result is one row of W in all lanes that hold it,
//     so the lane that unpacks a row's codes also has the scales that its sums take.
//
// In both a group's sum is finished in float32 and takes its scale in one fma.
// Measured with groups of 128: 1 x 896 x 896 2.6 us, a round trip to memory and the
// launch; 8 x 151936 x 896 20 us, 3.8 TB/s of codes, scales and y.
#include <type_traits>

#include "common.h"

namespace pesti {

struct I4Matrix {
  const uint8_t* packed;
  const uint16_t* scales;
  const uint8_t* zeros;
};
struct I4Op {
  I4Matrix a, b;   // b: the up projection of a paired launch
  const float* x;
  float* y;
  const float* bias;
  int64_t out;
  int32_t in;
  int32_t groups;
};
struct I4Args {
  I4Op op[PESTI_MAX_GROUP];
  int32_t shift;          // log2 of the group size
  int32_t batch;
  int32_t k_waves;        // wavefronts that share a tile's row length
  int32_t phase_chunks;   // chunks of x staged at once
  int32_t batch_magic;    // ceil(2^16 / batch)
  int32_t joints;         // buffers for the wavefronts' sums of a tile in LDS
};

// Sum over groups of L lanes, in every lane: rows of 16 by DPP, then exchanges
// of quarters and halves of the wavefront.
template <int L>
__device__ __forceinline__ float row_sum(float v) {
#ifdef __HIP_DEVICE_COMPILE__
  v = group_sum<16>(v);
  auto add = [](auto h) {
    return __builtin_bit_cast(float, static_cast<uint32_t>(h[0])) + __builtin_bit_cast(float, static_cast<uint32_t>(h[1]));
  };
  if constexpr (L >= 32) {
    const uint32_t b = __builtin_bit_cast(uint32_t, v);
    v = add(__builtin_amdgcn_permlane16_swap(b, b, false, false));
  }
  if constexpr (L >= 64) {
    const uint32_t b = __builtin_bit_cast(uint32_t, v);
    v = add(__builtin_amdgcn_permlane32_swap(b, b, false, false));
  }
#endif
  return v;
}

__device__ __forceinline__ float i4_scale(const I4Matrix& m, int64_t row, int32_t groups, int32_t g) {
  return f16_lo(m.scales[row * groups + g]);
}
__device__ __forceinline__ int i4_zero(const I4Matrix& m, int64_t row, int32_t groups, int32_t g) {
  return m.zeros ? m.zeros[row * groups + g] : 8;
}

constexpr int kChunk = 128;        // weights of a row that a wavefront takes at once
constexpr int kI4MaxWaves = 8;
// LDS bytes of a chunk of x in operand order: 16 runs (step, lane group) of the
// parts of the columns, one unused place behind each run so that the 16 lanes
// that write a chunk do not meet in one bank.
constexpr int chunk_bytes(int batch) { return 256 * (2 * batch + 1); }

#ifdef __HIP_DEVICE_COMPILE__
typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2a __attribute__((ext_vector_type(2), aligned(8)));
typedef uint32_t u32x2u1 __attribute__((ext_vector_type(2), aligned(1)));
typedef uint32_t u32x4u2 __attribute__((ext_vector_type(4), aligned(2)));

// -(1024 + z) twice, of byte i of z; i4_operand's zero.
__device__ __forceinline__ h2 i4_zero_pair(uint32_t z, int i) {
  return __builtin_bit_cast(h2, __builtin_amdgcn_perm(0xE4E4E4E4u, z, 0x04000400u | i | i << 16));
}

// q - z of 8 codes, in the order 0 4 1 5 2 6 3 7.
__device__ __forceinline__ h8 i4_operand(uint32_t w, h2 zero, uint32_t magic) {
  const h2 sixteenth = {static_cast<_Float16>(0.0625f), static_cast<_Float16>(0.0625f)};
  const h2 zero16 = zero + h2{static_cast<_Float16>(960.f), static_cast<_Float16>(960.f)};   // -(64 + z)
  auto low = [&](uint32_t v) { return __builtin_bit_cast(h2, (v & 0x000F000Fu) | magic) + zero; };
  auto high = [&](uint32_t v) {
    return __builtin_elementwise_fma(__builtin_bit_cast(h2, (v & 0x00F000F0u) | magic), sixteenth, zero16);
  };
  const h2 a = low(w), b = high(w), c = low(w >> 8), d = high(w >> 8);
  return h8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// 0x64006400 in a register, so that mask and exponent are one instruction
// (v_and_or_b32 takes no literals).
__device__ __forceinline__ uint32_t i4_magic() {
  uint32_t v = 0x64006400u;
  asm volatile("" : "+v"(v));
  return v;
}

// The sum of both parts' products.  An infinity of the first stands: an infinite
// scale makes infinities of any sign, or NaN, of the second's sums.
__device__ __forceinline__ float both_parts(float hi, float lo) {
  return __builtin_fabsf(hi) == INFINITY ? hi : fmaf(lo, 0x1p-11f, hi);
}
#endif

// ---------------------------------------------------------------------------
// Few products: L lanes per row, J dwords (8 weights) a lane, R rows a lane group
// (PAIR: a row of each matrix), B columns, other workgroups for the next ones.  A lane's dwords lie L apart, so a
// load of codes, and of the 32 bytes of x behind each, is one run of memory.
// Rows longer than 8 J L weights (L = 64) are walked in passes.  A workgroup
// takes slabs of rows in turn; the next slab's codes are in flight under the
// arithmetic of this one.
// ---------------------------------------------------------------------------
template <int B, int L, int J, int R, bool PAIR>
__global__ __launch_bounds__(256) void gemv_i4group_few_kernel(I4Args p) {
#ifdef __HIP_DEVICE_COMPILE__
  static_assert(!PAIR || R == 2, "a pair is two rows");
  constexpr int kGroups = 4 * 64 / L, kRows = PAIR ? kGroups : kGroups * R;   // lane groups, rows of y per slab
  const I4Op o = p.op[blockIdx.y];
  const int col0 = blockIdx.z * B, cols = p.batch - col0;   // the last workgroups of an odd batch have one column twice
  const int sub = threadIdx.x & (L - 1), mine = static_cast<int>(threadIdx.x / L);
  const int64_t slabs = (o.out + kRows - 1) / kRows;
  if (blockIdx.x >= slabs) return;
  const int dwords = o.in / 8, passes = (dwords + L * J - 1) / (L * J), shift = p.shift - 3;
  const uint32_t magic = i4_magic();

  struct Codes {
    uint32_t q, s, z;
  };
  Codes w[J][R];
  auto row_of = [&](int64_t slab, int r) {
    const int64_t row = slab * kRows + (PAIR ? mine : mine + kGroups * r);
    return row < o.out ? row : o.out - 1;
  };
  // Dwords past the row's end stand for dword 0 (x is zero there).
  auto load = [&](int64_t slab, int pass) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const I4Matrix& m = PAIR && r ? o.b : o.a;
      const int64_t row = row_of(slab, r), g0 = row * o.groups;
      const uint32_t* rp = reinterpret_cast<const uint32_t*>(m.packed + row * (o.in / 2));
#pragma unroll
      for (int j = 0; j < J; ++j) {
        int d = (pass * J + j) * L + sub;
        d = d < dwords ? d : 0;
        w[j][r].q = rp[d];
        w[j][r].s = m.scales[g0 + (d >> shift)];
        w[j][r].z = m.zeros ? m.zeros[g0 + (d >> shift)] : 8;
      }
    }
  };
  f32x4 x[B][J][2];
  auto load_x = [&](int pass) {
#pragma unroll
    for (int b = 0; b < B; ++b)
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const int d = (pass * J + j) * L + sub;
        x[b][j][0] = x[b][j][1] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (d < dwords) {
          const f32x4* src = reinterpret_cast<const f32x4*>(o.x + static_cast<int64_t>(col0 + (b < cols ? b : 0)) * o.in + 8 * d);
          x[b][j][0] = src[0];
          x[b][j][1] = src[1];
        }
      }
  };
  // One dword's sum of a row and column, and its scale, from memory.
  auto scale_of = [&](int64_t slab, int r, int d) {
    const I4Matrix& m = PAIR && r ? o.b : o.a;
    return i4_scale(m, row_of(slab, r), o.groups, d >> shift);
  };
  auto dot = [&](int64_t slab, int r, int b, int d) {
    const I4Matrix& m = PAIR && r ? o.b : o.a;
    const int64_t row = row_of(slab, r);
    const uint32_t q = load_u32(m.packed + row * (o.in / 2) + 4 * d);
    const int z = i4_zero(m, row, o.groups, d >> shift);
    const float* src = o.x + static_cast<int64_t>(col0 + (b < cols ? b : 0)) * o.in + 8 * d;
    float s = 0.f;
#pragma nounroll
    for (int e = 0; e < 8; ++e) s = fmaf(static_cast<float>(static_cast<int>(q >> (4 * e) & 15) - z), src[e], s);
    return s;
  };
  int64_t slab = blockIdx.x;
  load(slab, 0);
  if (passes == 1) load_x(0);
  for (; slab < slabs; slab += gridDim.x) {
    float acc[R][B], bias[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      bias[r] = !PAIR && o.bias ? o.bias[row_of(slab, r)] : 0.f;
#pragma unroll
      for (int b = 0; b < B; ++b) acc[r][b] = 0.f;
    }
    for (int pass = 0; pass < passes; ++pass) {
      if (passes > 1) load_x(pass);
      Codes now[J][R];
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int r = 0; r < R; ++r) now[j][r] = w[j][r];
      if (pass + 1 < passes) load(slab, pass + 1);
      else if (slab + gridDim.x < slabs) load(slab + gridDim.x, 0);
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const h8 q = i4_operand(now[j][r].q, i4_zero_pair(now[j][r].z, 0), magic);
          const float scale = f16_lo(now[j][r].s);
#pragma unroll
          for (int b = 0; b < B; ++b) {
            float s = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) s = fmaf(static_cast<float>(q[2 * (e % 4) + e / 4]), x[b][j][e / 4][e % 4], s);
            acc[r][b] = fmaf(s, scale, acc[r][b]);
          }
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int b = 0; b < B; ++b) acc[r][b] = row_sum<L>(acc[r][b]);
    bool none = false;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int b = 0; b < B; ++b) none |= acc[r][b] != acc[r][b];
    if (__any(none)) {   // a NaN, perhaps of a stand-in's zeros times an infinite scale: without those
#pragma nounroll
      for (int i = 0; i < R * B; ++i) {
        const int r = i / B, b = i % B;
        float v = 0.f;
#pragma nounroll
        for (int d = sub; d < dwords; d += L) v = fmaf(dot(slab, r, b, d), scale_of(slab, r, d), v);
        v = row_sum<L>(v);
#pragma unroll
        for (int k = 0; k < R * B; ++k)
          if (k == i) acc[k / B][k % B] = acc[k / B][k % B] != acc[k / B][k % B] ? v : acc[k / B][k % B];
      }
    }
    if (sub == 0) {
      if constexpr (PAIR) {
        const int64_t row = slab * kRows + mine;
        if (row < o.out)
#pragma unroll
          for (int b = 0; b < B; ++b)
            if (b < cols) o.y[(col0 + b) * o.out + row] = acc[0][b] / (1.f + expf(-acc[0][b])) * acc[R - 1][b];
      } else {
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const int64_t row = slab * kRows + mine + kGroups * r;
          if (row < o.out)
#pragma unroll
            for (int b = 0; b < B; ++b)
              if (b < cols) o.y[(col0 + b) * o.out + row] = acc[r][b] + bias[r];
        }
      }
    }
  }
#endif
}

// ---------------------------------------------------------------------------
// More columns, on the matrix cores.
//
//   codes   a lane loads 16 bytes, 32 weights of its row; four lane groups hold
//           128 (a chunk).  Two exchanges of halves and two of quarters of the
//           wavefront (v_permlane32_swap, v_permlane16_swap) turn that into one
//           32-weight step per register, so a step lies in one group.
//   x       staged in LDS in operand order; each 128-weight chunk of a column is
//           scaled by a power of two for itself, which its sums get back.
// ---------------------------------------------------------------------------
#ifdef __HIP_DEVICE_COMPILE__
// Register s of a lane becomes the 8 codes that its lane group has of step s.
__device__ __forceinline__ void steps_of(const u32x4& q, uint32_t (&w)[4]) {
  const auto a = __builtin_amdgcn_permlane32_swap(q.x, q.z, false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(q.y, q.w, false, false);
  const auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  const auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  w[0] = c[0];
  w[1] = c[1];
  w[2] = d[0];
  w[3] = d[1];
}
#endif

// Scales and zero points of a tile pass through LDS in windows of 32 groups of
// 16 rows: a lane loads 8 groups of a row at once (a load per chunk would fetch
// each row's line again and again), and reads its row's back by chunk.
[[maybe_unused]] constexpr int kWindow = 32;
constexpr int kScaleRow = 80, kZeroRow = 40;   // LDS bytes of a row's window, padded against bank conflicts
constexpr int kWindowBytes = 16 * (kScaleRow + kZeroRow);

// How the work is dealt out (cut_of): few columns on the vector ALUs (the kernel
// above); or a wavefront takes tiles of 16 rows by itself; or a workgroup's
// wavefronts share a tile's chunks and join their sums in LDS (two wavefronts at
// least: 128 threads store the tile); or they do so with x staged in phases.
enum Way { kFew, kRows, kDeal, kPhases };

// Tiles of 16 rows (PAIR: of both matrices) in turn, U chunks in flight.  GS:
// groups of a chunk (1 where a group is 128 weights or more).
//
// Loads are unconditional, from stand-in places where there is nothing to load:
// the compiler then knows how many are younger than the one that it waits for.
template <int GS, bool PAIR, Way WAY, int U>
__global__ __launch_bounds__(64 * kI4MaxWaves) __attribute__((amdgpu_waves_per_eu(PAIR ? 2 : 4)))
void gemv_i4group_kernel(I4Args p) {
#ifdef __HIP_DEVICE_COMPILE__
  extern __shared__ uint8_t lds[];
  constexpr int R = PAIR ? 2 : 1, kWindowChunks = kWindow / GS;
  constexpr bool ROWS = WAY == kRows, PHASES = WAY == kPhases;
  static_assert(kWindowChunks % U == 0, "a window is whole rounds");
  const I4Op o = p.op[blockIdx.y];
  asm volatile("" ::"s"(o.a.packed), "s"(o.a.scales), "s"(o.a.zeros), "s"(o.x), "s"(o.y), "s"(o.bias), "s"(o.out), "s"(o.in),
               "s"(o.groups), "s"(p.shift), "s"(p.batch), "s"(p.phase_chunks), "s"(p.batch_magic));
  if constexpr (PAIR) asm volatile("" ::"s"(o.b.packed), "s"(o.b.scales), "s"(o.b.zeros));
  const int tid = threadIdx.x, waves = blockDim.x >> 6;
  const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n = lane & 15, g = lane >> 4;
  const int batch = p.batch, in = o.in, chunks = (in + kChunk - 1) / kChunk;
  const int phase = PHASES ? p.phase_chunks : chunks;
  const int64_t out = o.out;
  const int32_t tiles = static_cast<int32_t>((out + 15) / 16);
  int32_t tile = ROWS ? blockIdx.x * waves + wave : blockIdx.x;
  if (ROWS ? static_cast<int64_t>(blockIdx.x) * waves >= tiles : tile >= tiles) return;   // the whole workgroup
  const int stride = 2 * batch + 1;
  const uint32_t magic = i4_magic();

  // LDS: x in operand order [step][lane group][part, column], what its chunks'
  // sums are scaled by [chunk][8], windows of the wavefronts, partial sums.
  float* lower = reinterpret_cast<float*>(lds + phase * chunk_bytes(batch));
  uint8_t* window = reinterpret_cast<uint8_t*>(lower + 8 * phase) + wave * R * kWindowBytes;
  float* joint = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(lower + 8 * phase) + waves * R * kWindowBytes);
  const int slot = n < 8 ? (n < batch ? n : batch - 1) : batch + (n - 8 < batch ? n - 8 : batch - 1);

  // count chunks of x from c0 on, into the places from pos on: 16 lanes take a chunk
  // of a column.  Where chunks are dealt out a wavefront stages those that it
  // multiplies itself, into places of its own, and waits for no other.
  auto stage = [&](int c0, int pos, int count) {
    constexpr int kAhead = 4;
    const int items = count * batch, start = ROWS ? wave * 4 + g : g, apart = ROWS ? waves * 4 : 4;
    for (int base = start; base - g < items; base += apart * kAhead) {
      f32x4 v[kAhead][2];
      int at[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int item = base + k * apart;
        const int c = item * p.batch_magic >> 16, b = item - c * batch, i = (c0 + c) * kChunk + 8 * n;
        at[k] = item < items ? (pos + c) * 16 + n : -1;
        v[k][0] = v[k][1] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (item < items && i < in) {
          const f32x4* src = reinterpret_cast<const f32x4*>(o.x + static_cast<int64_t>(b) * in + i);
          v[k][0] = src[0];
          v[k][1] = src[1];
        }
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        if (base - g + k * apart >= items) break;   // the same for the wavefront
        const int item = base + k * apart;
        const int c = item * p.batch_magic >> 16, b = item - c * batch;
        auto chunk_max = [](float m) {   // over the 16 lanes
          m = fmaxf(m, dpp<0xB1>(m));
          m = fmaxf(m, dpp<0x4E>(m));
          m = fmaxf(m, dpp<0x141>(m));
          return fmaxf(m, dpp<0x140>(m));
        };
        float top = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) top = fmaxf(top, __builtin_fabsf(v[k][j / 4][j % 4]));
        top = chunk_max(top);
        const bool endless = __any(top == INFINITY);
        if (endless) {   // the largest finite one
          top = 0.f;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float m = __builtin_fabsf(v[k][j / 4][j % 4]);
            top = m < INFINITY && m > top ? m : top;
          }
          top = chunk_max(top);
        }
        const uint32_t bits = __builtin_bit_cast(uint32_t, top);
        int up = 14 + 127 - static_cast<int>(bits >> 23);   // brings the largest to [2^14, 2^15)
        up = bits == 0 ? 0 : (up > 126 ? 126 : up);
        const float lift = __builtin_bit_cast(float, static_cast<uint32_t>(up + 127) << 23);
        h8 hi, lo;
        // Two at once (v_cvt_pk_f16_f32, to nearest even).
        typedef float f2 __attribute__((ext_vector_type(2)));
#pragma unroll
        for (int j = 0; j < 4; ++j) {   // codes j and j + 4 share a register
          const float x0 = v[k][0][j] * lift, x1 = v[k][1][j] * lift;
          const h2 h = __builtin_convertvector((f2{x0, x1}), h2);
          float r0 = (x0 - static_cast<float>(h[0])) * 0x1p11f, r1 = (x1 - static_cast<float>(h[1])) * 0x1p11f;
          if (endless) {   // an infinity is all in the first part
            r0 = r0 - r0 == 0.f ? r0 : 0.f;
            r1 = r1 - r1 == 0.f ? r1 : 0.f;
          }
          hi[2 * j] = h[0];
          hi[2 * j + 1] = h[1];
          const h2 l = __builtin_convertvector((f2{r0, r1}), h2);
          lo[2 * j] = l[0];
          lo[2 * j + 1] = l[1];
        }
        if (at[k] >= 0) {
          h8* x = reinterpret_cast<h8*>(lds) + at[k] * stride + b;
          x[0] = hi;
          x[batch] = lo;
          if (n == 0) lower[8 * (pos + c) + b] = __builtin_bit_cast(float, static_cast<uint32_t>(127 - up) << 23);
        }
      }
    }
    if constexpr (ROWS) __syncthreads();
    else __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  };

  const int64_t all_groups = out * o.groups;   // 8 at least
  const uint8_t* packed[R] = {o.a.packed};
  const uint16_t* scales[R] = {o.a.scales};
  const uint8_t* zeros[R] = {o.a.zeros};
  if constexpr (PAIR) {
    packed[R - 1] = o.b.packed;
    scales[R - 1] = o.b.scales;
    zeros[R - 1] = o.b.zeros;
  }
  // Offsets within a tile fit 32 bits; its start is the same in all lanes.
  const int half = in / 2;
  auto row_in = [&](int32_t t) {   // the lane's row of the tile; past the last one, that
    const int64_t left = out - 1 - static_cast<int64_t>(t) * 16;
    return left < n ? static_cast<int>(left) : n;
  };
  // Codes of chunk c of the lane's row; past the row's end (x is zero there) its
  // last ones.
  auto load = [&](int32_t t, int row_at, int c, u32x4 (&d)[R]) {
    int at = c * 64 + 16 * g;
    at = row_at + (at < half - 16 ? at : half - 16);
#pragma unroll
    for (int r = 0; r < R; ++r) d[r] = load_u32x4_a16(packed[r] + static_cast<int64_t>(t) * 16 * half + static_cast<uint32_t>(at));
  };

  // Groups g0 + 8 g .. + 7 of the lane's row.  At the arrays' end the load
  // starts earlier, and the values are moved down when they are put in place.
  u32x4 ws[R];
  u32x2 wz[R];
  auto fetch = [&](int32_t t, int row, int g0) {
    const int64_t start = static_cast<int64_t>(t) * 16 * o.groups, base = start < all_groups - 8 ? start : all_groups - 8;
    const int64_t room = all_groups - 8 - base;
    const int most = room < (1 << 30) ? static_cast<int>(room) : 1 << 30;
    int at = row * o.groups + g0 + 8 * g + static_cast<int>(start - base);
    at = at < most ? at : most;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      ws[r] = *reinterpret_cast<const u32x4u2*>(scales[r] + base + static_cast<uint32_t>(at));
      wz[r] = *reinterpret_cast<const u32x2u1*>((zeros[r] ? zeros[r] : reinterpret_cast<const uint8_t*>(scales[r])) + base +
                                                static_cast<uint32_t>(at));
    }
  };
  auto place = [&](int32_t t, int row, int g0) {
    const int64_t start = static_cast<int64_t>(t) * 16 * o.groups;
    if (start + 16 * o.groups + kWindow > all_groups) {   // the same in all lanes
      const int64_t past = start + row * o.groups + g0 + 8 * g - (all_groups - 8);
      const int k = past <= 0 ? 0 : (past < 8 ? static_cast<int>(past) : 7);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const uint64_t lo = ws[r].x | static_cast<uint64_t>(ws[r].y) << 32, hi = ws[r].z | static_cast<uint64_t>(ws[r].w) << 32;
        const int s = 16 * (k & 3);
        uint64_t a = k & 4 ? hi >> s : lo >> s, b = k & 4 ? 0 : hi >> s;
        if (s && !(k & 4)) a |= hi << (64 - s);
        ws[r] = u32x4{static_cast<uint32_t>(a), static_cast<uint32_t>(a >> 32), static_cast<uint32_t>(b), static_cast<uint32_t>(b >> 32)};
        const uint64_t z = (wz[r].x | static_cast<uint64_t>(wz[r].y) << 32) >> (8 * k);
        wz[r] = u32x2{static_cast<uint32_t>(z), static_cast<uint32_t>(z >> 32)};
      }
    }
    // Groups of a row's last chunk may lie past its end.  Their sums are 0 (x is zero
    // there), but the places hold the next row's scales, perhaps infinities or NaN.
    const int left = o.groups - g0 - 8 * g;   // groups of the row from the lane's first on
    if ((o.groups & (GS - 1)) != 0 && left < 8) {
      const int lo = left < 0 ? 0 : (left < 4 ? left : 4), hi = left < 4 ? 0 : left - 4;
      const uint64_t lo_mask = lo == 4 ? ~uint64_t{0} : (uint64_t{1} << 16 * lo) - 1, hi_mask = (uint64_t{1} << 16 * hi) - 1;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        ws[r].x &= static_cast<uint32_t>(lo_mask);
        ws[r].y &= static_cast<uint32_t>(lo_mask >> 32);
        ws[r].z &= static_cast<uint32_t>(hi_mask);
        ws[r].w &= static_cast<uint32_t>(hi_mask >> 32);
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (!zeros[r]) wz[r] = u32x2{0x08080808u, 0x08080808u};
      *reinterpret_cast<u32x4a*>(window + r * kWindowBytes + n * kScaleRow + 16 * g) = ws[r];
      *reinterpret_cast<u32x2a*>(window + r * kWindowBytes + 16 * kScaleRow + n * kZeroRow + 8 * g) = wz[r];
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  };

  float total[R][4];
  auto clear = [&]() {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i) total[r][i] = 0.f;
  };
  // c: place of the chunk; gw: its first group within the window
  auto multiply = [&](int c, int gw, const u32x4 (&d)[R]) {
    const h8* x = reinterpret_cast<const h8*>(lds) + (c * 16 + g) * stride + slot;
    h8 xf[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) xf[s] = x[s * 4 * stride];
    const f32x4 low = *reinterpret_cast<const f32x4*>(lower + 8 * c + (4 * g & 7));
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const uint8_t* sp = window + r * kWindowBytes + n * kScaleRow + 2 * gw;
      const uint8_t* zp = window + r * kWindowBytes + 16 * kScaleRow + n * kZeroRow + gw;
      uint32_t sc[(GS + 1) / 2], z;
      if constexpr (GS == 1) {
        sc[0] = *reinterpret_cast<const uint16_t*>(sp);
        z = *zp;
      } else if constexpr (GS == 2) {
        sc[0] = *reinterpret_cast<const uint32_t*>(sp);
        z = *reinterpret_cast<const uint16_t*>(zp);
      } else {
        const u32x2a v = *reinterpret_cast<const u32x2a*>(sp);
        sc[0] = v.x;
        sc[(GS - 1) / 2] = v.y;
        z = *reinterpret_cast<const uint32_t*>(zp);
      }
      uint32_t q[4];
      steps_of(d[r], q);
      f32x4 part;
      float acc[4];
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const int gi = s * GS / 4;
        if (s * GS % 4 == 0) part = f32x4{0.f, 0.f, 0.f, 0.f};
        part = __builtin_amdgcn_mfma_f32_16x16x32_f16(xf[s], i4_operand(q[s], i4_zero_pair(z, gi), magic), part, 0, 0, 0);
        if ((s + 1) * GS % 4 == 0) {
          const float scale = gi % 2 ? f16_hi(sc[gi / 2]) : f16_lo(sc[gi / 2]);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[i] = gi == 0 ? part[i] * scale : fmaf(part[i], scale, acc[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) total[r][i] = fmaf(acc[i], low[i], total[r][i]);
    }
  };

  // The thread's element of a tile that the wavefronts join.
  const int eb = tid >> 4 & 7, en = tid & 15;
  const bool mine = !ROWS && tid < 128 && eb < batch;
  auto bias_of = [&](int32_t t) {
    const int64_t row = static_cast<int64_t>(t) * 16 + (ROWS ? n : en);
    return *(o.bias && row < out ? o.bias + row : o.x);
  };
  auto store_rows = [&](int32_t t, float bias) {
    float y[R][4];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t v = __builtin_bit_cast(uint32_t, total[r][i]);
        const auto h = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        y[r][i] = both_parts(__builtin_bit_cast(float, static_cast<uint32_t>(h[0])),
                             __builtin_bit_cast(float, static_cast<uint32_t>(h[1])));
      }
    const int64_t row = static_cast<int64_t>(t) * 16 + n;
    if (g >= 2 || row >= out) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int b = 4 * g + i;
      if (b < batch) o.y[b * out + row] = PAIR ? y[0][i] / (1.f + expf(-y[0][i])) * y[R - 1][i] : (o.bias ? y[0][i] + bias : y[0][i]);
    }
  };
  auto keep = [&](float* at) {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i) at[((wave * R + r) * 4 + i) * 64 + lane] = total[r][i];
  };
  auto resume = [&](const float* at) {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int i = 0; i < 4; ++i) total[r][i] = at[((wave * R + r) * 4 + i) * 64 + lane];
  };
  auto join = [&](int32_t t, const float* at, float bias) {
    const int64_t row = static_cast<int64_t>(t) * 16 + en;
    if (!mine || row >= out) return;
    float y[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float hi = 0.f, lo = 0.f;
#pragma unroll
      for (int j = 0; j < kI4MaxWaves; ++j) {
        const float* src = at + (((j < waves ? j : 0) * R + r) * 4 + eb % 4) * 64 + eb / 4 * 16 + en;
        const float a = src[0], b = src[32];
        hi += j < waves ? a : 0.f;
        lo += j < waves ? b : 0.f;
      }
      y[r] = both_parts(hi, lo);
    }
    o.y[eb * out + row] = PAIR ? y[0] / (1.f + expf(-y[0])) * y[R - 1] : (o.bias ? y[0] + bias : y[0]);
  };

  // The workgroup takes tiles in turn, for each phase of x again: between
  // phases the tiles' sums wait in LDS.  A wavefront's chunks of a phase are
  // first .. first + count - 1.
  const int32_t apart = ROWS ? gridDim.x * waves : gridDim.x;
  const int slot_size = waves * R * 256;
  u32x4 w[U][R];
  if (tile >= tiles) tile = -1;   // no tiles for this wavefront: it stages x only
  float bias = bias_of(tile < 0 ? 0 : tile);
  for (int c0 = 0; c0 < chunks; c0 += phase) {
    const int here = chunks - c0 < phase ? chunks - c0 : phase;
    const int share = ROWS ? here : (here + waves - 1) / waves, first = ROWS ? 0 : wave * share;
    const int count = here - first < share ? (here - first > 0 ? here - first : 0) : share;
    const int pos = PHASES ? wave * (phase / waves) : first;
    const int g_first = (c0 + first) * kChunk >> p.shift;
    int32_t here_tile = tile < 0 ? 0 : tile;
    int row = row_in(here_tile), turn = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) load(here_tile, row * half, c0 + first + u, w[u]);
    fetch(here_tile, row, g_first);
    stage(c0 + first, pos, count);
    if (tile < 0) break;
    while (true) {
      const int32_t next = here_tile + apart < tiles ? here_tile + apart : here_tile;
      const int next_row = row_in(next);
      float* slot = joint + turn * slot_size;
      if (PHASES && c0 > 0) resume(slot);
      else clear();
      for (int w0 = 0; w0 < count; w0 += kWindowChunks) {
        const int gw0 = (c0 + first + w0) * kChunk >> p.shift;
        place(here_tile, row, gw0);
        const bool more = w0 + kWindowChunks < count;
        fetch(more ? here_tile : next, more ? row : next_row, more ? (c0 + first + w0 + kWindowChunks) * kChunk >> p.shift : g_first);
        const int end = more ? w0 + kWindowChunks : count;
        for (int i = w0; i < end; i += U) {
#pragma unroll
          for (int u = 0; u < U; ++u) {
            if (i + u >= end) break;
            multiply(pos + i + u, ((c0 + first + i + u) * kChunk >> p.shift) - gw0, w[u]);
            const bool same = i + u + U < count;
            load(same ? here_tile : next, (same ? row : next_row) * half, c0 + first + (same ? i + u + U : u), w[u]);
            __builtin_amdgcn_sched_barrier(0);   // (steps side by side cost registers, and wavefronts)
          }
        }
      }
      if constexpr (ROWS) {
        store_rows(here_tile, bias);
      } else if constexpr (PHASES) {
        keep(slot);
        ++turn;
      } else {
        if (p.joints == 1) __syncthreads();   // the tile before has been read
        keep(slot);
        __syncthreads();
        join(here_tile, slot, bias);
        if (p.joints > 1) turn ^= 1;
      }
      if (here_tile + apart >= tiles) break;
      here_tile = next;
      row = next_row;
      if constexpr (!PHASES) bias = bias_of(here_tile);
    }
  }
  if constexpr (PHASES) {
    __syncthreads();
    for (const float* slot = joint; tile < tiles; tile += apart, slot += slot_size) join(tile, slot, bias_of(tile));
  }
#endif
}

__global__ __launch_bounds__(256) void i4group_bias_kernel(I4Args p) {   // rows of no columns
  const I4Op& o = p.op[blockIdx.y];
  const int64_t n = o.out * p.batch;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n; i += static_cast<int64_t>(gridDim.x) * 256)
    o.y[i] = o.bias ? o.bias[i % o.out] : 0.f;
}

// Eight weights of one dword per thread.
__global__ __launch_bounds__(256) void dequant_i4group_kernel(I4Matrix m, int64_t rows, int32_t in, int32_t groups,
                                                              int32_t shift, float* w) {
  const int64_t n = rows * (in / 8);
  for (int64_t d = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; d < n; d += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t row = d / (in / 8);
    const int32_t g = static_cast<int32_t>(d - row * (in / 8)) * 8 >> shift;
    const uint32_t v = load_u32(m.packed + 4 * d);
    const float s = i4_scale(m, row, groups, g);
    const int z = i4_zero(m, row, groups, g);
    f32x4 lo, hi;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      lo[e] = s * static_cast<float>(static_cast<int>(v >> (4 * e) & 15) - z);
      hi[e] = s * static_cast<float>(static_cast<int>(v >> (4 * e + 16) & 15) - z);
    }
    reinterpret_cast<f32x4*>(w)[2 * d] = lo;
    reinterpret_cast<f32x4*>(w)[2 * d + 1] = hi;
  }
}

}  // namespace pesti

namespace {

using pesti::I4Args;
using pesti::I4Matrix;
using pesti::I4Op;

bool group_ok(int64_t group) {
  return group >= 32 && group <= PESTI_MAX_IN_FEATURES && (group & (group - 1)) == 0;
}

// PESTI_OK, an error, or 1 for nothing to do.
int check_op(const pesti_gemv_i4group_op& o, int32_t batch) {
  if (o.out_features < 0 || o.in_features < 0) return PESTI_ERR_SHAPE;
  if (o.out_features == 0 || batch == 0) return 1;
  if (o.in_features % 32 != 0 || o.in_features > PESTI_MAX_IN_FEATURES || o.out_features >= int64_t{1} << 31)
    return PESTI_ERR_SHAPE;
  const bool has_in = o.in_features > 0;
  if (!o.y || (has_in && (!o.packed || !o.scales || !o.x))) return PESTI_ERR_NULL;
  if (!pesti_host::aligned(o.y, 16) || !pesti_host::aligned(o.packed, 16) || !pesti_host::aligned(o.x, 16) ||
      !pesti_host::aligned(o.scales, 2) || !pesti_host::aligned(o.bias, 4))
    return PESTI_ERR_ALIGN;
  return PESTI_OK;
}

I4Op op_of(const pesti_gemv_i4group_op& o, int64_t group) {
  I4Op r{};
  r.a = I4Matrix{static_cast<const uint8_t*>(o.packed), o.scales, o.zeros};
  r.x = o.x;
  r.y = o.y;
  r.bias = o.bias;
  r.out = o.out_features;
  r.in = static_cast<int32_t>(o.in_features);
  r.groups = static_cast<int32_t>((o.in_features + group - 1) / group);
  return r;
}

int device() {
  int dev = 0;
  size_t lds = 0;
  return pesti_host::current_device(&dev, &lds);
}

// How an op is computed: it depends on the op and the batch alone, so an op of a
// group has the bits of its single call.  Measured with groups of 128, in us:
//   few products  (columns in pairs on the vector ALUs) 896 x 896, one column 2.8,
//     4.4 on the matrix cores, eight: 3.7 and 5.3; 2432 x 896, four: 4.2 and 4.7,
//     eight: 6.0 and 5.4; 4864 x 896, four: 6.1 and 5.7; 2048 x 4096, two: 5.3 and
//     6.5, three: 8.6 and 7.0; 512 x 16384, eight, few workgroups on the matrix
//     cores: 15 and 35
//   short rows    4864 x 896, four columns: 6.0 a wavefront a tile, 6.4 dealt
//     out; 2432 x 896: 6.0 and 4.8; 24576 x 896: 7.3 with four wavefronts a
//     workgroup, 6.7 with eight; gate and up of 9728 x 896: 8.0 with four, 9.9
//     with eight, 12.7 dealt out
//   longer rows   16384 x 2048, four columns: 10.9 a wavefront a tile, 10.1 dealt
//     out; 32768 x 2048, eight: 12.4 and 17.8; 100000 x 1536: 26 and 46; where x
//     leaves room for one workgroup a compute unit only if its wavefronts' rounds
//     are full (40000 x 3200, 1.2 rounds: 34.4 and 32.5)
//   long rows     14336 x 8192, eight columns: 40 in phases with four tiles of a
//     workgroup, 89 with one; 73 where the columns were split over three launches
using pesti::kDeal;
using pesti::kFew;
using pesti::kPhases;
using pesti::kRows;
struct Cut {
  pesti::Way way;
  int waves, phase, each;   // chunks staged at once (kFew: dwords of a pass); tiles of a workgroup, where x comes in phases
  bool operator==(const Cut& c) const { return way == c.way && waves == c.waves && phase == c.phase && each == c.each; }
};
constexpr int64_t kMost = 160 * 1024;   // LDS of a workgroup
int64_t x_bytes(int chunks, int columns) { return int64_t{chunks} * (pesti::chunk_bytes(columns) + 32); }
int64_t wave_bytes(int waves, bool pair, int joints) { return int64_t{waves} * (pair ? 2 : 1) * (pesti::kWindowBytes + 1024 * joints); }

Cut cut_of(const I4Op& o, int batch, bool pair) {
  const int chunks = (o.in + pesti::kChunk - 1) / pesti::kChunk, dwords = o.in / 8;
  const int64_t tiles = (o.out + 15) / 16, products = o.out * o.in * batch * (pair ? 2 : 1);
  const int64_t few = (chunks <= 8 ? 12 : (tiles > 64 ? 20 : (tiles > 32 ? 32 : 64))) << 20;
  // (the matrix kernel loads eight groups' scales at once)
  if (products <= few || o.out * o.groups < 8) {
    int span = 32;   // dwords per lane group and pass: 32 x 1, 2, 4 or 64 x 4, 8
    while (span < dwords && span < 512) span *= 2;
    return Cut{kFew, 4, span, 0};
  }
  if (tiles >= (chunks <= 8 ? 256 : 2048)) {
    const int64_t x = x_bytes(chunks, batch), rounds = (tiles + 2047) / 2048;   // of one workgroup a compute unit
    if (x <= 64 * 1024) return Cut{kRows, pair || tiles < 1024 ? 4 : 8, chunks, 0};
    if (x <= kMost - wave_bytes(8, pair, 0) && 4 * tiles >= 3 * 2048 * rounds) return Cut{kRows, 8, chunks, 0};
  }
  // 128 threads store a tile of eight columns
  const int waves = chunks < 2 ? 2 : (chunks < pesti::kI4MaxWaves ? chunks : pesti::kI4MaxWaves);
  if (x_bytes(chunks, batch) <= kMost - wave_bytes(waves, pair, 1)) return Cut{kDeal, waves, chunks, 0};
  // Tiles whose sums wait in LDS for the next phase: the more a workgroup has,
  // the fewer times x is staged, and the less of it at once.
  const int64_t most = pair ? 4 : 8, per_unit = (tiles + 255) / 256;
  const int each = static_cast<int>(per_unit < most ? per_unit : most);
  const int phase = static_cast<int>((kMost - wave_bytes(waves, pair, each)) / x_bytes(1, batch));
  return Cut{kPhases, waves, phase / waves * waves, each};   // (8 chunks of 8 columns are 35 KiB of the 64 that are left at least)
}

int64_t most_rows(const I4Args& p, int n_ops) {
  int64_t rows = 0;
  for (int i = 0; i < n_ops; ++i) rows = p.op[i].out > rows ? p.op[i].out : rows;
  return rows;
}

int submit(const void* kernel, I4Args& p, int64_t blocks, int n_ops, int threads, size_t lds, hipStream_t st, int columns = 1) {
  void* params[] = {&p};
  const hipError_t e = hipLaunchKernel(kernel, dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(n_ops), static_cast<unsigned>(columns)),
                                       dim3(threads), params, lds, st);
  return e == hipSuccess ? PESTI_OK : PESTI_ERR_LAUNCH;
}

template <int B, int L, int J, bool PAIR>
int launch_few(I4Args& p, int n_ops, hipStream_t st) {
  const int64_t groups = 4 * 64 / L, rows = most_rows(p, n_ops);
  auto run = [&](auto r) {
    constexpr int R = decltype(r)::value;
    const int64_t slabs = (rows + groups * (PAIR ? 1 : R) - 1) / (groups * (PAIR ? 1 : R));
    return submit(reinterpret_cast<const void*>(&pesti::gemv_i4group_few_kernel<B, L, J, R, PAIR>), p, slabs < 2048 ? slabs : 2048,
                  n_ops, 256, 0, st, (p.batch + B - 1) / B);
  };
  if constexpr (PAIR) {
    return run(std::integral_constant<int, 2>{});
  } else {
    if (rows >= 1024 * groups) return run(std::integral_constant<int, 2>{});
    return run(std::integral_constant<int, 1>{});
  }
}

template <int B, bool PAIR>
int launch_few_span(I4Args& p, int n_ops, int span, hipStream_t st) {
  if (span == 32) return launch_few<B, 32, 1, PAIR>(p, n_ops, st);
  if (span == 64) return launch_few<B, 32, 2, PAIR>(p, n_ops, st);
  if (span == 128) return launch_few<B, 32, 4, PAIR>(p, n_ops, st);
  if (span == 256) return launch_few<B, 64, 4, PAIR>(p, n_ops, st);
  return launch_few<B, 64, 8, PAIR>(p, n_ops, st);
}

template <int GS, bool PAIR>
int launch_many(I4Args& p, int n_ops, const Cut& c, hipStream_t st) {
  const int64_t tiles = (most_rows(p, n_ops) + 15) / 16;
  p.phase_chunks = c.phase;
  p.batch_magic = (65536 + p.batch - 1) / p.batch;
  const int64_t x = x_bytes(c.phase, p.batch);
  if (c.way == kRows) {
    const int64_t blocks = (tiles + c.waves - 1) / c.waves;
    return submit(reinterpret_cast<const void*>(&pesti::gemv_i4group_kernel<GS, PAIR, kRows, 2>), p, blocks < 512 ? blocks : 512,
                  n_ops, 64 * c.waves, x + wave_bytes(c.waves, PAIR, 0), st);
  }
  if (c.way == kPhases) {
    p.joints = c.each;
    return submit(reinterpret_cast<const void*>(&pesti::gemv_i4group_kernel<GS, PAIR, kPhases, 2>), p, (tiles + c.each - 1) / c.each,
                  n_ops, 64 * c.waves, x + wave_bytes(c.waves, PAIR, c.each), st);
  }
  // Workgroups that are resident together stage x once and take tiles in turn.
  p.joints = x + wave_bytes(c.waves, PAIR, 2) > kMost ? 1 : 2;
  const int64_t lds = x + wave_bytes(c.waves, PAIR, p.joints), resident = 256 * (lds > kMost / 2 ? 1 : 2);
  return submit(reinterpret_cast<const void*>(&pesti::gemv_i4group_kernel<GS, PAIR, kDeal, 2>), p, tiles < resident ? tiles : resident,
                n_ops, 64 * c.waves, lds, st);
}

template <bool PAIR>
int launch_cut(I4Args& p, int n_ops, const Cut& c, hipStream_t st) {
  if (c.way == kFew)
    return p.batch == 1 ? launch_few_span<1, PAIR>(p, n_ops, c.phase, st) : launch_few_span<2, PAIR>(p, n_ops, c.phase, st);
  if (p.shift == 5) return launch_many<4, PAIR>(p, n_ops, c, st);
  if (p.shift == 6) return launch_many<2, PAIR>(p, n_ops, c, st);
  return launch_many<1, PAIR>(p, n_ops, c, st);
}

// Ops of one cut share a launch.
int launch(const I4Args& all, int n_ops, bool pair, hipStream_t st) {
  bool taken[PESTI_MAX_GROUP] = {};
  for (int i = 0; i < n_ops; ++i) {
    if (taken[i]) continue;
    I4Args p = all;
    int n = 0;
    const bool empty = all.op[i].in == 0;
    const Cut c = empty ? Cut{} : cut_of(all.op[i], all.batch, pair);
    for (int j = i; j < n_ops; ++j) {
      if (taken[j] || (all.op[j].in == 0) != empty) continue;
      if (!empty && !(cut_of(all.op[j], all.batch, pair) == c)) continue;
      taken[j] = true;
      p.op[n++] = all.op[j];
    }
    int r;
    if (empty) {
      void* params[] = {&p};
      r = hipLaunchKernel(reinterpret_cast<const void*>(&pesti::i4group_bias_kernel), dim3(64, static_cast<unsigned>(n)), dim3(256),
                          params, 0, st) == hipSuccess ? PESTI_OK : PESTI_ERR_LAUNCH;
    } else {
      r = pair ? launch_cut<true>(p, n, c, st) : launch_cut<false>(p, n, c, st);
    }
    if (r != PESTI_OK) return r;
  }
  return PESTI_OK;
}

}  // namespace

extern "C" {

int pesti_gemv_group_i4group(int32_t n_ops, const pesti_gemv_i4group_op* ops, int64_t group, int32_t batch, void* stream) {
  if (n_ops < 0 || n_ops > PESTI_MAX_GROUP || !group_ok(group)) return PESTI_ERR_SHAPE;
  if (n_ops > 0 && !ops) return PESTI_ERR_NULL;
  if (batch < 0 || batch > PESTI_MAX_BATCH) return PESTI_ERR_BATCH;
  I4Args p{};
  int n = 0;
  for (int i = 0; i < n_ops; ++i) {
    const int st = check_op(ops[i], batch);
    if (st < 0) return st;
    if (st == PESTI_OK) p.op[n++] = op_of(ops[i], group);
  }
  if (n == 0) return PESTI_OK;
  const int st = device();
  if (st != PESTI_OK) return st;
  p.shift = __builtin_ctzll(static_cast<unsigned long long>(group));
  p.batch = batch;
  return launch(p, n, false, static_cast<hipStream_t>(stream));
}

int pesti_gemv_i4group(int64_t out_features, int64_t in_features, int64_t group, const void* packed, const uint16_t* scales,
                       const uint8_t* zeros, const float* x, float* y, const float* bias, int32_t batch, void* stream) {
  const pesti_gemv_i4group_op o{out_features, in_features, packed, scales, zeros, x, y, bias};
  return pesti_gemv_group_i4group(1, &o, group, batch, stream);
}

int pesti_gemv_i4group_swiglu(int64_t out_features, int64_t in_features, int64_t group, const void* gate_packed,
                              const uint16_t* gate_scales, const uint8_t* gate_zeros, const void* up_packed,
                              const uint16_t* up_scales, const uint8_t* up_zeros, const float* x, float* h,
                              int32_t batch, void* stream) {
  if (!group_ok(group)) return PESTI_ERR_SHAPE;
  if (batch < 0 || batch > PESTI_MAX_BATCH) return PESTI_ERR_BATCH;
  const pesti_gemv_i4group_op gate{out_features, in_features, gate_packed, gate_scales, gate_zeros, x, h, nullptr};
  const pesti_gemv_i4group_op up{out_features, in_features, up_packed, up_scales, up_zeros, x, h, nullptr};
  int st = check_op(gate, batch);
  if (st < 0) return st;
  const int st_up = check_op(up, batch);
  if (st_up < 0) return st_up;
  if (st == 1) return PESTI_OK;
  if ((st = device()) != PESTI_OK) return st;
  I4Args p{};
  p.op[0] = op_of(gate, group);
  p.op[0].b = op_of(up, group).a;
  p.shift = __builtin_ctzll(static_cast<unsigned long long>(group));
  p.batch = batch;
  return launch(p, 1, true, static_cast<hipStream_t>(stream));
}

int pesti_dequant_i4group(int64_t rows, int64_t in_features, int64_t group, const void* packed, const uint16_t* scales,
                          const uint8_t* zeros, float* w_out, void* stream) {
  if (!group_ok(group) || rows < 0 || in_features < 0 || in_features % 32 != 0 || in_features > PESTI_MAX_IN_FEATURES)
    return PESTI_ERR_SHAPE;
  if (rows == 0 || in_features == 0) return PESTI_OK;
  if (!packed || !scales || !w_out) return PESTI_ERR_NULL;
  if (!pesti_host::aligned(packed, 16) || !pesti_host::aligned(w_out, 16) || !pesti_host::aligned(scales, 2))
    return PESTI_ERR_ALIGN;
  const int st = device();
  if (st != PESTI_OK) return st;
  I4Matrix m{static_cast<const uint8_t*>(packed), scales, zeros};
  int32_t in = static_cast<int32_t>(in_features), groups = static_cast<int32_t>((in_features + group - 1) / group);
  int32_t shift = __builtin_ctzll(static_cast<unsigned long long>(group));
  void* params[] = {&m, &rows, &in, &groups, &shift, &w_out};
  const hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(&pesti::dequant_i4group_kernel),
                                       dim3(pesti_host::grid_for((rows * (in_features / 8) + 255) / 256, 8192)), dim3(256),
                                       params, 0, static_cast<hipStream_t>(stream));
  return e == hipSuccess ? PESTI_OK : PESTI_ERR_LAUNCH;
}

}  // extern "C"
