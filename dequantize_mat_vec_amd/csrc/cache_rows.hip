// New tokens' K and V into their places in the paged key-value cache: a row of
// head_dim values is rounded to binary16, or to 8 bits with a scale of its own
// by the rule of quant_i8token.hip (scale = max / 127, codes the exact quotient
// rounded half away from zero), and written once.
//
// A group of lanes serves a row, 8 values per lane: one page number, one or two
// 16-byte loads and one store each.  All rows of a call are on their way at once
// (2042 rows of 8 heads of 128: eight wavefronts on a SIMD), each behind its own
// sequence, length and page: the values are asked for with the row's place, the page
// with the length, and into 8 bits the exact rounding's cases are looked at only
// where a residual says so (that call 7.1 us, 8.6 with them always; one row of each
// of 64 sequences 2.9).  Counted over that call, the vector ALUs are busy for 60% of
// the time in which a compute unit has wavefronts, and those wait for 64% of theirs.
#include "i8_round.h"
#include "kv_cache.h"

namespace pesti {

struct AppendArgs {
  KvArgs kv;
  const void* x[2];        // K and V, [rows][stride]
  int64_t stride;
  const int32_t* seq_ids;
  const int32_t* positions;
  int64_t items;           // rows * 2 * kv_heads
};

typedef _Float16 f16x8 __attribute__((ext_vector_type(8), aligned(16)));

// Largest of a group of LANES.
template <int LANES>
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
#ifdef __HIP_DEVICE_COMPILE__
  auto with = [&](uint32_t o) { v = v > o ? v : o; };
  with(__builtin_amdgcn_update_dpp(0u, v, 0xB1, 0xF, 0xF, true));    // quads
  with(__builtin_amdgcn_update_dpp(0u, v, 0x4E, 0xF, 0xF, true));
  if constexpr (LANES >= 8) with(__builtin_amdgcn_update_dpp(0u, v, 0x141, 0xF, 0xF, true));    // halves of a row mirrored
  if constexpr (LANES >= 16) with(__builtin_amdgcn_update_dpp(0u, v, 0x140, 0xF, 0xF, true));   // a row mirrored
  if constexpr (LANES >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = r[0] > r[1] ? r[0] : r[1];
  }
#endif
  return v;
}

// T: type of x; LANES per row: head_dim / 8 rounded up to a power of two.
template <typename T, bool I8, int LANES>
__global__ __launch_bounds__(256) void append_kernel(AppendArgs p) {
  const KvArgs& a = p.kv;
  const int lane = threadIdx.x % LANES;
  constexpr int kRows = 256 / LANES;
  // whole groups of lanes take a row or pass over it together
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / LANES; i < p.items;
       i += static_cast<int64_t>(gridDim.x) * kRows) {
    const uint32_t item = static_cast<uint32_t>(i), rest = item / static_cast<uint32_t>(a.kv_heads);   // below 2^31
    const int32_t head = static_cast<int32_t>(item - rest * a.kv_heads);
    const int64_t row = rest >> 1;
    const int which = static_cast<int>(rest & 1);
    const int64_t s = p.seq_ids ? p.seq_ids[row] : row;
    int32_t pos = p.positions ? p.positions[row] : 0;
    const bool live = lane * 8 < a.head_dim;
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = 0.f;
    if (live) {
      const T* src = static_cast<const T*>(p.x[which]) + row * p.stride + static_cast<int64_t>(head) * a.head_dim + lane * 8;
      if constexpr (sizeof(T) == 4) {
        const f32x4 lo = reinterpret_cast<const f32x4*>(src)[0], hi = reinterpret_cast<const f32x4*>(src)[1];
#pragma unroll
        for (int e = 0; e < 4; ++e) { x[e] = lo[e]; x[e + 4] = hi[e]; }
      } else {
        const f16x8 v = *reinterpret_cast<const f16x8*>(src);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = static_cast<float>(v[e]);
      }
    }
    if (s < 0 || s >= a.seqs) continue;
    const int32_t* pages = a.table + s * a.width;
    const auto listed = [&](int32_t t) { return t >= 0 && t >> a.page_shift < a.width; };   // (else past the length too)
    const int32_t length = kv_length(a, static_cast<int32_t>(s));
    int32_t page = p.positions && listed(pos) ? pages[pos >> a.page_shift] : -1;
    if (!p.positions) {
      pos = length - 1;
      if (listed(pos)) page = pages[pos >> a.page_shift];
    }
    if (pos < 0 || pos >= length || !kv_page_ok(a, page)) continue;
    const int64_t at = page * a.page_rows + (static_cast<int64_t>(head) << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
    uint8_t* pool = which ? a.v : a.k;
    if constexpr (!I8) {
      if (!live) continue;
      f16x8 v;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = static_cast<_Float16>(x[e]);   // to nearest even
      reinterpret_cast<f16x8*>(pool)[(at * a.head_dim >> 3) + lane] = v;
    } else {
      // magnitudes compare as bit patterns: infinities and NaN lie above
      uint32_t m = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t u = __builtin_bit_cast(uint32_t, x[e]) & 0x7FFFFFFFu;
        m = m > u ? m : u;
      }
      m = row_max<LANES>(m);
      const bool finite = m < 0x7F800000u;
      float scale = finite ? __builtin_bit_cast(float, m) / 127.f : __builtin_nanf("");
      if (lane == 0) (which ? a.v_scales : a.k_scales)[at] = scale;
      uint32_t w[2];
      // The integer nearest to x / scale is the low byte of x inv + 1.5 2^23, and it
      // is that integer for certain where the exact residual is below half a scale,
      // however inv was rounded.
      const float magic = 12582912.f, inv = __builtin_amdgcn_rcpf(scale);
      float most = 0.f, t[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        t[e] = __builtin_fmaf(x[e], inv, magic);
        most = fmaxf(most, __builtin_fabsf(__builtin_fmaf(magic - t[e], scale, x[e])));
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        auto bits = [&](int e) { return __builtin_bit_cast(uint32_t, t[4 * h + e]); };
        w[h] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(bits(3), bits(2), 0x0C0C0400u),
                                     __builtin_amdgcn_perm(bits(1), bits(0), 0x0C0C0400u), 0x05040100u);
      }
      const bool sure = scale >= 0x1p-100f && 2.f * most < scale;   // false for a NaN
      if (__any(live && !sure)) {
        // (Near) ties, and rows whose 1 / scale overflows or whose scale has few bits,
        // as a subnormal: there both sides of the quotient take a power of two.
        const bool some = finite && scale > 0.f;
        const float up = scale < 0x1p-100f ? 0x1p100f : 1.f;
        const float s = some ? scale * up : 1.f, one = some ? 1.f / s : 0.f;
        w[0] = w[1] = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          w[e / 4] |= static_cast<uint32_t>(code_of(some ? x[e] * up : 0.f, one, s) & 0xFF) << (8 * (e % 4));
      }
      if (live) reinterpret_cast<uint2*>(pool)[(at * a.head_dim >> 3) + lane] = make_uint2(w[0], w[1]);
    }
  }
}

}  // namespace pesti

namespace {

template <typename T, bool I8, int LANES>
int launch(const pesti::AppendArgs& p, hipStream_t st) {
  pesti::AppendArgs args = p;
  void* params[] = {&args};
  return pesti_kv::launch(reinterpret_cast<const void*>(&pesti::append_kernel<T, I8, LANES>),
                          dim3(pesti_host::grid_for((p.items * LANES + 255) / 256, 1 << 20)), dim3(256), params, 0, st);
}

template <typename T, bool I8>
int launch_lanes(const pesti::AppendArgs& p, hipStream_t st) {
  if (p.kv.head_dim <= 32) return launch<T, I8, 4>(p, st);
  if (p.kv.head_dim <= 64) return launch<T, I8, 8>(p, st);
  if (p.kv.head_dim <= 128) return launch<T, I8, 16>(p, st);
  return launch<T, I8, 32>(p, st);
}

}  // namespace

extern "C" int pesti_cache_append(const pesti_kv_cache* cache, const pesti_kv_table* table, int64_t layer, int64_t rows,
                                  int32_t x_format, const void* k, const void* v, int64_t stride,
                                  const int32_t* seq_ids, const int32_t* positions, void* stream) {
  int st = pesti_kv::check_sizes(cache);
  if (st == PESTI_OK) st = pesti_kv::check_table_sizes(cache, table);
  if (st != PESTI_OK) return st;
  if (layer < 0 || layer >= cache->layers) return PESTI_ERR_SHAPE;
  if (x_format != PESTI_FMT_F16 && x_format != PESTI_FMT_F32) return PESTI_ERR_SHAPE;
  if (rows < 0 || rows > PESTI_MAX_TOKENS) return PESTI_ERR_BATCH;
  if (stride < cache->kv_heads * cache->head_dim || stride > (int64_t{1} << 40)) return PESTI_ERR_SHAPE;
  if (rows == 0) return PESTI_OK;
  if (!k || !v) return PESTI_ERR_NULL;
  if ((st = pesti_kv::check_table(cache, table, false)) != PESTI_OK) return st;
  if ((st = pesti_kv::check_pages(cache)) != PESTI_OK) return st;
  const int64_t size = x_format == PESTI_FMT_F32 ? 4 : 2;
  if (!pesti_host::aligned(k, 16) || !pesti_host::aligned(v, 16) || (stride * size) % 16 != 0 ||
      !pesti_host::aligned(seq_ids, 4) || !pesti_host::aligned(positions, 4))
    return PESTI_ERR_ALIGN;
  int dev = 0;
  size_t lds = 0;
  if ((st = pesti_host::current_device(&dev, &lds)) != PESTI_OK) return st;
  pesti::AppendArgs p{pesti_kv::args_of(cache, table), {k, v}, stride, seq_ids, positions, rows * 2 * cache->kv_heads};
  const int64_t page0 = layer * cache->pages;
  p.kv.k += page0 * p.kv.page_bytes;
  p.kv.v += page0 * p.kv.page_bytes;
  const hipStream_t sh = static_cast<hipStream_t>(stream);
  const bool f32 = x_format == PESTI_FMT_F32;
  if (cache->format == PESTI_FMT_F16) return f32 ? launch_lanes<float, false>(p, sh) : launch_lanes<_Float16, false>(p, sh);
  p.kv.k_scales += page0 * p.kv.page_rows;
  p.kv.v_scales += page0 * p.kv.page_rows;
  return f32 ? launch_lanes<float, true>(p, sh) : launch_lanes<_Float16, true>(p, sh);
}
