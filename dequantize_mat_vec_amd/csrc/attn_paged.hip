// Entry points of the paged attention (kernel in attn_impl.h, instantiated per
// format in attn_f16.hip and attn_i8.hip), the split of a sequence into parts,
// and the kernel that joins them.
#include "attn_impl.h"

namespace pesti {

constexpr int kMaxParts = 256;
constexpr int kManyRows = 16;

// y of one row and head from its parts, in part order: part i counts 2^(max_i -
// max) times.  D4: head_dim / 4 rounded up to a power of two; as many threads
// take a part, so several parts are in flight.
template <int D4>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs p) {
  __shared__ float weight[kMaxParts], sums[4], tops[4];
  __shared__ f32x4 joint[256 / D4][D4];
  const int tid = threadIdx.x, d = p.kv.head_dim;
  const int64_t row = blockIdx.y, slot0 = (row * p.heads + blockIdx.x) * p.splits;
  int64_t seq;
  const int32_t length = attn_length(p, row, &seq);
  const int32_t parts = attn_parts(length, attn_part_tiles(length, p.splits, p.part_tiles));
  if (parts <= 1) return;   // written already
  float m = -INFINITY, l = 0.f;
  if (tid < parts) {
    m = p.stats[2 * (slot0 + tid)];
    l = p.stats[2 * (slot0 + tid) + 1];
  }
  float top = m;
#pragma unroll
  for (int o = 1; o < 64; o *= 2) top = fmaxf(top, __shfl_xor(top, o, 64));
  if ((tid & 63) == 0) tops[tid >> 6] = top;
  __syncthreads();
  top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
  const float w = m == -INFINITY ? (l == l ? 0.f : 1.f) : exp2f(m - top);   // a NaN without a maximum stays
  weight[tid] = w;
  float total = w * l;
#pragma unroll
  for (int o = 1; o < 64; o *= 2) total += __shfl_xor(total, o, 64);
  if ((tid & 63) == 0) sums[tid >> 6] = total;
  __syncthreads();
  total = (sums[0] + sums[1]) + (sums[2] + sums[3]);
  constexpr int kGroups = 256 / D4;
  const int e = tid % D4, first = tid / D4;
  const bool live = 4 * e < d;
  f32x4 y = {0.f, 0.f, 0.f, 0.f};
  if (live) {
    const f32x4* src = reinterpret_cast<const f32x4*>(p.parts + slot0 * d) + e;
#pragma unroll 8
    for (int i = first; i < parts; i += kGroups) {
      const f32x4 v = src[static_cast<int64_t>(i) * (d / 4)];
      const float f = weight[i];
#pragma unroll
      for (int j = 0; j < 4; ++j) y[j] = fmaf(f, v[j], y[j]);
    }
  }
  joint[first][e] = y;
  __syncthreads();
  if (first > 0 || !live) return;
  for (int k = 1; k < kGroups; ++k)
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] += joint[k][e][j];
  const int64_t at = (row * p.heads + blockIdx.x) * d + 4 * e;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float r = total == 0.f ? 0.f : y[j] / total;
    if (p.y_f32) static_cast<float*>(p.y)[at + j] = r;
    else static_cast<_Float16*>(p.y)[at + j] = static_cast<_Float16>(r);
  }
}

}  // namespace pesti

namespace {

int check(const pesti_kv_cache* cache, int64_t rows, int64_t heads, int64_t max_length) {
  const int st = pesti_kv::check_sizes(cache);
  if (st != PESTI_OK) return st;
  if (rows < 0 || rows > PESTI_MAX_SEQS) return PESTI_ERR_BATCH;
  if (heads < 1 || heads > PESTI_MAX_HEADS || heads % cache->kv_heads != 0) return PESTI_ERR_SHAPE;
  if (max_length < 1 || max_length > int64_t{1} << 30) return PESTI_ERR_SHAPE;
  return PESTI_OK;
}

// Workgroups per KV head, and parts that a sequence of up to max_length tokens
// is split into, none of under kMinPartTiles tiles.  Few rows: about four
// workgroups a compute unit, all resident at once (one row of 131071 binary16
// tokens, 8 KV heads of 128: 104 us so, 111 at nine).  Many rows, whose lengths
// differ: about nine, so that what ends early makes room (48 rows up to 8191 in 8
// bits: 102 us so, 106 at four).
int64_t head_blocks(const pesti_kv_cache* cache, int64_t heads) {
  const int64_t group = heads / cache->kv_heads, each = 8 * pesti_attn::head_tiles(group, cache->head_dim);
  return (group + each - 1) / each;
}
int64_t splits_of(const pesti_kv_cache* cache, int64_t rows, int64_t heads, int64_t max_length) {
  const int64_t base = rows * cache->kv_heads * head_blocks(cache, heads);
  const int64_t most = (max_length + pesti::kTile * pesti::kMinPartTiles - 1) / (pesti::kTile * pesti::kMinPartTiles);
  const int64_t target = rows >= pesti::kManyRows ? 2304 : 1024;
  int64_t s = base > 0 ? (target + base - 1) / base : 1;
  s = s < most ? s : most;
  return s < pesti::kMaxParts ? s : pesti::kMaxParts;
}
int64_t workspace_of(const pesti_kv_cache* cache, int64_t rows, int64_t heads, int64_t splits) {
  return splits <= 1 ? 0 : rows * heads * splits * (cache->head_dim + 2) * 4;
}

template <int D4>
int join(const pesti::AttnArgs& p, int64_t rows, hipStream_t st) {
  pesti::AttnArgs args = p;
  void* params[] = {&args};
  return pesti_kv::launch(reinterpret_cast<const void*>(&pesti::attn_join_kernel<D4>),
                          dim3(static_cast<unsigned>(p.heads), static_cast<unsigned>(rows)), dim3(256), params, 0, st);
}

}  // namespace

extern "C" {

int64_t pesti_attn_paged_workspace_bytes(const pesti_kv_cache* cache, int64_t rows, int64_t heads, int64_t max_length) {
  const int st = check(cache, rows, heads, max_length);
  return st != PESTI_OK ? st : workspace_of(cache, rows, heads, splits_of(cache, rows, heads, max_length));
}

int pesti_attn_paged(const pesti_kv_cache* cache, const pesti_kv_table* table, int64_t layer, int64_t rows, int64_t heads,
                     const int32_t* seq_ids, int32_t q_format, const void* q, int64_t q_stride, int32_t y_format,
                     void* y, float scale, int64_t max_length, void* workspace, int64_t workspace_bytes, void* stream) {
  int st = check(cache, rows, heads, max_length);
  if (st == PESTI_OK) st = pesti_kv::check_table_sizes(cache, table);
  if (st != PESTI_OK) return st;
  if (layer < 0 || layer >= cache->layers) return PESTI_ERR_SHAPE;
  if ((q_format != PESTI_FMT_F16 && q_format != PESTI_FMT_F32) || (y_format != PESTI_FMT_F16 && y_format != PESTI_FMT_F32))
    return PESTI_ERR_SHAPE;
  if (q_stride < heads * cache->head_dim || q_stride > (int64_t{1} << 40)) return PESTI_ERR_SHAPE;
  if (rows == 0) return PESTI_OK;
  if (!q || !y) return PESTI_ERR_NULL;
  if ((st = pesti_kv::check_table(cache, table, false)) != PESTI_OK) return st;
  if ((st = pesti_kv::check_pages(cache)) != PESTI_OK) return st;
  if (!pesti_host::aligned(q, 16) || !pesti_host::aligned(y, 16) ||
      (q_stride * (q_format == PESTI_FMT_F32 ? 4 : 2)) % 16 != 0 || !pesti_host::aligned(seq_ids, 4))
    return PESTI_ERR_ALIGN;
  const int64_t splits = splits_of(cache, rows, heads, max_length), need = workspace_of(cache, rows, heads, splits);
  if (need > 0) {
    if (!workspace || workspace_bytes < need) return PESTI_ERR_WORKSPACE;
    if (!pesti_host::aligned(workspace, 16)) return PESTI_ERR_ALIGN;
  }
  int dev = 0;
  size_t lds = 0;
  if ((st = pesti_host::current_device(&dev, &lds)) != PESTI_OK) return st;
  pesti::AttnArgs p{};
  p.kv = pesti_kv::args_of(cache, table);
  const int64_t page0 = layer * cache->pages;
  p.kv.k += page0 * p.kv.page_bytes;
  p.kv.v += page0 * p.kv.page_bytes;
  const bool i8 = cache->format == PESTI_FMT_I8ROW;
  if (i8) {
    p.kv.k_scales += page0 * p.kv.page_rows;
    p.kv.v_scales += page0 * p.kv.page_rows;
  }
  p.seq_ids = seq_ids;
  p.q = q;
  p.q_stride = q_stride;
  p.y = y;
  p.parts = static_cast<float*>(workspace);
  p.stats = p.parts + rows * heads * splits * cache->head_dim;
  p.scale = scale * 1.44269504088896340736f;   // exponentials are taken to base 2
  p.heads = static_cast<int32_t>(heads);
  p.group = static_cast<int32_t>(heads / cache->kv_heads);
  p.head_blocks = static_cast<int32_t>(head_blocks(cache, heads));
  p.splits = static_cast<int32_t>(splits);
  const int64_t tiles = (max_length + pesti::kTile - 1) / pesti::kTile, part = (tiles + splits - 1) / splits;
  p.part_tiles = static_cast<int32_t>(part > pesti::kMinPartTiles ? part : pesti::kMinPartTiles);
  p.q_f32 = q_format == PESTI_FMT_F32;
  p.y_f32 = y_format == PESTI_FMT_F32;
  const hipStream_t sh = static_cast<hipStream_t>(stream);
  st = i8 ? pesti_attn::launch_i8(p, rows, sh) : pesti_attn::launch_f16(p, rows, sh);
  if (st != PESTI_OK || splits <= 1) return st;
  if (cache->head_dim <= 32) return join<8>(p, rows, sh);
  if (cache->head_dim <= 64) return join<16>(p, rows, sh);
  return cache->head_dim <= 128 ? join<32>(p, rows, sh) : join<64>(p, rows, sh);
}

}  // extern "C"
