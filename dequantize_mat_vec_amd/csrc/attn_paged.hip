// Entry points of the paged attention (kernel in attn_impl.h, instantiated per
// format in attn_f16.hip and attn_i8.hip), the split of a sequence into parts,
// and the kernel that joins them.
#include "attn_impl.h"

namespace pesti {

constexpr int kMaxParts = 256;
constexpr int kFewParts = 8;
constexpr int kManyRows = 32;

// y of one row and head from its parts: part i counts 2^(max_i - max) times, one
// whose every score is -infinity 0 times.  Zero times an infinity or NaN of its
// values is NaN, as in one part; a part without tokens, whose values are not
// written, is left out.  The parts are added in an order that the launch fixes.
__device__ __forceinline__ float part_weight(float m, float l, float top) {
  return m == -INFINITY ? (l == l ? 0.f : 1.f) : exp2f(m - top);   // a NaN without a maximum stays
}

// Few parts: a thread takes four dimensions of all of them.
__global__ __launch_bounds__(256) void attn_join_few_kernel(AttnArgs p, int64_t threads) {
  const int64_t at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (at >= threads) return;
  const int quads = p.kv.head_dim / 4, parts = p.splits;
  const int64_t head = at / quads, slot0 = head * parts;
  const int e = static_cast<int>(at - head * quads);
  const float* src = p.parts + slot0 * p.kv.head_dim + 4 * e;
  float m[kFewParts], l[kFewParts], top = -INFINITY, total = 0.f;
  f32x4 v[kFewParts], y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < kFewParts; ++i) {
    if (i >= parts) break;
    m[i] = p.stats[2 * (slot0 + i)];
    l[i] = p.stats[2 * (slot0 + i) + 1];
    v[i] = *reinterpret_cast<const f32x4*>(src + static_cast<int64_t>(i) * p.kv.head_dim);
  }
#pragma unroll
  for (int i = 0; i < kFewParts; ++i) top = i < parts ? fmaxf(top, m[i]) : top;
#pragma unroll
  for (int i = 0; i < kFewParts; ++i) {
    if (i >= parts) break;
    const float w = part_weight(m[i], l[i], top);
    const bool none = l[i] == kNoPart;
    total = fmaf(w, l[i], total);
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = none ? y[j] : fmaf(w, v[i][j], y[j]);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) y[j] = total == 0.f ? 0.f : y[j] / total;
  store_y(p, 4 * at, y);
}

// More: a workgroup has 4 * LANES dimensions of a row and head.  LANES threads
// take a part, all parts are in flight while the maxima are: with that many
// LANES at most that eight parts a thread are enough (256 parts of heads of 128
// with one workgroup a head: 28.5 us with the attention, with four: 17.6).
template <int LANES>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnArgs p) {
  constexpr int kGroups = 256 / LANES, kAhead = 8;
  __shared__ float weight[kMaxParts], sums[4], tops[4];   // (a weight of -1: no part)
  __shared__ f32x4 joint[kGroups][LANES];
  const int tid = threadIdx.x, d = p.kv.head_dim, parts = p.splits;
  const int64_t row = blockIdx.z, head = row * p.heads + blockIdx.y, slot0 = head * parts;
  const int e = tid % LANES, first = tid / LANES, at = blockIdx.x * 4 * LANES + 4 * e;
  const bool live = at < d;
  const float* src = p.parts + slot0 * d + (live ? at : 0);
  const int has = tid < parts ? tid : 0;
  float m = p.stats[2 * (slot0 + has)], l = p.stats[2 * (slot0 + has) + 1];
  f32x4 v[kAhead];
#pragma unroll
  for (int k = 0; k < kAhead; ++k) {
    const int i = first + k * kGroups;
    v[k] = *reinterpret_cast<const f32x4*>(src + static_cast<int64_t>(i < parts ? i : 0) * d);
  }
  if (tid >= parts) {
    m = -INFINITY;
    l = kNoPart;
  }
  float top = m;
#pragma unroll
  for (int o = 1; o < 64; o *= 2) top = fmaxf(top, __shfl_xor(top, o, 64));
  if ((tid & 63) == 0) tops[tid >> 6] = top;
  __syncthreads();
  top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3]));
  const float w = part_weight(m, l, top);
  weight[tid] = l == kNoPart ? -1.f : w;
  float total = w * l;
#pragma unroll
  for (int o = 1; o < 64; o *= 2) total += __shfl_xor(total, o, 64);
  if ((tid & 63) == 0) sums[tid >> 6] = total;
  __syncthreads();
  total = (sums[0] + sums[1]) + (sums[2] + sums[3]);
  f32x4 y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int k = 0; k < kAhead; ++k) {
    const float f = weight[first + k * kGroups];
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = f < 0.f ? y[j] : fmaf(f, v[k][j], y[j]);
  }
  joint[first][e] = y;
  __syncthreads();
  if (tid >= LANES || !live) return;
#pragma unroll
  for (int k = 1; k < kGroups; ++k)
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] += joint[k][e][j];
#pragma unroll
  for (int j = 0; j < 4; ++j) y[j] = total == 0.f ? 0.f : y[j] / total;
  store_y(p, head * d + at, y);
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

// Workgroups per KV head.
int64_t head_blocks(const pesti_kv_cache* cache, int64_t heads) {
  const int64_t group = heads / cache->kv_heads, each = 8 * pesti_attn::head_tiles(group, cache->head_dim);
  return (group + each - 1) / each;
}
// Parts that a sequence of up to max_length tokens is split into, and wavefronts
// of a workgroup.  In us, joining included, 8 KV heads of 128 in binary16 unless
// said:
//   whole   short sequences are one part and need no joining: longer ones the more
//     workgroups there are (512 tokens of 2 heads of 64: 7.5, 7.8 in parts, 700: 8.9
//     and 8.0; 64 rows up to 512: 19.4 and 28, up to 1500: 48 and 57, up to 5000: 143
//     and 133), in eight wavefronts where each has a compute unit to itself (64 rows
//     up to 300, two to a unit: 18.3 with eight, 13.3 with four; 40 rows up to 600 of
//     4 heads of 96: 9.4 and 9.8)
//   parts   of eight tiles, two of each of four wavefronts; of four tiles where the
//     launch has no more workgroups than compute units that way (2048 tokens: 10.2,
//     11.9 with eight); else as many parts as bring the launch to two workgroups a
//     compute unit, all resident at once (131071 tokens: 98, 101 at four; 32768: 31.5
//     and 36); three for some rows of different lengths (8 rows up to 4096: 22, 24 at
//     two and 26 at four), nine for many, so that what ends early makes room (48 rows
//     up to 8191 in 8 bits: 97, 98.5 at four, 114 at three)
struct Split {
  int64_t parts, part_tiles;
  int waves;
};
Split split_of(const pesti_kv_cache* cache, int64_t rows, int64_t heads, int64_t max_length) {
  const int64_t base = rows * cache->kv_heads * head_blocks(cache, heads), tiles = (max_length + pesti::kTile - 1) / pesti::kTile;
  const int64_t nt = pesti_attn::head_tiles(heads / cache->kv_heads, cache->head_dim);
  const int most_waves = pesti::attn_most_waves(static_cast<int>(cache->head_dim), static_cast<int>(nt));
  const int64_t whole = base <= 64 ? 1024 / cache->head_dim : (base < 256 ? 24 : 64);
  if (tiles <= whole) return Split{1, tiles, tiles > 4 && base <= 256 ? most_waves : 4};
  const int64_t least = base * ((tiles + 3) / 4) <= 256 ? 4 : 8, most = (tiles + least - 1) / least;
  const int64_t target = rows <= 2 ? 512 : (rows < pesti::kManyRows ? 768 : 2304);
  int64_t s = base > 0 ? (target + base - 1) / base : 1;
  s = s < most ? s : most;
  s = s < pesti::kMaxParts ? s : pesti::kMaxParts;
  const int64_t part = (tiles + s - 1) / s;
  return Split{s, part > least ? part : least, 4};
}
int64_t workspace_of(const pesti_kv_cache* cache, int64_t rows, int64_t heads, int64_t splits) {
  return splits <= 1 ? 0 : rows * heads * splits * (cache->head_dim + 2) * 4;
}

// The most that calls of up to so many rows and so long a bound need, so that a
// buffer of a program's largest call serves it as sequences finish: fewer rows have
// more parts each, and a bound just past the longest in parts of four tiles has half
// as many as that.
int64_t most_workspace(const pesti_kv_cache* cache, int64_t rows, int64_t heads, int64_t max_length) {
  int64_t most = 0;
  for (int64_t r = 1; r <= rows; ++r) {
    const int64_t four = 256 / (r * cache->kv_heads * head_blocks(cache, heads)) * 4 * pesti::kTile;   // longest in parts of four
    for (const int64_t bound : {four < max_length ? four : max_length, max_length}) {
      if (bound < 1) continue;
      const int64_t bytes = workspace_of(cache, r, heads, split_of(cache, r, heads, bound).parts);
      most = bytes > most ? bytes : most;
    }
  }
  return most;
}

int join(const pesti::AttnArgs& p, int64_t rows, hipStream_t st) {
  pesti::AttnArgs args = p;
  int64_t threads = rows * p.heads * (p.kv.head_dim / 4);
  void* params[] = {&args, &threads};
  if (p.splits <= pesti::kFewParts)
    return pesti_kv::launch(reinterpret_cast<const void*>(&pesti::attn_join_few_kernel), dim3(static_cast<unsigned>((threads + 255) / 256)),
                            dim3(256), params, 0, st);
  const int d = p.kv.head_dim, lanes = d > 64 && p.splits <= 64 ? 32 : (d > 32 && p.splits <= 128 ? 16 : 8);
  const void* kernel = lanes == 32 ? reinterpret_cast<const void*>(&pesti::attn_join_kernel<32>)
                                   : (lanes == 16 ? reinterpret_cast<const void*>(&pesti::attn_join_kernel<16>)
                                                  : reinterpret_cast<const void*>(&pesti::attn_join_kernel<8>));
  return pesti_kv::launch(kernel, dim3(static_cast<unsigned>((d + 4 * lanes - 1) / (4 * lanes)), static_cast<unsigned>(p.heads),
                                       static_cast<unsigned>(rows)),
                          dim3(256), params, 0, st);
}

}  // namespace

extern "C" {

int64_t pesti_attn_paged_workspace_bytes(const pesti_kv_cache* cache, int64_t rows, int64_t heads, int64_t max_length) {
  const int st = check(cache, rows, heads, max_length);
  return st != PESTI_OK ? st : most_workspace(cache, rows, heads, max_length);
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
  const Split split = split_of(cache, rows, heads, max_length);
  const int64_t splits = split.parts, need = workspace_of(cache, rows, heads, splits);
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
  p.part_tiles = static_cast<int32_t>(split.part_tiles);
  p.waves = split.waves;
  p.q_f32 = q_format == PESTI_FMT_F32;
  p.y_f32 = y_format == PESTI_FMT_F32;
  const hipStream_t sh = static_cast<hipStream_t>(stream);
  st = i8 ? pesti_attn::launch_i8(p, rows, sh) : pesti_attn::launch_f16(p, rows, sh);
  return st != PESTI_OK || splits <= 1 ? st : join(p, rows, sh);
}

}  // extern "C"
