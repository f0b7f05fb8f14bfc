// Attention of one new token per sequence over the paged key-value cache
// ("PESTI ..." README, "Conformance" and "Current Status": grouped-query
// attention, paged attention during generation):
//   y[h] = sum_t p_t v[t] / sum_t p_t,  p_t = exp(scale q[h] . k[t] - max)
//
// The plainest form: a wavefront per row and query head walks the sequence 64
// tokens at a time, a token per lane for the scores, then 64 values of y per
// step, with the running maximum and sum of the softmax.
#include "kv_cache.h"

namespace pesti {

struct AttnArgs {
  KvArgs kv;
  const int32_t* seq_ids;
  const void* q;
  int64_t q_stride;
  void* y;
  float scale;
  int32_t heads;
  int32_t q_f32, y_f32, i8;
};

__global__ __launch_bounds__(64) void attn_kernel(AttnArgs p) {
  __shared__ float q[256], w[64];
  __shared__ int64_t at[64];
  const KvArgs& a = p.kv;
  const int h = blockIdx.x, lane = threadIdx.x, d = a.head_dim;
  const int64_t row = blockIdx.y;
  const int kvh = h / (p.heads / a.kv_heads);
  const int64_t s = p.seq_ids ? p.seq_ids[row] : row;
  const int32_t length = s >= 0 && s < a.seqs ? kv_length(a, static_cast<int32_t>(s)) : 0;
  for (int i = lane; i < d; i += 64) {
    const int64_t e = row * p.q_stride + h * d + i;
    q[i] = p.scale * (p.q_f32 ? static_cast<const float*>(p.q)[e] : static_cast<float>(static_cast<const _Float16*>(p.q)[e]));
  }
  __syncthreads();
  auto value = [&](const uint8_t* pool, const float* scales, int64_t r, int i) {
    if (p.i8) return scales[r] * static_cast<float>(reinterpret_cast<const int8_t*>(pool)[r * d + i]);
    return static_cast<float>(reinterpret_cast<const _Float16*>(pool)[r * d + i]);
  };
  float most = -INFINITY, sum = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int32_t t0 = 0; t0 < length; t0 += 64) {
    const int32_t t = t0 + lane;
    float score = -INFINITY;
    at[lane] = -1;
    if (t < length) {
      const int32_t page = a.table[s * a.width + (t >> a.page_shift)];
      if (kv_page_ok(a, page)) {
        const int64_t r = page * a.page_rows + (static_cast<int64_t>(kvh) << a.page_shift) + (t & ((1 << a.page_shift) - 1));
        at[lane] = r;
        score = 0.f;
        for (int i = 0; i < d; ++i) score = fmaf(q[i], value(a.k, a.k_scales, r, i), score);
      }
    }
    float m = score;
    for (int o = 1; o < 64; o *= 2) m = fmaxf(m, __shfl_xor(m, o, 64));
    const bool nan = __any(score != score);
    const float now = nan ? __builtin_nanf("") : fmaxf(most, m);
    const float base = now == -INFINITY ? 0.f : now;
    const float old = expf(most - base), e = expf(score - base);
    w[lane] = e;
    float all = e;
    for (int o = 1; o < 64; o *= 2) all += __shfl_xor(all, o, 64);
    sum = sum * old + all;
    most = now;
    __syncthreads();
    for (int j = 0; j < 4 && lane + 64 * j < d; ++j) {
      float v = acc[j] * old;
      for (int i = 0; i < 64; ++i)
        if (at[i] >= 0) v = fmaf(w[i], value(a.v, a.v_scales, at[i], lane + 64 * j), v);
      acc[j] = v;
    }
    __syncthreads();
  }
  for (int j = 0; j < 4 && lane + 64 * j < d; ++j) {
    const float v = sum == 0.f ? 0.f : acc[j] / sum;
    const int64_t e = (row * p.heads + h) * d + lane + 64 * j;
    if (p.y_f32) static_cast<float*>(p.y)[e] = v;
    else static_cast<_Float16*>(p.y)[e] = static_cast<_Float16>(v);
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

}  // namespace

extern "C" {

int64_t pesti_attn_paged_workspace_bytes(const pesti_kv_cache* cache, int64_t rows, int64_t heads, int64_t max_length) {
  return check(cache, rows, heads, max_length);
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
  int dev = 0;
  size_t lds = 0;
  if ((st = pesti_host::current_device(&dev, &lds)) != PESTI_OK) return st;
  pesti::AttnArgs p{pesti_kv::args_of(cache, table), seq_ids, q, q_stride, y, scale, static_cast<int32_t>(heads),
                    q_format == PESTI_FMT_F32, y_format == PESTI_FMT_F32, cache->format == PESTI_FMT_I8ROW};
  const int64_t page0 = layer * cache->pages;
  p.kv.k += page0 * p.kv.page_bytes;
  p.kv.v += page0 * p.kv.page_bytes;
  if (p.i8) {
    p.kv.k_scales += page0 * p.kv.page_rows;
    p.kv.v_scales += page0 * p.kv.page_rows;
  }
  void* params[] = {&p};
  return pesti_kv::launch(reinterpret_cast<const void*>(&pesti::attn_kernel),
                          dim3(static_cast<unsigned>(heads), static_cast<unsigned>(rows)), dim3(64), params, 0,
                          static_cast<hipStream_t>(stream));
}

}  // extern "C"
