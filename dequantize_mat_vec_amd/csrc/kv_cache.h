// The paged key-value cache as its kernels see it, and the checks that its
// entry points share.
#pragma once

#include <cstdint>

#include "common.h"

namespace pesti {

// One pool of K or V pages [layers][pages][kv_heads][page_size][head_dim]
// with scales [layers][pages][kv_heads][page_size] in 8 bits (else null), and
// the sequences' tables.  page_size is 1 << page_shift.
struct KvArgs {
  uint8_t* k;
  uint8_t* v;
  float* k_scales;
  float* v_scales;
  int32_t* table;
  int32_t* lengths;
  int32_t* refs;
  int32_t pages;
  int32_t page_shift;
  int32_t kv_heads;
  int32_t head_dim;
  int32_t layers;
  int32_t seqs;
  int32_t width;
  int64_t page_bytes;     // K (or V) of one page of one layer
  int64_t page_rows;      // kv_heads * page_size: rows of one page, and its scales
};

// Tokens of sequence s, within its row of the table.
__device__ __forceinline__ int32_t kv_length(const KvArgs& a, int32_t s) {
  const int64_t n = a.lengths[s], most = static_cast<int64_t>(a.width) << a.page_shift;
  return static_cast<int32_t>(n < 0 ? 0 : (n > most ? most : n));
}
__device__ __forceinline__ int32_t kv_pages_of(const KvArgs& a, int32_t tokens) {
  return (tokens + (1 << a.page_shift) - 1) >> a.page_shift;
}
__device__ __forceinline__ bool kv_page_ok(const KvArgs& a, int32_t page) {
  return static_cast<uint32_t>(page) < static_cast<uint32_t>(a.pages);
}

}  // namespace pesti

namespace pesti_kv {

inline int size_of(int64_t format) { return format == PESTI_FMT_F16 ? 2 : 1; }

// The cache's sizes (no pointers).
inline int check_sizes(const pesti_kv_cache* c) {
  if (!c) return PESTI_ERR_NULL;
  if (c->format != PESTI_FMT_F16 && c->format != PESTI_FMT_I8ROW) return PESTI_ERR_SHAPE;
  if (c->layers < 1 || c->layers > PESTI_MAX_LAYERS || c->pages < 0 || c->pages > PESTI_MAX_PAGES) return PESTI_ERR_SHAPE;
  if (c->page_size < 8 || c->page_size > 1024 || (c->page_size & (c->page_size - 1))) return PESTI_ERR_SHAPE;
  if (c->kv_heads < 1 || c->kv_heads > PESTI_MAX_HEADS) return PESTI_ERR_SHAPE;
  if (c->head_dim < 32 || c->head_dim > 256 || c->head_dim % 32) return PESTI_ERR_SHAPE;
  return PESTI_OK;
}

inline int check_table_sizes(const pesti_kv_cache* c, const pesti_kv_table* t) {
  if (!t) return PESTI_ERR_NULL;
  if (t->seqs < 0 || t->seqs > PESTI_MAX_SEQS || t->width < 0 || t->width > (int64_t{1} << 30) / c->page_size)
    return PESTI_ERR_SHAPE;
  return PESTI_OK;
}

// The arrays of pages.
inline int check_pages(const pesti_kv_cache* c) {
  if (c->pages == 0) return PESTI_OK;
  const bool i8 = c->format == PESTI_FMT_I8ROW;
  if (!c->k || !c->v || (i8 && (!c->k_scales || !c->v_scales))) return PESTI_ERR_NULL;
  if (!pesti_host::aligned(c->k, 16) || !pesti_host::aligned(c->v, 16) ||
      (i8 && (!pesti_host::aligned(c->k_scales, 16) || !pesti_host::aligned(c->v_scales, 16))))
    return PESTI_ERR_ALIGN;
  return PESTI_OK;
}

// The sequences' arrays.
inline int check_table(const pesti_kv_cache* c, const pesti_kv_table* t, bool refs) {
  if (t->seqs > 0 && (!t->lengths || (t->width > 0 && !t->table))) return PESTI_ERR_NULL;
  if (refs && c->pages > 0 && !t->refs) return PESTI_ERR_NULL;
  if (!pesti_host::aligned(t->table, 4) || !pesti_host::aligned(t->lengths, 4) || !pesti_host::aligned(t->refs, 4))
    return PESTI_ERR_ALIGN;
  return PESTI_OK;
}

inline pesti::KvArgs args_of(const pesti_kv_cache* c, const pesti_kv_table* t) {
  pesti::KvArgs a{};
  const bool i8 = c->format == PESTI_FMT_I8ROW;
  a.k = static_cast<uint8_t*>(c->k);
  a.v = static_cast<uint8_t*>(c->v);
  a.k_scales = i8 ? c->k_scales : nullptr;
  a.v_scales = i8 ? c->v_scales : nullptr;
  if (t) {
    a.table = t->table;
    a.lengths = t->lengths;
    a.refs = t->refs;
    a.seqs = static_cast<int32_t>(t->seqs);
    a.width = static_cast<int32_t>(t->width);
  }
  a.pages = static_cast<int32_t>(c->pages);
  a.page_shift = __builtin_ctzll(static_cast<unsigned long long>(c->page_size));
  a.kv_heads = static_cast<int32_t>(c->kv_heads);
  a.head_dim = static_cast<int32_t>(c->head_dim);
  a.layers = static_cast<int32_t>(c->layers);
  a.page_rows = c->kv_heads * c->page_size;
  a.page_bytes = a.page_rows * c->head_dim * size_of(c->format);
  return a;
}

inline int launch(const void* kernel, dim3 grid, dim3 block, void** params, size_t lds, hipStream_t st) {
  return hipLaunchKernel(kernel, grid, block, params, lds, st) == hipSuccess ? PESTI_OK : PESTI_ERR_LAUNCH;
}

}  // namespace pesti_kv
