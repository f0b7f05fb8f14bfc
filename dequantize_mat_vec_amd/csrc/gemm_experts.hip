// Linear layers grouped by expert: the rows of X, sorted by the expert that a
// router sent them to, each times its own expert's matrix, in one launch for
// all experts; and the joined gate and up products of the experts'
// feed-forward block ("PESTI ..." README, "Conformance": SwiGLU = silu(gate)
// * up).  The binary16 instances of the kernels in gemm_tile.h, and the
// entry points of both element types.
#include "gemm_tile.h"

int pesti_host::gemm_tiles_f16(const pesti::TileArgs& a, bool gated, hipStream_t st) {
  return gated ? launch_any<pesti::ElemF16, true>(a, st) : launch_any<pesti::ElemF16, false>(a, st);
}

namespace {

bool off(const void* p, uintptr_t a) { return p && !pesti_host::aligned(p, a); }

int run(int32_t format, pesti::TileArgs a, int64_t experts, int64_t in_features, int32_t y_format, bool gated,
        void* stream) {
  const bool i8 = format == PESTI_FMT_I8ROW;
  if (!i8 && format != PESTI_FMT_F16) return PESTI_ERR_SHAPE;
  if (y_format != PESTI_FMT_F32 && y_format != PESTI_FMT_F16) return PESTI_ERR_SHAPE;
  if (a.n < 0 || a.n > INT32_MAX || in_features < 0 || in_features % 32 != 0 || in_features > PESTI_MAX_IN_FEATURES)
    return PESTI_ERR_SHAPE;
  if (experts < 0 || experts > PESTI_MAX_EXPERTS) return PESTI_ERR_SHAPE;
  if (a.rows < 0 || a.rows > PESTI_MAX_TOKENS || a.x_tokens < 0 || a.x_tokens > PESTI_MAX_TOKENS)
    return PESTI_ERR_BATCH;
  if (!a.x_rows && a.x_tokens < a.rows) return PESTI_ERR_BATCH;
  if (a.x_rows && a.x_tokens * in_features * (i8 ? 1 : 2) > UINT32_MAX - 15) return PESTI_ERR_SHAPE;
  if (a.rows == 0 || a.n == 0 || experts == 0) return PESTI_OK;
  const bool data = in_features > 0 && a.x_tokens > 0;
  if (!a.y || !a.offsets) return PESTI_ERR_NULL;
  if (data && (!a.w || !a.x || (gated && !a.w2))) return PESTI_ERR_NULL;
  if (i8 && (!a.ws || (gated && !a.ws2) || (a.x_tokens > 0 && !a.xs))) return PESTI_ERR_NULL;
  if (off(a.y, 16) || off(a.w, 16) || off(a.w2, 16) || off(a.x, 16) || off(a.ws, 4) || off(a.ws2, 4) ||
      off(a.xs, 4) || off(a.bias, 4) || off(a.offsets, 4) || off(a.x_rows, 4))
    return PESTI_ERR_ALIGN;
  int dev = 0;
  size_t lds = 0;
  const int st = pesti_host::current_device(&dev, &lds);
  if (st != PESTI_OK) return st;
  a.experts = static_cast<int32_t>(experts);
  // without a row of X every row of Y is the product of a row of zeros
  a.kbytes = data ? static_cast<int32_t>(in_features * (i8 ? 1 : 2)) : 0;
  a.y_f16 = y_format == PESTI_FMT_F16;
  const hipStream_t sh = static_cast<hipStream_t>(stream);
  return i8 ? pesti_host::gemm_tiles_i8(a, gated, sh) : pesti_host::gemm_tiles_f16(a, gated, sh);
}

}  // namespace

extern "C" {

int pesti_gemm_experts(int32_t format, int64_t rows, int64_t experts, int64_t out_features, int64_t in_features,
                       const int32_t* offsets, const void* w, const float* w_scales, int64_t x_tokens, const void* x,
                       const float* x_scales, const int32_t* x_rows, int32_t y_format, void* y, const float* bias,
                       void* stream) {
  pesti::TileArgs a{};
  a.w = static_cast<const uint8_t*>(w);
  a.ws = w_scales;
  a.x = static_cast<const uint8_t*>(x);
  a.xs = x_scales;
  a.x_rows = x_rows;
  a.offsets = offsets;
  a.y = y;
  a.bias = bias;
  a.rows = rows;
  a.x_tokens = x_tokens;
  a.n = out_features;
  return run(format, a, experts, in_features, y_format, false, stream);
}

int pesti_gemm_experts_swiglu(int32_t format, int64_t rows, int64_t experts, int64_t out_features, int64_t in_features,
                              const int32_t* offsets, const void* w_gate, const void* w_up, const float* gate_scales,
                              const float* up_scales, int64_t x_tokens, const void* x, const float* x_scales,
                              const int32_t* x_rows, int32_t h_format, void* h, void* stream) {
  pesti::TileArgs a{};
  a.w = static_cast<const uint8_t*>(w_gate);
  a.w2 = static_cast<const uint8_t*>(w_up);
  a.ws = gate_scales;
  a.ws2 = up_scales;
  a.x = static_cast<const uint8_t*>(x);
  a.xs = x_scales;
  a.x_rows = x_rows;
  a.offsets = offsets;
  a.y = h;
  a.rows = rows;
  a.x_tokens = x_tokens;
  a.n = out_features;
  return run(format, a, experts, in_features, h_format, true, stream);
}

}  // extern "C"
