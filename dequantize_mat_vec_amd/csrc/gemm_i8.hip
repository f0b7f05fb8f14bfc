// Linear layer on 8-bit integers with a scale per token and per channel,
// Y = (X W^T) * (token scale) * (channel scale) + b: the prompt-width product
// ("inferno" README, "Benchmarks": x @ w + b at prompt width) on the per-row
// int8 weights ("Project scaffold ...", quant.rs), X quantized by
// pesti_quant_i8token.  The 8-bit instances of the kernels in gemm_tile.h.
#include "gemm_tile.h"

int pesti_host::gemm_tiles_i8(const pesti::TileArgs& a, bool gated, hipStream_t st) {
  return gated ? launch_any<pesti::ElemI8, true>(a, st) : launch_any<pesti::ElemI8, false>(a, st);
}

extern "C" int pesti_gemm_i8row_i8token(int64_t m, int64_t out_features, int64_t in_features, const int8_t* codes,
                                        const float* row_scales, const int8_t* x_codes, const float* x_scales,
                                        int32_t y_format, void* y, const float* bias, void* stream) {
  if (y_format != PESTI_FMT_F32 && y_format != PESTI_FMT_F16) return PESTI_ERR_SHAPE;
  if (out_features < 0 || out_features > INT32_MAX || in_features < 0 || in_features % 32 != 0 ||
      in_features > PESTI_MAX_IN_FEATURES)
    return PESTI_ERR_SHAPE;
  if (m < 0 || m > PESTI_MAX_TOKENS) return PESTI_ERR_BATCH;
  if (m == 0 || out_features == 0) return PESTI_OK;
  if (!y || !row_scales || !x_scales || (in_features > 0 && (!codes || !x_codes))) return PESTI_ERR_NULL;
  if (!pesti_host::aligned(y, 16) || (codes && !pesti_host::aligned(codes, 16)) ||
      (x_codes && !pesti_host::aligned(x_codes, 16)) || !pesti_host::aligned(row_scales, 4) ||
      !pesti_host::aligned(x_scales, 4) || (bias && !pesti_host::aligned(bias, 4)))
    return PESTI_ERR_ALIGN;
  int dev = 0;
  size_t lds = 0;
  const int st = pesti_host::current_device(&dev, &lds);
  if (st != PESTI_OK) return st;
  pesti::TileArgs a{};
  a.w = reinterpret_cast<const uint8_t*>(codes);
  a.ws = row_scales;
  a.x = reinterpret_cast<const uint8_t*>(x_codes);
  a.xs = x_scales;
  a.y = y;
  a.bias = bias;
  a.rows = a.x_tokens = m;
  a.n = out_features;
  a.kbytes = static_cast<int32_t>(in_features);
  a.experts = 1;
  a.y_f16 = y_format == PESTI_FMT_F16;
  return pesti_host::gemm_tiles_i8(a, false, static_cast<hipStream_t>(stream));
}
