// Per-token symmetric 8-bit quantization of activations: the rule of the
// per-row int8 weights ("Project scaffold ...", quant.rs: per-row symmetric
// quantization) applied to rows of X, so that the prompt-width product runs
// on 8-bit integers (csrc/gemm_i8.hip).
//
//   s[t] = max_i |x[t][i]| / 127            one float32 rounding
//   c[t][i] = x[t][i] / s[t]                rounded half away from zero
//
// One pass: a row stays in the registers of the 64, 256 or 1024 lanes that
// serve it between its maximum and its codes, so X is read once.
//
// The codes are those of the exact quotient.  t = x * (1 / s) is within a
// few ulps of x / s, so q = rint(t) is off by one at most; the residual
// r = x - q s is exact in one fma (both terms are multiples of ulp(s) or
// finer with |r| below 2 s, so r needs no more than 24 bits), and comparing
// 2 |r| with s moves q by one exactly where the quotient lies on the other
// side of a border, ties away from zero.
#include "common.h"

namespace pesti {

struct QuantArgs {
  const void* x;
  int8_t* codes;
  float* scales;
  int64_t m;
  int64_t k;
};

// Elements of one 16-byte load as float32.
template <typename T>
struct Vec;
template <>
struct Vec<_Float16> {
  static constexpr int kN = 8;
  typedef _Float16 h8 __attribute__((ext_vector_type(8)));
  __device__ __forceinline__ static void load(const void* p, int64_t i, float* v) {
    const h8 h = reinterpret_cast<const h8*>(p)[i];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = static_cast<float>(h[e]);
  }
};
template <>
struct Vec<float> {
  static constexpr int kN = 4;
  __device__ __forceinline__ static void load(const void* p, int64_t i, float* v) {
    const f32x4 f = reinterpret_cast<const f32x4*>(p)[i];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = f[e];
  }
};

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

__device__ __forceinline__ int code_of(float x, float inv, float s) {
  float q = __builtin_rintf(x * inv);
  const float r = __builtin_fmaf(-q, s, x);
  const float d = 2.f * __builtin_fabsf(r);
  // A tie (d == s) moves away from zero only from the side nearer to it.
  if (d > s || (d == s && (r > 0.f) == (x > 0.f))) q += r > 0.f ? 1.f : -1.f;
  q = q > 127.f ? 127.f : (q < -127.f ? -127.f : q);
  return static_cast<int>(q);
}

// LANES lanes per row (64: four rows per workgroup), NV 16-byte vectors per
// lane at most.
template <typename T, int LANES, int NV>
__global__ __launch_bounds__(LANES < 256 ? 256 : LANES) void quant_i8token_kernel(QuantArgs a) {
  constexpr int kN = Vec<T>::kN;
  constexpr int kRows = LANES < 256 ? 256 / LANES : 1;
  __shared__ uint32_t wave_max[LANES / 64 < 1 ? 1 : LANES / 64];
  const int lane = threadIdx.x % LANES;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / LANES;
  if (LANES == 64 && row >= a.m) return;
  const int nv = static_cast<int>(a.k / kN);
  const uint8_t* xr = static_cast<const uint8_t*>(a.x) + row * a.k * static_cast<int64_t>(sizeof(T));

  float v[NV][kN];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int i = lane + LANES * j;
    if (i < nv) {
      Vec<T>::load(xr, i, v[j]);
    } else {
#pragma unroll
      for (int e = 0; e < kN; ++e) v[j][e] = 0.f;
    }
  }
  // Magnitudes compare as their bit patterns, with infinities and then NaN
  // above every finite value, so one integer maximum finds both.
  uint32_t mx = 0;
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < kN; ++e) mx = umax(mx, __builtin_bit_cast(uint32_t, v[j][e]) & 0x7FFFFFFFu);
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) mx = umax(mx, static_cast<uint32_t>(__shfl_xor(static_cast<int>(mx), d, 64)));
  if constexpr (LANES > 64) {
    if ((threadIdx.x & 63) == 0) wave_max[threadIdx.x >> 6] = mx;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < LANES / 64; ++w) mx = umax(mx, wave_max[w]);
  }

  const float amax = __builtin_bit_cast(float, mx);
  const bool finite = mx < 0x7F800000u;
  float s = finite ? amax / 127.f : __builtin_nanf("");
  if (lane == 0) a.scales[row] = s;
  const bool live = finite && s > 0.f;
  // 1 / s overflows below 2^-128 and s has few bits among the subnormals:
  // there both sides of the quotient are scaled by an exact power of two.
  const float up = s < 0x1p-100f ? 0x1p100f : 1.f;
  s = live ? s * up : 1.f;
  const float inv = live ? 1.f / s : 0.f;
  int8_t* cr = a.codes + row * a.k;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int i = lane + LANES * j;
    uint32_t packed[kN / 4];
#pragma unroll
    for (int w = 0; w < kN / 4; ++w) {
      uint32_t p = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x = live ? v[j][4 * w + e] * up : 0.f;
        p |= static_cast<uint32_t>(code_of(x, inv, s) & 0xFF) << (8 * e);
      }
      packed[w] = p;
    }
    if (i < nv) {
      if constexpr (kN == 8)
        reinterpret_cast<uint2*>(cr)[i] = make_uint2(packed[0], packed[1]);
      else
        reinterpret_cast<uint32_t*>(cr)[i] = packed[0];
    }
  }
}

}  // namespace pesti

namespace {

template <typename T, int LANES, int NV>
int launch(const pesti::QuantArgs& a, hipStream_t st) {
  constexpr int kRows = LANES < 256 ? 256 / LANES : 1;
  pesti::QuantArgs args = a;
  void* params[] = {&args};
  const hipError_t e = hipLaunchKernel(
      reinterpret_cast<const void*>(&pesti::quant_i8token_kernel<T, LANES, NV>),
      dim3(static_cast<unsigned>((a.m + kRows - 1) / kRows)), dim3(LANES < 256 ? 256 : LANES), params, 0, st);
  return e == hipSuccess ? PESTI_OK : PESTI_ERR_LAUNCH;
}

template <typename T, int LANES>
int launch_nv(const pesti::QuantArgs& a, hipStream_t st) {
  const int64_t per = (a.k / pesti::Vec<T>::kN + LANES - 1) / LANES;
  if (per <= 1) return launch<T, LANES, 1>(a, st);
  if (per <= 2) return launch<T, LANES, 2>(a, st);
  if (per <= 4) return launch<T, LANES, 4>(a, st);
  return launch<T, LANES, 8>(a, st);
}

// Lanes per row: a wavefront per row once the rows fill the chip and a row
// is at most 8 vectors per lane; else 256 lanes; rows too long for those
// take 1024 (PESTI_MAX_IN_FEATURES float32 are 8 vectors per lane).
template <typename T>
int launch_rows(const pesti::QuantArgs& a, hipStream_t st) {
  const int64_t nv = a.k / pesti::Vec<T>::kN;
  if (a.m >= 1024 && nv <= 8 * 64) return launch_nv<T, 64>(a, st);
  if (nv <= 8 * 256) return launch_nv<T, 256>(a, st);
  return launch_nv<T, 1024>(a, st);
}

}  // namespace

extern "C" int pesti_quant_i8token(int32_t x_format, int64_t m, int64_t in_features, const void* x,
                                   int8_t* codes, float* scales, void* stream) {
  if (x_format != PESTI_FMT_F16 && x_format != PESTI_FMT_F32) return PESTI_ERR_SHAPE;
  if (m < 0 || m > PESTI_MAX_TOKENS) return PESTI_ERR_BATCH;
  if (in_features < 0 || in_features % 32 != 0 || in_features > PESTI_MAX_IN_FEATURES) return PESTI_ERR_SHAPE;
  if (m == 0) return PESTI_OK;
  if (!scales || (in_features > 0 && (!x || !codes))) return PESTI_ERR_NULL;
  if ((x && !pesti_host::aligned(x, 16)) || (codes && !pesti_host::aligned(codes, 16)) ||
      !pesti_host::aligned(scales, 4))
    return PESTI_ERR_ALIGN;
  int dev = 0;
  size_t lds = 0;
  const int st = pesti_host::current_device(&dev, &lds);
  if (st != PESTI_OK) return st;
  const pesti::QuantArgs a{x, codes, scales, m, in_features};
  const hipStream_t sh = static_cast<hipStream_t>(stream);
  return x_format == PESTI_FMT_F16 ? launch_rows<_Float16>(a, sh) : launch_rows<float>(a, sh);
}
