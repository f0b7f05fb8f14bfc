// Per-token symmetric 8-bit quantization of activations: the rule of the
// per-row int8 weights ("Project scaffold ...", quant.rs: per-row symmetric
// quantization) applied to rows of X, so that the prompt-width product runs
// on 8-bit integers (csrc/gemm_i8.hip).
//
//   s[t] = max_i |x[t][i]| / 127            one float32 rounding
//   c[t][i] = x[t][i] / s[t]                rounded half away from zero
//
// One pass: a row stays in the registers of the 64, 256 or 1024 lanes that
// serve it between its maximum and its codes, so X is read once.  What bounds
// long batches is memory and, close behind, vector ALU work: 4096 x 4864
// binary16 (60 MB) took 24 us with a division-free exact rounding of every
// element (17 operations), and takes 13 us with the one below (6), 4.6 TB/s;
// 8192 x 8192 36 us, 5.6 TB/s; float32 X 21 and 64 us, 4.8 and 5.2 TB/s.
//
// The codes are those of the exact quotient.  t = x * (1 / s) + 1.5 * 2^23 in
// one fma is the nearest integer of x * (1 / s), its low byte the code, and
// d = x * (1 / s) - q, the distance from it, shows where that may not be the
// nearest to x / s: 1 / s is within 2^-24 of its value, so the two lie within
// 127 * 2^-24 of each other.  Where some |d| of a wavefront's elements comes
// within 10^-5 of 1/2 (a few wavefronts in a hundred), all are done again
// exactly: the residual r = x - q s is exact in one fma (both terms are
// multiples of ulp(s) or finer with |r| below 2 s, so r needs no more than 24
// bits), and comparing 2 |r| with s moves q by one exactly where the quotient
// lies on the other side of a border, ties away from zero.
#include <type_traits>

#include "common.h"

namespace pesti {

struct QuantArgs {
  const void* x;
  int8_t* codes;
  float* scales;
  int64_t m;
  int64_t k;
};

// A 16-byte load: its elements as float32, and the largest magnitude's bits
// (as float32) so far.  Magnitudes compare as their bit patterns, with
// infinities and then NaN above every finite value, so one integer maximum
// finds them all.
template <typename T>
struct Vec;
template <>
struct Vec<_Float16> {
  static constexpr int kN = 8;
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  typedef u16x2 Max;
  __device__ __forceinline__ static Max zero() { return u16x2{0, 0}; }
  __device__ __forceinline__ static Max max(Max m, u32x4a v) {
#pragma unroll
    for (int w = 0; w < 4; ++w) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, v[w] & 0x7FFF7FFFu));
    return m;
  }
  __device__ __forceinline__ static uint32_t bits(Max m) {
    const uint16_t h = m.x > m.y ? m.x : m.y;
    return __builtin_bit_cast(uint32_t, static_cast<float>(__builtin_bit_cast(_Float16, h)));
  }
  __device__ __forceinline__ static float at(u32x4a v, int e) {
    typedef _Float16 h2 __attribute__((ext_vector_type(2)));
    const uint32_t w = v[e / 2];   // a copy: bit_cast of the element itself reads the vector's first
    return static_cast<float>(__builtin_bit_cast(h2, w)[e & 1]);
  }
};
template <>
struct Vec<float> {
  static constexpr int kN = 4;
  typedef uint32_t Max;
  __device__ __forceinline__ static Max zero() { return 0; }
  __device__ __forceinline__ static Max max(Max m, u32x4a v) {
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const uint32_t u = v[w] & 0x7FFFFFFFu;
      m = m > u ? m : u;
    }
    return m;
  }
  __device__ __forceinline__ static uint32_t bits(Max m) { return m; }
  __device__ __forceinline__ static float at(u32x4a v, int e) {
    const uint32_t w = v[e];
    return __builtin_bit_cast(float, w);
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

// Largest value of a wavefront, in a scalar register.
__device__ __forceinline__ uint32_t wave_umax(uint32_t v) {
  auto dpp = [](uint32_t x, auto ctrl) {
    return static_cast<uint32_t>(
        __builtin_amdgcn_update_dpp(0, static_cast<int>(x), decltype(ctrl)::value, 0xF, 0xF, false));
  };
  v = umax(v, dpp(v, std::integral_constant<int, 0xB1>{}));    // lane ^ 1
  v = umax(v, dpp(v, std::integral_constant<int, 0x4E>{}));    // lane ^ 2
  v = umax(v, dpp(v, std::integral_constant<int, 0x141>{}));   // mirror within 8
  v = umax(v, dpp(v, std::integral_constant<int, 0x140>{}));   // mirror within 16
  auto lane = [&](int l) { return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), l)); };
  return umax(umax(lane(0), lane(16)), umax(lane(32), lane(48)));
}

// Scale and codes of a row held by LANES lanes, NV vectors each.
template <typename T, int LANES, int NV>
__device__ __forceinline__ void one_row(const QuantArgs& a, int64_t row, int lane, int nv, const u32x4a (&v)[NV],
                                        uint32_t* wave_max) {
  typedef Vec<T> V;
  constexpr int kN = V::kN;
  typename V::Max m = V::zero();
#pragma unroll
  for (int j = 0; j < NV; ++j) m = V::max(m, v[j]);
  uint32_t mx = wave_umax(V::bits(m));
  if constexpr (LANES > 64) {
    if ((threadIdx.x & 63) == 0) wave_max[threadIdx.x >> 6] = mx;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < LANES / 64; ++w) mx = umax(mx, wave_max[w]);
  }

  const bool finite = mx < 0x7F800000u;
  float s = finite ? __builtin_bit_cast(float, mx) / 127.f : __builtin_nanf("");
  if (lane == 0) a.scales[row] = s;
  int8_t* cr = a.codes + row * a.k;
  auto store = [&](int j, const uint32_t* p) {
    const int i = lane + LANES * j;
    if (i >= nv) return;
    if constexpr (kN == 8)
      reinterpret_cast<uint2*>(cr)[i] = make_uint2(p[0], p[1]);
    else
      reinterpret_cast<uint32_t*>(cr)[i] = p[0];
  };
  uint32_t p[NV][kN / 4];
  float far = 0.f;
  const bool live = finite && s > 0.f;
  if (live && s >= 0x1p-100f) {
    const float inv = 1.f / s;
    constexpr float kRound = 12582912.f;   // 1.5 * 2^23: sums with it are integers, low byte first
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int w = 0; w < kN / 4; ++w) {
        uint32_t t[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x = V::at(v[j], 4 * w + e);
          const float q = __builtin_fmaf(x, inv, kRound);
          far = __builtin_fmaxf(far, __builtin_fabsf(__builtin_fmaf(x, inv, kRound - q)));
          t[e] = __builtin_bit_cast(uint32_t, q);
        }
        // low bytes of t[0..3]
        const uint32_t lo = __builtin_amdgcn_perm(t[1], t[0], 0x0C0C0400u);
        const uint32_t hi = __builtin_amdgcn_perm(t[3], t[2], 0x04000C0Cu);
        p[j][w] = lo | hi;
      }
    if (!__any(far > 0.5f - 1e-5f)) {
#pragma unroll
      for (int j = 0; j < NV; ++j) store(j, p[j]);
      return;
    }
  }
  // Every element exactly.  1 / s overflows below 2^-128 and s has few bits
  // among the subnormals: there both sides of the quotient are scaled by an
  // exact power of two.
  const float up = s < 0x1p-100f ? 0x1p100f : 1.f;
  s = live ? s * up : 1.f;
  const float inv = live ? 1.f / s : 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
#pragma unroll
    for (int w = 0; w < kN / 4; ++w) {
      p[j][w] = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x = live ? V::at(v[j], 4 * w + e) * up : 0.f;
        p[j][w] |= static_cast<uint32_t>(code_of(x, inv, s) & 0xFF) << (8 * e);
      }
    }
    store(j, p[j]);
  }
}

// LANES lanes per row (64: four rows per workgroup), NV 16-byte vectors per
// lane at most.  One row each: workgroups that take several, the next one's
// loads under the work on this one, measured slower (8192 x 8192 52 us
// against 40).
template <typename T, int LANES, int NV>
__global__ __launch_bounds__(LANES < 256 ? 256 : LANES) void quant_i8token_kernel(QuantArgs a) {
#ifdef __HIP_DEVICE_COMPILE__
  constexpr int kRows = LANES < 256 ? 256 / LANES : 1;
  __shared__ uint32_t wave_max[LANES / 64];
  const int lane = threadIdx.x % LANES;
  const int64_t row =
      static_cast<int64_t>(blockIdx.x) * kRows + __builtin_amdgcn_readfirstlane(threadIdx.x / LANES);
  if (LANES == 64 && row >= a.m) return;
  const int64_t bytes = a.k * static_cast<int64_t>(sizeof(T));
  const BufferRsrc x = buffer_of(static_cast<const uint8_t*>(a.x) + row * bytes, bytes);
  u32x4a v[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j)   // zeros past the row's end
    v[j] = __builtin_bit_cast(u32x4a, __builtin_amdgcn_raw_buffer_load_b128(x, 16 * (lane + LANES * j), 0, 0));
  one_row<T, LANES, NV>(a, row, lane, static_cast<int>(a.k / Vec<T>::kN), v, wave_max);
#endif
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

// 1024 lanes serve rows of more than 2048 vectors: at least 3 per lane, at
// most 4 in binary16.
template <typename T, int LANES>
int launch_nv(const pesti::QuantArgs& a, hipStream_t st) {
  const int64_t per = (a.k / pesti::Vec<T>::kN + LANES - 1) / LANES;
  if constexpr (LANES < 1024) {
    if (per <= 1) return launch<T, LANES, 1>(a, st);
    if (per <= 2) return launch<T, LANES, 2>(a, st);
  }
  if (per <= 3) return launch<T, LANES, 3>(a, st);
  if constexpr (LANES < 1024 || sizeof(T) == 4) {
    if (per > 6) return launch<T, LANES, 8>(a, st);
    if (per > 4) return launch<T, LANES, 6>(a, st);
  }
  return launch<T, LANES, 4>(a, st);
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
