// Mat-vec of 4-bit weights with a scale and a zero point per group:
//   y[b][o] = sum_i s[o][i / G] (q[o][i] - z[o][i / G]) x[b][i] + bias[o]
//
// The plainest form: a wavefront per row, 8 weights (a dword) per lane and step.
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
  int32_t shift;   // log2 of the group size
  int32_t batch;
  int32_t pair;
};

__device__ __forceinline__ float i4_scale(const I4Matrix& m, int64_t row, int32_t groups, int32_t g) {
  return f16_lo(m.scales[row * groups + g]);
}
__device__ __forceinline__ int i4_zero(const I4Matrix& m, int64_t row, int32_t groups, int32_t g) {
  return m.zeros ? m.zeros[row * groups + g] : 8;
}

__global__ __launch_bounds__(64) void gemv_i4group_kernel(I4Args p) {
  const I4Op& o = p.op[blockIdx.y];
  const int64_t row = blockIdx.x;
  if (row >= o.out) return;
  const int lane = threadIdx.x;
  for (int b = 0; b < p.batch; ++b) {
    float y[2] = {0.f, 0.f};
    for (int k = 0; k <= p.pair; ++k) {
      const I4Matrix& m = k ? o.b : o.a;
      float acc = 0.f;
      for (int i = 8 * lane; i < o.in; i += 512) {
        const uint32_t w = load_u32(m.packed + row * (o.in / 2) + i / 2);
        const int g = i >> p.shift, z = i4_zero(m, row, o.groups, g);
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          s = fmaf(static_cast<float>(static_cast<int>(w >> (4 * e) & 15) - z), o.x[static_cast<int64_t>(b) * o.in + i + e], s);
        acc = fmaf(s, i4_scale(m, row, o.groups, g), acc);
      }
      y[k] = group_sum<64>(acc);
    }
    if (lane == 0)
      o.y[b * o.out + row] = p.pair ? y[0] / (1.f + expf(-y[0])) * y[1] : y[0] + (o.bias ? o.bias[row] : 0.f);
  }
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

int launch(I4Args& p, int n_ops, hipStream_t st) {
  int64_t rows = 0;
  for (int i = 0; i < n_ops; ++i) rows = p.op[i].out > rows ? p.op[i].out : rows;
  void* params[] = {&p};
  const hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(&pesti::gemv_i4group_kernel),
                                       dim3(static_cast<unsigned>(rows), static_cast<unsigned>(n_ops)), dim3(64), params, 0, st);
  return e == hipSuccess ? PESTI_OK : PESTI_ERR_LAUNCH;
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
  return launch(p, n, static_cast<hipStream_t>(stream));
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
  p.pair = 1;
  return launch(p, 1, static_cast<hipStream_t>(stream));
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
