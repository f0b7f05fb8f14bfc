// The exact rounding of the symmetric 8-bit rule, for rows of X and of the
// key-value cache: the code of x / s, rounded half away from zero, from
// inv = 1 / s (rounded) and the residual r = x - q s, exact in one fma.
#pragma once

#include <hip/hip_runtime.h>

namespace pesti {

__device__ __forceinline__ int code_of(float x, float inv, float s) {
  float q = __builtin_rintf(x * inv);
  const float r = __builtin_fmaf(-q, s, x);
  const float d = 2.f * __builtin_fabsf(r);
  // A tie (d == s) moves away from zero only from the side nearer to it.
  if (d > s || (d == s && (r > 0.f) == (x > 0.f))) q += r > 0.f ? 1.f : -1.f;
  q = q > 127.f ? 127.f : (q < -127.f ? -127.f : q);
  return static_cast<int>(q);
}

}  // namespace pesti
