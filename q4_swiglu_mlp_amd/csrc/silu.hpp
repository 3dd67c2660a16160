// silu over fp32's whole range.
#pragma once

#include <hip/hip_runtime.h>

namespace zinc {

// silu(z) u = z u / (1 + e^-z).  e^-z as 2^t (1 + r ln 2) with t = -z log2(e) rounded and r what
// the rounding left, log2(e) in two parts: within a few units in the last place, and the reciprocal
// within one.  z is cut for t: at 64, where e^-z adds nothing to 1, and at kTail.
// From kTail on down (t > 119) the quotient is 2^-t, to 2^-119 of it, and soon leaves fp32's range,
// where a large u may bring the product back.  TAIL leaves 2^-120 to the reciprocal and takes the rest,
// 2^(120 - t), as two factors, u first, so that nothing falls out of range before the product does; for
// other z it gives the same bits.  (Under e^-1024 every u vanishes.)
constexpr float kTail = -83.0f;
template <bool TAIL = false>
__device__ __forceinline__ float silu_times(float z, float u) {
  constexpr float kHi = -0x1.715476p+0f, kLo = -0x1.4ae0cp-26f, kLn2 = 0x1.62e43p-1f;
  const float c = __builtin_amdgcn_fmed3f(z, TAIL ? -1024.0f : kTail, 64.0f);
  const float t = c * kHi;
  const float r = fmaf(c, kLo, fmaf(c, kHi, -t));
  const float e2 = __builtin_amdgcn_exp2f(TAIL ? fminf(t, 120.0f) : t);
  const float s = z * __builtin_amdgcn_rcpf(1.0f + fmaf(e2, r * kLn2, e2));
  if constexpr (!TAIL) return s * u;
  const float f = __builtin_amdgcn_exp2f(fminf(120.0f - t, 0.0f) * 0.5f);
  return u * f * f * s;
}

// s = 1 / (1 + e^-z) as value factor^2, and 1 - s, by the same steps.  The factor is 2^-half, 1 down to
// z = -28, and value stays above 2^-42, so that z value u factor^2, one factor after u, loses nothing before the result
// does: u factor is the larger.  (Below 2^-149 the factor is zero, and so is the result.)  1 - s
// is e^-z s, which has no cancellation (z is cut where e^-z is zero, and not before: a large z times 1 - s has to
// vanish).
struct Sigmoid {
  float value, factor, rest;
  int half;
};
__device__ __forceinline__ Sigmoid sigmoid(float z) {
  constexpr float kHi = -0x1.715476p+0f, kLo = -0x1.4ae0cp-26f, kLn2 = 0x1.62e43p-1f;
  const float c = __builtin_amdgcn_fmed3f(z, -1024.0f, 200.0f);
  const float t = c * kHi;
  const float r = fmaf(c, kLo, fmaf(c, kHi, -t));
  const float half = rintf(fmaxf(t - 40.0f, 0.0f) * 0.5f);
  const float e2 = __builtin_amdgcn_exp2f(fmaf(half, -2.0f, t));
  const float e = fmaf(e2, r * kLn2, e2);
  const float value = __builtin_amdgcn_rcpf(1.0f + e);
  return {value, __builtin_amdgcn_ldexpf(1.0f, -(int)half), e * value, (int)half};
}

}  // namespace zinc
