// Device helpers shared by the expert layer's FP8 operators: 16-bit and fp32
// rows read as eight values at a time, and the block quantiser's arithmetic.
//
// A block of 128 values is stored as e4m3 (OCP: largest value 448) with one
// fp32 scale, the smallest power of two s with max|x| / s <= 448.  With a power
// of two, x / s is exact, so e4m3's own rounding (to nearest, ties to even) is
// the only one, and q * s is exact in fp32 and bf16.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace zinc {

typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bhalf8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

// Eight consecutive values, 16-byte aligned, as fp32.
__device__ __forceinline__ void load8(const _Float16* p, float (&v)[8]) {
  const half8_t h = *reinterpret_cast<const half8_t*>(p);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = (float)h[i];
}
__device__ __forceinline__ void load8(const __bf16* p, float (&v)[8]) {
  const bhalf8_t h = *reinterpret_cast<const bhalf8_t*>(p);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = (float)h[i];
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const f32x4_t a = *reinterpret_cast<const f32x4_t*>(p), b = *reinterpret_cast<const f32x4_t*>(p + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = a[i];
    v[4 + i] = b[i];
  }
}
// Eight consecutive values rounded to the row's type.  STREAMED: past the caches.
template <bool STREAMED = false, typename V>
__device__ __forceinline__ void store_vector(V* p, V v) {
  if constexpr (STREAMED)
    __builtin_nontemporal_store(v, p);
  else
    *p = v;
}
template <bool STREAMED = false>
__device__ __forceinline__ void store8(_Float16* p, const float (&v)[8]) {
  half8_t h;
#pragma unroll
  for (int i = 0; i < 8; ++i) h[i] = (_Float16)v[i];
  store_vector<STREAMED>(reinterpret_cast<half8_t*>(p), h);
}
template <bool STREAMED = false>
__device__ __forceinline__ void store8(__bf16* p, const float (&v)[8]) {
  bhalf8_t h;
#pragma unroll
  for (int i = 0; i < 8; ++i) h[i] = (__bf16)v[i];
  store_vector<STREAMED>(reinterpret_cast<bhalf8_t*>(p), h);
}
template <bool STREAMED = false>
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  store_vector<STREAMED>(reinterpret_cast<f32x4_t*>(p), f32x4_t{v[0], v[1], v[2], v[3]});
  store_vector<STREAMED>(reinterpret_cast<f32x4_t*>(p) + 1, f32x4_t{v[4], v[5], v[6], v[7]});
}

// The largest |v| of eight values as its bit pattern (patterns of non-negative
// floats order as the floats do), infinities and NaN left out.  They are looked
// for once, over the wave, and `whole` says that it holds none.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }
__device__ __forceinline__ uint32_t max_finite(const float (&v)[8], bool& whole) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, abs_bits(v[i]));
  whole = !__any(m >= 0x7F800000u);
  if (!whole) {
    m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, abs_bits(v[i]) < 0x7F800000u ? abs_bits(v[i]) : 0u);
  }
  return m;
}

// The scale of a block whose largest finite |x| has the bits `amax`: the
// exponent field of 2^e, e = exponent - 8, one more where the fraction is above
// 448's (1.75 x 2^8).  At least 2^-126 (so that 1 / s is finite too), and 1 for
// a block of zeros.
__device__ __forceinline__ uint32_t scale_field(uint32_t amax) {
  if (amax == 0u) return 127u;
  const int f = (int)(amax >> 23) - 8 + ((amax & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return (uint32_t)(f < 1 ? 1 : f);
}
__device__ __forceinline__ float scale_of(uint32_t field) { return __uint_as_float(field << 23); }
__device__ __forceinline__ float inverse_scale_of(uint32_t field) { return __uint_as_float((254u - field) << 23); }

// Eight values times `inv` as e4m3 bytes.  Infinities become NaN (e4m3 has none).
__device__ __forceinline__ uint2 to_e4m3(const float (&v)[8], float inv, bool whole) {
  float s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) s[i] = v[i] * inv;
  if (!whole) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (__builtin_isinf(v[i])) s[i] = __builtin_nanf("");
  }
  uint2 q;
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(s[0], s[1], 0, false);
  q.x = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(s[2], s[3], w, true);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(s[4], s[5], 0, false);
  q.y = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(s[6], s[7], w, true);
  return q;
}

// Maximum over the aligned group of 16 lanes that holds one row's block.
__device__ __forceinline__ uint32_t max16(uint32_t v) {
  auto step = [&](int o) { v = (uint32_t)o > v ? (uint32_t)o : v; };
  step(__builtin_amdgcn_update_dpp((int)v, (int)v, 0xB1, 0xF, 0xF, false));    // quad_perm [1,0,3,2]
  step(__builtin_amdgcn_update_dpp((int)v, (int)v, 0x4E, 0xF, 0xF, false));    // quad_perm [2,3,0,1]
  step(__builtin_amdgcn_update_dpp((int)v, (int)v, 0x141, 0xF, 0xF, false));   // row_half_mirror
  step(__builtin_amdgcn_update_dpp((int)v, (int)v, 0x140, 0xF, 0xF, false));   // row_mirror
  return v;
}

__device__ __forceinline__ float wave_sum_f32(float v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

}  // namespace zinc
