// Device-side pieces shared by the operators around the MLP block.
#pragma once
#include "kcommon.h"
#include "layer.h"

namespace ocq {

typedef float v2f __attribute__((ext_vector_type(2)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef int v2i __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {   // nearest even, NaN kept
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f{a, b}), v2bf));
}

__device__ __forceinline__ v4i pack8_bf16(const float* f) {
  return v4i{(int)pack_bf16(f[0], f[1]), (int)pack_bf16(f[2], f[3]), (int)pack_bf16(f[4], f[5]),
             (int)pack_bf16(f[6], f[7])};
}

__device__ __forceinline__ void unpack8_bf16(const v4i& u, float* f) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[2 * j] = __uint_as_float((uint32_t)u[j] << 16);
    f[2 * j + 1] = __uint_as_float((uint32_t)u[j] & 0xFFFF0000u);
  }
}

// The larger of m and |v|, NaN if either is one (fmaxf would skip it).
__device__ __forceinline__ float max_mag(float m, float v) { return __builtin_elementwise_maximum(m, fabsf(v)); }
// The scale of an E4M3 row whose largest magnitude is m; NaN (with codes 0) if one
// of its values is not finite, so that whoever reads the row sees it.
__device__ __forceinline__ float e4m3_scale(float m) { return m < __builtin_inff() ? m / 448.0f : __builtin_nanf(""); }

// What e4m3x8_quot takes for a row of scale s: s and its reciprocal (0 for a zero
// row), of the values times `up`.  up is 1 but for scales below 2^-126: from 2^-128
// down the reciprocal would overflow, so values and scale grow by 2^64 first,
// which is exact and leaves the quotients as they are.
struct Quot {
  float s, rcp, up;
};
__device__ __forceinline__ Quot e4m3_quot_of(float s) {
  const float up = s > 0.0f && s < 0x1p-126f ? 0x1p64f : 1.0f;
  return Quot{s * up, s > 0.0f ? 1.0f / (s * up) : 0.0f, up};
}

}  // namespace ocq
