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

// What e4m3x8_quot takes for the N values of a lane whose row has scale s > 0: s and
// its reciprocal.  Where that would overflow (s below 2^-128) values and scale
// grow by 2^64 first, which is exact and leaves the quotients as they are.
struct Quot {
  float s, rcp;
};
template <int N>
__device__ __forceinline__ Quot e4m3_quot_of(float s, float (&v)[N][8]) {
  Quot q{s, 1.0f / s};
  if (q.rcp == __builtin_inff() && s > 0.0f) {
    asm volatile("");   // a branch that is hardly ever taken
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] *= 0x1p64f;
    q.s = s * 0x1p64f;
    q.rcp = 1.0f / q.s;
  }
  return q;
}

}  // namespace ocq
