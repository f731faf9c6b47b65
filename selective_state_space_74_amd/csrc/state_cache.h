// The quantised state cache's number formats (see ssm_cache_format): block
// scales and codes, shared by the cache's write and read and by the decode
// update that keeps its states there.
#pragma once

#include "ssm_internal.h"

namespace ssm {

constexpr int kCacheBlock = SSM_CACHE_BLOCK;

// A format's largest code value is (1 + kMant / 2^23) 2^kLead.
template <int F> struct CacheFormat;
template <> struct CacheFormat<SSM_CACHE_INT8> {
  static constexpr uint32_t kLead = 6, kMant = 0x7e0000;   // 127
};
template <> struct CacheFormat<SSM_CACHE_FP8> {
  static constexpr uint32_t kLead = 8, kMant = 0x600000;   // 448
};
template <> struct CacheFormat<SSM_CACHE_FP4> {
  static constexpr uint32_t kLead = 2, kMant = 0x400000;   // 6
};

// The magnitude bits of a float order like its magnitude, with infinity and
// then NaN above every finite value: an integer maximum loses no NaN.
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// The block's scale byte from its largest magnitude.  Where the exponent field
// is below kLead the scale is clamped to 2^-127, and the magnitude is below
// 2^(kLead - 127), so it is in range without the mantissa's comparison.
template <int F>
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
  const uint32_t field = amax >> 23;
  uint32_t e = 0;
  if (field >= CacheFormat<F>::kLead)
    e = field - CacheFormat<F>::kLead + ((amax & 0x7fffffu) > CacheFormat<F>::kMant ? 1u : 0u);
  return amax >= 0x7f800000u ? 255u : e;
}

// 2^(E - 127), NaN for 255.
__device__ __forceinline__ float scale_value(uint32_t e) {
  return __uint_as_float(e == 255u ? 0x7fc00000u : e == 0u ? 0x00400000u : e << 23);
}

// 2^(127 - E); 0 for 255 (the codes of such a block are of no account).
__device__ __forceinline__ float scale_inverse(uint32_t e) {
  return __uint_as_float(e == 255u ? 0u : (254u - e) << 23);
}

// Adding 1.5 * 2^23 leaves the nearest integer (ties to even) of a small
// product in the low bits, in one rounding: the product with a power of two is
// exact.
constexpr float kIntMagic = 12582912.0f;
__device__ __forceinline__ uint32_t nearest_bits(float v, float unit) {
  return __float_as_uint(fmaf(v, unit, kIntMagic));
}

// Two values to two codes: int8 and fp8 in the low two bytes, fp4 in the low
// byte.
template <int F>
__device__ __forceinline__ uint32_t encode2(float v0, float v1, float inv) {
  if constexpr (F == SSM_CACHE_INT8) {
    return (nearest_bits(v0, inv) & 0xffu) | ((nearest_bits(v1, inv) & 0xffu) << 8);
  } else if constexpr (F == SSM_CACHE_FP8) {
    return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(v0 * inv, v1 * inv, 0, false)) & 0xffffu;
  } else {
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, v0 * inv, v1 * inv, 1.0f, 0) & 0xffu;
  }
}

// The inverse: the values the codes stand for, unscaled.
template <int F>
__device__ __forceinline__ void decode2(uint32_t bits, float& v0, float& v1) {
  if constexpr (F == SSM_CACHE_INT8) {
    v0 = static_cast<float>(static_cast<int8_t>(bits & 0xffu));
    v1 = static_cast<float>(static_cast<int8_t>((bits >> 8) & 0xffu));
  } else if constexpr (F == SSM_CACHE_FP8) {
    const auto r = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(bits), false);
    v0 = r[0];
    v1 = r[1];
  } else {
    const auto r = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(bits, 1.0f, 0);
    v0 = r[0];
    v1 = r[1];
  }
}

// Philox-4x32 (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy
// as 1, 2, 3", 2011) with 7 rounds, the fewest that paper found to pass its
// tests: 16 random bytes for a counter and a 64-bit key.
__device__ __forceinline__ void philox7(uint32_t (&c)[4], uint64_t seed) {
  uint32_t k0 = static_cast<uint32_t>(seed), k1 = static_cast<uint32_t>(seed >> 32);
#pragma unroll
  for (int r = 0; r < 7; ++r) {
    const uint64_t p0 = static_cast<uint64_t>(0xD2511F53u) * c[0];
    const uint64_t p1 = static_cast<uint64_t>(0xCD9E8D57u) * c[2];
    c[0] = static_cast<uint32_t>(p1 >> 32) ^ c[1] ^ k0;
    c[1] = static_cast<uint32_t>(p1);
    c[2] = static_cast<uint32_t>(p0 >> 32) ^ c[3] ^ k1;
    c[3] = static_cast<uint32_t>(p0);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
}

}  // namespace ssm
