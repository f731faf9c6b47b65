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

// Byte n of each of four words, in order.
template <int BYTE>
__device__ __forceinline__ uint32_t gather_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  // byte n of the second operand, then of the first; 0x0c gives zero
  constexpr uint32_t kPick = (4u + BYTE) << 8 | BYTE;
  return __builtin_amdgcn_perm(b, a, 0x0c0c0000u | kPick) | __builtin_amdgcn_perm(d, c, kPick << 16 | 0x0c0cu);
}

// Four values to four codes: int8 and fp8 in 32 bits, fp4 in the low 16.
template <int F>
__device__ __forceinline__ uint32_t encode4(const float (&v)[4], float inv) {
  if constexpr (F == SSM_CACHE_INT8) {
    return gather_bytes<0>(nearest_bits(v[0], inv), nearest_bits(v[1], inv), nearest_bits(v[2], inv),
                           nearest_bits(v[3], inv));
  } else if constexpr (F == SSM_CACHE_FP8) {
    const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] * inv, v[1] * inv, 0, false);
    return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(v[2] * inv, v[3] * inv, lo, true));
  } else {
    const uint32_t lo = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, v[0] * inv, v[1] * inv, 1.0f, 0);
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(lo, v[2] * inv, v[3] * inv, 1.0f, 1) & 0xffffu;
  }
}

// Four int8 codes to their values times unit.
__device__ __forceinline__ void decode4_int8(uint32_t codes, float unit, float (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = static_cast<float>(static_cast<int8_t>(codes >> (8 * i))) * unit;
}

template <int F>
__device__ __forceinline__ void decode4(uint32_t codes, float unit, float (&v)[4]) {
  if constexpr (F == SSM_CACHE_INT8) {
    decode4_int8(codes, unit, v);
  } else if constexpr (F == SSM_CACHE_FP8) {
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(codes), false);
    const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(codes), true);
    v[0] = lo[0] * unit; v[1] = lo[1] * unit; v[2] = hi[0] * unit; v[3] = hi[1] * unit;
  } else {
    const auto lo = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 0);
    const auto hi = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 1);
    v[0] = lo[0] * unit; v[1] = lo[1] * unit; v[2] = hi[0] * unit; v[3] = hi[1] * unit;
  }
}

// Philox-4x32 (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy
// as 1, 2, 3", 2011) with 7 rounds, the fewest that paper found to pass its
// tests: 16 random bytes for a counter and a 64-bit key.
__device__ __forceinline__ uint32_t xor3(uint32_t a, uint32_t b, uint32_t c) {
  return __builtin_amdgcn_bitop3_b32(a, b, c, 0x96);   // the truth table of a ^ b ^ c
}
__device__ __forceinline__ void philox7(uint32_t (&c)[4], uint64_t seed) {
  uint32_t k0 = static_cast<uint32_t>(seed), k1 = static_cast<uint32_t>(seed >> 32);
#pragma unroll
  for (int r = 0; r < 7; ++r) {
    const uint64_t p0 = static_cast<uint64_t>(0xD2511F53u) * c[0];
    const uint64_t p1 = static_cast<uint64_t>(0xCD9E8D57u) * c[2];
    c[0] = xor3(static_cast<uint32_t>(p1 >> 32), c[1], k0);
    c[1] = static_cast<uint32_t>(p1);
    c[2] = xor3(static_cast<uint32_t>(p0 >> 32), c[3], k1);
    c[3] = static_cast<uint32_t>(p0);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
}

}  // namespace ssm
