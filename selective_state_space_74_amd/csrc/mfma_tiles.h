// Tiles of the matrix cores as the SSD kernels use them: operand fragments of
// 16-wide tiles, products, and sums over a wavefront.
#pragma once

#include <type_traits>

#include "ssm_internal.h"

namespace ssm {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef short v8s __attribute__((ext_vector_type(8)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef unsigned int v4u __attribute__((ext_vector_type(4)));
typedef unsigned int v2u __attribute__((ext_vector_type(2)));

// Storage of one IO element in LDS and its widening.
template <typename T> struct Lds;
template <> struct Lds<float> {
  using E = float;
  __device__ static __forceinline__ float f(E v) { return v; }
  __device__ static __forceinline__ E from(float v) { return v; }
};
template <> struct Lds<uint16_t> {
  using E = uint16_t;
  __device__ static __forceinline__ float f(E v) { return bf16_to_f32(v); }
  // round to nearest even in hardware (v_cvt_pk_bf16_f32)
  __device__ static __forceinline__ E from(float v) {
    return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
  }
};

// A lane's operand fragment of one 16x16 tile step over a 16-wide k block:
// four consecutive k values (k = 4 (l/16) + i) of its A row or B column, as
// the product instruction takes them (four bf16, or four fp32).
template <typename T> struct Frag;
template <> struct Frag<uint16_t> { using V = v4s; };
template <> struct Frag<float> { using V = v4f; };

// Sums of the bf16 k = 16 form, a type of their own: they must not go on from the
// k = 32 form's directly.  The compiler puts no wait between the two where the second
// reads the first's result as its sum, and the shorter one then takes part of it too
// early: with small integers 128 of 256 values were wrong right behind each other, none
// with 16 wait states between, nor the other way round or within one form, whichever
// registers hold the sums.
struct Sum16 {
  v4f v;
};
template <typename T> struct SumOf { using V = v4f; };
template <> struct SumOf<uint16_t> { using V = Sum16; };
__device__ __forceinline__ float value_of(const v4f& c, int i) { return c[i]; }
__device__ __forceinline__ float value_of(const Sum16& c, int i) { return c.v[i]; }

template <typename T>
__device__ __forceinline__ typename SumOf<T>::V mma16(typename Frag<T>::V a, typename Frag<T>::V b, typename SumOf<T>::V c) {
  if constexpr (sizeof(T) == 2) {
    return Sum16{__builtin_amdgcn_mfma_f32_16x16x16bf16_1k(a, b, c.v, 0, 0, 0)};
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i], b[i], c, 0, 0, 0);
    return c;
  }
}
// Sums made some other way, to go on with in mma16.
template <typename T>
__device__ __forceinline__ typename SumOf<T>::V go_on_16(v4f c) {
  if constexpr (sizeof(T) == 2) {
    asm volatile("s_nop 15" : "+v"(c));
    return Sum16{c};
  } else {
    return c;
  }
}

// bf16, k = 32 (v_mfma_f32_16x16x32_bf16, twice the work of the k = 16 form
// at the same issue rate on gfx950).  The instruction sums over its 32 k
// slots, pairing slot v of A's lane 16 g + i with slot v of B's lane
// 16 g + j, so any placement of the k values into (lane group, slot) that A
// and B share gives the same sum: two k = 16 fragments side by side (slots
// 0-3 and 4-7) give the sum of their two k = 16 products, and eight
// consecutive k values per lane (slots 0-7 of lane group g holding k = 8 g
// .. 8 g + 7) one 32-wide k block.
__device__ __forceinline__ v4f mma32(v8s a, v8s b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b),
                                                 c, 0, 0, 0);
}
__device__ __forceinline__ v4f mma32(v4s a0, v4s a1, v4s b0, v4s b1, v4f c) {
  return mma32(__builtin_shufflevector(a0, a1, 0, 1, 2, 3, 4, 5, 6, 7),
               __builtin_shufflevector(b0, b1, 0, 1, 2, 3, 4, 5, 6, 7), c);
}

// One form's sums are not the other's argument.
static_assert(!std::is_convertible_v<v4f, Sum16> && !std::is_convertible_v<Sum16, v4f>);

// Four consecutive LDS elements (8 or 16 bytes, aligned) as a fragment.
template <typename T>
__device__ __forceinline__ typename Frag<T>::V ldsf(const typename Lds<T>::E* p) {
  return *reinterpret_cast<const typename Frag<T>::V*>(p);
}

// bf16 operand fragment through the LDS transpose read (ds_read_b64_tr_b16).
// Within each group of 16 lanes, lane i receives element k from the chunk
// (four consecutive elements) that lane 4k + i / 4 of the group addresses,
// its element i % 4 (lane layout checked on the device with an in-bounds
// probe).  So when lane r of group g addresses row 4g + r / 4, columns
// 4 (r % 4) .. + 3 of a row-major tile X[k][c], lane 16 g + i receives
// X[4g + k][i] for k = 0..3: the operand fragment of column i (k = 4g + k')
// of a 16x16x16 product, equally the A fragment of row i of X^T.
__device__ __forceinline__ v4s lds_tr(const uint16_t* row_chunk) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (v4s __attribute__((address_space(3)))*)(row_chunk));
}

// Two fp32 values rounded to bf16 (nearest even) in one word, a low.
__device__ __forceinline__ uint32_t pack_bf16x2(float a, float b) {
  typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
  const bf2 v = {static_cast<__bf16>(a), static_cast<__bf16>(b)};
  return __builtin_bit_cast(uint32_t, v);
}

// Four LDS elements (already in the fragment's element type) as a fragment.
template <typename T>
__device__ __forceinline__ typename Frag<T>::V tofrag_bits(typename Lds<T>::E a, typename Lds<T>::E b,
                                                           typename Lds<T>::E c, typename Lds<T>::E d) {
  if constexpr (sizeof(T) == 2) {
    v4s v;
    v[0] = static_cast<short>(a); v[1] = static_cast<short>(b);
    v[2] = static_cast<short>(c); v[3] = static_cast<short>(d);
    return v;
  } else {
    return v4f{a, b, c, d};
  }
}

// Four fp32 values as a fragment (rounded to bf16 for bf16 IO).
template <typename T>
__device__ __forceinline__ typename Frag<T>::V tofrag(float a, float b, float c, float d) {
  if constexpr (sizeof(T) == 2) {
    v4s v;
    v[0] = __builtin_bit_cast(short, static_cast<__bf16>(a));
    v[1] = __builtin_bit_cast(short, static_cast<__bf16>(b));
    v[2] = __builtin_bit_cast(short, static_cast<__bf16>(c));
    v[3] = __builtin_bit_cast(short, static_cast<__bf16>(d));
    return v;
  } else {
    return v4f{a, b, c, d};
  }
}

// One DPP step on a float: lanes outside the row and bank masks, and lanes
// whose source lies outside their row, read 0.
template <int kCtrl, int kRowMask = 0xf>
__device__ __forceinline__ float dpp0(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), kCtrl, kRowMask, 0xf, true));
}

// Inclusive prefix sums over each 16 lanes: row shifts by 1, 2, 4 and 8.
__device__ __forceinline__ float row_prefix_sum(float v) {
  v += dpp0<0x111>(v);         // row_shr:1
  v += dpp0<0x112>(v);         // row_shr:2
  v += dpp0<0x114>(v);         // row_shr:4
  return v + dpp0<0x118>(v);   // row_shr:8
}

// The same from each 16 lanes' end: row shifts the other way.
__device__ __forceinline__ float row_suffix_sum(float v) {
  v += dpp0<0x101>(v);         // row_shl:1
  v += dpp0<0x102>(v);         // row_shl:2
  v += dpp0<0x104>(v);         // row_shl:4
  return v + dpp0<0x108>(v);   // row_shl:8
}

// Inclusive prefix sum over the 64 lanes of a wavefront in registers: each
// 16-lane row, then row_bcast:15 adds row 0's total to row 1 and row 2's to
// row 3, and row_bcast:31 adds lane 31's (rows 0 and 1) to rows 2 and 3.
__device__ __forceinline__ float wave_prefix_sum(float v) {
  v = row_prefix_sum(v);
  v += dpp0<0x142, 0xa>(v);    // row_bcast:15 into rows 1 and 3
  v += dpp0<0x143, 0xc>(v);    // row_bcast:31 into rows 2 and 3
  return v;
}

// Sums over the lanes up to each, in 64 bits.
template <int kCtrl, int kRows = 0xf>
__device__ __forceinline__ double dpp0(double v) {
  const v2u w = __builtin_bit_cast(v2u, v);
  return __builtin_bit_cast(double, v2u{static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(w[0]), kCtrl, kRows, 0xf, true)),
                                        static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(w[1]), kCtrl, kRows, 0xf, true))});
}
__device__ __forceinline__ double wave_prefix_sum64(double v) {
  v += dpp0<0x111>(v);
  v += dpp0<0x112>(v);
  v += dpp0<0x114>(v);
  v += dpp0<0x118>(v);
  v += dpp0<0x142, 0xa>(v);
  v += dpp0<0x143, 0xc>(v);
  return v;
}
__device__ __forceinline__ double lane_value(double v, int lane) {
  const v2u w = __builtin_bit_cast(v2u, v);
  return __builtin_bit_cast(double, v2u{static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(w[0]), lane)),
                                        static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(w[1]), lane))});
}

// A sum of steps as it is kept in LDS, a float and what its rounding leaves: the
// difference of two is then rounded once, and the sums' own sizes do not matter.
struct TwoFloats {
  float v, rest;
};
__device__ __forceinline__ TwoFloats two_floats(double v) {
  const float f = static_cast<float>(v);
  return TwoFloats{f, static_cast<float>(v - f)};
}
__device__ __forceinline__ float decay_between(float to, float to_rest, const TwoFloats& from) {
  return __builtin_amdgcn_exp2f((to - from.v) + (to_rest - from.rest));
}

// The decay between two sums of steps times their rate, in units of log 2.
__device__ __forceinline__ float decay_of(double difference) { return __builtin_amdgcn_exp2f(static_cast<float>(difference)); }

}  // namespace ssm
