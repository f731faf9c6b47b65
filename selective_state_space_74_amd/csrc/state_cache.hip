// state_cache.hip -- writing recurrent states to a quantised cache and reading
// them back, for gfx950.  Formats: state_cache.h.
//
// Both move 4 bytes (fp32) against 1 or 1/2 a value, and a scale byte a block.  A lane takes 4 consecutive values of a block, so
// that the lanes of a block (8 for 32 values, fewer for shorter rows) read or
// write 16 bytes each in one run, and the block's maximum is two or three DPP
// steps.  Which row of the batch a workgroup has comes from the grid; only the
// row's place in the cache waits for its slot.  64 x 5120 x 16 fp32 states to
// int8: 7.7 us written and 6.5 us read (27 MB, 3.4 and 4.1 TB/s); 24 x 2048 x 128
// to e2m1 8.6 and 7.8 us.  About 2.6 us of each are the way from the slot to the
// values, there with next to no data too; the rest is memory traffic: 256 x 5120 x
// 16 to int8 take 22.9 and 17.3 us (106 MB, 4.6 and 6.1 TB/s).
#include "state_cache.h"

namespace ssm {
namespace {

constexpr int kThreads = 256;

struct CacheParams {
  uint8_t* codes; uint8_t* scales; void* states; const int32_t* slots;
  int64_t cs, ss, vs;
  int batch, nslots;
  uint32_t inner, nblk, blocks;   // blocks: of one state
  int lane_bits;                  // log2 of the lanes of a block
};

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), CTRL, 0xf, 0xf, true));
}
// The maximum over groups of 2^bits lanes.
__device__ __forceinline__ uint32_t group_max(uint32_t v, int bits) {
  // quads: lanes (1,0,3,2), then (2,3,0,1); then each half row of 8, mirrored
  if (bits > 0) v = max(v, dpp<0xB1>(v));
  if (bits > 1) v = max(v, dpp<0x4E>(v));
  if (bits > 2) v = max(v, dpp<0x141>(v));
  return v;
}

// Where a lane's 4 values are: the block's number in the state, the values'
// offset in the state, and how many of the 4 there are.
struct Place {
  uint32_t block;
  int64_t at;
  int count;
};
__device__ __forceinline__ Place place(const CacheParams& p, uint32_t thread) {
  Place r;
  r.block = thread >> p.lane_bits;
  const uint32_t first = (thread & ((1u << p.lane_bits) - 1)) * 4;
  const uint32_t o = p.nblk == 1 ? r.block : r.block / p.nblk, k = r.block - o * p.nblk;
  const uint32_t in_row = k * kCacheBlock + first;
  r.at = static_cast<int64_t>(o) * p.inner + in_row;
  const uint32_t end = min(p.inner, (k + 1) * kCacheBlock);
  r.count = r.block < p.blocks && in_row < end ? static_cast<int>(min(4u, end - in_row)) : 0;
  return r;
}

template <typename T, bool VEC>
__device__ __forceinline__ void load4(const T* q, int count, float (&v)[4]) {
  if constexpr (VEC) {
    v[0] = v[1] = v[2] = v[3] = 0.0f;
    if (count) {
      if constexpr (sizeof(T) == 4) {
        const float4 f = *reinterpret_cast<const float4*>(q);
        v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
      } else {
        const uint2 f = *reinterpret_cast<const uint2*>(q);
        v[0] = __uint_as_float(f.x << 16); v[1] = __uint_as_float(f.x & 0xffff0000u);
        v[2] = __uint_as_float(f.y << 16); v[3] = __uint_as_float(f.y & 0xffff0000u);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = i < count ? io<T>::load(q + i) : 0.0f;
  }
}

// VEC: rows of a multiple of 4 values, all of them aligned for accesses of 4.
template <int F, typename T, bool VEC>
__global__ __launch_bounds__(kThreads) void cache_write_kernel(CacheParams p) {
  const int b = blockIdx.y;
  const Place w = place(p, blockIdx.x * kThreads + threadIdx.x);
  float v[4];
  load4<T, VEC>(static_cast<const T*>(p.states) + b * p.vs + w.at, w.count, v);
  const int slot = p.slots ? p.slots[b] : b;
  if (p.slots) {
    // the last row of a slot is the one written
    bool later = false;
    for (int j = b + 1 + (threadIdx.x & 63); j < p.batch; j += 64) later |= p.slots[j] == slot;
    if (__any(later) || slot < 0 || slot >= p.nslots) return;
  }
  const uint32_t amax = group_max(max(max(magnitude(v[0]), magnitude(v[1])), max(magnitude(v[2]), magnitude(v[3]))), p.lane_bits);
  const uint32_t e = scale_byte<F>(amax);
  const uint32_t q = encode4<F>(v, scale_inverse(e));
  if (w.count == 0) return;
  if ((threadIdx.x & ((1u << p.lane_bits) - 1)) == 0) p.scales[slot * p.ss + w.block] = static_cast<uint8_t>(e);
  if constexpr (F == SSM_CACHE_FP4) {
    uint8_t* const c = p.codes + slot * p.cs + w.at / 2;
    if constexpr (VEC) {
      *reinterpret_cast<uint16_t*>(c) = static_cast<uint16_t>(q);
    } else {
      c[0] = static_cast<uint8_t>(q);
      if (w.count > 2) c[1] = static_cast<uint8_t>(q >> 8);
    }
  } else {
    uint8_t* const c = p.codes + slot * p.cs + w.at;
    if constexpr (VEC) {
      *reinterpret_cast<uint32_t*>(c) = q;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < w.count) c[i] = static_cast<uint8_t>(q >> (8 * i));
    }
  }
}

template <int F, typename T, bool VEC>
__global__ __launch_bounds__(kThreads) void cache_read_kernel(CacheParams p) {
  const int b = blockIdx.y;
  const Place w = place(p, blockIdx.x * kThreads + threadIdx.x);
  if (w.count == 0) return;
  const int slot = p.slots ? p.slots[b] : b;
  float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (slot >= 0 && slot < p.nslots) {
    const float unit = scale_value(p.scales[slot * p.ss + w.block]);
    uint32_t q = 0;
    if constexpr (F == SSM_CACHE_FP4) {
      const uint8_t* const c = p.codes + slot * p.cs + w.at / 2;
      if constexpr (VEC) q = *reinterpret_cast<const uint16_t*>(c);
      else q = c[0] | (w.count > 2 ? c[1] << 8 : 0);
    } else {
      const uint8_t* const c = p.codes + slot * p.cs + w.at;
      if constexpr (VEC) {
        q = *reinterpret_cast<const uint32_t*>(c);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i < w.count) q |= static_cast<uint32_t>(c[i]) << (8 * i);
      }
    }
    decode4<F>(q, unit, v);
  }
  T* const out = static_cast<T*>(p.states) + b * p.vs + w.at;
  if constexpr (VEC) {
    if constexpr (sizeof(T) == 4) {
      *reinterpret_cast<float4*>(out) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
      *reinterpret_cast<uint2*>(out) = make_uint2(f32_to_bf16(v[0]) | static_cast<uint32_t>(f32_to_bf16(v[1])) << 16,
                                                  f32_to_bf16(v[2]) | static_cast<uint32_t>(f32_to_bf16(v[3])) << 16);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < w.count) io<T>::store(out + i, v[i]);
  }
}

template <int F, typename T, bool VEC>
void launch_v(bool write, dim3 grid, const CacheParams& p, hipStream_t stream) {
  if (write) cache_write_kernel<F, T, VEC><<<grid, kThreads, 0, stream>>>(p);
  else cache_read_kernel<F, T, VEC><<<grid, kThreads, 0, stream>>>(p);
}

template <int F, typename T>
hipError_t launch(bool write, const ssm_state_cache_args& a, hipStream_t stream) {
  CacheParams p{a.codes, a.scales, a.states, a.slots, a.codes_slot_stride, a.scales_slot_stride, a.states_batch_stride,
                static_cast<int>(a.batch), static_cast<int>(a.nslots < 0x7fffffff ? a.nslots : 0x7fffffff),
                static_cast<uint32_t>(a.inner), static_cast<uint32_t>((a.inner + kCacheBlock - 1) / kCacheBlock), 0, 0};
  p.blocks = static_cast<uint32_t>(a.outer * p.nblk);
  while (p.lane_bits < 3 && (4u << p.lane_bits) < p.inner) ++p.lane_bits;
  auto fits = [](const void* q, int64_t stride, int64_t bytes) {
    return reinterpret_cast<uintptr_t>(q) % static_cast<uintptr_t>(bytes) == 0 && stride % bytes == 0;
  };
  const int64_t esz = sizeof(T), held = F == SSM_CACHE_FP4 ? 2 : 4;
  const bool vec = a.inner % 4 == 0 && fits(a.states, a.states_batch_stride * esz, 4 * esz) &&
                   fits(a.codes, a.codes_slot_stride, held);
  const dim3 grid(static_cast<unsigned>(((static_cast<int64_t>(p.blocks) << p.lane_bits) + kThreads - 1) / kThreads),
                  static_cast<unsigned>(a.batch));
  if (vec) launch_v<F, T, true>(write, grid, p, stream);
  else launch_v<F, T, false>(write, grid, p, stream);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_format(bool write, const ssm_state_cache_args& a, hipStream_t stream) {
  switch (a.format) {
    case SSM_CACHE_INT8: return launch<SSM_CACHE_INT8, T>(write, a, stream);
    case SSM_CACHE_FP8: return launch<SSM_CACHE_FP8, T>(write, a, stream);
    default: return launch<SSM_CACHE_FP4, T>(write, a, stream);
  }
}

}  // namespace

hipError_t launch_cache_write(const ssm_state_cache_args& a, hipStream_t stream) {
  return a.io_dtype == SSM_BF16 ? launch_format<uint16_t>(true, a, stream) : launch_format<float>(true, a, stream);
}

hipError_t launch_cache_read(const ssm_state_cache_args& a, hipStream_t stream) {
  return a.io_dtype == SSM_BF16 ? launch_format<uint16_t>(false, a, stream) : launch_format<float>(false, a, stream);
}

}  // namespace ssm
