// state_cache.hip -- writing recurrent states to a quantised cache and reading
// them back, for gfx950.  Formats: state_cache.h.
#include "state_cache.h"

namespace ssm {
namespace {

constexpr int kThreads = 256;

struct CacheParams {
  uint8_t* codes; uint8_t* scales; void* states; const int32_t* slots;
  int64_t cs, ss, vs, batch, nslots, outer, inner, nblk;
};

// One thread a block of 32 values.
template <int F, typename T>
__global__ __launch_bounds__(kThreads) void cache_write_kernel(CacheParams p) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= p.outer * p.nblk) return;
  const int64_t b = blockIdx.y, o = i / p.nblk, k = i % p.nblk;
  const int64_t slot = p.slots ? p.slots[b] : b;
  if (slot < 0 || slot >= p.nslots) return;
  if (p.slots)   // the last row of a slot is the one written
    for (int64_t j = b + 1; j < p.batch; ++j)
      if (p.slots[j] == slot) return;
  const int n = static_cast<int>(min(static_cast<int64_t>(kCacheBlock), p.inner - k * kCacheBlock));
  const T* v = static_cast<const T*>(p.states) + b * p.vs + o * p.inner + k * kCacheBlock;
  uint32_t amax = 0;
  for (int j = 0; j < n; ++j) amax = max(amax, magnitude(io<T>::load(v + j)));
  const uint32_t e = scale_byte<F>(amax);
  const float inv = scale_inverse(e);
  p.scales[slot * p.ss + i] = static_cast<uint8_t>(e);
  const bool nan = e == 255u;
  for (int j = 0; j < n; j += 2) {
    const float v0 = nan ? 0.0f : io<T>::load(v + j), v1 = nan || j + 1 >= n ? 0.0f : io<T>::load(v + j + 1);
    const uint32_t q = encode2<F>(v0, v1, inv);
    if constexpr (F == SSM_CACHE_FP4) {
      p.codes[slot * p.cs + (o * p.inner + k * kCacheBlock + j) / 2] = static_cast<uint8_t>(q);
    } else {
      uint8_t* c = p.codes + slot * p.cs + o * p.inner + k * kCacheBlock + j;
      c[0] = static_cast<uint8_t>(q);
      if (j + 1 < n) c[1] = static_cast<uint8_t>(q >> 8);
    }
  }
}

template <int F, typename T>
__global__ __launch_bounds__(kThreads) void cache_read_kernel(CacheParams p) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= p.outer * p.nblk) return;
  const int64_t b = blockIdx.y, o = i / p.nblk, k = i % p.nblk;
  const int64_t slot = p.slots ? p.slots[b] : b;
  const bool held = slot >= 0 && slot < p.nslots;
  const int n = static_cast<int>(min(static_cast<int64_t>(kCacheBlock), p.inner - k * kCacheBlock));
  T* v = static_cast<T*>(p.states) + b * p.vs + o * p.inner + k * kCacheBlock;
  const float unit = held ? scale_value(p.scales[slot * p.ss + i]) : 0.0f;
  for (int j = 0; j < n; j += 2) {
    float v0 = 0.0f, v1 = 0.0f;
    if (held) {
      if constexpr (F == SSM_CACHE_FP4) {
        decode2<F>(p.codes[slot * p.cs + (o * p.inner + k * kCacheBlock + j) / 2], v0, v1);
      } else {
        const uint8_t* c = p.codes + slot * p.cs + o * p.inner + k * kCacheBlock + j;
        decode2<F>(c[0] | (j + 1 < n ? c[1] << 8 : 0), v0, v1);
      }
    }
    io<T>::store(v + j, v0 * unit);
    if (j + 1 < n) io<T>::store(v + j + 1, v1 * unit);
  }
}

CacheParams params(const ssm_state_cache_args& a) {
  return CacheParams{a.codes, a.scales, a.states, a.slots, a.codes_slot_stride, a.scales_slot_stride,
                     a.states_batch_stride, a.batch, a.nslots, a.outer, a.inner,
                     (a.inner + kCacheBlock - 1) / kCacheBlock};
}

template <int F, typename T>
void launch(bool write, const CacheParams& p, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>((p.outer * p.nblk + kThreads - 1) / kThreads),
                  static_cast<unsigned>(p.batch));
  if (write) cache_write_kernel<F, T><<<grid, kThreads, 0, stream>>>(p);
  else cache_read_kernel<F, T><<<grid, kThreads, 0, stream>>>(p);
}

template <typename T>
hipError_t launch_format(bool write, const ssm_state_cache_args& a, hipStream_t stream) {
  switch (a.format) {
    case SSM_CACHE_INT8: launch<SSM_CACHE_INT8, T>(write, params(a), stream); break;
    case SSM_CACHE_FP8: launch<SSM_CACHE_FP8, T>(write, params(a), stream); break;
    default: launch<SSM_CACHE_FP4, T>(write, params(a), stream); break;
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_cache_write(const ssm_state_cache_args& a, hipStream_t stream) {
  return a.io_dtype == SSM_BF16 ? launch_format<uint16_t>(true, a, stream) : launch_format<float>(true, a, stream);
}

hipError_t launch_cache_read(const ssm_state_cache_args& a, hipStream_t stream) {
  return a.io_dtype == SSM_BF16 ? launch_format<uint16_t>(false, a, stream) : launch_format<float>(false, a, stream);
}

}  // namespace ssm
