// cached_update.hip -- the decode update of state_update.hip on states held in
// an int8 cache (state_cache.h): dequantise, step, read out, quantise again.
#include "state_cache.h"

namespace ssm {
namespace {

constexpr int kThreads = 64;

struct CachedParams {
  uint8_t* codes; uint8_t* scales;
  const void* x; const void* dt; const void* z; const void* B; const void* C;
  const float* A; const float* D; const float* bias; void* out;
  const int32_t* slots; const int64_t* seed;
  int64_t cs, ss, xb, dtb, zb, Bb, Bg, Cb, Cg, Ad, ob, batch, nslots, dim, cpg;
  int N, softplus;
};

// One thread a channel of a row.
template <typename T>
__global__ __launch_bounds__(kThreads) void cached_update_kernel(CachedParams p) {
  const int64_t d = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t b0 = blockIdx.y;
  if (d >= p.dim) return;
  const int64_t slot = p.slots ? p.slots[b0] : b0;
  if (slot < 0 || slot >= p.nslots) {
    io<T>::store(static_cast<T*>(p.out) + b0 * p.ob + d, 0.0f);
    return;
  }
  if (p.slots)   // the first row of a slot takes every row of it, in order
    for (int64_t i = 0; i < b0; ++i)
      if (p.slots[i] == slot) return;
  const int nblk = (p.N + kCacheBlock - 1) / kCacheBlock;
  uint8_t* codes = p.codes + slot * p.cs + d * p.N;
  uint8_t* scales = p.scales + slot * p.ss + d * nblk;
  const int64_t g = d / p.cpg;
  for (int64_t b = b0; b < p.batch; ++b) {
    if (b > b0) {
      if (!p.slots) break;
      if (p.slots[b] != slot) continue;
    }
    const float x = io<T>::load(static_cast<const T*>(p.x) + b * p.xb + d);
    float dl = io<T>::load(static_cast<const T*>(p.dt) + b * p.dtb + d) + (p.bias ? p.bias[d] : 0.0f);
    if (p.softplus) dl = softplus_f32(dl);
    float y = 0.0f;
    for (int k = 0; k < nblk; ++k) {
      const int n = min(kCacheBlock, p.N - k * kCacheBlock);
      const float unit = scale_value(scales[k]);
      float h[kCacheBlock];
      uint32_t amax = 0;
      for (int j = 0; j < n; ++j) {
        const int i = k * kCacheBlock + j;
        h[j] = static_cast<float>(static_cast<int8_t>(codes[i])) * unit;
        h[j] = fmaf(__builtin_amdgcn_exp2f(dl * (p.A[d * p.Ad + i] * kLog2e)), h[j],
                    dl * x * io<T>::load(static_cast<const T*>(p.B) + b * p.Bb + g * p.Bg + i));
        y = fmaf(io<T>::load(static_cast<const T*>(p.C) + b * p.Cb + g * p.Cg + i), h[j], y);
        amax = max(amax, magnitude(h[j]));
      }
      const uint32_t e = scale_byte<SSM_CACHE_INT8>(amax);
      const float inv = scale_inverse(e);
      scales[k] = static_cast<uint8_t>(e);
      uint32_t r[4];
      for (int j = 0; j < n; ++j) {
        const float v = e == 255u ? 0.0f : h[j];
        uint32_t q;
        if (p.seed) {
          if (j % 16 == 0) {
            r[0] = static_cast<uint32_t>(d); r[1] = static_cast<uint32_t>(b);
            r[2] = static_cast<uint32_t>(k * 2 + j / 16); r[3] = 0;
            philox7(r, static_cast<uint64_t>(*p.seed));
          }
          const uint32_t w = j % 16 < 4 ? r[0] : j % 16 < 8 ? r[1] : j % 16 < 12 ? r[2] : r[3];
          q = (nearest_bits(v * inv, 256.0f) + ((w >> (8 * (j & 3))) & 0xffu)) >> 8;
        } else {
          q = nearest_bits(v, inv);
        }
        codes[k * kCacheBlock + j] = static_cast<uint8_t>(q);
      }
    }
    y = fmaf(p.D ? p.D[d] : 0.0f, x, y);
    if (p.z) y *= silu_f32(io<T>::load(static_cast<const T*>(p.z) + b * p.zb + d));
    io<T>::store(static_cast<T*>(p.out) + b * p.ob + d, y);
  }
}

}  // namespace

hipError_t launch_cached_update(const ssm_cached_update_args& a, hipStream_t stream) {
  const int64_t G = a.ngroups > 1 ? a.ngroups : 1;
  CachedParams p{a.codes, a.scales, a.x, a.dt, a.z, a.B, a.C, a.A, a.D, a.dt_bias, a.out, a.slots, a.seed,
                 a.codes_slot_stride, a.scales_slot_stride, a.x_batch_stride, a.dt_batch_stride,
                 a.z_batch_stride, a.B_batch_stride, G > 1 ? a.B_group_stride : 0, a.C_batch_stride,
                 G > 1 ? a.C_group_stride : 0, a.A_dim_stride, a.out_batch_stride, a.batch, a.nslots,
                 a.dim, a.dim / G, static_cast<int>(a.dstate), a.dt_softplus ? 1 : 0};
  const dim3 grid(static_cast<unsigned>((a.dim + kThreads - 1) / kThreads), static_cast<unsigned>(a.batch));
  if (a.io_dtype == SSM_BF16) cached_update_kernel<uint16_t><<<grid, kThreads, 0, stream>>>(p);
  else cached_update_kernel<float><<<grid, kThreads, 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace ssm
