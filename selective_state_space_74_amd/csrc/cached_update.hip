// cached_update.hip -- the decode update of state_update.hip on states held in
// an int8 cache (state_cache.h): dequantise, step, read out, quantise again,
// with the state in registers in between.
//
// A lane has one channel and all its states: 16 codes are one 16-byte access,
// and a wavefront's are one run of 1 KB.  (The fp32 update spreads a channel
// over four lanes for the same reason.)  The readout and the block's maximum
// then need no exchange between lanes.  B and C, the same for every lane where
// the wavefront is inside one B/C group, come through scalar loads and are
// unpacked by scalar instructions.  (Several batch rows a thread, to load A once
// for them, measured 19.7 us with two and 21.5 with four against 20.0 at
// 256 x 5120 x 16; A's rows come from L2 anyway.)
//
// 256 x 5120 x 16 states move 55 MB a step, 9.3 us of memory time, where the
// fp32 update moves 179 MB; 327 vector instructions a wavefront, a fifth of them
// the generator's, are 11 us of issue.  A wavefront loads, computes and stores
// once, seven of them a SIMD: 19.1 us, 17.4 rounded to nearest.  With 32 states 36.4
// us (97 MB); with 64, four or two wavefronts a SIMD for a lane's 109 to 212
// registers, 87.6 (184 MB).
#include "slots.h"
#include "state_cache.h"

namespace ssm {
namespace {

constexpr int kThreads = 256;

struct CachedParams {
  uint8_t* codes; uint8_t* scales;
  const void* x; const void* dt; const void* z; const void* B; const void* C;
  const float* A; const float* D; const float* bias; void* out;
  const int32_t* slots; const int64_t* seed;
  int64_t cs, ss, xb, dtb, zb, Bb, Bg, Cb, Cg, Ad, ob, dim, cpg;
  int batch, nslots, N, softplus;
};

// Uniform values read through the scalar cache (the memory is not written by
// the kernel).
template <typename U>
using Uniform = const __attribute__((address_space(4))) U;

template <typename T>
__device__ __forceinline__ float uniform_value(const T* p, int i) {
  if constexpr (sizeof(T) == 4) {
    return reinterpret_cast<Uniform<float>*>(reinterpret_cast<uintptr_t>(p))[i];
  } else {
    const uint32_t w = reinterpret_cast<Uniform<uint32_t>*>(reinterpret_cast<uintptr_t>(p))[i / 2];
    return __uint_as_float(i % 2 ? w & 0xffff0000u : w << 16);
  }
}

// A value in a branch that is hardly ever taken: keeps the branch from being
// computed on every path (56 vector instructions of 327 a wavefront).
__device__ __forceinline__ float rarely(float v) {
  asm volatile("" : "+v"(v));
  return v;
}

// CH: 16-state chunks of a channel.  WIDTH: states of an access to the codes:
// 16 (N = 16 CH), 4 (N and every row a multiple of 4) or 1.  With 16 and 4 a
// wavefront is in one B/C group, whose rows come in 32-bit words.  SEEDED:
// stochastic rounding.
template <typename T, int CH, int WIDTH, bool SEEDED>
struct Channel {
  static constexpr int NS = 16 * CH, NB = (CH + 1) / 2;
  uint32_t q[4 * CH];   // codes
  uint32_t e[NB];       // scale bytes
  static constexpr bool kUniform = WIDTH > 1;
  // whether the channel has states from n on (uniform; always with whole chunks)
  __device__ static __forceinline__ bool has(const CachedParams& p, int n) { return WIDTH == 16 || n < p.N; }

  // the channel's row of A
  __device__ static __forceinline__ void load_a(const CachedParams& p, int64_t d, float (&a)[NS]) {
#pragma unroll
    for (int n = 0; n < NS; n += 4) {
      if constexpr (WIDTH > 1) {
        const float4 f = has(p, n) ? *reinterpret_cast<const float4*>(p.A + d * p.Ad + n) : make_float4(0, 0, 0, 0);
        a[n] = f.x; a[n + 1] = f.y; a[n + 2] = f.z; a[n + 3] = f.w;
      } else {
#pragma unroll
        for (int i = n; i < n + 4; ++i) a[i] = i < p.N ? p.A[d * p.Ad + i] : 0.0f;
      }
    }
  }

  __device__ __forceinline__ void load(const CachedParams& p, int64_t slot, int64_t d) {
    const uint8_t* const c = p.codes + slot * p.cs + d * p.N;
    const int nb = (p.N + kCacheBlock - 1) / kCacheBlock;
#pragma unroll
    for (int k = 0; k < NB; ++k) e[k] = p.scales[slot * p.ss + d * nb + k];
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      if constexpr (WIDTH == 16) {
        const uint4 w = reinterpret_cast<const uint4*>(c)[k];
        q[4 * k] = w.x; q[4 * k + 1] = w.y; q[4 * k + 2] = w.z; q[4 * k + 3] = w.w;
      } else if constexpr (WIDTH == 4) {
#pragma unroll
        for (int w = 4 * k; w < 4 * k + 4; ++w) q[w] = has(p, 4 * w) ? reinterpret_cast<const uint32_t*>(c)[w] : 0u;
      } else {
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          q[4 * k + w] = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (16 * k + 4 * w + i < p.N) q[4 * k + w] |= static_cast<uint32_t>(c[16 * k + 4 * w + i]) << (8 * i);
        }
      }
    }
  }

  __device__ __forceinline__ void store(const CachedParams& p, int64_t slot, int64_t d) const {
    uint8_t* const c = p.codes + slot * p.cs + d * p.N;
    const int nb = (p.N + kCacheBlock - 1) / kCacheBlock;
#pragma unroll
    for (int k = 0; k < NB; ++k) p.scales[slot * p.ss + d * nb + k] = static_cast<uint8_t>(e[k]);
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      if constexpr (WIDTH == 4) {
#pragma unroll
        for (int w = 4 * k; w < 4 * k + 4; ++w)
          if (has(p, 4 * w)) reinterpret_cast<uint32_t*>(c)[w] = q[w];
      } else if constexpr (WIDTH == 16) {
        reinterpret_cast<uint4*>(c)[k] = make_uint4(q[4 * k], q[4 * k + 1], q[4 * k + 2], q[4 * k + 3]);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (16 * k + i < p.N) c[16 * k + i] = static_cast<uint8_t>(q[4 * k + i / 4] >> (8 * (i % 4)));
      }
    }
  }

  // One step of row b (B/C group g) on the state in q, e; returns sum_n C s'.
  // (B and C are read here and not ahead of the slot: the scalar registers for
  // that cost more than the wait, 20.9 us against 19.3.)
  __device__ __forceinline__ float step(const CachedParams& p, int b, int64_t g, int64_t d, const float (&a)[NS], float dl,
                                        float x, uint64_t seed) {
    const T* const Bp = static_cast<const T*>(p.B) + b * p.Bb + g * p.Bg;
    const T* const Cp = static_cast<const T*>(p.C) + b * p.Cb + g * p.Cg;
    auto bc = [&](const T* v, int n) -> float {
      if constexpr (kUniform) return uniform_value(v, n);
      else return n < p.N ? io<T>::load(v + n) : 0.0f;
    };
    float h[NS];
    const float dlx = dl * x, dl2 = dl * kLog2e;
    float y = 0.0f;
#pragma unroll
    for (int k = 0; k < 4 * CH; ++k) {
      if (!has(p, 4 * k)) {
        h[4 * k] = h[4 * k + 1] = h[4 * k + 2] = h[4 * k + 3] = 0.0f;
        continue;
      }
      float s[4];
      decode4_int8(q[k], scale_value(e[k / 8]), s);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int n = 4 * k + i;
        h[n] = fmaf(__builtin_amdgcn_exp2f(dl2 * a[n]), s[i], dlx * bc(Bp, n));
        y = fmaf(bc(Cp, n), h[n], y);
      }
    }
    // Largest magnitudes.  fmax drops a NaN; but a state that is not finite
    // makes y so too, and then the magnitudes' bits are compared.
    const bool odd = __any(magnitude(y) >= 0x7f800000u);
#pragma unroll
    for (int k = 0; k < NB; ++k) {
      constexpr int kIn = NS < kCacheBlock ? NS : kCacheBlock;
      float m = 0.0f;
#pragma unroll
      for (int n = k * kCacheBlock; n < k * kCacheBlock + kIn && n < NS; ++n) m = fmaxf(m, fabsf(h[n]));
      uint32_t bits = __float_as_uint(m);
      if (odd) {
#pragma unroll
        for (int n = k * kCacheBlock; n < k * kCacheBlock + kIn && n < NS; ++n) bits = max(bits, magnitude(rarely(h[n])));
      }
      e[k] = scale_byte<SSM_CACHE_INT8>(bits);
    }
    // 256 2^(127 - E) is no fp32 number for E < 8 (states below 2^-112): scale in
    // two steps there
    bool tiny = false;
#pragma unroll
    for (int k = 0; k < NB; ++k) tiny |= e[k] < 8u;
    const bool two = SEEDED && __any(tiny);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      if (!has(p, 16 * c)) continue;
      const uint32_t eb = e[c / 2];
      const float inv = scale_inverse(eb);
      uint32_t t[16];
      if constexpr (SEEDED) {
        uint32_t r[4] = {static_cast<uint32_t>(d), static_cast<uint32_t>(b), static_cast<uint32_t>(c), 0u};
        philox7(r, seed);
        const float fine = 256.0f * inv;
#pragma unroll
        for (int i = 0; i < 16; ++i) t[i] = nearest_bits(h[16 * c + i], fine);
        if (two) {
#pragma unroll
          for (int i = 0; i < 16; ++i) t[i] = nearest_bits(rarely(h[16 * c + i]) * inv, 256.0f);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) t[i] += (r[i / 4] >> (8 * (i % 4))) & 0xffu;
#pragma unroll
        for (int w = 0; w < 4; ++w) q[4 * c + w] = gather_bytes<1>(t[4 * w], t[4 * w + 1], t[4 * w + 2], t[4 * w + 3]);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) t[i] = nearest_bits(h[16 * c + i], inv);
#pragma unroll
        for (int w = 0; w < 4; ++w) q[4 * c + w] = gather_bytes<0>(t[4 * w], t[4 * w + 1], t[4 * w + 2], t[4 * w + 3]);
      }
    }
    return y;
  }
};

template <typename T, int CH, int WIDTH, bool SEEDED>
__global__ __launch_bounds__(kThreads) void cached_update_kernel(CachedParams p) {
  const int lane = threadIdx.x & 63;
  const int64_t d0 = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t wave0 = static_cast<int64_t>(blockIdx.x) * kThreads + (threadIdx.x & ~63);
  if (wave0 >= p.dim) return;
  const bool live = d0 < p.dim;
  const int64_t d = live ? d0 : p.dim - 1;   // lanes past the channels repeat the last one, and store nothing
  const int row = blockIdx.y;
  using Ch = Channel<T, CH, WIDTH, SEEDED>;
  // the channel's B/C group, a scalar where the wavefront is in one
  int64_t g = 0;
  if (p.cpg != p.dim) {
    if constexpr (Ch::kUniform)
      g = __builtin_amdgcn_readfirstlane(static_cast<int>(static_cast<uint32_t>(wave0) / static_cast<uint32_t>(p.cpg)));
    else g = static_cast<uint32_t>(d) / static_cast<uint32_t>(p.cpg);
  }

  Ch ch;
  float a[Ch::NS], xv, dtv, zv;
  int slot = p.slots ? p.slots[row] : row;
  if (slot < 0 || slot >= p.nslots) slot = -1;
  const uint64_t seed = SEEDED ? static_cast<uint64_t>(*p.seed) : 0;
  auto inputs = [&](int b) {
    xv = io<T>::load(static_cast<const T*>(p.x) + b * p.xb + d);
    dtv = io<T>::load(static_cast<const T*>(p.dt) + b * p.dtb + d);
    zv = p.z ? io<T>::load(static_cast<const T*>(p.z) + b * p.zb + d) : 0.0f;
  };
  // what does not wait for the slot goes first
  inputs(row);
  Ch::load_a(p, d, a);
  const float bias = p.bias ? p.bias[d] : 0.0f, Dd = p.D ? p.D[d] : 0.0f;
  T* const out = static_cast<T*>(p.out) + d;
  if (slot >= 0) ch.load(p, slot, d);
  // the first row of a slot takes every row of it, in order
  bool before;
  int next;
  slot_order(p.slots, row, p.batch, slot, lane, before, next);
  if (slot < 0) {   // a padding row
    if (live) io<T>::store(out + row * p.ob, 0.0f);
    return;
  }
  if (before) return;

  for (int b = row;;) {
    float dl = dtv + bias;
    if (p.softplus) dl = softplus_close_f32(dl);
    float y = fmaf(Dd, xv, ch.step(p, b, g, d, a, dl, xv, seed));
    if (p.z) y *= silu_f32(zv);
    if (live) io<T>::store(out + b * p.ob, y);
    b = b == row ? next : named_next(p.slots, b, p.batch, slot, lane);
    if (b >= p.batch) break;
    inputs(b);
  }
  if (live) ch.store(p, slot, d);
}

template <typename T, int CH, int WIDTH>
void launch_w(const CachedParams& p, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>((p.dim + kThreads - 1) / kThreads), static_cast<unsigned>(p.batch));
  if (p.seed) cached_update_kernel<T, CH, WIDTH, true><<<grid, kThreads, 0, stream>>>(p);
  else cached_update_kernel<T, CH, WIDTH, false><<<grid, kThreads, 0, stream>>>(p);
}

template <typename T, int CH>
void launch_c(int width, const CachedParams& p, hipStream_t stream) {
  if (width == 16) launch_w<T, CH, 16>(p, stream);
  else if (width == 4) launch_w<T, CH, 4>(p, stream);
  else launch_w<T, CH, 1>(p, stream);
}

template <typename T>
void launch_t(int width, const CachedParams& p, hipStream_t stream) {
  switch ((p.N + 15) / 16) {
    case 1: launch_c<T, 1>(width, p, stream); break;
    case 2: launch_c<T, 2>(width, p, stream); break;
    case 3: launch_c<T, 3>(width, p, stream); break;
    default: launch_c<T, 4>(width, p, stream); break;
  }
}

}  // namespace

hipError_t launch_cached_update(const ssm_cached_update_args& a, hipStream_t stream) {
  const int64_t G = a.ngroups > 1 ? a.ngroups : 1;
  const CachedParams p{a.codes, a.scales, a.x, a.dt, a.z, a.B, a.C, a.A, a.D, a.dt_bias, a.out, a.slots, a.seed,
                       a.codes_slot_stride, a.scales_slot_stride, a.x_batch_stride, a.dt_batch_stride,
                       a.z_batch_stride, a.B_batch_stride, G > 1 ? a.B_group_stride : 0, a.C_batch_stride,
                       G > 1 ? a.C_group_stride : 0, a.A_dim_stride, a.out_batch_stride, a.dim, a.dim / G,
                       static_cast<int>(a.batch), static_cast<int>(a.nslots < 0x7fffffff ? a.nslots : 0x7fffffff),
                       static_cast<int>(a.dstate), a.dt_softplus ? 1 : 0};
  auto al = [](const void* q, int64_t bytes) { return reinterpret_cast<uintptr_t>(q) % static_cast<uintptr_t>(bytes) == 0; };
  const int64_t w = a.io_dtype == SSM_BF16 ? 2 : 1;   // elements of a 32-bit word
  const bool uniform = (G == 1 || p.cpg % 64 == 0) && al(a.B, 4) && al(a.C, 4) && p.Bb % w == 0 && p.Cb % w == 0 &&
                       p.Bg % w == 0 && p.Cg % w == 0;
  auto fits = [&](int64_t n) { return p.N % n == 0 && al(a.codes, n) && a.codes_slot_stride % n == 0; };
  const int width = !uniform || !al(a.A, 16) || a.A_dim_stride % 4 != 0 ? 1 : fits(16) ? 16 : fits(4) ? 4 : 1;
  if (a.io_dtype == SSM_BF16) launch_t<uint16_t>(width, p, stream);
  else launch_t<float>(width, p, stream);
  return hipGetLastError();
}

}  // namespace ssm
