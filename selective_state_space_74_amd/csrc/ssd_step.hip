// ssd_step.hip -- the single-token step of the Mamba-2 SSM (SSD layer), gfx950.
//
// Per batch row b, head h, head channel p and state n, on the fp32 state of the
// row's slot:
//   Delta = softplus(dt[b,h] + bias[h])
//   S[p,n] = exp(Delta A[h]) S[p,n] + Delta x[b,h,p] B[b,g,n]     (in place)
//   out = (sum_n C[b,g,n] S[p,n] + D[h] x) silu(z)
//
// Bound by memory: a state is read and written once, 8 bytes a value, for six
// operations.  LPR lanes share a row of N states in pieces of 4 (16 bytes): 8 lanes
// cover 128 bytes, a cache line, and a wavefront 8 rows of a head at a time, so
// every access is made of whole lines.  A wavefront stays with one head, whose
// decay and whose B and C it keeps in registers, for up to kMostSets such sets of
// rows, the next set's loads in flight while one is computed.  256 x 80 x 64 x 128
// bf16: 270 us, 5.0 TB/s, a large copy's rate.
#include "ssm_internal.h"
#include "slots.h"

namespace ssm {
namespace {

constexpr int kWaves = 4;
constexpr int kMostSets = 8;

struct StepParams {
  float* state;
  const void* x;
  const void* dt;
  const void* z;
  const void* B;
  const void* C;
  const float* A;
  const float* D;
  const float* bias;
  const int32_t* slots;
  void* out;
  int64_t ss, xb, xh, db, zb, zh, Bb, Bg, Cb, Cg, ob, oh;
  int H, P, N, per_group, batch, nslots, softplus;
  int sets, parts;   // sets of rows of a wavefront, wavefronts of a head
};

// Four consecutive values, those from `left` on zero; kVec: all there, one access.
template <typename T, bool kVec>
__device__ __forceinline__ void load4(const T* p, int left, float (&v)[4]) {
  struct alignas(4 * sizeof(T)) Pack { T e[4]; };
  if constexpr (kVec) {
    if (left <= 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = 0.0f;
      return;
    }
    const Pack q = *reinterpret_cast<const Pack*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = io<T>::load(&q.e[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = i < left ? io<T>::load(p + i) : 0.0f;
  }
}
template <bool kVec>
__device__ __forceinline__ void store4(float* p, int left, const float (&v)[4]) {
  if constexpr (kVec) {
    if (left > 0) *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < left) p[i] = v[i];
  }
}

template <int kCtrl>
__device__ __forceinline__ float moved(float v) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), kCtrl, 0xf, 0xf, true));
}
// Sum over the 4 or 8 lanes of a row: quad permutations, then the half rows mirrored.
template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
  v += moved<0xB1>(v);
  v += moved<0x4E>(v);
  if constexpr (LPR == 8) v += moved<0x141>(v);
  return v;
}

template <typename T, int LPR, int NV, bool kVec>
__global__ __launch_bounds__(64 * kWaves) void ssd_step_kernel(StepParams p) {
  constexpr int kRows = 64 / LPR;
  const int lane = threadIdx.x & 63;
  const int task = blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (task >= p.H * p.parts) return;
  const int h = task / p.parts, part = task - h * p.parts, g = h / p.per_group;
  const int row = blockIdx.y;
  int slot = p.slots ? p.slots[row] : row;
  if (slot < 0 || slot >= p.nslots) slot = -1;
  bool before;
  int next;
  slot_order(p.slots, row, p.batch, slot, lane, before, next);
  if (before && slot >= 0) return;
  const int j = lane % LPR;
  const int first = part * p.sets * kRows + lane / LPR;
  const int end = min(p.P, (part + 1) * p.sets * kRows);
  const float A = p.A[h], Dh = p.D ? p.D[h] : 0.0f, bias = p.bias ? p.bias[h] : 0.0f;
  float* const st = p.state + max(slot, 0) * p.ss + static_cast<int64_t>(h) * p.P * p.N + 4 * j;
  const int left = p.N - 4 * j;   // states from this lane's first on

  for (int b = row;;) {
    T* const out = static_cast<T*>(p.out) + b * p.ob + h * p.oh;
    if (slot < 0) {
      for (int r = first; r < end; r += kRows)
        if (j == 0) io<T>::store(out + r, 0.0f);
      return;
    }
    const T* const x = static_cast<const T*>(p.x) + b * p.xb + h * p.xh;
    const T* const z = p.z ? static_cast<const T*>(p.z) + b * p.zb + h * p.zh : nullptr;
    float s[NV][4], bv[NV][4], cv[NV][4];
    auto load_state = [&](int r, float (&v)[NV][4]) {
      if (r >= end) return;
#pragma unroll
      for (int k = 0; k < NV; ++k)
        load4<float, kVec>(st + static_cast<int64_t>(r) * p.N + 4 * LPR * k, left - 4 * LPR * k, v[k]);
    };
    load_state(first, s);
    float xr = first < end ? io<T>::load(x + first) : 0.0f;
    float zr = z && first < end ? io<T>::load(z + first) : 0.0f;
    float delta = io<T>::load(static_cast<const T*>(p.dt) + b * p.db + h) + bias;
    if (p.softplus) delta = softplus_close_f32(delta);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      load4<T, kVec>(static_cast<const T*>(p.B) + b * p.Bb + g * p.Bg + 4 * j + 4 * LPR * k, left - 4 * LPR * k, bv[k]);
      load4<T, kVec>(static_cast<const T*>(p.C) + b * p.Cb + g * p.Cg + 4 * j + 4 * LPR * k, left - 4 * LPR * k, cv[k]);
    }
    const float decay = __builtin_amdgcn_exp2f(delta * A * kLog2e);
    for (int r = first; r < end; r += kRows) {
      float s1[NV][4], x1 = 0.0f, z1 = 0.0f;
      load_state(r + kRows, s1);
      if (r + kRows < end) {
        x1 = io<T>::load(x + r + kRows);
        if (z) z1 = io<T>::load(z + r + kRows);
      }
      const float in = delta * xr;
      float y = 0.0f;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[k][i] = fmaf(decay, s[k][i], in * bv[k][i]);
          y = fmaf(cv[k][i], s[k][i], y);
        }
        store4<kVec>(st + static_cast<int64_t>(r) * p.N + 4 * LPR * k, left - 4 * LPR * k, s[k]);
      }
      y = fmaf(Dh, xr, row_sum<LPR>(y));
      if (z) y *= silu_f32(zr);
      if (j == 0) io<T>::store(out + r, y);
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[k][i] = s1[k][i];
      xr = x1;
      zr = z1;
    }
    b = b == row ? next : named_next(p.slots, b, p.batch, slot, lane);
    if (b >= p.batch) return;
  }
}

template <typename T, int LPR, int NV>
void launch(StepParams p, bool vec, hipStream_t stream) {
  // as many sets of rows a wavefront as leave 4096 wavefronts (16 a compute unit)
  const int sets = (p.P + 64 / LPR - 1) / (64 / LPR);
  p.sets = std::min(sets, kMostSets);
  while (p.sets > 1 && static_cast<int64_t>(p.batch) * p.H * ((sets + p.sets - 1) / p.sets) < 4096) p.sets = (p.sets + 1) / 2;
  p.parts = (sets + p.sets - 1) / p.sets;
  const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(p.H) * p.parts + kWaves - 1) / kWaves),
                  static_cast<unsigned>(p.batch));
  if (vec) ssd_step_kernel<T, LPR, NV, true><<<grid, 64 * kWaves, 0, stream>>>(p);
  else ssd_step_kernel<T, LPR, NV, false><<<grid, 64 * kWaves, 0, stream>>>(p);
}

template <typename T>
void launch_for(const StepParams& p, bool vec, hipStream_t stream) {
  if (p.N <= 16) launch<T, 4, 1>(p, vec, stream);
  else if (p.N <= 32) launch<T, 8, 1>(p, vec, stream);
  else if (p.N <= 64) launch<T, 8, 2>(p, vec, stream);
  else if (p.N <= 128) launch<T, 8, 4>(p, vec, stream);
  else launch<T, 8, 8>(p, vec, stream);
}

}  // namespace

hipError_t launch_ssd_step(const ssm_ssd_update_args& a, hipStream_t stream) {
  const int64_t G = a.ngroups > 1 ? a.ngroups : 1, esz = a.io_dtype == SSM_BF16 ? 2 : 4;
  StepParams p{a.state, a.x, a.dt, a.z, a.B, a.C, a.A, a.D, a.dt_bias, a.slots, a.out, a.state_slot_stride,
               a.x_batch_stride, a.x_head_stride, a.dt_batch_stride, a.z_batch_stride, a.z_head_stride,
               a.B_batch_stride, G > 1 ? a.B_group_stride : 0, a.C_batch_stride, G > 1 ? a.C_group_stride : 0,
               a.out_batch_stride, a.out_head_stride, static_cast<int>(a.nheads), static_cast<int>(a.headdim),
               static_cast<int>(a.dstate), static_cast<int>(a.nheads / G), static_cast<int>(a.batch),
               static_cast<int>(a.nslots < 0x7fffffff ? a.nslots : 0x7fffffff), a.dt_softplus != 0, 0, 0};
  auto fits = [](const void* q, int64_t s0, int64_t s1, int64_t bytes) {
    return reinterpret_cast<uintptr_t>(q) % static_cast<uintptr_t>(4 * bytes) == 0 && s0 % 4 == 0 && s1 % 4 == 0;
  };
  const bool vec = a.dstate % 4 == 0 && fits(a.state, a.state_slot_stride, 0, 4) && fits(a.B, p.Bb, p.Bg, esz) &&
                   fits(a.C, p.Cb, p.Cg, esz);
  if (a.io_dtype == SSM_BF16) launch_for<uint16_t>(p, vec, stream);
  else launch_for<float>(p, vec, stream);
  return hipGetLastError();
}

}  // namespace ssm
