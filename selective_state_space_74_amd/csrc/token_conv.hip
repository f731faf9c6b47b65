// token_conv.hip -- the causal depthwise convolution over tokens (token-major),
// and its single-token step, on gfx950.
//
//   pre_t = bias[d] + sum_k weight[d,k] x_{t-(K-1)+k},   out_t = silu(pre_t)
//
// A lane has 4 channels of a token and walks a run of tokens with the last K - 1
// inputs in registers, so a token is read once but for the K - 1 that each run
// reads again (from L2).  16 lanes lie side by side (whole cache lines of a row),
// 16 runs of tokens one after the other, four tokens' loads in flight at a time.
// Four tokens within one sequence take a path without checks.  Bound by memory, one
// read and one write: 16,411 x 2176 bf16 in 36 us, 3.9 TB/s (a large copy: 5.06).
// Loads four tokens further ahead cost registers and with them wavefronts: 43 us.
#include "token_conv.h"
#include "slots.h"

namespace ssm {
namespace {

struct ConvParams {
  const void* x;
  const float* w;
  const float* bias;
  const int32_t* cu;
  const float* state_in;
  float* state_out;
  void* out;
  int64_t xb, xs, ob, os, L, D, nseq, runs;   // runs: of tokens, in all rows
  uint32_t per_row, cols, groups;             // runs of a row, columns and workgroups that have tokens
  int run;                                    // tokens of a run
  int silu, zero_outside;
};

// Workgroups past those with tokens: the states of sequences without any.
__device__ __forceinline__ void carry_empty(const int32_t* cu, int64_t L, int64_t nseq, const float* from, float* to,
                                            int64_t n, uint32_t at, uint32_t stride) {
  if (!to) return;
  for (int64_t k = at; k < nseq; k += stride) {
    if (cu && L > 0) {
      const int64_t lo = min(max(int64_t{cu[k]}, int64_t{0}), L), hi = min(max(int64_t{cu[k + 1]}, int64_t{0}), L);
      if (hi > lo) continue;
    }
    for (int64_t i = threadIdx.x; i < n; i += blockDim.x) to[k * n + i] = from ? from[k * n + i] : 0.0f;
  }
}

template <typename T, int K, bool kVec>
__global__ __launch_bounds__(kConvThreads) void conv_fwd_kernel(ConvParams p) {
  constexpr int V = kConvV, kAhead = 4;
  __shared__ int32_t held[kConvBounds];
  if (blockIdx.x >= p.groups) {
    carry_empty(p.cu, p.L, p.nseq, p.state_in, p.state_out, p.D * K, blockIdx.x - p.groups, gridDim.x - p.groups);
    return;
  }
  const int64_t run = static_cast<int64_t>(blockIdx.x / p.cols) * kConvRuns + threadIdx.x / kConvLanes;
  const int64_t c = (static_cast<int64_t>(blockIdx.x % p.cols) * kConvLanes + threadIdx.x % kConvLanes) * V;
  int step = 0;
  if (p.cu) {
    step = hold_bounds(p.cu, static_cast<int>(p.nseq), held);
    __syncthreads();
  }
  if (c >= p.D || run >= p.runs) return;
  const int nv = static_cast<int>(min(int64_t{V}, p.D - c));
  const int64_t b = run / p.per_row;
  const int t0 = static_cast<int>(run - b * p.per_row) * p.run;
  const int t1 = static_cast<int>(min(int64_t{t0} + p.run, p.L));
  const T* x = static_cast<const T*>(p.x) + b * p.xb + c;
  T* out = static_cast<T*>(p.out) + b * p.ob + c;

  float w[K][V], bias[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int64_t d = c + min(v, nv - 1);
    bias[v] = p.bias ? p.bias[d] : 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) w[k][v] = p.w[d * K + k];
  }
  Walk walk;
  if (p.cu) walk.find(p.cu, static_cast<int>(p.nseq), static_cast<int>(p.L), held, step, t0);
  else walk.whole(static_cast<int>(b), static_cast<int>(p.L));

  // h[K - 1 + i]: the input of token t + i, those before it its history
  float h[K - 1 + kAhead][V];
  // an input before the sequence: position `back` (-(K-1) .. -1) from its first token
  auto from_state = [&](int back, float (&v)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      v[i] = p.state_in && i < nv ? p.state_in[(walk.k * p.D + c + i) * K + K + back] : 0.0f;
  };
  if (walk.inside() && t0 >= walk.lo) {
#pragma unroll
    for (int j = 1; j < K; ++j) {
      if (t0 - j >= walk.lo) load_channels<T, V, kVec>(x + (t0 - j) * p.xs, nv).widen(h[K - 1 - j]);
      else from_state(t0 - j - walk.lo, h[K - 1 - j]);
    }
  }
  // four tokens from xt on; short runs and ends: the last token again, not used
  Channels<T, V> next[kAhead];
  const T* xt = x + t0 * p.xs;
  T* ot = out + t0 * p.os;
  auto load = [&](const T* from, int left) {
    if (left >= kAhead) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) next[i] = load_channels<T, V, kVec>(from + i * p.xs, nv);
    } else {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) next[i] = load_channels<T, V, kVec>(from + min(i, left - 1) * p.xs, nv);
    }
  };
  auto value = [&](int i, float (&y)[V]) {   // out of token t + i
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float pre = bias[v];
#pragma unroll
      for (int k = 0; k < K; ++k) pre = fmaf(w[k][v], h[i + k][v], pre);
      y[v] = p.silu ? silu_f32(pre) : pre;
    }
  };
  for (int t = t0; t < t1; t += kAhead) {
    load(xt, t1 - t);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) next[i].widen(h[K - 1 + i]);
    xt += kAhead * p.xs;
    if (t + kAhead <= t1 && walk.inside() && t >= walk.lo && t + kAhead < walk.hi) {   // four tokens within a sequence
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        float y[V];
        value(i, y);
        store_channels<T, V, kVec>(ot + i * p.os, nv, y);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int u = t + i;
        if (u >= t1) break;
        if (walk.reach(u) && walk.inside()) {
#pragma unroll
          for (int j = 1; j < K; ++j) from_state(-j, h[K - 1 + i - j]);
        }
        const bool in = walk.inside() && u >= walk.lo && u < walk.hi;
        if (!in && !p.zero_outside) continue;
        float y[V] = {};
        if (in) value(i, y);
        store_channels<T, V, kVec>(ot + i * p.os, nv, y);
        if (p.state_out && in && u == walk.hi - 1) {
#pragma unroll
          for (int v = 0; v < V; ++v) {
            if (v >= nv) continue;
            float* s = p.state_out + (walk.k * p.D + c + v) * K;
#pragma unroll
            for (int k = 0; k < K; ++k) s[k] = h[i + k][v];
          }
        }
      }
    }
    ot += kAhead * p.os;
#pragma unroll
    for (int j = 0; j < K - 1; ++j)
#pragma unroll
      for (int v = 0; v < V; ++v) h[j][v] = h[j + kAhead][v];
  }
}

template <typename T, int K>
void launch_fwd(const ConvParams& p, bool vec, dim3 grid, hipStream_t stream) {
  if (vec) conv_fwd_kernel<T, K, true><<<grid, kConvThreads, 0, stream>>>(p);
  else conv_fwd_kernel<T, K, false><<<grid, kConvThreads, 0, stream>>>(p);
}

// ---- the step ----------------------------------------------------------------

struct StepParams {
  float* state;
  const void* x;
  const float* w;
  const float* bias;
  const int32_t* slots;
  void* out;
  int64_t ss, xb, ob, D;
  int batch, nslots, silu;
};

// A lane has one channel, its K inputs one access where they are aligned.  Bound
// by the pool's K fp32 a channel, read and written: 256 x 5376 x 4 in 10.4 us, 4.8
// TB/s, and by the call's own 10 us.
template <typename T, int K, bool kVec>
__global__ __launch_bounds__(kConvThreads) void conv_step_kernel(StepParams p) {
  struct alignas(kVec ? 4 * K : 4) Held { float v[K]; };
  const int lane = threadIdx.x & 63;
  const int64_t c0 = static_cast<int64_t>(blockIdx.x) * kConvThreads + threadIdx.x;
  const bool live = c0 < p.D;
  const int64_t c = live ? c0 : p.D - 1;   // lanes past the channels repeat the last one, and store nothing
  const int row = blockIdx.y;
  int slot = p.slots ? p.slots[row] : row;
  if (slot < 0 || slot >= p.nslots) slot = -1;
  const T* x = static_cast<const T*>(p.x) + c;
  T* out = static_cast<T*>(p.out) + c;
  float xv = io<T>::load(x + row * p.xb);
  Held* const at = reinterpret_cast<Held*>(p.state + max(slot, 0) * p.ss + c * K);
  Held h{};
  if (slot >= 0) h = *at;
  const Held w = *reinterpret_cast<const Held*>(p.w + c * K);
  const float bias = p.bias ? p.bias[c] : 0.0f;
  bool before;
  int next;
  slot_order(p.slots, row, p.batch, slot, lane, before, next);
  if (before && slot >= 0) return;
  for (int b = row;;) {
    float y = 0.0f;
    if (slot >= 0) {
      float pre = bias;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        h.v[k] = k < K - 1 ? h.v[k < K - 1 ? k + 1 : k] : xv;
        pre = fmaf(w.v[k], h.v[k], pre);
      }
      y = p.silu ? silu_f32(pre) : pre;
    }
    if (live) io<T>::store(out + b * p.ob, y);
    if (slot < 0) return;
    b = b == row ? next : named_next(p.slots, b, p.batch, slot, lane);
    if (b >= p.batch) break;
    xv = io<T>::load(x + b * p.xb);
  }
  if (live) *at = h;
}

template <typename T, int K>
void launch_step(const StepParams& p, hipStream_t stream) {
  auto fits = [](const void* q) { return reinterpret_cast<uintptr_t>(q) % 16 == 0; };
  const dim3 grid(static_cast<unsigned>((p.D + kConvThreads - 1) / kConvThreads), static_cast<unsigned>(p.batch));
  if (K == 4 && fits(p.state) && fits(p.w) && p.ss % 4 == 0)
    conv_step_kernel<T, K, K == 4><<<grid, kConvThreads, 0, stream>>>(p);
  else conv_step_kernel<T, K, false><<<grid, kConvThreads, 0, stream>>>(p);
}

// f(std::integral_constant<int, K>) for the width of a call.
template <typename F>
void with_width(int K, F&& f) {
  switch (K) {
    case 1: f(std::integral_constant<int, 1>{}); break;
    case 2: f(std::integral_constant<int, 2>{}); break;
    case 3: f(std::integral_constant<int, 3>{}); break;
    case 4: f(std::integral_constant<int, 4>{}); break;
    case 5: f(std::integral_constant<int, 5>{}); break;
    case 6: f(std::integral_constant<int, 6>{}); break;
    case 7: f(std::integral_constant<int, 7>{}); break;
    default: f(std::integral_constant<int, 8>{}); break;
  }
}

}  // namespace

hipError_t launch_token_conv_fwd(const ssm_token_conv_args& a, hipStream_t stream) {
  constexpr int64_t V = kConvV;
  const int64_t esz = a.io_dtype == SSM_BF16 ? 2 : 4;
  const bool packed = a.cu_seqlens != nullptr;
  ConvParams p;
  p.x = a.x; p.w = a.weight; p.bias = a.bias; p.cu = a.cu_seqlens; p.state_in = a.state_in; p.state_out = a.state_out;
  p.out = a.out;
  p.xb = a.x_batch_stride; p.xs = a.x_seq_stride; p.ob = a.out_batch_stride; p.os = a.out_seq_stride;
  p.L = a.seqlen; p.D = a.dim; p.nseq = packed ? a.nseq : a.batch;
  p.cols = static_cast<uint32_t>((a.dim + kConvLanes * V - 1) / (kConvLanes * V));
  // runs of 32 tokens, shorter ones where that leaves the machine short of work
  // (16,411 packed x 2176 bf16: 36 us, and 39 with runs of 16)
  p.run = 32;
  while (p.run > 4 && a.batch * ((a.seqlen + p.run - 1) / p.run) * p.cols < 1024 * kConvRuns) p.run /= 2;
  p.per_row = static_cast<uint32_t>((a.seqlen + p.run - 1) / p.run);
  p.runs = a.batch * p.per_row;
  p.groups = static_cast<uint32_t>((p.runs + kConvRuns - 1) / kConvRuns * p.cols);
  p.silu = a.conv_silu != 0; p.zero_outside = a.zero_outside != 0;
  // sequences without tokens: some of a packed row, or all
  const int64_t more = a.state_out && (packed || a.seqlen == 0) ? std::min<int64_t>(p.nseq, 256) : 0;
  if (p.groups + more == 0) return hipSuccess;
  const dim3 grid(static_cast<unsigned>(p.groups + more));
  auto fits = [&](const void* q, int64_t sb, int64_t ss) {
    return reinterpret_cast<uintptr_t>(q) % static_cast<uintptr_t>(V * esz) == 0 && sb % V == 0 && ss % V == 0;
  };
  const bool vec = a.dim % V == 0 && fits(a.x, a.x_batch_stride, a.x_seq_stride) &&
                   fits(a.out, a.out_batch_stride, a.out_seq_stride);
  with_width(a.d_conv, [&](auto k) {
    if (a.io_dtype == SSM_BF16) launch_fwd<uint16_t, k.value>(p, vec, grid, stream);
    else launch_fwd<float, k.value>(p, vec, grid, stream);
  });
  return hipGetLastError();
}

hipError_t launch_token_conv_update(const ssm_token_conv_update_args& a, hipStream_t stream) {
  const StepParams p{a.state, a.x, a.weight, a.bias, a.slots, a.out, a.state_slot_stride, a.x_batch_stride,
                     a.out_batch_stride, a.dim, static_cast<int>(a.batch),
                     static_cast<int>(a.nslots < 0x7fffffff ? a.nslots : 0x7fffffff), a.conv_silu != 0};
  with_width(a.d_conv, [&](auto k) {
    if (a.io_dtype == SSM_BF16) launch_step<uint16_t, k.value>(p, stream);
    else launch_step<float, k.value>(p, stream);
  });
  return hipGetLastError();
}

}  // namespace ssm
