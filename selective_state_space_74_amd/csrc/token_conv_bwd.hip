// token_conv_bwd.hip -- gradients of the causal convolution over tokens, gfx950.
//
// With e_t = dout_t silu'(pre_t), silu'(v) = s (1 + v (1 - s)), s = sigmoid(v):
//   dx_q        = sum_k weight[d,k] e_{q+(K-1)-k}   over tokens of q's sequence
//   dweight[d,k] = sum_t e_t x_{t-(K-1)+k},   dbias[d] = sum_t e_t
// and an input from the state gets its gradient the same way.
//
// A lane has 4 channels and walks a run of tokens, computing pre again, with
// the last K - 1 inputs and the K - 1 gradients that are not complete yet in
// registers; it goes on for K - 1 tokens into the next run (their x and dout
// come from L2).  Bound by memory, two reads and one write, and by the 160 registers
// that leave 12 wavefronts a compute unit: 8 x 2048 x 2176 bf16 in 62 us, 3.5 TB/s.
// dweight and dbias: sums of a run in registers, of a workgroup's 16 runs by shuffles
// and LDS, and of all workgroups by a second kernel, in a fixed order.
//
// Registers grow with K, 26 a tap; with 8 they are held to 256, so that two wavefronts
// a SIMD remain (4 x 2000 x 2176 bf16 forward and backward, K 4, 5, 6, 7 and 8: 58, 75,
// 85, 113 and 110 us; K 8 without the bound 149).  The lambdas are always inline: called,
// they kept a lane's arrays in memory (K 5: 240 us).
#include "token_conv.h"

namespace ssm {
namespace {

struct ConvBwdParams {
  const void* x;
  const void* dout;
  const float* w;
  const float* bias;
  const int32_t* cu;
  const float* state_in;
  const float* dstate_out;
  void* dx;
  float* dstate_in;
  float* part;                    // [group of runs][K + 1][D]
  int64_t xb, xs, eb, es, gb, gs, L, D, nseq, runs;
  uint32_t per_row, cols, groups;
  int run, silu;
};

template <typename T, int K, bool kVec>
__global__ __launch_bounds__(kConvThreads, K > 7 ? 2 : 1) void conv_bwd_kernel(ConvBwdParams p) {
  constexpr int V = kConvV;
  __shared__ int32_t held[kConvBounds];
  __shared__ float sums[kConvThreads / 64][kConvLanes][(K + 1) * V];
  if (blockIdx.x >= p.groups) {   // sequences without tokens: their state goes through
    const int64_t n = p.D * K;
    for (int64_t k = blockIdx.x - p.groups; k < p.nseq; k += gridDim.x - p.groups) {
      if (p.cu && p.L > 0) {
        const int64_t lo = min(max(int64_t{p.cu[k]}, int64_t{0}), p.L), hi = min(max(int64_t{p.cu[k + 1]}, int64_t{0}), p.L);
        if (hi > lo) continue;
      }
      for (int64_t i = threadIdx.x; i < n; i += blockDim.x)
        p.dstate_in[k * n + i] = p.dstate_out ? p.dstate_out[k * n + i] : 0.0f;
    }
    return;
  }
  const uint32_t group = blockIdx.x / p.cols;
  const int lane16 = threadIdx.x % kConvLanes;
  const int64_t run = static_cast<int64_t>(group) * kConvRuns + threadIdx.x / kConvLanes;
  const int64_t c = (static_cast<int64_t>(blockIdx.x % p.cols) * kConvLanes + lane16) * V;
  int step = 0;
  if (p.cu) {
    step = hold_bounds(p.cu, static_cast<int>(p.nseq), held);
    __syncthreads();
  }
  float dw[K + 1][V];   // the last one: dbias
#pragma unroll
  for (int k = 0; k <= K; ++k)
#pragma unroll
    for (int v = 0; v < V; ++v) dw[k][v] = 0.0f;

  if (c < p.D && run < p.runs) {
    const int nv = static_cast<int>(min(int64_t{V}, p.D - c));
    const int64_t b = run / p.per_row;
    const int t0 = static_cast<int>(run - b * p.per_row) * p.run;
    const int t1 = static_cast<int>(min(int64_t{t0} + p.run, p.L));
    const T* x = static_cast<const T*>(p.x) + b * p.xb + c;
    const T* dout = static_cast<const T*>(p.dout) + b * p.eb + c;
    T* dx = static_cast<T*>(p.dx) + b * p.gb + c;
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

    float h[K][V];      // inputs of tokens u - (K-1) .. u
    float pend[K][V];   // gradients of the inputs at u - (K-1) .. u, not complete yet
#pragma unroll
    for (int j = 0; j < K; ++j)
#pragma unroll
      for (int v = 0; v < V; ++v) h[j][v] = pend[j][v] = 0.0f;
    auto state_at = [&](int back) { return (walk.k * p.D + c) * K + K + back; };
    auto from_state = [&](int back, float (&v)[V]) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = p.state_in && i < nv ? p.state_in[state_at(back) + i * K] : 0.0f;
    };
    // the gradient of the input at token q of the walk's sequence (before its
    // first token: of the state) is complete
    auto emit = [&](int q, float (&g)[V]) __attribute__((always_inline)) {
      if (!walk.inside()) return;
      const bool token = q >= walk.lo;
      if (token ? q < t0 || q >= t1 : !p.dstate_in || walk.lo < t0 || walk.lo >= t1) return;
      const int kept = q - (walk.hi - K);   // its place in the state that the sequence leaves
      if (p.dstate_out && kept >= 0) {
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (i < nv) g[i] += p.dstate_out[state_at(kept - K) + i * K];
      }
      if (token) {
        store_channels<T, V, kVec>(dx + q * p.gs, nv, g);
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (i < nv) p.dstate_in[state_at(q - walk.lo) + i * K] = g[i];
      }
    };
    // the walk's sequence ends before token u: so are all its gradients
    auto flush = [&](int u) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < K - 1; ++j) emit(u - (K - 1) + j, pend[j]);
    };
    auto begin = [&]() __attribute__((always_inline)) {   // a sequence's first token
#pragma unroll
      for (int j = 0; j < K - 1; ++j) {
        if (walk.inside()) from_state(j - (K - 1), h[j + 1]);
#pragma unroll
        for (int v = 0; v < V; ++v) pend[j][v] = 0.0f;
      }
      if (walk.inside() && p.dstate_in) {   // the oldest of the state is no tap of any token
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (i < nv) p.dstate_in[state_at(-K) + i * K] = 0.0f;
      }
    };
    // token u, its input and upstream gradient; own: one of the run's.  Leaves in
    // `done` the gradient of the input at u - (K - 1), now complete.
    auto add = [&](const float (&xu)[V], const float (&eu)[V], bool own, float (&done)[V]) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < K - 1; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v) h[j][v] = h[j + 1][v];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        h[K - 1][v] = xu[v];
        pend[K - 1][v] = 0.0f;
        float pre = bias[v];
#pragma unroll
        for (int k = 0; k < K; ++k) pre = fmaf(w[k][v], h[k][v], pre);
        float e = eu[v];
        if (p.silu) {
          const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-pre * kLog2e));
          e *= s * fmaf(pre, 1.0f - s, 1.0f);
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
          pend[k][v] = fmaf(w[k][v], e, pend[k][v]);
          if (own) dw[k][v] = fmaf(e, h[k][v], dw[k][v]);
        }
        if (own) dw[K][v] += e;
        done[v] = pend[0][v];
      }
#pragma unroll
      for (int j = 0; j < K - 1; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v) pend[j][v] = pend[j + 1][v];
    };
    auto token = [&](int u, const float (&xu)[V], const float (&eu)[V], bool own) __attribute__((always_inline)) {
      float done[V];
      add(xu, eu, own, done);
      emit(u - (K - 1), done);
    };

    if (walk.inside() && t0 >= walk.lo) {
      if (t0 == walk.lo) {
        begin();
      } else {
#pragma unroll
        for (int j = 1; j < K; ++j) {
          if (t0 - j >= walk.lo) load_channels<T, V, kVec>(x + (t0 - j) * p.xs, nv).widen(h[K - j]);
          else from_state(t0 - j - walk.lo, h[K - j]);
        }
      }
    }
    constexpr int kAhead = 4;
    Channels<T, V> xn[kAhead], en[kAhead];
    const T* xt = x + t0 * p.xs;
    const T* et = dout + t0 * p.es;
    T* dt = dx + (t0 - (K - 1)) * p.gs;   // where the gradient that token t completes goes
    auto load = [&](int left) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {   // past the run: its last token again, not used
        const int at = left >= kAhead ? i : min(i, left - 1);
        xn[i] = load_channels<T, V, kVec>(xt + at * p.xs, nv);
        en[i] = load_channels<T, V, kVec>(et + at * p.es, nv);
      }
    };
    for (int t = t0; t < t1; t += kAhead) {
      load(t1 - t);
      xt += kAhead * p.xs;
      et += kAhead * p.es;
      // four tokens within a sequence that complete gradients of the run's own
      // tokens, none of them among the last K, which the state holds
      if (t + kAhead <= t1 && walk.inside() && t - (K - 1) >= max(walk.lo, t0) && t + kAhead <= walk.hi &&
          (!p.dstate_out || t + kAhead <= walk.hi - K)) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          float xu[V], eu[V], done[V];
          xn[i].widen(xu);
          en[i].widen(eu);
          add(xu, eu, true, done);
          store_channels<T, V, kVec>(dt + i * p.gs, nv, done);
        }
      } else {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const int u = t + i;
          if (u >= t1) break;
          if (u >= walk.hi && walk.cu) {
            flush(u);
            walk.reach(u);
            begin();
          }
          if (walk.inside() && u >= walk.lo && u < walk.hi) {
            float xu[V], eu[V];
            xn[i].widen(xu);
            en[i].widen(eu);
            token(u, xu, eu, true);
          } else {
            const float none[V] = {};
            store_channels<T, V, kVec>(dx + u * p.gs, nv, none);
          }
        }
      }
      dt += kAhead * p.gs;
    }
    // the tokens after the run that its last ones reach
    int u = t1;
    if (walk.inside() && t1 > walk.lo) {
      for (; u < t1 + K - 1 && u < walk.hi; ++u) {
        float xu[V], eu[V];
        load_channels<T, V, kVec>(x + u * p.xs, nv).widen(xu);
        load_channels<T, V, kVec>(dout + u * p.es, nv).widen(eu);
        token(u, xu, eu, false);
      }
      if (u < t1 + K - 1) flush(u);
    }
  }

  // dweight and dbias of the workgroup
#pragma unroll
  for (int k = 0; k <= K; ++k)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float s = dw[k][v];
      s += __shfl_xor(s, 16, 64);
      s += __shfl_xor(s, 32, 64);
      if ((threadIdx.x & 63) < kConvLanes) sums[threadIdx.x / 64][lane16][k * V + v] = s;
    }
  __syncthreads();
  for (int i = threadIdx.x; i < kConvLanes * (K + 1) * V; i += kConvThreads) {
    const int v = i % V, l = i / V % kConvLanes, k = i / (V * kConvLanes);
    const int64_t d = (static_cast<int64_t>(blockIdx.x % p.cols) * kConvLanes + l) * V + v;
    if (d >= p.D) continue;
    float s = 0.0f;
#pragma unroll
    for (int q = 0; q < kConvThreads / 64; ++q) s += sums[q][l][k * V + v];
    p.part[(static_cast<int64_t>(group) * (K + 1) + k) * p.D + d] = s;
  }
}

// Sums of the groups' parts: 64 channels a workgroup, the groups in 4 strands.
__global__ __launch_bounds__(256) void conv_param_kernel(const float* part, int64_t groups, int64_t D, int K, float* dweight,
                                                         float* dbias) {
  __shared__ float strands[4][64];
  const int64_t d = static_cast<int64_t>(blockIdx.x) * 64 + threadIdx.x % 64;
  const int k = blockIdx.y, strand = threadIdx.x / 64;
  float s = 0.0f;
  if (d < D)
#pragma unroll 8
    for (int64_t g = strand; g < groups; g += 4) s += part[(g * (K + 1) + k) * D + d];
  strands[strand][threadIdx.x % 64] = s;
  __syncthreads();
  if (strand == 0 && d < D) {
    s = (strands[0][threadIdx.x] + strands[1][threadIdx.x]) + (strands[2][threadIdx.x] + strands[3][threadIdx.x]);
    if (k < K) dweight[d * K + k] = s;
    else if (dbias) dbias[d] = s;
  }
}

struct ConvBwdPlan {
  int run;
  int64_t per_row, runs, cols, groups;   // groups: of kConvRuns runs
};

// Runs of 32 tokens, shorter ones where that leaves the machine short of work.
ConvBwdPlan plan_of(const ssm_token_conv_bwd_args& a) {
  ConvBwdPlan q;
  q.cols = (a.dim + kConvLanes * kConvV - 1) / (kConvLanes * kConvV);
  q.run = 32;
  while (q.run > 8 && a.batch * ((a.seqlen + q.run - 1) / q.run) * q.cols < 1024 * kConvRuns) q.run /= 2;
  q.per_row = (a.seqlen + q.run - 1) / q.run;
  q.runs = a.batch * q.per_row;
  q.groups = (q.runs + kConvRuns - 1) / kConvRuns;
  return q;
}

template <typename T>
void launch_bwd(const ConvBwdParams& p, int K, bool vec, dim3 grid, hipStream_t stream) {
  auto go = [&](auto k) {
    if (vec) conv_bwd_kernel<T, k.value, true><<<grid, kConvThreads, 0, stream>>>(p);
    else conv_bwd_kernel<T, k.value, false><<<grid, kConvThreads, 0, stream>>>(p);
  };
  switch (K) {
    case 1: go(std::integral_constant<int, 1>{}); break;
    case 2: go(std::integral_constant<int, 2>{}); break;
    case 3: go(std::integral_constant<int, 3>{}); break;
    case 4: go(std::integral_constant<int, 4>{}); break;
    case 5: go(std::integral_constant<int, 5>{}); break;
    case 6: go(std::integral_constant<int, 6>{}); break;
    case 7: go(std::integral_constant<int, 7>{}); break;
    default: go(std::integral_constant<int, 8>{}); break;
  }
}

}  // namespace

size_t token_conv_bwd_workspace_bytes(const ssm_token_conv_bwd_args& a) {
  return static_cast<size_t>(plan_of(a).groups) * (a.d_conv + 1) * a.dim * 4;
}

hipError_t launch_token_conv_bwd(const ssm_token_conv_bwd_args& a, hipStream_t stream) {
  const ConvBwdPlan q = plan_of(a);
  const bool packed = a.cu_seqlens != nullptr;
  ConvBwdParams p;
  p.x = a.x; p.dout = a.dout; p.w = a.weight; p.bias = a.bias; p.cu = a.cu_seqlens; p.state_in = a.state_in;
  p.dstate_out = a.dstate_out; p.dx = a.dx; p.dstate_in = a.dstate_in; p.part = static_cast<float*>(a.workspace);
  p.xb = a.x_batch_stride; p.xs = a.x_seq_stride; p.eb = a.dout_batch_stride; p.es = a.dout_seq_stride;
  p.gb = a.dx_batch_stride; p.gs = a.dx_seq_stride;
  p.L = a.seqlen; p.D = a.dim; p.nseq = packed ? a.nseq : a.batch; p.runs = q.runs;
  p.per_row = static_cast<uint32_t>(q.per_row); p.cols = static_cast<uint32_t>(q.cols);
  p.groups = static_cast<uint32_t>(q.groups * q.cols); p.run = q.run; p.silu = a.conv_silu != 0;
  const int64_t more = a.dstate_in && (packed || a.seqlen == 0) ? std::min<int64_t>(p.nseq, 256) : 0;
  const int64_t esz = a.io_dtype == SSM_BF16 ? 2 : 4;
  auto fits = [&](const void* ptr, int64_t sb, int64_t ss) {
    return reinterpret_cast<uintptr_t>(ptr) % static_cast<uintptr_t>(kConvV * esz) == 0 && sb % kConvV == 0 && ss % kConvV == 0;
  };
  const bool vec = a.dim % kConvV == 0 && fits(a.x, a.x_batch_stride, a.x_seq_stride) &&
                   fits(a.dout, a.dout_batch_stride, a.dout_seq_stride) && fits(a.dx, a.dx_batch_stride, a.dx_seq_stride);
  if (p.groups + more > 0) {
    const dim3 grid(static_cast<unsigned>(p.groups + more));
    if (a.io_dtype == SSM_BF16) launch_bwd<uint16_t>(p, a.d_conv, vec, grid, stream);
    else launch_bwd<float>(p, a.d_conv, vec, grid, stream);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  conv_param_kernel<<<dim3(static_cast<unsigned>((a.dim + 63) / 64), static_cast<unsigned>(a.d_conv + 1)), 256, 0, stream>>>(
      p.part, q.groups, a.dim, a.d_conv, a.dweight, a.dbias);
  return hipGetLastError();
}

}  // namespace ssm
