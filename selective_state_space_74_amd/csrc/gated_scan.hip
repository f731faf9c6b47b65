// gated_scan.hip -- the gated linear recurrence for gfx950: prefill and the
// single-token step.
//   a_t = exp(-s sigma(gate_a_t)), s = c softplus(lam)
//   h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigma(gate_x_t) x_t
#include <type_traits>

#include "gated_tile.h"
#include "slots.h"

namespace ssm {
namespace {

constexpr int kThreads = 256;   // of the single-token step

// The tile kernel (gated_tile.h says how tiles are joined): (a, b) of every token
// in registers, then one product and one sum a token with the state that
// entered.  16 tokens a wavefront: with 8, halves as many bytes would be on
// their way a workgroup, and twice the pairs to hand on.
struct FwdParams {
  const void* x; const void* ga; const void* gx;
  const float* lam; const float* h0;
  float* last; void* out; float* ck;
  const int32_t* marks;
  uint32_t* ticket; uint64_t* words;
  int64_t xb, xs, gab, gas, gxb, gxs, ob, os;
  int64_t L, D, nck, nseq;
  uint32_t batch, tiles, cols;
  int shift;   // narrow calls: log2 of the channels
  float c;
  int zero_outside;
};

template <typename T, int V, bool PACKED, bool CHAIN, bool NARROW, int CACHE>
__global__ __launch_bounds__(64 * kMaxWaves) void gated_fwd_kernel(FwdParams p) {
  constexpr int W = 64 * V;
  __shared__ float2 pairs[kMaxWaves][W];
  constexpr int kGroup = chain_group(NARROW);
  __shared__ ChainShared<CHAIN ? W : 1, kGroup> before;
  __shared__ float initial[PACKED ? 1 : W];
  __shared__ uint32_t taken;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = blockDim.x >> 6;

  uint32_t id = blockIdx.x;
  if constexpr (CHAIN) {
    if (threadIdx.x == 0) taken = atomicAdd(p.ticket, 1u);
    __syncthreads();
    id = __builtin_amdgcn_readfirstlane(taken);
    if (id >= p.tiles * p.cols * p.batch) return;   // only if another call reset the counter
  }
  // along the channels first, then the batch: neighbours read neighbouring bytes
  const uint32_t col = id % p.cols, row = id / p.cols % p.batch, tile = id / p.cols / p.batch;
  // A wavefront has 16 tokens of 64 V channels; in a narrow call each stretch of
  // 2^shift lanes has 16 tokens of its own.
  constexpr int kBytes = V * sizeof(T);
  const int shift = NARROW ? p.shift : V == 2 ? 7 : 6;
  const int width = 1 << shift, subs = NARROW ? 64 >> shift : 1;
  const int sub = NARROW ? lane >> shift : 0, c = NARROW ? lane & (width - 1) : lane;
  const int64_t b = row, wave_t0 = (static_cast<int64_t>(tile) * waves + wave) * (kWaveTokens * subs);
  const int64_t t0 = wave_t0 + sub * kWaveTokens;
  const int n = static_cast<int>(min(static_cast<int64_t>(kWaveTokens), max(int64_t{0}, p.L - t0)));
  const bool some = NARROW ? wave_t0 < p.L : n > 0;   // of the wavefront
  const int64_t ch = static_cast<int64_t>(col) * W + c * V;
  const bool live = ch < p.D;
  const int64_t d = live ? ch : p.D - V;   // per-channel values: lanes past the channels repeat the last ones
  // a lane's offset from the wavefront's row j of a tensor
  auto at = [&](int64_t stride) {
    if constexpr (NARROW) return live ? static_cast<uint32_t>((c + sub * kWaveTokens * stride) * sizeof(T)) : kNowhere;
    else return static_cast<uint32_t>(ch) * static_cast<uint32_t>(sizeof(T));
  };

  Rate s[V];
  float a[kWaveTokens][V], u[kWaveTokens][V], P[V], H[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    s[v] = Rate(p.c, p.lam[d + v]);
    P[v] = 1.0f;
    H[v] = 0.0f;
  }
  // Wavefronts of 16 tokens of one sequence, none of them its first or last,
  // take a path without branches; the others ask for their tokens' marks, which
  // one load brings, as scalars.  (One path with a branch a token, as in the
  // backward, measured slower here: 598 us against 574 at 262144 x 1536 bf16.
  // So did fetching the rows before the marks that decide the path are known:
  // the rows' uses then wait together.)
  int32_t marks = 0, each[NARROW ? kWaveTokens : 1];
  auto mark_at = [&](int64_t t) {
    const int32_t m = p.marks[t];
    return m >> 2 < p.nseq ? m : kOutside;
  };
  if constexpr (PACKED && !NARROW) marks = some ? mark_at(t0 + lane % kWaveTokens) : kOutside;
  if constexpr (PACKED && NARROW)
    for (int i = c; i < n; i += width) marks |= mark_at(t0 + i);   // kOutside sets every bit
  auto mark = [&](int j) { return NARROW ? each[NARROW ? j : 0] : __builtin_amdgcn_readlane(marks, j); };

  // tokens to (a, b) of h = a h + b; past the end of the row (1, 0)
  auto tokens = [&](auto every) {
    constexpr bool PLAIN = decltype(every)::value;
    constexpr bool MARKED = PACKED && !PLAIN;
    uint32_t rx[kWaveTokens], ra[kWaveTokens], rg[kWaveTokens];
    const TokenRows x = token_rows<T>(p.x, b * p.xb + wave_t0 * p.xs, p.xs, p.D, subs),
                    ga = token_rows<T>(p.ga, b * p.gab + wave_t0 * p.gas, p.gas, p.D, subs),
                    gx = token_rows<T>(p.gx, b * p.gxb + wave_t0 * p.gxs, p.gxs, p.D, subs);
#pragma unroll
    for (int j = 0; j < kWaveTokens; ++j) {
      const int jj = PLAIN || NARROW ? j : min(j, n - 1);
      const bool in = PLAIN || !NARROW || j < n;
      ra[j] = ga.load<kBytes, CACHE>(jj, in ? at(p.gas) : kNowhere);
      rg[j] = gx.load<kBytes, CACHE>(jj, in ? at(p.gxs) : kNowhere);
      rx[j] = x.load<kBytes, CACHE>(jj, in ? at(p.xs) : kNowhere);
    }
#pragma unroll
    for (int j = 0; j < kWaveTokens; ++j) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float sa = sigmoid_f32(widen<T, V>(ra[j], v));
        float aj = __builtin_amdgcn_exp2f(s[v].log2a * sa);
        float bj = __builtin_amdgcn_sqrtf(one_minus_square(aj, s[v].u * sa)) *
                   (sigmoid_f32(widen<T, V>(rg[j], v)) * widen<T, V>(rx[j], v));
        if constexpr (MARKED) {
          if (mark(j) & 1) {   // first token of its sequence, or in none
            const float h0 = mark(j) >= 0 && p.h0 ? p.h0[static_cast<int64_t>(mark(j) >> 2) * p.D + d + v] : 0.0f;
            bj = mark(j) >= 0 ? fmaf(aj, h0, bj) : 0.0f;
          }
        }
        if constexpr (!PLAIN) {
          aj = j < n ? aj : 1.0f;
          bj = j < n ? bj : 0.0f;
        }
        a[j][v] = aj;
        u[j][v] = bj;
        P[v] *= aj;
        H[v] = MARKED && (mark(j) & 1) ? bj : fmaf(aj, H[v], bj);
      }
    }
  };
  bool plain;
  if constexpr (NARROW) plain = __all(n == kWaveTokens) && !__any(marks < 0 || (marks & 3));
  else plain = n == kWaveTokens && (!PACKED || __ballot(marks < 0 || (marks & 3)) == 0);
  if (plain) tokens(std::true_type{});
  if (!plain && some) {
    if constexpr (PACKED && NARROW) {
#pragma unroll
      for (int j = 0; j < kWaveTokens; ++j) each[j] = j < n ? mark_at(t0 + j) : kOutside;
      marks = 0;   // of the lane's own stretch now
#pragma unroll
      for (int j = 0; j < kWaveTokens; ++j) marks |= j < n ? each[j] : 0;
    }
    tokens(std::false_type{});
  }
  if constexpr (PACKED) {
    if (NARROW ? !plain && (marks & 1) : some && __ballot(marks & 1)) {
#pragma unroll
      for (int v = 0; v < V; ++v) P[v] = kCut;
    }
  }

  if constexpr (NARROW) {
    const float2 all = wave_stretches<PACKED, false>(shift, P[0], H[0]);
    if (sub == subs - 1) pairs[wave][c] = all;
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) pairs[wave][lane * V + v] = make_float2(P[v], H[v]);
  }
  // last_state may be h0 itself: h0 has therefore been read, into LDS, before the
  // tile's first barrier.  The state is stored behind that barrier or, by another
  // tile, behind words that this one publishes there.  (A packed sequence's first
  // token takes its h0 into the pair.)  Of a chain, the first group's tiles start
  // from h0.  (Read here: a register that holds it through the tokens would be the
  // 65th in fp32, and cost a workgroup a compute unit.)
  if constexpr (!PACKED) {
    if (wave == 0 && sub == 0 && (!CHAIN || tile < static_cast<uint32_t>(kGroup))) {
#pragma unroll
      for (int v = 0; v < V; ++v) initial[c * V + v] = p.h0 ? p.h0[b * p.D + d + v] : 0.0f;
    }
  }
  __syncthreads();
  float h[V];
  if constexpr (CHAIN) {
    // the words of (row, col): tiles, then groups
    const int64_t ngroups = (p.tiles + kGroup - 1) / kGroup;
    uint64_t* const base = p.words + (static_cast<int64_t>(row) * p.cols + col) * (p.tiles + ngroups) * width;
    const Chain chain{base, base + static_cast<int64_t>(p.tiles) * width, width};
    // thread i of the first 2^shift has channel i of the group
    const float first = PACKED ? 0.0f : initial[threadIdx.x & (width - 1)];   // of the first group's tiles
    chain_carry<PACKED, W, kGroup, chain_mine(NARROW, V)>(chain, tile, p.tiles, pairs, before, shift, first,
                                                             [](int w) { return w; });
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = before.entering[c * V + v];
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = PACKED ? 0.0f : initial[c * V + v];
  }
  if (!some) return;
  for (int w = 0; w < wave; ++w)
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float2 q = pairs[w][c * V + v];
      h[v] = chain_apply<PACKED>(q.x, q.y, h[v]);
    }
  if constexpr (NARROW) h[0] = chain_apply<PACKED>(P[0], H[0], h[0]);   // the stretches before this one
  // the state entering token j, for the backward
  auto checkpoint = [&](int j) {
    float* const ck = p.ck + (b * p.nck + (t0 + j) / kGatedCkpt) * p.D + d;
#pragma unroll
    for (int v = 0; v < V; ++v) ck[v] = h[v];
  };
  const TokenRows out = token_rows<T>(p.out, b * p.ob + wave_t0 * p.os, p.os, p.D, subs);
  auto outputs = [&](auto every) {
    constexpr bool PLAIN = decltype(every)::value;
    constexpr bool MARKED = PACKED && !PLAIN;
#pragma unroll
    for (int j = 0; j < kWaveTokens; ++j) {
      if (!PLAIN && !NARROW && j >= n) continue;
      if (j % kGatedCkpt == 0 && p.ck && live && (PLAIN || !NARROW || j < n)) checkpoint(j);
#pragma unroll
      for (int v = 0; v < V; ++v) h[v] = MARKED && (mark(j) & 1) ? u[j][v] : fmaf(a[j][v], h[v], u[j][v]);
      if constexpr (MARKED) {
        if (mark(j) >= 0 && (mark(j) & 2) && p.last && live) {
#pragma unroll
          for (int v = 0; v < V; ++v) p.last[static_cast<int64_t>(mark(j) >> 2) * p.D + d + v] = h[v];
        }
      }
      const bool write = (!MARKED || mark(j) >= 0 || p.zero_outside) && (PLAIN || !NARROW || j < n);
      if (NARROW || write) out.store<kBytes, CACHE>(j, write ? at(p.os) : kNowhere, narrow<T, V>(h));
    }
  };
  if (plain) outputs(std::true_type{});
  else outputs(std::false_type{});
  if constexpr (!PACKED) {
    if (p.last && live && n > 0 && t0 + n == p.L) {
#pragma unroll
      for (int v = 0; v < V; ++v) p.last[b * p.D + d + v] = h[v];
    }
  }
}

struct StepParams {
  float* state; const void* x; const void* ga; const void* gx;
  const float* lam; const int32_t* slots; void* out;
  int64_t ss, xb, gab, gxb, ob, D;
  int batch, nslots;
  float c;
};

// A lane has V channels of a row: 16 bytes of its fp32 state.  256 x 5120 bf16
// take 6 us (21 MB); what is left is the way from the slot to the state.
template <typename T, int V>
__global__ __launch_bounds__(kThreads) void gated_step_kernel(StepParams p) {
  struct alignas(sizeof(T) * V) Vec { T v[V]; };
  struct alignas(4 * V) State { float v[V]; };
  const int lane = threadIdx.x & 63;
  const int64_t d0 = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) * V;
  const bool live = d0 < p.D;
  const int64_t d = live ? d0 : p.D - V;   // lanes past the channels repeat the last ones, and store nothing
  const int row = blockIdx.y;
  int slot = p.slots ? p.slots[row] : row;
  if (slot < 0 || slot >= p.nslots) slot = -1;
  auto at = [&](const void* q, int64_t stride, int64_t b) {
    return *reinterpret_cast<const Vec*>(static_cast<const T*>(q) + b * stride + d);
  };
  Vec x = at(p.x, p.xb, row), ga = at(p.ga, p.gab, row), gx = at(p.gx, p.gxb, row);
  State h{};
  if (slot >= 0) h = *reinterpret_cast<const State*>(p.state + slot * p.ss + d);
  Rate s[V];
#pragma unroll
  for (int v = 0; v < V; ++v) s[v] = Rate(p.c, p.lam[d + v]);
  bool before;
  int next;
  slot_order(p.slots, row, p.batch, slot, lane, before, next);
  if (before && slot >= 0) return;

  for (int b = row;;) {
    Vec o{};
    if (slot >= 0) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float sa = sigmoid_f32(io<T>::load(&ga.v[v])), g = sigmoid_f32(io<T>::load(&gx.v[v]));
        const float a = __builtin_amdgcn_exp2f(s[v].log2a * sa);
        h.v[v] = fmaf(a, h.v[v], __builtin_amdgcn_sqrtf(one_minus_square(a, s[v].u * sa)) * (g * io<T>::load(&x.v[v])));
        io<T>::store(&o.v[v], h.v[v]);
      }
    }
    if (live) *reinterpret_cast<Vec*>(static_cast<T*>(p.out) + b * p.ob + d) = o;
    if (slot < 0) return;
    b = b == row ? next : named_next(p.slots, b, p.batch, slot, lane);
    if (b >= p.batch) break;
    x = at(p.x, p.xb, b);
    ga = at(p.ga, p.gab, b);
    gx = at(p.gx, p.gxb, b);
  }
  if (live) *reinterpret_cast<State*>(p.state + slot * p.ss + d) = h;
}

template <typename T>
void launch_step(const StepParams& p, hipStream_t stream) {
  // 4 channels a lane where every row allows accesses of 4
  constexpr int64_t esz = sizeof(T);
  auto fits = [](const void* q, int64_t stride, int64_t bytes) {
    return reinterpret_cast<uintptr_t>(q) % static_cast<uintptr_t>(4 * bytes) == 0 && stride % 4 == 0;
  };
  const bool four = p.D % 4 == 0 && fits(p.state, p.ss, 4) && fits(p.x, p.xb, esz) && fits(p.ga, p.gab, esz) &&
                    fits(p.gx, p.gxb, esz) && fits(p.out, p.ob, esz);
  const int64_t lanes = four ? p.D / 4 : p.D;
  const dim3 grid(static_cast<unsigned>((lanes + kThreads - 1) / kThreads), static_cast<unsigned>(p.batch));
  if (four) gated_step_kernel<T, 4><<<grid, kThreads, 0, stream>>>(p);
  else gated_step_kernel<T, 1><<<grid, kThreads, 0, stream>>>(p);
}

}  // namespace

namespace {

// A lane takes 4 bytes of a row: one fp32 channel, or two bf16 ones where every
// row allows 4-byte accesses.  Measured at 262,144 x 1536 bf16: 596 us, and 684
// us with one channel (2 bytes) a lane.  Two fp32 channels (8 bytes) cost
// registers and with them a workgroup a compute unit: 128 us against 99 at
// 16,411 x 1536, in the kernel's first form (84 us now).
int channels_per_lane(const ssm_gated_args& a) {
  auto ok = [&](const void* p, int64_t sb, int64_t ss) {
    return reinterpret_cast<uintptr_t>(p) % 4 == 0 && sb % 2 == 0 && ss % 2 == 0;
  };
  return a.io_dtype == SSM_BF16 && a.dim % 2 == 0 && ok(a.x, a.x_batch_stride, a.x_seq_stride) &&
                 ok(a.gate_a, a.gate_a_batch_stride, a.gate_a_seq_stride) &&
                 ok(a.gate_x, a.gate_x_batch_stride, a.gate_x_seq_stride) &&
                 ok(a.out, a.out_batch_stride, a.out_seq_stride)
             ? 2 : 1;
}

GatedPlan plan(const ssm_gated_args& a, int V, int shift) {
  return gated_plan(a.batch, a.seqlen, a.dim, a.cu_seqlens != nullptr, V, kWaveTokens, shift, 0);
}

int shift_of(const ssm_gated_args& a) {
  const int64_t esz = a.io_dtype == SSM_BF16 ? 2 : 4;
  for (int64_t stride : {a.x_seq_stride, a.gate_a_seq_stride, a.gate_x_seq_stride, a.out_seq_stride})
    if (!narrow_fits(a.dim, stride, esz)) return 0;
  return narrow_shift(a.dim);
}

template <typename T, int V, bool NARROW, int CACHE>
void launch_fwd(const FwdParams& p, const GatedPlan& q, bool packed, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(q.tiles * q.cols * p.batch)), block(64 * q.waves);
  if (packed) {
    if (q.words) gated_fwd_kernel<T, V, true, true, NARROW, CACHE><<<grid, block, 0, stream>>>(p);
    else gated_fwd_kernel<T, V, true, false, NARROW, CACHE><<<grid, block, 0, stream>>>(p);
  } else {
    if (q.words) gated_fwd_kernel<T, V, false, true, NARROW, CACHE><<<grid, block, 0, stream>>>(p);
    else gated_fwd_kernel<T, V, false, false, NARROW, CACHE><<<grid, block, 0, stream>>>(p);
  }
}

}  // namespace

// No output has rows 0 elements apart, but one of a single token.
size_t gated_workspace_bytes(const ssm_gated_args& a) {
  return gated_bytes(shift_of(a), a.out_seq_stride != 0, [&](int V, int shift) { return plan(a, V, shift); });
}

hipError_t launch_gated_fwd(const ssm_gated_args& a, hipStream_t stream) {
  const int shift = shift_of(a);
  const int V = shift ? 1 : channels_per_lane(a);
  const GatedPlan q = plan(a, V, shift);
  char* const ws = static_cast<char*>(a.workspace);
  const bool packed = a.cu_seqlens != nullptr;
  const int64_t nseq = packed ? a.nseq : a.batch;
  if (packed || q.words || (a.seqlen == 0 && a.last_state)) {
    const hipError_t e = launch_gated_prep(
        PrepParams{q.words ? reinterpret_cast<uint32_t*>(ws) : nullptr, reinterpret_cast<uint64_t*>(ws + q.words_at), q.words,
                   a.cu_seqlens, packed ? reinterpret_cast<int32_t*>(ws + q.marks_at) : nullptr, a.h0,
                   packed || a.seqlen == 0 ? a.last_state : nullptr, a.seqlen, nseq, a.dim}, stream);
    if (e != hipSuccess || a.seqlen == 0) return e;
  }
  if (a.seqlen == 0) return hipSuccess;
  const FwdParams p{a.x, a.gate_a, a.gate_x, a.lam, a.h0, a.last_state, a.out, a.checkpoints,
                    reinterpret_cast<const int32_t*>(ws + q.marks_at), reinterpret_cast<uint32_t*>(ws),
                    reinterpret_cast<uint64_t*>(ws + q.words_at),
                    a.x_batch_stride, a.x_seq_stride, a.gate_a_batch_stride, a.gate_a_seq_stride,
                    a.gate_x_batch_stride, a.gate_x_seq_stride, a.out_batch_stride, a.out_seq_stride,
                    a.seqlen, a.dim, (a.seqlen + kGatedCkpt - 1) / kGatedCkpt, nseq, static_cast<uint32_t>(a.batch),
                    static_cast<uint32_t>(q.tiles), static_cast<uint32_t>(q.cols), q.shift, a.c, a.zero_outside};
  const int64_t esz = a.io_dtype == SSM_BF16 ? 2 : 4;
  const bool lines = on_lines(a.x, a.x_batch_stride, a.x_seq_stride, esz) &&
                     on_lines(a.gate_a, a.gate_a_batch_stride, a.gate_a_seq_stride, esz) &&
                     on_lines(a.gate_x, a.gate_x_batch_stride, a.gate_x_seq_stride, esz) &&
                     on_lines(a.out, a.out_batch_stride, a.out_seq_stride, esz);
  if (a.io_dtype == SSM_BF16) {
    if (shift) launch_fwd<uint16_t, 1, true, kPlain>(p, q, packed, stream);
    else if (V == 1) launch_fwd<uint16_t, 1, false, kPlain>(p, q, packed, stream);
    else if (lines) launch_fwd<uint16_t, 2, false, kStream>(p, q, packed, stream);
    else launch_fwd<uint16_t, 2, false, kPlain>(p, q, packed, stream);
  } else {
    if (shift) launch_fwd<float, 1, true, kPlain>(p, q, packed, stream);
    else if (lines) launch_fwd<float, 1, false, kStream>(p, q, packed, stream);
    else launch_fwd<float, 1, false, kPlain>(p, q, packed, stream);
  }
  return hipGetLastError();
}

hipError_t launch_gated_step(const ssm_gated_update_args& a, hipStream_t stream) {
  const StepParams p{a.state, a.x, a.gate_a, a.gate_x, a.lam, a.slots, a.out, a.state_slot_stride,
                     a.x_batch_stride, a.gate_a_batch_stride, a.gate_x_batch_stride, a.out_batch_stride, a.dim,
                     static_cast<int>(a.batch), static_cast<int>(a.nslots < 0x7fffffff ? a.nslots : 0x7fffffff), a.c};
  if (a.io_dtype == SSM_BF16) launch_step<uint16_t>(p, stream);
  else launch_step<float>(p, stream);
  return hipGetLastError();
}

}  // namespace ssm
