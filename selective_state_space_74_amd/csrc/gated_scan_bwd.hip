// gated_scan_bwd.hip -- the gradients of the gated linear recurrence for gfx950.
// With e_t the whole derivative on h_t, e_t = dout_t + a_{t+1} e_{t+1} (at a
// sequence's last token + dlast), g = sigma(gate_x), beta = sqrt(1 - a^2),
// v = -log a = s sigma(gate_a):
//   dx      = e beta g
//   dgate_x = e beta x g (1 - g)
//   dv      = e (g x a^2 / beta - a h_{t-1})
//   dgate_a = dv v (1 - sigma(gate_a))
//   dlam    = c sigma(lam) sum_t dv sigma(gate_a)
//   dh0     = a_first e_first
#include "gated_tile.h"

namespace ssm {
namespace {

struct BwdParams {
  const void* x; const void* ga; const void* gx; const void* dout;
  const float* lam; const float* h0; const float* ck; const float* dlast;
  void* dx; void* dga; void* dgx; float* dh0; float* part;
  const int32_t* marks;
  uint32_t* ticket; uint64_t* words;
  int64_t xb, xs, gab, gas, gxb, gxs, dob, dos, dxb, dxs, dgab, dgas, dgxb, dgxs;
  int64_t L, D, nck, nseq;
  uint32_t batch, tiles, cols;
  int shift;   // narrow calls: log2 of the channels
  float c;
};

// A tile as in the forward, taken from the end of the sequence to its start.
// The states before each token come forward from the wavefront's checkpoint,
// so the three gradients' factors of e are ready before e is known; only
// e_t = dout_t + a_{t+1} e_{t+1} waits for the tiles behind.
template <typename T, int V, bool PACKED, bool CHAIN, bool NARROW, int CACHE>
__global__ __launch_bounds__(64 * kMaxWaves, 4) void gated_bwd_kernel(BwdParams p) {
  constexpr int W = 64 * V;
  __shared__ float2 pairs[kMaxWaves][W];
  constexpr int kGroup = chain_group(NARROW);
  __shared__ ChainShared<CHAIN ? W : 1, kGroup> before;
  __shared__ uint32_t taken;
  constexpr int kTok = V == 2 ? kGatedCkpt : kWaveTokens;   // tokens of a wavefront
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
  const uint32_t col = id % p.cols, row = id / p.cols % p.batch, k = id / p.cols / p.batch;
  const uint32_t tile = p.tiles - 1 - k;
  // A wavefront has 16 tokens of 64 channels or 8 of 128 (its registers hold six
  // values for each); in a narrow call each stretch of 2^shift lanes has 16
  // tokens of its own.
  constexpr int kBytes = V * sizeof(T);
  const int shift = NARROW ? p.shift : V == 2 ? 7 : 6;
  const int width = 1 << shift, subs = NARROW ? 64 >> shift : 1;
  const int sub = NARROW ? lane >> shift : 0, c = NARROW ? lane & (width - 1) : lane;
  const int64_t b = row, wave_t0 = (static_cast<int64_t>(tile) * waves + wave) * (kTok * subs);
  const int64_t t0 = wave_t0 + sub * kTok;
  const int n = static_cast<int>(min(static_cast<int64_t>(kTok), max(int64_t{0}, p.L - t0)));
  const bool some = NARROW ? wave_t0 < p.L : n > 0;   // of the wavefront
  const int64_t ch = static_cast<int64_t>(col) * W + c * V;
  const bool live = ch < p.D;
  const int64_t d = live ? ch : p.D - V;   // per-channel values: lanes past the channels repeat the last ones
  // a lane's offset from the wavefront's row j of a tensor
  auto at = [&](int64_t stride) {
    if constexpr (NARROW)
      return live && n > 0 ? static_cast<uint32_t>((c + sub * kTok * stride) * sizeof(T)) : kNowhere;
    else return static_cast<uint32_t>(ch) * static_cast<uint32_t>(sizeof(T));
  };

  Rate s[V];
  float a[kTok][V], fx[kTok][V], fg[kTok][V], fa[kTok][V], fl[kTok][V],
      dout[kTok][V], P[V], Q[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    s[v] = Rate(p.c, p.lam[d + v]);
    P[v] = 1.0f;
    Q[v] = 0.0f;
  }
  // Which of the lane's tokens are a sequence's first or last, or in none (past
  // the end of the row, or of every packed sequence): a bit each.  A token that is
  // so for any lane (the any_ bits, scalars) has a branch over what it asks for.
  // With a path of its own for wavefronts that hold such tokens 30,011 x 1536
  // bf16, packed from 64 sequences, took 190 us, and from one 161 (now 151 and
  // 151): that path's code came from memory, and its registers were spilled.
  uint32_t firsts = 0, lasts = 0, outs = 0;
  auto mark_at = [&](int64_t t) {
    const int32_t m = p.marks[t];
    return m >> 2 < p.nseq ? m : kOutside;
  };
  int32_t marks = 0;
  if constexpr (!PACKED) {
    outs = ~0u << n;
  } else if constexpr (!NARROW) {
    marks = some ? mark_at(t0 + lane % kTok) : kOutside;
    firsts = static_cast<uint32_t>(__ballot(marks & 1));
    outs = static_cast<uint32_t>(__ballot(marks < 0));
    lasts = static_cast<uint32_t>(__ballot(marks & 2)) & ~outs;
  } else {
    // a stretch's lanes have a token's mark each, of 2^shift tokens at a time
    const uint64_t own = (uint64_t{1} << width) - 1;
    for (int i = 0; i < kTok; i += width) {
      const int32_t m = c + i >= kTok ? 0 : c + i < n ? mark_at(t0 + c + i) : kOutside;
      auto bits = [&](bool of) { return static_cast<uint32_t>(__ballot(of) >> (sub << shift) & own) << i; };
      firsts |= bits(m & 1);
      outs |= bits(m < 0);
      lasts |= bits(m >= 0 && (m & 2));
    }
  }
  uint32_t any_firsts = firsts, any_lasts = lasts, any_outs = outs;
  if constexpr (NARROW) {
    any_firsts = any_lasts = any_outs = 0;
    for (int i = 0; i < 64; i += width) {
      any_firsts |= __builtin_amdgcn_readlane(firsts, i);
      any_lasts |= __builtin_amdgcn_readlane(lasts, i);
      any_outs |= __builtin_amdgcn_readlane(outs, i);
    }
  }
  auto bit = [](uint32_t of, int j) { return (of >> j & 1) != 0; };
  // a packed token's row of h0, dlast or dh0; only of tokens in a sequence
  auto seq_row = [&](int j) {
    const int32_t m = NARROW ? mark_at(t0 + j) : __builtin_amdgcn_readlane(marks, j);
    return static_cast<int64_t>(max(m, 0) >> 2) * p.D + d;
  };

  if (some) {
    uint32_t rx[kTok], ra[kTok], rg[kTok], rd[kTok];
    const int64_t left = p.L - wave_t0;
    const TokenRows tx = token_rows<T>(p.x, b * p.xb + wave_t0 * p.xs, p.xs, p.D, subs, left),
                    ta = token_rows<T>(p.ga, b * p.gab + wave_t0 * p.gas, p.gas, p.D, subs, left),
                    tg = token_rows<T>(p.gx, b * p.gxb + wave_t0 * p.gxs, p.gxs, p.D, subs, left),
                    td = token_rows<T>(p.dout, b * p.dob + wave_t0 * p.dos, p.dos, p.D, subs, left);
    float h[V];
#pragma unroll
    for (int v = 0; v < V; ++v)
      h[v] = p.ck[(b * p.nck + (NARROW ? min(t0 / kGatedCkpt, p.nck - 1) : t0 / kGatedCkpt)) * p.D + d + v];
#pragma unroll
    for (int j = 0; j < kTok; ++j) {
      ra[j] = ta.load_within<kBytes, CACHE>(j, at(p.gas));
      rg[j] = tg.load_within<kBytes, CACHE>(j, at(p.gxs));
      rx[j] = tx.load_within<kBytes, CACHE>(j, at(p.xs));
      rd[j] = td.load_within<kBytes, CACHE>(j, at(p.dos));
    }
#pragma unroll
    for (int j = 0; j < kTok; ++j) {
      if (PACKED && bit(any_firsts, j)) [[unlikely]] {
#pragma unroll
        for (int v = 0; v < V; ++v)
          if (bit(firsts, j)) h[v] = !bit(outs, j) && p.h0 ? p.h0[seq_row(j) + v] : 0.0f;
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float x = widen<T, V>(rx[j], v), sa = sigmoid_f32(widen<T, V>(ra[j], v)),
                    g = sigmoid_f32(widen<T, V>(rg[j], v));
        const float aj = __builtin_amdgcn_exp2f(s[v].log2a * sa);
        const float q = one_minus_square(aj, s[v].u * sa);
        // 1 / beta, finite where beta is 0: the factors below have sigma(gate_a) or s,
        // one of which is then 0
        const float inv = __builtin_amdgcn_rsqf(fmaxf(q, 0x1p-126f));
        const float m = q * inv * g, mx = m * x;   // beta g, b
        const float dv = fmaf(g * x, aj * aj * inv, -aj * h[v]) * sa;
        h[v] = fmaf(aj, h[v], mx);
        a[j][v] = aj;
        fx[j][v] = m;
        fg[j][v] = fmaf(-mx, g, mx);
        fl[j][v] = dv;
        fa[j][v] = dv * fmaf(-s[v].s, sa, s[v].s);
        dout[j][v] = widen<T, V>(rd[j], v);
      }
      if (bit(any_outs | any_lasts, j)) [[unlikely]] {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          if (bit(outs, j)) {
            a[j][v] = PACKED ? 0.0f : 1.0f;
            fx[j][v] = fg[j][v] = fl[j][v] = fa[j][v] = dout[j][v] = 0.0f;
          } else if (PACKED && p.dlast && bit(lasts, j)) {   // dlast enters at a sequence's last token
            dout[j][v] += p.dlast[seq_row(j) + v];
          }
        }
      }
    }
#pragma unroll
    for (int j = kTok - 1; j >= 0; --j) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        P[v] *= a[j][v];
        Q[v] = a[j][v] * (dout[j][v] + Q[v]);
      }
      if (PACKED && bit(any_firsts, j)) [[unlikely]] {
#pragma unroll
        for (int v = 0; v < V; ++v) Q[v] = bit(firsts, j) ? 0.0f : Q[v];
      }
    }
    if (PACKED && firsts) {
#pragma unroll
      for (int v = 0; v < V; ++v) P[v] = kCut;
    }
  }

  if constexpr (NARROW) {
    const float2 all = wave_stretches<PACKED, true>(shift, P[0], Q[0]);
    if (sub == 0) pairs[wave][c] = all;
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) pairs[wave][lane * V + v] = make_float2(P[v], Q[v]);
  }
  __syncthreads();
  float e[V];
  if constexpr (CHAIN) {
    // the words of (row, col): tiles, then groups
    const int64_t ngroups = (p.tiles + kGroup - 1) / kGroup;
    uint64_t* const base = p.words + (static_cast<int64_t>(row) * p.cols + col) * (p.tiles + ngroups) * width;
    const Chain chain{base, base + static_cast<int64_t>(p.tiles) * width, width};
    // thread i of the first 2^shift has channel i of the group
    const int64_t di = min(static_cast<int64_t>(col) * W + (threadIdx.x & (width - 1)), p.D - 1);
    const float first = !PACKED && p.dlast ? p.dlast[b * p.D + di] : 0.0f;
    chain_carry<PACKED, W, kGroup, chain_mine(NARROW, V)>(chain, k, p.tiles, pairs, before, shift, first,
                                                             [](int w) { return kMaxWaves - 1 - w; });
#pragma unroll
    for (int v = 0; v < V; ++v) e[v] = before.entering[c * V + v];
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) e[v] = !PACKED && p.dlast ? p.dlast[b * p.D + d + v] : 0.0f;
  }
  float acc[V];
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = 0.0f;
  if (some) {
    for (int w = waves - 1; w > wave; --w)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float2 q = pairs[w][c * V + v];
        e[v] = chain_apply<PACKED>(q.x, q.y, e[v]);
      }
    if constexpr (NARROW) e[0] = chain_apply<PACKED>(P[0], Q[0], e[0]);   // the stretches behind this one
    const int64_t left = p.L - wave_t0;
    const TokenRows dx = token_rows<T>(p.dx, b * p.dxb + wave_t0 * p.dxs, p.dxs, p.D, subs, left),
                    dga = token_rows<T>(p.dga, b * p.dgab + wave_t0 * p.dgas, p.dgas, p.D, subs, left),
                    dgx = token_rows<T>(p.dgx, b * p.dgxb + wave_t0 * p.dgxs, p.dgxs, p.D, subs, left);
#pragma unroll
    for (int j = kTok - 1; j >= 0; --j) {
      // past the end e passes unchanged, be it an infinity; outside packed
      // sequences it is 0, and so are all the products
      if (!PACKED && !NARROW && bit(outs, j)) continue;
      float ox[V], oa[V], og[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float et = dout[j][v] + e[v];
        ox[v] = et * fx[j][v];
        og[v] = et * fg[j][v];
        oa[v] = et * fa[j][v];
        if (PACKED || !NARROW || !bit(any_outs, j)) acc[v] = fmaf(et, fl[j][v], acc[v]);
        else acc[v] = bit(outs, j) ? acc[v] : fmaf(et, fl[j][v], acc[v]);
        e[v] = a[j][v] * et;
      }
      if (PACKED && bit(any_firsts, j)) [[unlikely]] {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          if (!bit(firsts, j)) continue;
          if (p.dh0 && live && !bit(outs, j)) p.dh0[seq_row(j) + v] = e[v];
          e[v] = 0.0f;
        }
      }
      dx.store_within<kBytes, CACHE>(j, at(p.dxs), narrow<T, V>(ox));
      dga.store_within<kBytes, CACHE>(j, at(p.dgas), narrow<T, V>(oa));
      dgx.store_within<kBytes, CACHE>(j, at(p.dgxs), narrow<T, V>(og));
    }
    if constexpr (!PACKED) {
      if (p.dh0 && live && t0 == 0 && n > 0) {
#pragma unroll
        for (int v = 0; v < V; ++v) p.dh0[b * p.D + d + v] = e[v];
      }
    }
  }
  // the tile's part of dlam, wavefront by wavefront
  __syncthreads();
  if constexpr (NARROW) {
    for (int k = 32; k >= width; k >>= 1) acc[0] += __shfl_down(acc[0], k);
    if (sub == 0) pairs[wave][c].x = acc[0];
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) pairs[wave][lane * V + v].x = acc[v];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < width; i += blockDim.x) {
    float sum = 0.0f;
    for (int w = 0; w < waves; ++w) sum += pairs[w][i].x;
    const int64_t di = static_cast<int64_t>(col) * W + i;
    if (di < p.D) p.part[(static_cast<int64_t>(row) * p.tiles + tile) * p.D + di] = sum;
  }
}

// dlam: the tiles' parts, 32 channels a workgroup; 32 threads a channel each
// add every 32nd row, and the 32 sums are added in order.
constexpr int kSumCols = 32, kSumRows = 32;
__global__ __launch_bounds__(kSumCols * kSumRows) void gated_dlam_kernel(const float* part, int64_t rows, int64_t D,
                                                                        const float* lam, float c, float* dlam) {
  __shared__ float sums[kSumRows][kSumCols];
  const int x = threadIdx.x % kSumCols, y = threadIdx.x / kSumCols;
  const int64_t d = static_cast<int64_t>(blockIdx.x) * kSumCols + x;
  float acc = 0.0f;
  if (d < D)
#pragma unroll 8
    for (int64_t i = y; i < rows; i += kSumRows) acc += part[i * D + d];
  sums[y][x] = acc;
  __syncthreads();
  if (y == 0 && d < D) {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kSumRows; ++i) sum += sums[i][x];
    dlam[d] = c * sigmoid_f32(lam[d]) * sum;
  }
}

int shift_of(const ssm_gated_bwd_args& a) {
  const int64_t esz = a.io_dtype == SSM_BF16 ? 2 : 4;
  for (int64_t stride : {a.x_seq_stride, a.gate_a_seq_stride, a.gate_x_seq_stride, a.dout_seq_stride, a.dx_seq_stride,
                         a.dgate_a_seq_stride, a.dgate_x_seq_stride})
    if (!narrow_fits(a.dim, stride, esz)) return 0;
  return narrow_shift(a.dim);
}

// Two channels a lane as in the forward, where a call has at least four groups
// of 128 channels and more than one tile.  A tile is then 64 tokens and not 128:
// with fewer groups the carry through the tiles, about 0.9 tokens a nanosecond
// and group, would bound the call, and a second tile costs a launch.  Forward and
// backward with two against one: 367 against 419 us at 4 x 4096 x 5120 bf16, 250
// against 281 at 2 x 8587 x 2306; with one group, 280 against 200 at 250,095 x 40.
constexpr int64_t kMinGroups = 4;
int channels_per_lane(const ssm_gated_bwd_args& a) {
  auto ok = [&](const void* p, int64_t sb, int64_t ss) {
    return reinterpret_cast<uintptr_t>(p) % 4 == 0 && sb % 2 == 0 && ss % 2 == 0;
  };
  return a.io_dtype == SSM_BF16 && a.dim % 2 == 0 && a.seqlen > kMaxWaves * kWaveTokens &&
                 a.batch * ((a.dim + 127) / 128) >= kMinGroups &&
                 ok(a.x, a.x_batch_stride, a.x_seq_stride) && ok(a.gate_a, a.gate_a_batch_stride, a.gate_a_seq_stride) &&
                 ok(a.gate_x, a.gate_x_batch_stride, a.gate_x_seq_stride) &&
                 ok(a.dout, a.dout_batch_stride, a.dout_seq_stride) && ok(a.dx, a.dx_batch_stride, a.dx_seq_stride) &&
                 ok(a.dgate_a, a.dgate_a_batch_stride, a.dgate_a_seq_stride) &&
                 ok(a.dgate_x, a.dgate_x_batch_stride, a.dgate_x_seq_stride)
             ? 2 : 1;
}

GatedPlan plan(const ssm_gated_bwd_args& a, int V, int shift) {
  return gated_plan(a.batch, a.seqlen, a.dim, a.cu_seqlens != nullptr, V, V == 2 ? kGatedCkpt : kWaveTokens, shift, 1);
}

template <typename T, int V, bool NARROW, int CACHE>
void launch_bwd(const BwdParams& p, const GatedPlan& q, bool packed, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(q.tiles * q.cols * p.batch)), block(64 * q.waves);
  if (V == 2 || q.words) {
    if (packed) gated_bwd_kernel<T, V, true, true, NARROW, CACHE><<<grid, block, 0, stream>>>(p);
    else gated_bwd_kernel<T, V, false, true, NARROW, CACHE><<<grid, block, 0, stream>>>(p);
  } else if constexpr (V == 1) {   // two channels a lane: more than one tile
    if (packed) gated_bwd_kernel<T, V, true, false, NARROW, CACHE><<<grid, block, 0, stream>>>(p);
    else gated_bwd_kernel<T, V, false, false, NARROW, CACHE><<<grid, block, 0, stream>>>(p);
  }
}

template <typename T>
void launch_rows(const ssm_gated_bwd_args& a, const BwdParams& p, const GatedPlan& q, int V, bool packed,
                 hipStream_t stream) {
  constexpr int64_t esz = sizeof(T);
  const bool lines = on_lines(a.x, a.x_batch_stride, a.x_seq_stride, esz) &&
                     on_lines(a.gate_a, a.gate_a_batch_stride, a.gate_a_seq_stride, esz) &&
                     on_lines(a.gate_x, a.gate_x_batch_stride, a.gate_x_seq_stride, esz) &&
                     on_lines(a.dout, a.dout_batch_stride, a.dout_seq_stride, esz) &&
                     on_lines(a.dx, a.dx_batch_stride, a.dx_seq_stride, esz) &&
                     on_lines(a.dgate_a, a.dgate_a_batch_stride, a.dgate_a_seq_stride, esz) &&
                     on_lines(a.dgate_x, a.dgate_x_batch_stride, a.dgate_x_seq_stride, esz);
  if (q.shift) return launch_bwd<T, 1, true, kPlain>(p, q, packed, stream);
  if constexpr (sizeof(T) == 2) {
    if (V == 2) {
      if (lines) return launch_bwd<T, 2, false, kStream>(p, q, packed, stream);
      return launch_bwd<T, 2, false, kPlain>(p, q, packed, stream);
    }
  }
  if (lines) launch_bwd<T, 1, false, kStream>(p, q, packed, stream);
  else launch_bwd<T, 1, false, kPlain>(p, q, packed, stream);
}

}  // namespace

// No output has rows 0 elements apart, but one of a single token.
size_t gated_bwd_workspace_bytes(const ssm_gated_bwd_args& a) {
  return gated_bytes(shift_of(a), a.dx_seq_stride != 0, [&](int V, int shift) { return plan(a, V, shift); });
}

hipError_t launch_gated_bwd(const ssm_gated_bwd_args& a, hipStream_t stream) {
  const int shift = shift_of(a), V = shift ? 1 : channels_per_lane(a);
  const GatedPlan q = plan(a, V, shift);
  char* const ws = static_cast<char*>(a.workspace);
  const bool packed = a.cu_seqlens != nullptr;
  const int64_t nseq = packed ? a.nseq : a.batch;
  if (packed || q.words || (a.seqlen == 0 && a.dh0)) {
    const hipError_t e = launch_gated_prep(
        PrepParams{q.words ? reinterpret_cast<uint32_t*>(ws) : nullptr, reinterpret_cast<uint64_t*>(ws + q.words_at), q.words,
                   a.cu_seqlens, packed ? reinterpret_cast<int32_t*>(ws + q.marks_at) : nullptr, a.dlast,
                   packed || a.seqlen == 0 ? a.dh0 : nullptr, a.seqlen, nseq, a.dim}, stream);
    if (e != hipSuccess) return e;
  }
  const BwdParams p{a.x, a.gate_a, a.gate_x, a.dout, a.lam, a.h0, a.checkpoints, a.dlast,
                    a.dx, a.dgate_a, a.dgate_x, a.dh0, reinterpret_cast<float*>(ws + q.parts_at),
                    reinterpret_cast<const int32_t*>(ws + q.marks_at), reinterpret_cast<uint32_t*>(ws),
                    reinterpret_cast<uint64_t*>(ws + q.words_at),
                    a.x_batch_stride, a.x_seq_stride, a.gate_a_batch_stride, a.gate_a_seq_stride,
                    a.gate_x_batch_stride, a.gate_x_seq_stride, a.dout_batch_stride, a.dout_seq_stride,
                    a.dx_batch_stride, a.dx_seq_stride, a.dgate_a_batch_stride, a.dgate_a_seq_stride,
                    a.dgate_x_batch_stride, a.dgate_x_seq_stride,
                    a.seqlen, a.dim, (a.seqlen + kGatedCkpt - 1) / kGatedCkpt, nseq, static_cast<uint32_t>(a.batch),
                    static_cast<uint32_t>(q.tiles), static_cast<uint32_t>(q.cols), q.shift, a.c};
  const int64_t rows = q.tiles * a.batch;
  if (rows > 0) {
    if (a.io_dtype == SSM_BF16) launch_rows<uint16_t>(a, p, q, V, packed, stream);
    else launch_rows<float>(a, p, q, V, packed, stream);
  }
  gated_dlam_kernel<<<static_cast<unsigned>((a.dim + kSumCols - 1) / kSumCols), kSumCols * kSumRows, 0, stream>>>(
      p.part, rows, a.dim, a.lam, a.c, a.dlam);
  return hipGetLastError();
}

}  // namespace ssm
