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
#include <type_traits>

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
  int64_t L, D, nck;
  uint32_t batch, tiles, cols;
  float c;
};

// A tile as in the forward, taken from the end of the sequence to its start.
// The states before each token come forward from the wavefront's checkpoint,
// so the three gradients' factors of e are ready before e is known; only
// e_t = dout_t + a_{t+1} e_{t+1} waits for the tiles behind.
template <typename T, int V, bool PACKED, bool CHAIN>
__global__ __launch_bounds__(64 * kMaxWaves) void gated_bwd_kernel(BwdParams p) {
  constexpr int W = 64 * V;
  __shared__ float2 pairs[kMaxWaves][W];
  __shared__ float entering[W];
  __shared__ uint32_t taken;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = blockDim.x >> 6;

  uint32_t id = blockIdx.x;
  if constexpr (CHAIN) {
    if (threadIdx.x == 0) taken = atomicAdd(p.ticket, 1u);
    __syncthreads();
    id = __builtin_amdgcn_readfirstlane(taken);
  }
  const uint32_t col = id % p.cols, row = id / p.cols % p.batch, k = id / p.cols / p.batch;
  const uint32_t tile = p.tiles - 1 - k;
  const int64_t b = row, t0 = (static_cast<int64_t>(tile) * waves + wave) * kWaveTokens;
  const int n = static_cast<int>(min(static_cast<int64_t>(kWaveTokens), max(int64_t{0}, p.L - t0)));
  const int64_t col_at = static_cast<int64_t>(col) * W, ch = col_at + lane * V;
  const bool live = ch < p.D;
  const int64_t d = live ? ch : p.D - V;   // lanes past the channels repeat the last ones, and store nothing
  const uint32_t lane_bytes = static_cast<uint32_t>(d - col_at) * sizeof(T);

  // e's factors: dx = e fx, dgate_x = e fg, dgate_a = e fa, dlam's sum e fl
  float s[V], a[kWaveTokens][V], fx[kWaveTokens][V], fg[kWaveTokens][V], fa[kWaveTokens][V], fl[kWaveTokens][V],
      dout[kWaveTokens][V], P[V], Q[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    s[v] = p.c * softplus_f32(p.lam[d + v]);
    P[v] = 1.0f;
    Q[v] = 0.0f;
  }
  int32_t mark[kWaveTokens];
  if constexpr (PACKED) {
#pragma unroll
    for (int j = 0; j < kWaveTokens; ++j) mark[j] = n > 0 ? p.marks[t0 + j] : kOutside;
  }

  auto tokens = [&](auto full) {
    constexpr bool FULL = decltype(full)::value;
    Raw<T, V> rx[kWaveTokens], ra[kWaveTokens], rg[kWaveTokens], rd[kWaveTokens];
    const int64_t xo = b * p.xb + t0 * p.xs + col_at, ao = b * p.gab + t0 * p.gas + col_at,
                  go = b * p.gxb + t0 * p.gxs + col_at, eo = b * p.dob + t0 * p.dos + col_at;
    float h[V];
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = p.ck[(b * p.nck + t0 / kCkpt) * p.D + d + v];
#pragma unroll
    for (int j = 0; j < kWaveTokens; ++j) {
      const int jj = FULL ? j : min(j, n - 1);
      ra[j] = load_raw<T, V>(p.ga, ao + jj * p.gas, lane_bytes);
      rg[j] = load_raw<T, V>(p.gx, go + jj * p.gxs, lane_bytes);
      rx[j] = load_raw<T, V>(p.x, xo + jj * p.xs, lane_bytes);
      rd[j] = load_raw<T, V>(p.dout, eo + jj * p.dos, lane_bytes);
    }
#pragma unroll
    for (int j = 0; j < kWaveTokens; ++j) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if constexpr (PACKED) {
          if (mark[j] & 1)   // first token of its sequence, or in none
            h[v] = mark[j] >= 0 && p.h0 ? p.h0[static_cast<int64_t>(mark[j] >> 2) * p.D + d + v] : 0.0f;
        }
        const float x = widen<T>(rx[j].v[v]), sa = sigmoid_f32(widen<T>(ra[j].v[v])), g = sigmoid_f32(widen<T>(rg[j].v[v]));
        const float r = s[v] * sa;
        const float aj = __builtin_amdgcn_exp2f(-r * kLog2e);
        const float q = one_minus_square(aj, r);
        // below fp32's normal numbers the hardware's root takes q for 0
        const float inv = q >= 0x1p-126f ? __builtin_amdgcn_rsqf(q) : 0.0f;
        const float m = q * inv * g;               // beta g
        const float dv = fmaf(g * x, aj * aj * inv, -aj * h[v]) * sa;
        h[v] = fmaf(aj, h[v], m * x);
        a[j][v] = aj;
        fx[j][v] = m;
        fg[j][v] = m * x * (1.0f - g);
        fl[j][v] = dv;
        fa[j][v] = dv * s[v] * (1.0f - sa);
        dout[j][v] = widen<T>(rd[j].v[v]);
        if constexpr (PACKED) {
          // dlast enters at a sequence's last token
          if (mark[j] >= 0 && (mark[j] & 2) && p.dlast)
            dout[j][v] += p.dlast[static_cast<int64_t>(mark[j] >> 2) * p.D + d + v];
        }
        if constexpr (!FULL) {
          a[j][v] = j < n ? a[j][v] : 1.0f;
          dout[j][v] = j < n ? dout[j][v] : 0.0f;
        }
      }
    }
#pragma unroll
    for (int j = kWaveTokens - 1; j >= 0; --j)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        P[v] *= a[j][v];
        Q[v] = PACKED && (mark[j] & 1) && (FULL || j < n) ? 0.0f : a[j][v] * (dout[j][v] + Q[v]);
      }
  };
  if (n == kWaveTokens) tokens(std::true_type{});
  else if (n > 0) tokens(std::false_type{});
  if constexpr (PACKED) {
    int32_t any = 0;
#pragma unroll
    for (int j = 0; j < kWaveTokens; ++j) any |= mark[j];
    if (n > 0 && (any & 1)) {
#pragma unroll
      for (int v = 0; v < V; ++v) P[v] = kCut;
    }
  }

#pragma unroll
  for (int v = 0; v < V; ++v) pairs[wave][lane * V + v] = make_float2(P[v], Q[v]);
  __syncthreads();
  for (int c = threadIdx.x; c < W; c += blockDim.x) {   // once with eight wavefronts
    const int64_t dc = min(col_at + c, p.D - 1);
    float e = 0.0f;
    if (!PACKED && p.dlast) e = p.dlast[b * p.D + dc];
    if constexpr (CHAIN) {
      float tp = 1.0f, tq = 0.0f;
#pragma unroll
      for (int w = kMaxWaves - 1; w >= 0; --w) {
        const float2 q = pairs[w][c];
        tp = chain_product<PACKED>(tp, q.x);
        tq = chain_apply<PACKED>(q.x, q.y, tq);
      }
      const int64_t ngroups = (p.tiles + kChainGroup - 1) / kChainGroup;
      uint64_t* const base = p.words + (static_cast<int64_t>(row) * p.cols + col) * (p.tiles + ngroups) * W;
      e = chain_carry<PACKED>(Chain{base, base + static_cast<int64_t>(p.tiles) * W, W}, k, p.tiles, c, tp, tq, e);
    }
    entering[c] = e;
  }
  __syncthreads();

  float acc[V];
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = 0.0f;
  if (n > 0) {
    float e[V];
#pragma unroll
    for (int v = 0; v < V; ++v) e[v] = entering[lane * V + v];
    for (int w = waves - 1; w > wave; --w)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float2 q = pairs[w][lane * V + v];
        e[v] = chain_apply<PACKED>(q.x, q.y, e[v]);
      }
    constexpr int64_t esz = sizeof(T);
    char* const dx = static_cast<char*>(p.dx) + (b * p.dxb + t0 * p.dxs + col_at) * esz + lane_bytes;
    char* const dga = static_cast<char*>(p.dga) + (b * p.dgab + t0 * p.dgas + col_at) * esz + lane_bytes;
    char* const dgx = static_cast<char*>(p.dgx) + (b * p.dgxb + t0 * p.dgxs + col_at) * esz + lane_bytes;
#pragma unroll
    for (int j = kWaveTokens - 1; j >= 0; --j) {
      if (j >= n) continue;
      Raw<T, V> ox, oa, og;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const bool in = !PACKED || mark[j] >= 0;
        const float et = dout[j][v] + e[v];
        ox.v[v] = narrow<T>(in ? et * fx[j][v] : 0.0f);
        og.v[v] = narrow<T>(in ? et * fg[j][v] : 0.0f);
        oa.v[v] = narrow<T>(in ? et * fa[j][v] : 0.0f);
        if (in) acc[v] = fmaf(et, fl[j][v], acc[v]);
        e[v] = a[j][v] * et;
        if constexpr (PACKED) {
          if (mark[j] & 1) {
            if (in && p.dh0 && live) p.dh0[static_cast<int64_t>(mark[j] >> 2) * p.D + d + v] = e[v];
            e[v] = 0.0f;
          }
        }
      }
      if (live) {
        *reinterpret_cast<Raw<T, V>*>(dx + j * p.dxs * esz) = ox;
        *reinterpret_cast<Raw<T, V>*>(dga + j * p.dgas * esz) = oa;
        *reinterpret_cast<Raw<T, V>*>(dgx + j * p.dgxs * esz) = og;
      }
    }
    if constexpr (!PACKED) {
      if (p.dh0 && live && t0 == 0) {
#pragma unroll
        for (int v = 0; v < V; ++v) p.dh0[b * p.D + d + v] = e[v];
      }
    }
  }
  // the tile's part of dlam, wavefront by wavefront
  __syncthreads();
#pragma unroll
  for (int v = 0; v < V; ++v) pairs[wave][lane * V + v].x = acc[v];
  __syncthreads();
  for (int c = threadIdx.x; c < W; c += blockDim.x) {
    float sum = 0.0f;
    for (int w = 0; w < waves; ++w) sum += pairs[w][c].x;
    if (col_at + c < p.D) p.part[(static_cast<int64_t>(row) * p.tiles + tile) * p.D + col_at + c] = sum;
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

GatedPlan plan(const ssm_gated_bwd_args& a, int V) {
  return gated_plan(a.batch, a.seqlen, a.dim, a.cu_seqlens != nullptr, V, 1);
}

template <typename T, int V>
void launch_bwd(const BwdParams& p, const GatedPlan& q, bool packed, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(q.tiles * q.cols * p.batch)), block(64 * q.waves);
  if (packed) {
    if (q.words) gated_bwd_kernel<T, V, true, true><<<grid, block, 0, stream>>>(p);
    else gated_bwd_kernel<T, V, true, false><<<grid, block, 0, stream>>>(p);
  } else {
    if (q.words) gated_bwd_kernel<T, V, false, true><<<grid, block, 0, stream>>>(p);
    else gated_bwd_kernel<T, V, false, false><<<grid, block, 0, stream>>>(p);
  }
}

}  // namespace

size_t gated_bwd_workspace_bytes(const ssm_gated_bwd_args& a) { return static_cast<size_t>(plan(a, 1).bytes); }

hipError_t launch_gated_bwd(const ssm_gated_bwd_args& a, hipStream_t stream) {
  constexpr int V = 1;
  const GatedPlan q = plan(a, V);
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
                    a.seqlen, a.dim, (a.seqlen + kCkpt - 1) / kCkpt, static_cast<uint32_t>(a.batch),
                    static_cast<uint32_t>(q.tiles), static_cast<uint32_t>(q.cols), a.c};
  const int64_t rows = q.tiles * a.batch;
  if (rows > 0) {
    if (a.io_dtype == SSM_BF16) launch_bwd<uint16_t, V>(p, q, packed, stream);
    else launch_bwd<float, V>(p, q, packed, stream);
  }
  gated_dlam_kernel<<<static_cast<unsigned>((a.dim + kSumCols - 1) / kSumCols), kSumCols * kSumRows, 0, stream>>>(
      p.part, rows, a.dim, a.lam, a.c, a.dlam);
  return hipGetLastError();
}

}  // namespace ssm
