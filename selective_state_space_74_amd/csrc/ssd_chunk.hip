// ssd_chunk.hip -- the states of chunks, and the outputs from them: the
// chunk-parallel SSD prefill over packed sequences, gfx950 (see ssd_chunk.h).
#include <algorithm>

#include "ssd_chunk.h"

namespace ssm {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

// ---- the chunks of packed sequences --------------------------------------------

// Workgroup 0: each sequence's count of chunks, their sums, and the chunks.  The
// bounds are held to the row and the chunks to nc, whatever the bounds say.  The
// other workgroups clear rows of tokens outside every sequence.
constexpr int kTableThreads = 1024;
__global__ __launch_bounds__(kTableThreads) void chunk_table_kernel(const int32_t* cu, int64_t L, int64_t nseq, int nc,
                                                                    ChunkEntry* table, int32_t* seq_chunk, OutsideRows rows) {
  const int tid = threadIdx.x;
  auto bound = [&](int64_t i) { return min(max(int64_t{cu[i]}, int64_t{0}), L); };
  if (blockIdx.x > 0) {
    const int64_t lo = bound(0), hi = max(bound(nseq), lo), n = lo + (L - hi);
    for (int64_t i = blockIdx.x - 1; i < n; i += gridDim.x - 1) {
      const int64_t t = i < lo ? i : hi + (i - lo);
      for (int k = 0; k < rows.n; ++k) {
        const OutsideRows::Tensor& r = rows.t[k];
        for (int64_t h = 0; h < r.heads; ++h) {
          uint16_t* const q = reinterpret_cast<uint16_t*>(static_cast<char*>(r.p) + t * r.stride + h * r.head_stride);
          for (int64_t j = tid; j < r.bytes / 2; j += kTableThreads) q[j] = 0;
        }
      }
    }
    return;
  }
  __shared__ int32_t part[kTableThreads / 64];
  int64_t before = 0;   // chunks of the sequences done
  for (int64_t base = 0; base < nseq; base += kTableThreads) {
    const int64_t k = base + tid;
    int count = 0;
    if (k < nseq) {
      const int64_t lo = bound(k), hi = max(bound(k + 1), lo);
      count = static_cast<int>((hi - lo + kQ - 1) / kQ);
    }
    int sum = count;   // inclusive, over the wavefront and then the workgroup
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(sum, d, 64);
      if (tid % 64 >= d) sum += v;
    }
    if (tid % 64 == 63) part[tid / 64] = sum;
    __syncthreads();
    int64_t at = before + sum - count;
    int64_t all = 0;
    for (int w = 0; w < kTableThreads / 64; ++w) {
      if (w < tid / 64) at += part[w];
      all += part[w];
    }
    if (k < nseq) seq_chunk[k] = static_cast<int32_t>(min(at, int64_t{nc}));
    before += all;
    __syncthreads();
  }
  before = min(before, int64_t{nc});
  if (tid == 0) seq_chunk[nseq] = static_cast<int32_t>(before);
  __syncthreads();   // this workgroup's own stores to seq_chunk are read below
  for (int c = tid; c < nc; c += kTableThreads) {
    ChunkEntry e{0, 0};
    if (c < before) {
      int64_t a = 0, b = nseq;   // the last sequence that begins at or before chunk c
      while (b - a > 1) {
        const int64_t m = (a + b) / 2;
        if (seq_chunk[m] <= c) a = m; else b = m;
      }
      const int64_t lo = bound(a), hi = max(bound(a + 1), lo);
      const int64_t t0 = lo + int64_t{c - seq_chunk[a]} * kQ;
      e.t0 = static_cast<int32_t>(min(t0, L));
      e.len = static_cast<int32_t>(max(min(hi - t0, int64_t{kQ}), int64_t{0}));
    }
    table[c] = e;
  }
}

// ---- what a chunk adds to the state ------------------------------------------------

// Rows of x (or of dout, gated) times their weights into LDS, for bf16 in three parts
// (kParts arrays, one behind the other): the products are then of all 24 bits, and the last
// state and dh0 as exact as fp32 sums are.  With two parts, 16 bits, they were 2e-6 off.
template <typename T> constexpr int kParts = sizeof(T) == 2 ? 3 : 1;
template <typename T, bool kGate, int kN, typename W>
__device__ __forceinline__ void put_weighted(typename Lds<T>::E* sX, int pitch, const Pieces<T, kPB, kN>& x, [[maybe_unused]] const Pieces<T, kPB, kN>& z, W&& weight,
                                             int tid) {
  using Tokens = Pieces<T, kPB, kN>;
#pragma unroll
  for (int j = 0; j < Tokens::kN; ++j) {
    const int r = tid / Tokens::kPer + j * Tokens::kStep, at = r * pitch + tid % Tokens::kPer * kPiece<T>;
    const float w = weight(r);
    uint32_t s[kPiece<T>];
    [[maybe_unused]] uint32_t mid[kPiece<T>], rest[kPiece<T>];
#pragma unroll
    for (int e = 0; e < kPiece<T>; ++e) {
      float f = piece_f32<T>(x.v[j], e) * w;
      if constexpr (kGate) f *= silu_f32(piece_f32<T>(z.v[j], e));
      s[e] = __float_as_uint(f);
      if constexpr (sizeof(T) == 2) {   // 8 bits of the significand each, cut off and not rounded: every difference is exact
        f -= __uint_as_float(s[e] & 0xffff0000u);
        mid[e] = __float_as_uint(f);
        rest[e] = __float_as_uint(f - __uint_as_float(mid[e] & 0xffff0000u));
      }
    }
    if constexpr (sizeof(T) == 2) {
      auto put = [&](int part, const uint32_t (&v)[kPiece<T>]) {
        *reinterpret_cast<v4u*>(sX + part * kQ * pitch + at) = v4u{highs(v[0], v[1]), highs(v[2], v[3]), highs(v[4], v[5]), highs(v[6], v[7])};
      };
      put(0, s);
      put(1, mid);
      put(2, rest);
    } else {
      *reinterpret_cast<v4u*>(sX + at) = v4u{s[0], s[1], s[2], s[3]};
    }
  }
}

// A tile of those rows, 16 tokens by 16 channels, and its product with B's (C's).
template <typename T>
struct WeightedFrag {
  typename Frag<T>::V v[kParts<T>];
  __device__ __forceinline__ WeightedFrag(const typename Lds<T>::E* sX, int pitch, int k0, int c0, int lr, int lq) {
#pragma unroll
    for (int i = 0; i < kParts<T>; ++i) v[i] = frag_down<T>(sX + i * kQ * pitch, pitch, k0, c0, lr, lq);
  }
  __device__ __forceinline__ v4f times(const typename Frag<T>::V& mf, v4f acc) const {
    if constexpr (sizeof(T) == 2) return mma32(mf, mf, v[0], v[1], mma32(mf, mf, v[2], typename Frag<T>::V{}, acc));
    else return mma16<T>(mf, v[0], acc);
  }
};

// Workgroup: (chunk, heads of one group, direction).  B (C backward) of the chunk
// is staged once; then for each head the rows x_s (dy_t) times their weight.  A
// wavefront owns 16 channels of the state (fewer channels: a share of its columns).
// Bound by memory: the states written are 4 N bytes for 2 x (64 tokens) bytes of x
// read; 16,411 packed x 32 x 64 x 64 bf16, 23 sequences: 57 us, 3.7 TB/s.
template <typename T, int NMAX, bool kVec>
__global__ __launch_bounds__(kThreads) void ssd_states_kernel(ChunkParams p, int grid) {
  using E = typename Lds<T>::E;
  constexpr int kPad = 16 / sizeof(E), NP = NMAX + kPad, XP = kPB + kPad, NT = NMAX / 16;
  __shared__ __align__(16) E sM[kQ * NP];
  __shared__ __align__(16) E sX[kParts<T> * kQ * XP];
  __shared__ float sW[kMostHeads][kQ];
  const int tid = threadIdx.x, lane = tid & 63, lr = lane & 15, lq = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const bool back = blockIdx.y != 0;
  const int id = static_cast<int>(xcd_order(blockIdx.x, grid));
  const int c = id / (p.G * p.blocks), g = id / p.blocks % p.G, h0 = g * p.per_group + id % p.blocks * p.hb;
  const int heads = min(p.hb, (g + 1) * p.per_group - h0);
  const Chunk k = chunk_of(p, c);
  if (k.len == 0) return;

  for (int i = wave; i < heads; i += kWaves) {
    const Steps s = steps_of<T>(p, k, h0 + i, lane);
    const double end = lane_value(s.la, 63);
    sW[i][lane] = back ? decay_of(s.la) : decay_of(end - s.la) * s.delta;
    if (!back && lane == 0) p.lam[static_cast<int64_t>(c) * p.H + h0 + i] = decay_of(end);
  }
  const TokenTensor& m = back ? p.C : p.B;
  stage_rows<T, NMAX, kThreads, kVec>(sM, NP, rows_of<T>(m, k, g, 0, p.N), tid, p.bc_vec);
  __syncthreads();

  const TokenTensor& x = back ? p.dout : p.x;
  const bool gate = back && p.z.p;
  const int nt = (p.N + 15) / 16, kb = (k.len + 15) / 16;
  using Tokens = Pieces<T, kPB, kThreads>;
  Tokens xv, zv;
  auto load = [&](int i, int p0) {
    xv.template load<kVec>(rows_of<T>(x, k, h0 + i, p0, p.P), tid);
    if (gate) zv.template load<kVec>(rows_of<T>(p.z, k, h0 + i, p0, p.P), tid);
  };
  load(0, 0);
  for (int i = 0; i < heads; ++i) {
    for (int p0 = 0; p0 < p.P; p0 += kPB) {
      const int cols = p.P - p0;
      auto weight = [&](int r) { return sW[i][r]; };
      if (gate) put_weighted<T, true>(sX, XP, xv, zv, weight, tid);
      else put_weighted<T, false>(sX, XP, xv, zv, weight, tid);
      __syncthreads();
      // the next pass's loads are under way while this one is computed
      if (p0 + kPB < p.P) load(i, p0 + kPB);
      else if (i + 1 < heads) load(i + 1, 0);
      // channels' tiles of this pass (1, 2 or 4) and the wavefronts that share one
      const int pts = min(kPB, cols) > 32 ? 4 : min(kPB, cols) > 16 ? 2 : 1;
      const int pt = wave % pts, first = wave / pts, step = kWaves / pts;
      v4f acc[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) acc[n] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
      for (int q = 0; q < kb; ++q) {
        const WeightedFrag<T> xf(sX, XP, 16 * q, 16 * pt, lr, lq);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if (n % step != first || n >= nt) continue;
          acc[n] = xf.times(frag_down<T>(sM, NP, 16 * q, 16 * n, lr, lq), acc[n]);
        }
      }
      // lane: channel 16 pt + lr, states 16 n + 4 lq ..
      const int pp = p0 + 16 * pt + lr;
      if (pp < p.P) {
        float* const to = (back ? p.dstate : p.state) +
                          ((static_cast<int64_t>(c) * p.H + h0 + i) * p.P + pp) * p.N;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if (n % step != first) continue;
          const int s0 = 16 * n + 4 * lq;
          if constexpr (kVec) {
            if (s0 < p.N) *reinterpret_cast<v4f*>(to + s0) = acc[n];
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (s0 + e < p.N) to[s0 + e] = acc[n][e];
          }
        }
      }
      __syncthreads();
    }
  }
}

// ---- the carry from chunk to chunk -----------------------------------------------

struct CarryParams {
  const int32_t* seq_chunk;
  const float* lam;
  float* state[2];
  const float* from[2];
  float* to[2];
  int64_t nseq, elems;
  int per_row, H, head_elems;
};

// A lane has V values of a sequence's state and goes along its chunks (blockIdx.z
// = 1: from the end), kAhead chunks' loads in flight; in place of what a chunk adds
// it leaves the state that enters it.  Bound by memory, as fast as a copy: 283 MB of the same case in 52 us, 5.4 TB/s.
template <int V>
__global__ __launch_bounds__(kThreads) void ssd_carry_kernel(CarryParams p) {
  constexpr int kAhead = 8;
  struct alignas(4 * V) Pack { float e[V]; };
  const int64_t e0 = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) * V;
  if (e0 >= p.elems) return;
  const int dir = blockIdx.z;
  const int head = static_cast<int>(e0 / p.head_elems);   // V values are of one head
  for (int64_t s = blockIdx.y; s < p.nseq; s += gridDim.y) {
    const int lo = p.seq_chunk ? p.seq_chunk[s] : static_cast<int>(s) * p.per_row;
    const int hi = p.seq_chunk ? p.seq_chunk[s + 1] : lo + p.per_row;
    float h[V];
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = p.from[dir] ? p.from[dir][s * p.elems + e0 + v] : 0.0f;
    float* const base = p.state[dir] + e0;
    for (int c = 0; c < hi - lo; c += kAhead) {
      Pack add[kAhead];
      float lam[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (c + i >= hi - lo) break;
        const int at = dir ? hi - 1 - c - i : lo + c + i;
        add[i] = *reinterpret_cast<const Pack*>(base + at * p.elems);
        lam[i] = p.lam[static_cast<int64_t>(at) * p.H + head];
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (c + i >= hi - lo) break;
        const int at = dir ? hi - 1 - c - i : lo + c + i;
        Pack in;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          in.e[v] = h[v];
          h[v] = fmaf(lam[i], h[v], add[i].e[v]);
        }
        *reinterpret_cast<Pack*>(base + at * p.elems) = in;
      }
    }
    if (p.to[dir]) {
#pragma unroll
      for (int v = 0; v < V; ++v) p.to[dir][s * p.elems + e0 + v] = h[v];
    }
  }
}

// ---- both at once, where whole sequences keep the machine busy -------------------------

constexpr int kWalkThreads = 512;

struct WalkParams {
  const float* from[2];
  float* to[2];
  int split;   // workgroups of a head, up to 64 channels each
};

// Workgroup: (batch row, head, 64 of its channels, direction).  It goes along the
// row's chunks with the state in registers, so that the states are written once and
// not read and written again by the carry: loads are two chunks ahead, LDS in two
// halves makes do with one barrier a chunk.  Bound by the chain of chunks, 3.8 us
// each: 8 x 2048 x 32 x 64 x 64 bf16, both directions, 122 us, 3.4 TB/s.
template <typename T, int NMAX>
__global__ __launch_bounds__(kWalkThreads) void ssd_walk_kernel(ChunkParams p, WalkParams q) {
  using E = typename Lds<T>::E;
  constexpr int kPad = 16 / sizeof(E), NP = NMAX + kPad, XP = kPB + kPad, NT = NMAX / 16;
  constexpr int kHalf = kQ * NP + kParts<T> * kQ * XP;
  __shared__ __align__(16) E lds[2 * kHalf];
  const int tid = threadIdx.x, lane = tid & 63, lr = lane & 15, lq = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int dir = blockIdx.y, h = static_cast<int>(blockIdx.x / q.split) % p.H;
  const int b = static_cast<int>(blockIdx.x / q.split) / p.H, p0 = static_cast<int>(blockIdx.x % q.split) * kPB;
  const int last = min(p.P, p0 + kPB);   // channels p0 .. last - 1
  const bool gate = dir && p.z.p;
  const TokenTensor& x = dir ? p.dout : p.x;
  const TokenTensor& m = dir ? p.C : p.B;
  float* const state = dir ? p.dstate : p.state;
  const int g = h / p.per_group, nt = (p.N + 15) / 16;
  const StepHead steps = step_head(p, h);
  // channels' tiles (1, 2 or 4) and the wavefronts that share one, at least two: tiles
  // of states first, first + step ..; lane: channel 16 pt + lr, states 16 n + 4 lq ..
  const int pts = last - p0 > 32 ? 4 : last - p0 > 16 ? 2 : 1;
  const int pt = wave % pts, first = wave / pts, step = kWalkThreads / 64 / pts;
  constexpr int kMost = NT / 2;
  const int pp = p0 + 16 * pt + lr;
  // the lane's place in a head's state, or none
  auto place = [&](int j, int e) {
    const int s = 16 * (first + step * j) + 4 * lq + e;
    return pp < last && s < p.N ? (pp * p.N + s) * 4u : kNowhere;
  };
  auto head_of = [&](const float* t) {   // h0 and the like
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(t + (static_cast<int64_t>(b) * p.H + h) * p.P * p.N), 0, p.P * p.N * 4,
                                             kRsrcWord3);
  };

  v4f acc[kMost];
#pragma unroll
  for (int j = 0; j < kMost; ++j) {
    acc[j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    if (q.from[dir]) {
      const __amdgpu_buffer_rsrc_t from = head_of(q.from[dir]);
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[j][e] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(from, place(j, e), 0, 0));
    }
  }
  // what a chunk needs, loaded two chunks ahead; past the row its last chunk again.
  // Loads and stores are issued whether or not a lane has any (their offsets then
  // lie nowhere): a wait can then count them and leave the latest in flight.
  struct Ahead {
    Pieces<T, kPB, kWalkThreads> x, z;
    Pieces<T, NMAX, kWalkThreads> m;
    uint32_t raw;   // the lane's step, before its bias
    int len;
  } ahead[2];
  auto load = [&](int i, Ahead& a) {
    i = min(i, p.per_row - 1);
    const int t0 = (dir ? p.per_row - 1 - i : i) * kQ;
    const Chunk k{b, t0, min(kQ, p.L - t0)};
    a.len = k.len;
    const T* const dt = static_cast<const T*>(p.dt) + k.b * p.dtb + k.t0 * p.dts + h;
    a.raw = Elem<T>::load(__builtin_amdgcn_make_buffer_rsrc(const_cast<T*>(dt), 0, 0x7fffffff, kRsrcWord3),
                          lane < k.len ? lane * static_cast<uint32_t>(p.dts) * static_cast<uint32_t>(sizeof(T)) : kNowhere);
    a.x.template load<true>(rows_of<T>(x, k, h, p0, last), tid);
    if (gate) a.z.template load<true>(rows_of<T>(p.z, k, h, p0, last), tid);
    a.m.template load<true>(rows_of<T>(m, k, g, 0, p.N), tid);
  };
  auto chunk = [&](int i, Ahead& a) {
    E* const sM = lds + (i % 2) * kHalf;
    E* const sX = sM + kQ * NP;
    const int len = a.len;
    const Steps s = steps_from(steps, Elem<T>::f32(a.raw), len, lane);
    const double end = lane_value(s.la, 63);
    const float w = dir ? decay_of(s.la) : decay_of(end - s.la) * s.delta;
    a.m.put(sM, NP, tid);
    auto weight = [&](int r) { return __shfl(w, r, 64); };
    if (gate) put_weighted<T, true>(sX, XP, a.x, a.z, weight, tid);
    else put_weighted<T, false>(sX, XP, a.x, a.z, weight, tid);
    __syncthreads();
    load(i + 2, a);
    // the state that enters the chunk
    const int64_t c = static_cast<int64_t>(b) * p.per_row + (dir ? p.per_row - 1 - i : i);
    const __amdgpu_buffer_rsrc_t to =
        __builtin_amdgcn_make_buffer_rsrc(state + (c * p.H + h) * p.P * p.N, 0, p.P * p.N * 4, kRsrcWord3);
    const float through = decay_of(end);
#pragma unroll
    for (int j = 0; j < kMost; ++j) {
      v4u v;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = __float_as_uint(acc[j][e]);
      __builtin_amdgcn_raw_buffer_store_b128(v, to, place(j, 0), 0, 0);
      acc[j] *= through;
    }
    const int kb = (len + 15) / 16;
#pragma unroll
    for (int t = 0; t < kQ / 16; ++t) {
      if (t >= kb) continue;
      const WeightedFrag<T> xf(sX, XP, 16 * t, 16 * pt, lr, lq);
#pragma unroll
      for (int j = 0; j < kMost; ++j) {
        const int n = first + step * j;
        if (n >= nt) continue;
        acc[j] = xf.times(frag_down<T>(sM, NP, 16 * t, 16 * n, lr, lq), acc[j]);
      }
    }
  };
  load(0, ahead[0]);
  load(1, ahead[1]);
  for (int i = 0; i < p.per_row; i += 2) {
    chunk(i, ahead[0]);
    if (i + 1 < p.per_row) chunk(i + 1, ahead[1]);
  }
  if (q.to[dir]) {
    const __amdgpu_buffer_rsrc_t to = head_of(q.to[dir]);
#pragma unroll
    for (int j = 0; j < kMost; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(acc[j][e]), to, place(j, e), 0, 0);
  }
}

// ---- outputs ------------------------------------------------------------------------

// Workgroup: (chunk, heads of one group); two of its 8 wavefronts share 16 of the
// tokens, each with every other 16 channels of a head.  The scores C_t . B_s of the
// chunk are computed once and stay in registers for all heads; the next heads' loads
// are under way while one is computed.  Tiles lie so that a lane has four channels
// of one token.  Bound by the latency of a pass (stage, barrier, products, barrier;
// 46% of a wavefront's cycles are waits) with 16 wavefronts a compute unit: the case
// above, gated, in 106 us, 3.3 TB/s (102 while the carry left the states split, which
// held them to 16 bits for the gradients too).  Loads one pass ahead and not two were 9 us
// slower, four wavefronts, each with all channels of 16 tokens, 67.
// kDz: the gate's gradient dout y silu'(z) in place of the output.
// Two workgroups a compute unit (128 registers); rows by elements then keep up to 24
// registers in scratch, which costs less than one workgroup without any (5000 packed x 32
// x 33 x 128 bf16 167 us, 174; x 64 fp32 118, 135), but for the gate's gradient with 128
// states (79 registers: gradients of 4 x 1000 x 32 x 33 x 128 bf16 369, 347).
constexpr int kOutThreads = 512;

// Four values of a row from column c on (of `cols`), as they lie.
template <typename T, bool kVec>
struct Four {
  uint32_t w[sizeof(T)];
  __device__ __forceinline__ void load(const Rows64& r, int row, int c) {
    const uint32_t off = row * r.stride + c * static_cast<uint32_t>(sizeof(T));
    if constexpr (!kVec) {
      uint32_t v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        v[e] = Elem<T>::load(r.r, row < r.len && c + e < r.cols ? off + e * static_cast<uint32_t>(sizeof(T)) : kNowhere);
#pragma unroll
      for (int e = 0; e < static_cast<int>(sizeof(T)); ++e) w[e] = sizeof(T) == 4 ? v[e] : v[2 * e % 4] | v[(2 * e + 1) % 4] << 16;
    } else {
      const uint32_t at = ((row < r.len) & (c < r.cols)) ? off : kNowhere;
      if constexpr (sizeof(T) == 4) __builtin_memcpy(w, &static_cast<const v4u&>(__builtin_amdgcn_raw_buffer_load_b128(r.r, at, 0, 0)), 16);
      else __builtin_memcpy(w, &static_cast<const v2u&>(__builtin_amdgcn_raw_buffer_load_b64(r.r, at, 0, 0)), 8);
    }
  }
  __device__ __forceinline__ void store(const Rows64& r, int row, int c) const {
    const uint32_t off = row * r.stride + c * static_cast<uint32_t>(sizeof(T));
    if constexpr (!kVec) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        Elem<T>::store(r.r, row < r.len && c + e < r.cols ? off + e * static_cast<uint32_t>(sizeof(T)) : kNowhere, (*this)[e]);
    } else {
      const uint32_t at = ((row < r.len) & (c < r.cols)) ? off : kNowhere;
      if constexpr (sizeof(T) == 4) __builtin_amdgcn_raw_buffer_store_b128(v4u{w[0], w[1], w[2], w[3]}, r.r, at, 0, 0);
      else __builtin_amdgcn_raw_buffer_store_b64(v2u{w[0], w[1]}, r.r, at, 0, 0);
    }
  }
  __device__ __forceinline__ float operator[](int e) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[e]);
    else return __uint_as_float(e % 2 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
  }
  __device__ __forceinline__ void set(const float (&v)[4]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = __float_as_uint(v[e]);
    } else {
      w[0] = pack_bf16x2(v[0], v[1]);
      w[1] = pack_bf16x2(v[2], v[3]);
    }
  }
};

template <typename T, int NMAX, bool kDz, bool kVec>
__global__ __launch_bounds__(kOutThreads, kDz && !kVec && NMAX == 128 ? 2 : 4) void ssd_outputs_kernel(ChunkParams p, ChunkOut o, int grid) {
  using E = typename Lds<T>::E;
  constexpr bool kBF = sizeof(T) == 2;
  constexpr int kPad = 16 / sizeof(E), NP = NMAX + kPad, XP = kPB + kPad, NT = NMAX / 16, QB = kQ / 16;
  constexpr int kScores = 2 * kQ * NP, kHead = kQ * XP + (kBF ? 2 : 1) * kPB * NP;
  struct Shared {
    float la[kMostHeads][kQ], lr[kMostHeads][kQ], dl[kMostHeads][kQ], D[kMostHeads];
    alignas(16) E tiles[kScores > kHead ? kScores : kHead];
  };
  __shared__ __align__(16) Shared sh;
  const int tid = threadIdx.x, lane = tid & 63, lr = lane & 15, lq = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), tok = wave % QB, half = wave / QB;
  const int id = static_cast<int>(xcd_order(blockIdx.x, grid));
  const int c = id / (p.G * p.blocks), g = id / p.blocks % p.G, h0 = g * p.per_group + id % p.blocks * p.hb;
  const int heads = min(p.hb, (g + 1) * p.per_group - h0);
  const Chunk k = chunk_of(p, c);
  if (k.len == 0) return;

  for (int i = wave; i < heads; i += kOutThreads / 64) {
    const Steps s = steps_of<T>(p, k, h0 + i, lane);
    sh.dl[i][lane] = s.delta;
    const TwoFloats la = two_floats(s.la);
    sh.la[i][lane] = la.v;
    sh.lr[i][lane] = la.rest;
    if (lane == 0) sh.D[i] = p.D ? p.D[h0 + i] : 0.0f;
  }
  E* const sB = sh.tiles;
  E* const sC = sh.tiles + kQ * NP;
  stage_rows<T, NMAX, kOutThreads, kVec>(sB, NP, rows_of<T>(p.B, k, g, 0, p.N), tid, p.bc_vec);
  stage_rows<T, NMAX, kOutThreads, kVec>(sC, NP, rows_of<T>(p.C, k, g, 0, p.N), tid, p.bc_vec);
  __syncthreads();
  // scores[sb]: lane holds s = 16 sb + 4 lq + e, t = own
  const int own = 16 * tok + lr;
  v4f scores[QB];
  typename Frag<T>::V cf[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) cf[n] = frag_along<T>(sC, NP, 16 * tok, 16 * n, lr, lq);
#pragma unroll
  for (int sb = 0; sb < QB; ++sb) {
    scores[sb] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    if (sb > tok) continue;
    if constexpr (kBF) {
#pragma unroll
      for (int n = 0; n < NT; n += 2)
        scores[sb] = mma32(frag_along<T>(sB, NP, 16 * sb, 16 * n, lr, lq), frag_along<T>(sB, NP, 16 * sb, 16 * n + 16, lr, lq),
                           cf[n], cf[n + 1], scores[sb]);
    } else {
#pragma unroll
      for (int n = 0; n < NT; ++n) scores[sb] = mma16<T>(frag_along<T>(sB, NP, 16 * sb, 16 * n, lr, lq), cf[n], scores[sb]);
    }
  }
  __syncthreads();   // the scores' operands make room for the heads'

  E* const sX = sh.tiles;
  E* const sH = sh.tiles + kQ * XP;
  [[maybe_unused]] E* const sHL = sH + kPB * NP;
  const int nt = (p.N + 15) / 16;
  // what a pass (64 channels of a head) needs, loaded kDepth passes ahead.  Loads and
  // stores are issued whether or not there is anything to take or leave (their offsets
  // then lie nowhere), so that a wait can count them and leave the later ones in flight.
  // Two ahead where 128 registers hold them: not for rows by elements (5000 packed x 16
  // x 33 x 64 bf16: whole call 111 us for 77) nor with dout besides (104 and 108 us at
  // 8 x 2048 x 32 x 64 x 64).
  constexpr int kDepth = kBF && NMAX == 64 && kVec && !kDz ? 2 : 1;
  constexpr int kTiles = kPB / 32;
  const int of_head = (p.P + kPB - 1) / kPB, passes = heads * of_head;
  struct Ahead {
    Pieces<T, kPB, kOutThreads> x;
    StatePieces<T, NMAX, kOutThreads> s;
    Four<T, kVec> z[kTiles], up[kDz ? kTiles : 1];
  } ahead[kDepth];
  const bool gated = p.z.p != nullptr;
  const TokenTensor zt = gated ? p.z : p.x;
  auto load = [&](int s, Ahead& a) {
    const bool any = s < passes;
    s = any ? s : 0;
    const int h = h0 + s / of_head, p0 = s % of_head * kPB;
    const Rows64 x = rows_of<T>(p.x, k, h, p0, p.P, any), z = rows_of<T>(zt, k, h, p0, p.P, any && gated);
    const StateRows st = state_rows(p.state, ((static_cast<int64_t>(c) * p.H + h) * p.P + p0) * p.N, any ? min(kPB, p.P - p0) : 0, p.N);
    a.x.template load<kVec>(x, tid);
    a.s.template load<kVec>(st, tid);
#pragma unroll
    for (int j = 0; j < kTiles; ++j) a.z[j].load(z, own, 16 * (2 * j + half) + 4 * lq);
    if constexpr (kDz) {
      const Rows64 up = rows_of<T>(p.dout, k, h, p0, p.P, any);
#pragma unroll
      for (int j = 0; j < kTiles; ++j) a.up[j].load(up, own, 16 * (2 * j + half) + 4 * lq);
    }
  };
  typename Frag<T>::V mf[QB];
  float ea = 0.0f, Dh = 0.0f;
  auto pass = [&](int s, Ahead& a) {
    const int i = s / of_head, h = h0 + i, p0 = s % of_head * kPB, cols = s < passes ? p.P - p0 : 0;
    if (p0 == 0 && cols > 0) {
      // weighted scores of the head, as operands; those above the diagonal are zero
      const float la_t = sh.la[i][own], lr_t = sh.lr[i][own];
#pragma unroll
      for (int sb = 0; sb < QB; ++sb) {
        mf[sb] = tofrag<T>(0.0f, 0.0f, 0.0f, 0.0f);
        if (sb > tok) continue;
        const v4f la_s = *reinterpret_cast<const v4f*>(&sh.la[i][16 * sb + 4 * lq]);
        const v4f lr_s = *reinterpret_cast<const v4f*>(&sh.lr[i][16 * sb + 4 * lq]);
        const v4f dl_s = *reinterpret_cast<const v4f*>(&sh.dl[i][16 * sb + 4 * lq]);
        float m[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) m[e] = scores[sb][e] * decay_between(la_t, lr_t, TwoFloats{la_s[e], lr_s[e]}) * dl_s[e];
        if (sb == tok) {
#pragma unroll
          for (int e = 0; e < 4; ++e) m[e] = 4 * lq + e <= lr ? m[e] : 0.0f;
        }
        mf[sb] = tofrag<T>(m[0], m[1], m[2], m[3]);
      }
      ea = __builtin_amdgcn_exp2f(la_t);
      Dh = sh.D[i];
    }
    a.x.put(sX, XP, tid);
    a.s.template put<kBF ? 2 : 1>(sH, kPB * NP, NP, tid);
    float by[kTiles][4];   // what the sums are multiplied by
#pragma unroll
    for (int j = 0; j < kTiles; ++j) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float z = a.z[j][e];
        if constexpr (kDz) {
          const float g = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-z * kLog2e));
          by[j][e] = a.up[j][e] * (g * fmaf(z, 1.0f - g, 1.0f));
        } else {
          by[j][e] = gated ? silu_f32(z) : 1.0f;
        }
        asm volatile("" : "+v"(by[j][e]));   // here, and not behind the next loads: a copy of z would wait for them
      }
    }
    __syncthreads();
    load(s + kDepth, a);
    const Rows64 to = rows_of<T>(TokenTensor{kDz ? o.dz : o.out, o.sb, o.ss, o.sh, kVec}, k, h, p0, p.P, cols > 0);
#pragma unroll
    for (int j = 0; j < kTiles; ++j) {
      const int pt = 2 * j + half, c0 = 16 * pt + 4 * lq;
      Four<T, kVec> out{};
      if (16 * pt < cols) {
        v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if (n >= nt) continue;
          const auto hf = frag_along<T>(sH, NP, 16 * pt, 16 * n, lr, lq);
          if constexpr (kBF) acc = mma32(hf, frag_along<T>(sHL, NP, 16 * pt, 16 * n, lr, lq), cf[n], cf[n], acc);
          else acc = mma16<T>(hf, cf[n], acc);
        }
        acc *= ea;
        if constexpr (kBF) {
#pragma unroll
          for (int sb = 0; sb < QB; sb += 2)
            if (sb <= tok)
              acc = mma32(frag_down<T>(sX, XP, 16 * sb, 16 * pt, lr, lq), frag_down<T>(sX, XP, 16 * sb + 16, 16 * pt, lr, lq), mf[sb],
                          mf[sb + 1], acc);
        } else {
#pragma unroll
          for (int sb = 0; sb < QB; ++sb)
            if (sb <= tok) acc = mma16<T>(frag_down<T>(sX, XP, 16 * sb, 16 * pt, lr, lq), mf[sb], acc);
        }
        // token own, channels c0 ..
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] = fmaf(Dh, Lds<T>::f(sX[own * XP + c0 + e]), acc[e]) * by[j][e];
        out.set(y);
      }
      out.store(to, own, c0);
    }
    __syncthreads();
  };
  if constexpr (kDepth == 1) {
    load(0, ahead[0]);
    for (int s = 0; s < passes; ++s) pass(s, ahead[0]);
  } else {
    load(0, ahead[0]);
    load(1, ahead[1]);
    // always two: with an exit between them the waits could not count on both
    for (int s = 0; s < passes; s += 2) {
      pass(s, ahead[0]);
      pass(s + 1, ahead[1]);
    }
  }
}

template <typename T, int NMAX>
void launch_states(ChunkParams p, bool backward, hipStream_t stream) {
  // half of more than 4 heads a workgroup where the grid is less than one and a half
  // times what the machine holds at once (1024 workgroups), so that its end leaves
  // less of it idle: 16,411 packed x 32 x 64 x 64 bf16, 8 heads 62 us and 4 heads 56
  // (the outputs 102 with either); from 4 to 2 B is staged too often
  if (p.hb > 4 && static_cast<int64_t>(p.nc) * p.G * p.blocks < 1536) {
    p.hb = (p.hb + 1) / 2;
    p.blocks = (p.per_group + p.hb - 1) / p.hb;
  }
  const int grid = p.nc * p.G * p.blocks;
  if (p.vec) ssd_states_kernel<T, NMAX, true><<<dim3(grid, backward ? 2 : 1), kThreads, 0, stream>>>(p, grid);
  else ssd_states_kernel<T, NMAX, false><<<dim3(grid, backward ? 2 : 1), kThreads, 0, stream>>>(p, grid);
}

template <typename T, int NMAX>
void launch_outputs(const ChunkParams& p, const ChunkOut& o, hipStream_t stream) {
  const int grid = p.nc * p.G * p.blocks;
  auto go = [&](auto dz, auto vec) {
    ssd_outputs_kernel<T, NMAX, dz.value, vec.value><<<grid, kOutThreads, 0, stream>>>(p, o, grid);
  };
  if (o.dz && p.vec) go(std::true_type{}, std::true_type{});
  else if (o.dz) go(std::true_type{}, std::false_type{});
  else if (p.vec) go(std::false_type{}, std::true_type{});
  else go(std::false_type{}, std::false_type{});
}

}  // namespace

// Heads of a workgroup: as many as share the chunk's B and C (up to 8) while
// three workgroups a compute unit remain.
ChunkPlan chunk_plan(int64_t batch, int64_t L, int64_t nseq, bool packed, int64_t H, int64_t G) {
  ChunkPlan q;
  q.per_row = (L + kQ - 1) / kQ;
  q.nc = packed ? (L ? L / kQ + std::min(nseq, L) : 0) : batch * q.per_row;
  const int64_t per_group = H / G;
  q.hb = std::min<int64_t>(kMostHeads, per_group);
  while (q.hb > 1 && q.nc * G * ((per_group + q.hb - 1) / q.hb) < 768) q.hb = (q.hb + 1) / 2;
  q.blocks = (per_group + q.hb - 1) / q.hb;
  return q;
}

hipError_t launch_chunk_table(const int32_t* cu, int64_t L, int64_t nseq, int64_t nc, ChunkEntry* table, int32_t* seq_chunk,
                              const OutsideRows& rows, hipStream_t stream) {
  chunk_table_kernel<<<rows.n ? 64 : 1, kTableThreads, 0, stream>>>(cu, L, nseq, static_cast<int>(nc), table, seq_chunk, rows);
  return hipGetLastError();
}

namespace {

template <typename T, int NMAX>
void launch_walk(const ChunkParams& p, const WalkParams& q, bool backward, int64_t rows, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(rows * p.H * q.split), backward ? 2 : 1);
  ssd_walk_kernel<T, NMAX><<<grid, kWalkThreads, 0, stream>>>(p, q);
}

}  // namespace

hipError_t launch_chunk_states(const ChunkParams& p, bool bf16, bool backward, int64_t nseq, const float* h0, float* last,
                               const float* dlast, float* dh0, hipStream_t stream) {
  // batch rows of equal length: a workgroup goes along a whole row where that gives at
  // least three of four compute units one.  Gradients of rows x 32 heads of 64 channels, L 2048,
  // us chunk by chunk and by the walk:
  //   rows         1 (64)     2 (128)     3 (192)     4 (256)     8 (512)    16 (1024 workgroups)
  //   N 64 bf16    71, 96     97, 106    129, 121    166, 148    319, 256    639, 487
  //   N 128 bf16  126, 163   191, 203    247, 226    331, 278    625, 499   1234, 985
  //   N 64 fp32   117, 157   174, 196    229, 231    300, 283    549, 493   1102, 969
  // and alike with L 8192 and 64 heads.  Cutting a head's 64 channels over more
  // workgroups stages B and C again and never won (8 rows, N 64: 298 in halves).  Heads
  // of 16 channels leave too little to a wavefront (4 x 64, N 128: 330, 354).  Rows of
  // 16-byte pieces only: by elements the walk waits for its loads, 4 x 1000 x 16 x 64 x
  // 100 bf16 51 us, 168.
  if (!p.table && p.nc > 0 && p.vec && p.bc_vec && p.P > 16) {
    WalkParams q{{h0, dlast}, {last, dh0}, (p.P + kPB - 1) / kPB};
    const int64_t groups = nseq * p.H * q.split, all = groups * (backward ? 2 : 1);
    // (its windows hold a head's state and a chunk of dt, its grid 2^32 threads)
    if (all >= 192 && groups < (int64_t{1} << 23) && static_cast<int64_t>(p.P) * p.N < (int64_t{1} << 29) && p.dts < (int64_t{1} << 23)) {
      if (!bf16) launch_walk<float, 64>(p, q, backward, nseq, stream);
      else if (p.N > 64) launch_walk<uint16_t, 128>(p, q, backward, nseq, stream);
      else launch_walk<uint16_t, 64>(p, q, backward, nseq, stream);
      return hipGetLastError();
    }
  }
  if (p.nc > 0) {
    if (!bf16) launch_states<float, 64>(p, backward, stream);
    else if (p.N > 64) launch_states<uint16_t, 128>(p, backward, stream);
    else launch_states<uint16_t, 64>(p, backward, stream);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (nseq == 0) return hipSuccess;
  CarryParams q{p.seq_chunk, p.lam, {p.state, p.dstate}, {h0, dlast}, {last, dh0}, nseq,
                static_cast<int64_t>(p.H) * p.P * p.N, p.per_row, p.H, p.P * p.N};
  const bool four = p.P * p.N % 4 == 0;
  const int64_t lanes = four ? q.elems / 4 : q.elems;
  const dim3 grid(static_cast<unsigned>((lanes + kThreads - 1) / kThreads), static_cast<unsigned>(std::min<int64_t>(nseq, 4096)),
                  backward ? 2 : 1);
  if (four) ssd_carry_kernel<4><<<grid, kThreads, 0, stream>>>(q);
  else ssd_carry_kernel<1><<<grid, kThreads, 0, stream>>>(q);
  return hipGetLastError();
}

hipError_t launch_chunk_outputs(const ChunkParams& p, const ChunkOut& o, bool bf16, hipStream_t stream) {
  if (p.nc == 0) return hipSuccess;
  if (!bf16) launch_outputs<float, 64>(p, o, stream);
  else if (p.N > 64) launch_outputs<uint16_t, 128>(p, o, stream);
  else launch_outputs<uint16_t, 64>(p, o, stream);
  return hipGetLastError();
}

}  // namespace ssm
