// What the chunk-parallel SSD kernels share (packed prefill and gradients).
//
// A sequence is cut into chunks of kQ tokens, each of one sequence.  With Delta_t
// the step sizes, a_t = A (Delta_0 + ... + Delta_t) within a chunk, S_in the state
// that enters it and dS_out the gradient on the one that leaves it:
//   S_out  = e^{a_end} S_in  + sum_s e^{a_end - a_s} Delta_s x_s B_s^T
//   dS_in  = e^{a_end} dS_out + sum_t e^{a_t} dy_t C_t^T
// so both directions are one kernel of sums over a chunk (ssd_states) and one
// that carries a state from chunk to chunk (ssd_carry); everything else of a chunk
// is computed from S_in and dS_out by one workgroup, chunks independently.
#pragma once

#include "mfma_tiles.h"
#include "ssm_internal.h"

namespace ssm {

constexpr int kQ = 64;        // tokens of a chunk
constexpr int kPB = 64;       // head channels of a pass
constexpr int kMostHeads = 8; // heads of a workgroup

// Chunk c of a packed row: tokens t0 .. t0 + len - 1 (none: not a chunk).
struct ChunkEntry {
  int32_t t0, len;
};

// A token-major tensor: batch, token and head (or group) strides in elements.
struct TokenTensor {
  const void* p;
  int64_t sb, ss, sh;
  bool vec;   // rows of 16-byte pieces
};

struct ChunkParams {
  TokenTensor x, z, B, C, dout;
  const void* dt;
  int64_t dtb, dts;
  const float* A;
  const float* D;
  const float* bias;
  const ChunkEntry* table;     // packed: chunks; NULL: per_row chunks of each row
  const int32_t* seq_chunk;    // packed: each sequence's first chunk, nseq + 1 entries
  int L, H, P, G, N, per_group, softplus;
  int nc, per_row;             // chunks; of a row
  int hb, blocks;              // heads of a workgroup, workgroups of a group
  bool vec;                    // rows of the heads' tensors and of states are made of 16-byte pieces
  bool bc_vec;                 // rows of B and C are
  float* lam;                  // [nc][H] decay over a chunk
  float* state;                // [nc][H][P][N] what a chunk adds; then S_in
  float* dstate;               // the same backward; then dS_out
};

struct Chunk {
  int64_t b;
  int t0, len;
};

__device__ __forceinline__ Chunk chunk_of(const ChunkParams& p, int c) {
  Chunk k;
  if (p.table) {
    const ChunkEntry e = p.table[c];
    k.b = 0;
    k.t0 = e.t0;
    k.len = e.len;
  } else {
    k.b = c / p.per_row;
    k.t0 = (c - static_cast<int>(k.b) * p.per_row) * kQ;
    k.len = min(kQ, p.L - k.t0);
  }
  return k;
}

// A chunk's rows of one head (or group) as a byte window: rows are addressed by
// 32-bit offsets from it, and what is to be left out by one that lies past it.
struct Rows64 {
  __amdgpu_buffer_rsrc_t r;
  uint32_t stride;   // bytes from token to token
  int len, cols;     // real rows and columns
};
constexpr uint32_t kNowhere = 0x80000000u;

// any = false: a window of nothing.
template <typename T>
__device__ __forceinline__ Rows64 rows_of(const TokenTensor& t, const Chunk& k, int head, int first, int inner, bool any = true) {
  const T* const base = static_cast<const T*>(t.p) + k.b * t.sb + k.t0 * t.ss + head * t.sh + first;
  Rows64 w;
  w.stride = static_cast<uint32_t>(t.ss) * sizeof(T);
  w.len = k.len;
  w.cols = inner - first;
  w.r = __builtin_amdgcn_make_buffer_rsrc(const_cast<T*>(base), 0,
                                          any ? static_cast<int>((k.len - 1) * w.stride + w.cols * sizeof(T)) : 0, kRsrcWord3);
  return w;
}

// Step sizes of a chunk, one token a lane: Delta (0 past the end), and the sums of
// A Delta up to each token in units of log 2.  These are of 64 bits: a decay is a
// difference of two, and one large step (a model that drops its state) would take the
// low bits of every later sum of the chunk in 32 (after a step of 1000 at A = -16
// outputs 1.4e-4 off, and 2.4e-7 now).
struct Steps {
  float delta;
  double la;
};
// What they take of a head, read once: a load within a loop would wait for those
// ahead of it.
struct StepHead {
  double a2;
  float bias;
  int softplus;
};
__device__ __forceinline__ StepHead step_head(const ChunkParams& p, int h) {
  return StepHead{p.A[h] * 1.4426950408889634, p.bias ? p.bias[h] : 0.0f, p.softplus};
}
// v: the lane's step before its bias.
__device__ __forceinline__ Steps steps_from(const StepHead& q, float v, int len, int lane) {
  Steps s;
  v += q.bias;
  s.delta = lane < len ? (q.softplus ? softplus_close_f32(v) : v) : 0.0f;
  s.la = wave_prefix_sum64(s.delta) * q.a2;
  return s;
}
template <typename T>
__device__ __forceinline__ Steps steps_of(const ChunkParams& p, const Chunk& k, int h, int lane) {
  float v = 0.0f;
  if (lane < k.len) v = io<T>::load(static_cast<const T*>(p.dt) + k.b * p.dtb + (k.t0 + lane) * p.dts + h);
  return steps_from(step_head(p, h), v, k.len, lane);
}
// softplus'(v) from Delta = softplus(v): sigmoid(v) = 1 - e^-Delta, by its series where
// the difference would cancel (Delta < 1/4: the first term left out is below 2^-26 of it).
__device__ __forceinline__ float slope_of(float delta) {
  float s = fmaf(delta, -1.0f / 5040, 1.0f / 720);
  s = fmaf(-delta, s, 1.0f / 120);
  s = fmaf(-delta, s, 1.0f / 24);
  s = fmaf(-delta, s, 1.0f / 6);
  s = fmaf(-delta, s, 0.5f);
  s = delta * fmaf(-delta, s, 1.0f);
  return delta < 0.25f ? s : 1.0f - __builtin_amdgcn_exp2f(-delta * kLog2e);
}
__device__ __forceinline__ float lane_value(float v, int lane) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}
__device__ __forceinline__ float wave_sum(float v) { return lane_value(wave_prefix_sum(v), 63); }

// ---- tiles in LDS ---------------------------------------------------------------

// A thread's number that the compiler takes for a new one: offsets made from it are
// computed where they are used, and not kept in registers around a loop.
__device__ __forceinline__ int anew(int tid) {
  asm volatile("" : "+v"(tid));
  return tid;
}

template <typename V>
__device__ __forceinline__ V anew_words(V v) {
  if constexpr (sizeof(V) == 8) {
    v2u w = __builtin_bit_cast(v2u, v);
    asm volatile("" : "+v"(w));
    return __builtin_bit_cast(V, w);
  } else {
    return v;
  }
}

// 16 bytes of a row as registers hold them.
template <typename T> constexpr int kPiece = 16 / sizeof(T);

// A thread's piece of a row: columns col .. of row r; zeros past the real ones.
// kVec: rows are made of whole 16-byte pieces (of all tensors of a kind); else
// element by element.
template <typename T, bool kVec>
__device__ __forceinline__ v4u load_piece(const Rows64& w, int r, int col) {
  const uint32_t off = r * w.stride + col * static_cast<uint32_t>(sizeof(T));
  if constexpr (kVec) return __builtin_amdgcn_raw_buffer_load_b128(w.r, r < w.len && col < w.cols ? off : kNowhere, 0, 0);
  v4u v = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < kPiece<T>; ++i) {
    const uint32_t e = Elem<T>::load(w.r, r < w.len && col + i < w.cols ? off + i * static_cast<uint32_t>(sizeof(T)) : kNowhere);
    if constexpr (sizeof(T) == 4) v[i] = e;
    else v[i / 2] |= e << (16 * (i % 2));
  }
  return v;
}
template <typename T>
__device__ __forceinline__ float piece_f32(const v4u& v, int i) {
  if constexpr (sizeof(T) == 4) return __uint_as_float(v[i]);
  else return __uint_as_float(i % 2 ? v[i / 2] & 0xffff0000u : v[i / 2] << 16);
}

// Rows of a chunk (kQ rows of W columns) in a workgroup's registers, on their way to
// LDS; zeros past the chunk's tokens and past the real columns.
template <typename T, int W, int kThreads>
struct Pieces {
  static constexpr int kPer = W / kPiece<T>, kStep = kThreads / kPer, kN = kQ / kStep;
  static_assert(kThreads % kPer == 0 && kQ % kStep == 0, "whole rows a step");
  v4u v[kN];
  template <bool kVec>
  __device__ __forceinline__ void load(const Rows64& w, int tid) {
    tid = anew(tid);
#pragma unroll
    for (int i = 0; i < kN; ++i) v[i] = load_piece<T, kVec>(w, tid / kPer + i * kStep, tid % kPer * kPiece<T>);
  }
  __device__ __forceinline__ void put(typename Lds<T>::E* dst, int pitch, int tid) const {
#pragma unroll
    for (int i = 0; i < kN; ++i) *reinterpret_cast<v4u*>(dst + (tid / kPer + i * kStep) * pitch + tid % kPer * kPiece<T>) = v[i];
  }
};
// vec: as kVec, found out here (a chunk's B and C are staged once for several heads,
// and 100 states a row do not make 16-byte pieces of bf16).
template <typename T, int W, int kThreads, bool kVec>
__device__ __forceinline__ void stage_rows(typename Lds<T>::E* dst, int pitch, const Rows64& w, int tid, bool vec) {
  Pieces<T, W, kThreads> q;
  if (kVec && vec) q.template load<true>(w, tid);
  else q.template load<false>(w, tid);
  q.put(dst, pitch, tid);
}

// Four states n .. n + 3 of row r of a chunk's state.
// rows of the window: the head's channels from a pass's first on.
struct StateRows {
  __amdgpu_buffer_rsrc_t r;
  int N;
};
__device__ __forceinline__ StateRows state_rows(const float* state, int64_t at, int rows, int N) {
  return StateRows{__builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(state + at), 0, rows * N * 4, kRsrcWord3), N};
}
template <bool kVec>
__device__ __forceinline__ v4u load_states(const StateRows& w, int r, int n) {
  const uint32_t off = (r * w.N + n) * 4u;
  if constexpr (kVec) return __builtin_amdgcn_raw_buffer_load_b128(w.r, n < w.N ? off : kNowhere, 0, 0);
  v4u v;
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = __builtin_amdgcn_raw_buffer_load_b32(w.r, n + e < w.N ? off + 4 * e : kNowhere, 0, 0);
  return v;
}

// The high halves of two words, the first one's low.
__device__ __forceinline__ uint32_t highs(uint32_t a, uint32_t b) { return a >> 16 | (b & 0xffff0000u); }

// Two fp32 values as kParts bf16 parts, each the nearest to what the ones before it
// leave: 8 bits more a part, the second value in the high halves.
template <int kParts>
__device__ __forceinline__ void split_bf16(float a, float b, uint32_t (&w)[kParts]) {
#pragma unroll
  for (int i = 0; i < kParts; ++i) {
    w[i] = pack_bf16x2(a, b);
    if (i + 1 == kParts) break;
    a -= __uint_as_float(w[i] << 16);
    b -= __uint_as_float(w[i] & 0xffff0000u);
  }
}

// kPB rows of a state, likewise; bf16: as kParts parts in as many arrays of LDS, `part`
// elements apart.
template <typename T, int NMAX, int kThreads>
struct StatePieces {
  static constexpr int kPer = NMAX / 4, kStep = kThreads / kPer, kN = kPB / kStep;
  v4u v[kN];
  template <bool kVec>
  __device__ __forceinline__ void load(const StateRows& w, int tid) {
    tid = anew(tid);
#pragma unroll
    for (int i = 0; i < kN; ++i) v[i] = load_states<kVec>(w, tid / kPer + i * kStep, tid % kPer * 4);
  }
  template <int kParts>
  __device__ __forceinline__ void put(typename Lds<T>::E* dst, [[maybe_unused]] int part, int pitch, int tid) const {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int at = (tid / kPer + i * kStep) * pitch + tid % kPer * 4;
      if constexpr (sizeof(T) == 2) {
        uint32_t a[kParts], b[kParts];
        split_bf16(__uint_as_float(v[i][0]), __uint_as_float(v[i][1]), a);
        split_bf16(__uint_as_float(v[i][2]), __uint_as_float(v[i][3]), b);
#pragma unroll
        for (int k = 0; k < kParts; ++k) *reinterpret_cast<v2u*>(dst + k * part + at) = v2u{a[k], b[k]};
      } else {
        *reinterpret_cast<v4u*>(dst + at) = v[i];
      }
    }
  }
};

// A 16-wide tile's fragment down the rows of LDS: X[k0 + 4 lq + i][c0 + lr].
template <typename T>
__device__ __forceinline__ typename Frag<T>::V frag_down(const typename Lds<T>::E* X, int pitch, int k0, int c0, int lr, int lq) {
  if constexpr (sizeof(T) == 2) {
    return lds_tr(X + (k0 + 4 * lq + lr / 4) * pitch + c0 + 4 * (lr % 4));
  } else {
    const float* q = X + (k0 + 4 * lq) * pitch + c0 + lr;
    return v4f{q[0], q[pitch], q[2 * pitch], q[3 * pitch]};
  }
}
// The fragment along a row: X[r0 + lr][k0 + 4 lq + i].
template <typename T>
__device__ __forceinline__ typename Frag<T>::V frag_along(const typename Lds<T>::E* X, int pitch, int r0, int k0, int lr, int lq) {
  return ldsf<T>(X + (r0 + lr) * pitch + k0 + 4 * lq);
}

// Element e of a fragment as fp32.
template <typename T>
__device__ __forceinline__ float elem(const typename Frag<T>::V& v, int e) {
  if constexpr (sizeof(T) == 2) return bf16_to_f32(static_cast<uint16_t>(v[e]));
  else return v[e];
}

// Rows of 16 lanes, two at a time: the first and the second of each pair, in both
// (kOver 16: rows 0 and 1, 2 and 3; 32: rows 0 and 2, 1 and 3).
struct RowPair {
  float first, second;
};
template <int kOver>
__device__ __forceinline__ RowPair row_pair(float v) {
  const uint32_t w = __float_as_uint(v);
  if constexpr (kOver == 16) {
    const auto q = __builtin_amdgcn_permlane16_swap(w, w, false, false);
    return RowPair{__uint_as_float(q[0]), __uint_as_float(q[1])};
  } else {
    const auto q = __builtin_amdgcn_permlane32_swap(w, w, false, false);
    return RowPair{__uint_as_float(q[0]), __uint_as_float(q[1])};
  }
}
// Sum over the four lanes that hold a tile's column (or row), 16 lanes apart.
__device__ __forceinline__ float quarter_sum(float v) {
  const RowPair near = row_pair<16>(v), far = row_pair<32>(near.first + near.second);
  return far.first + far.second;
}

// Four values a lane, summed over each 16-lane row: lane lr gets value lr % 4.
__device__ __forceinline__ float row_sums(const v4f& v, int lane) {
  const bool odd = lane & 1, high = lane & 2;
  auto dpp = [](float f, auto ctrl) {
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(f), decltype(ctrl)::value, 0xf, 0xf, true));
  };
  using Swap1 = std::integral_constant<int, 0xB1>;
  using Swap2 = std::integral_constant<int, 0x4E>;
  using Ror4 = std::integral_constant<int, 0x124>;
  using Ror8 = std::integral_constant<int, 0x128>;
  const float a = (odd ? v[1] : v[0]) + dpp(odd ? v[0] : v[1], Swap1{});
  const float b = (odd ? v[3] : v[2]) + dpp(odd ? v[2] : v[3], Swap1{});
  float s = (high ? b : a) + dpp(high ? a : b, Swap2{});
  s += dpp(s, Ror4{});
  return s + dpp(s, Ror8{});
}

// ---- launches shared by the packed prefill and the gradients ------------------

struct ChunkPlan {
  int64_t nc, per_row;
  int64_t hb, blocks;   // heads of a workgroup, workgroups of a group
};
ChunkPlan chunk_plan(int64_t batch, int64_t L, int64_t nseq, bool packed, int64_t H, int64_t G);

// Rows of tensors that belong to tokens of no sequence: `heads` runs of `bytes`.
struct OutsideRows {
  struct Tensor {
    void* p;
    int64_t bytes, stride, heads, head_stride;
  } t[6];
  int n = 0;
  void add(void* p, int64_t bytes, int64_t stride, int64_t heads = 1, int64_t head_stride = 0) {
    t[n++] = Tensor{p, bytes, stride, heads, head_stride};
  }
};
hipError_t launch_chunk_table(const int32_t* cu, int64_t L, int64_t nseq, int64_t nc, ChunkEntry* table, int32_t* seq_chunk,
                              const OutsideRows& rows, hipStream_t stream);
// What each chunk adds to the state (and, with backward, to the gradient's), and
// the carry along each sequence.
hipError_t launch_chunk_states(const ChunkParams& p, bool bf16, bool backward, int64_t nseq, const float* h0, float* last,
                               const float* dlast, float* dh0, hipStream_t stream);
// The outputs from S_in; with dz given, the gradient of the gate instead.
struct ChunkOut {
  void* out;
  int64_t sb, ss, sh;
  void* dz;
};
hipError_t launch_chunk_outputs(const ChunkParams& p, const ChunkOut& o, bool bf16, hipStream_t stream);

}  // namespace ssm
