// ssd_bwd.hip -- gradients of the Mamba-2 SSM prefill on gfx950, chunk by chunk on
// the matrix cores (see ssd_chunk.h for S_in and dS_out, which two kernels there
// leave for every chunk and head).
//
// Within a chunk, with dy_t = dout_t silu(z_t), L[t,s] = e^{a_t - a_s} for s <= t (else
// 0), G = C B^T (one for all heads of a group) and M = dy x^T:
//   dx_s  = Delta_s (sum_t (G L)[t,s] dy_t + e^{a_end - a_s} dS_out B_s) + D dy_s
//   dC_t  = sum_h sum_s (M L)[t,s] Delta_s B_s + e^{a_t} S_in^T dy_t
//   dB_s  = sum_h sum_t (M L)[t,s] Delta_s C_t + e^{a_end - a_s} Delta_s dS_out^T x_s
// The gradients of the steps need no further product.  With K = G L M (elementwise;
// what of the output at t comes from the input at s, times dy_t, over Delta_s), and
//   r_t = e^{a_t} C_t . (S_in^T dy_t),   c_s = e^{a_end - a_s} B_s . (dS_out^T x_s)
// the gradient that flows through the decay of step s is everything from before s
// to s or after:
//   g_s = sum_{t >= s} sum_{u < s} K[t,u] Delta_u + sum_{t >= s} r_t + sum_{u < s} c_u Delta_u
//         + e^{a_end} <S_in, dS_out>
//   dDelta_s = sum_{t >= s} K[t,s] + c_s + A g_s,   dA = sum Delta_s g_s,
// Every term of g_s has the decay of step s in it.  All 64 could be had as running sums
// of row and column sums of K, but a step that drops the state would then leave the
// rounding of the whole chunk where next to nothing flows (with every 8th step 100 at
// A = -16, dA 4e-4 off).  So nothing is subtracted: the rectangle t >= s, u < s of K
// Delta is made of row sums over the 16 u of a block, added over t >= s (blocks of u
// before s's), column sums over the blocks of t after s's, added over u < s, and of the
// tile on the diagonal, where sums down its columns are added along its rows.
//   ddt = dDelta softplus'(dt + bias),   dD = sum_t M[t,t]
// For bf16 IO K comes from products of the inputs as they are, and dy, where it is gated,
// and the states S_in and dS_out enter as three bf16 parts, 24 bits (with two, 16 bits, dA
// and the bias's gradient were 2 to 5e-6 off, and 8 x 2048 x 32 x 64 x 64 took 252 us for
// 266, gated 414 for 483); so these sums are as good as fp32's.  Rounded to bf16 are, where
// they enter the products for dx, dB and dC, which are rounded to bf16 themselves, G L and
// M L, and dS_out where it enters dx; a gated dy enters dx in two parts.
//
// A workgroup takes a chunk and up to 8 heads of a group.  Two of its 8 wavefronts
// share 16 of the chunk's tokens, as s for dx and dB and as t for dC: each has every
// other tile of G and M, half of the states for dB and dC and half of the channels
// for dx.  G, the sum over the heads of M L Delta, and dB and dC stay in registers
// from head to head, so dB and dC cost one product with C and B for all heads; the
// next head's loads are under way while one is computed.  Bound by memory and the
// latency of a head's five stages between barriers (55% of a wavefront's cycles are
// waits): 8 x 2048 x 32 x 64 x 64 bf16 in 152 us, 3.1 TB/s of x, dout, both states and
// dx; one wavefront a token block was 39 us slower.
#include <algorithm>

#include "abi_checks.h"
#include "ssd_chunk.h"

namespace ssm {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kGradThreads = 512;
constexpr int QB = kQ / 16;        // blocks of 16 tokens
constexpr int kTiles = QB / 2;     // tiles of a wavefront, of its tokens as s

struct GradParams {
  void* dx;          // contiguous (row, token, H, P)
  void* ddt;         // contiguous (row, token, H)
  void* dB;          // contiguous (row, token, G, N), where a group has one workgroup
  void* dC;
  float* parts;      // [3][H][nc] sums of dA, ddt_bias and dD
  float* dBparts;    // [block][row, token][G][N], where it has several
  float* dCparts;
  int64_t tokens;    // of all rows
};

// Wavefronts a SIMD: four (two workgroups a compute unit, 128 registers) for up to 64
// states in bf16 without a gate, though only the form of 16-byte rows and one pass fits
// them; the others keep 8 to 26 registers in scratch, which costs less than half the
// wavefronts.  Gradients with four and, without scratch, two, us: 8 x 2048 x 32 x 64 x 64
// 266, 325; 4 x 2048 x 16 x 128 180, 196; 4 x 2048 x 32 x 36 by elements 238, 259; 4 x
// 2048 x 16 x 132 391, 427.  A gate's dy in three parts leaves LDS for one workgroup; with
// B and C in registers instead there was room for two and 32 to 60 registers in scratch
// (8 x 2048 x 32 x 64 x 64 485 -> 517, 4 x 2048 x 32 x 36 434 -> 482).
template <typename T, int NMAX, bool kGate>
constexpr int kGradWaves = sizeof(T) == 2 && NMAX == 64 && !kGate ? 4 : 2;

// kOne: a head's channels are one pass.
template <typename T, int NMAX, bool kGate, bool kVec, bool kOne>
__global__ __launch_bounds__(kGradThreads, (kGradWaves<T, NMAX, kGate>)) void ssd_grad_kernel(ChunkParams p, GradParams q, int grid) {
  using E = typename Lds<T>::E;
  using F = typename Frag<T>::V;
  constexpr bool kBF = sizeof(T) == 2;
  constexpr int kPad = 16 / sizeof(E), NP = NMAX + kPad, XP = kPB + kPad, GP = kQ + kPad, NT = NMAX / 16, NH = NT / 2;
  // bf16: a state in three parts, a gated dout too, 24 bits together
  constexpr int kSP = kBF ? 3 : 1, kYP = kBF && kGate ? 3 : 1, kPartS = kPB * NP, kPartY = kQ * XP;
  // heads: x, dy, a state, (G L)^T; before and after them: B and C, and the sum over
  // the heads
  constexpr int kX = 0, kDy = kQ * XP, kS = kDy + kYP * kPartY;
  constexpr int kGl = kS + kSP * kPartS, kHead = kGl + kQ * GP, kEnds = 2 * kQ * NP + kQ * GP;
  // kKeep: B and C stay in LDS, next to the heads' operands; their fragments are read
  // again and again, which leaves the registers for two workgroups a compute unit
  // (128 of them).  Else they make room, and their fragments stay in registers.
  constexpr bool kKeep = kBF && NMAX == 64;
  constexpr int kB = kKeep ? kHead : 0, kC = kB + kQ * NP, kG = kKeep ? 0 : 2 * kQ * NP;
  // the small arrays first: their addresses are then offsets in the instruction
  struct Shared {
    float la[kMostHeads][kQ], lr[kMostHeads][kQ], dl[kMostHeads][kQ], A[kMostHeads], D[kMostHeads];
    // of a token: K Delta of its block's rectangle; sums over K's column in its block, and
    // below (by the wavefronts' halves); M's diagonal, where that gives dD
    float in_block[kQ], col[kQ], below[2][kQ], m[kGate && kBF ? 1 : kQ], pairs[kGradThreads / 64], dd[kGradThreads / 64];
    alignas(16) E tiles[kKeep ? kHead + 2 * kQ * NP : kHead > kEnds ? kHead : kEnds];
  };
  __shared__ __align__(16) Shared sh;
  E* const lds = sh.tiles;
  const int tid = threadIdx.x, lane = tid & 63, lr = lane & 15, lq = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), tok = wave % QB, half = wave / QB;
  const int id = static_cast<int>(xcd_order(blockIdx.x, grid));
  const int c = id / (p.G * p.blocks), g = id / p.blocks % p.G, block = id % p.blocks, h0 = g * p.per_group + block * p.hb;
  const int heads = min(p.hb, (g + 1) * p.per_group - h0);
  const Chunk k = chunk_of(p, c);
  if (k.len == 0) {   // not a chunk: nothing to the sums
    for (int i = tid; i < 3 * heads; i += kGradThreads)
      q.parts[(static_cast<int64_t>(i % 3) * p.H + h0 + i / 3) * p.nc + c] = 0.0f;
    return;
  }
  for (int i = wave; i < heads; i += kGradThreads / 64) {
    const Steps s = steps_of<T>(p, k, h0 + i, lane);
    sh.dl[i][lane] = s.delta;
    const TwoFloats la = two_floats(s.la);
    sh.la[i][lane] = la.v;
    sh.lr[i][lane] = la.rest;
    if (lane == 0) {
      sh.A[i] = p.A[h0 + i];
      sh.D[i] = p.D ? p.D[h0 + i] : 0.0f;
    }
  }
  E* const sB = lds + kB;
  E* const sC = lds + kC;
  auto stage_bc = [&]() {
    stage_rows<T, NMAX, kGradThreads, kVec>(sB, NP, rows_of<T>(p.B, k, g, 0, p.N), tid, p.bc_vec);
    stage_rows<T, NMAX, kGradThreads, kVec>(sC, NP, rows_of<T>(p.C, k, g, 0, p.N), tid, p.bc_vec);
  };
  stage_bc();
  __syncthreads();

  // the lane's token, as s and as t; its B, and of B and C the states of the
  // wavefront's half: tiles n0 .. n0 + NH - 1, lane: states 16 n + 4 lq ..
  const int own = 16 * tok + lr, n0 = half * NH, nt = (p.N + 15) / 16;
  F bf[kKeep ? 1 : NT], bh[kKeep ? 1 : NH], cf[kKeep ? 1 : NH];
  auto frag_b = [&](int n) { return frag_along<T>(sB, NP, 16 * tok, 16 * n, lr, lq); };
  auto frag_c = [&](int n) { return frag_along<T>(sC, NP, 16 * tok, 16 * n, lr, lq); };
  if constexpr (!kKeep) {
#pragma unroll
    for (int n = 0; n < NT; ++n) bf[n] = frag_b(n);
#pragma unroll
    for (int n = 0; n < NH; ++n) {
      bh[n] = frag_b(n0 + n);
      cf[n] = frag_c(n0 + n);
    }
  }
  auto own_b = [&](int n) {
    if constexpr (kKeep) return frag_b(n);
    else return bf[n];
  };
  auto half_b = [&](int n) {
    if constexpr (kKeep) return frag_b(n0 + n);
    else return anew_words(bh[n]);
  };
  auto half_c = [&](int n) {
    if constexpr (kKeep) return frag_c(n0 + n);
    else return anew_words(cf[n]);
  };
  // tiles of G and of the sum over the heads: t block tok + half + 2 j, lane holds
  // t = 16 tb + 4 lq + e, s = own
  auto block_of = [&](int j) { return tok + half + 2 * j; };
  v4f G[kTiles], sum[kTiles], dB[NH], dC[NH];
#pragma unroll
  for (int j = 0; j < kTiles; ++j) {
    G[j] = sum[j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    const int tb = block_of(j);
    if (tb >= QB) continue;
    if constexpr (kBF) {
#pragma unroll
      for (int n = 0; n < NT; n += 2)
        G[j] = mma32(frag_along<T>(sC, NP, 16 * tb, 16 * n, lr, lq), frag_along<T>(sC, NP, 16 * tb, 16 * n + 16, lr, lq), own_b(n),
                     own_b(n + 1), G[j]);
    } else {
#pragma unroll
      for (int n = 0; n < NT; ++n) G[j] = mma16<T>(frag_along<T>(sC, NP, 16 * tb, 16 * n, lr, lq), own_b(n), G[j]);
    }
  }
#pragma unroll
  for (int n = 0; n < NH; ++n) dB[n] = dC[n] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  __syncthreads();

  E* const sX = lds + kX;
  E* const sY = lds + kDy;
  E* const sS = lds + kS;
  E* const sGl = lds + kGl;   // [s][t]
  // four more sums a token lie behind its rows (two workgroups then fit a compute unit):
  // r and c of both halves behind x, K Delta's row over each block before it behind dy
  auto sums_rc = [&](int t) { return reinterpret_cast<float*>(sX + t * XP + kPB); };
  auto sums_row = [&](int t) { return reinterpret_cast<float*>(sY + t * XP + kPB); };
  static_assert(kPad * sizeof(E) == 4 * sizeof(float), "four floats behind a row");
  using Tokens = Pieces<T, kPB, kGradThreads>;
  using States = StatePieces<T, NMAX, kGradThreads>;
  Tokens xv, yv, zv;
  States sv;
  auto load_y = [&](int h, int p0) {
    yv.template load<kVec>(rows_of<T>(p.dout, k, h, p0, p.P), tid);
    if constexpr (kGate) zv.template load<kVec>(rows_of<T>(p.z, k, h, p0, p.P), tid);
  };
  auto load_state = [&](const float* state, int h, int p0) {
    sv.template load<kVec>(state_rows(state, ((static_cast<int64_t>(c) * p.H + h) * p.P + p0) * p.N, min(kPB, p.P - p0), p.N), tid);
  };
  auto load_head = [&](int h, int p0) {
    xv.template load<kVec>(rows_of<T>(p.x, k, h, p0, p.P), tid);
    load_y(h, p0);
    load_state(p.state, h, p0);
  };
  // dy = dout, or dout silu(z), bf16 then in parts; and what it gives dD, of a bf16 gate
  constexpr bool kOwnD = kGate && kBF;
  [[maybe_unused]] float dd_own = 0.0f;
  auto put_y = [&](auto first) {
    if constexpr (!kGate) {
      yv.put(sY, XP, tid);
    } else {
#pragma unroll
      for (int j = 0; j < Tokens::kN; ++j) {
        const int at = (tid / Tokens::kPer + j * Tokens::kStep) * XP + tid % Tokens::kPer * kPiece<T>;
        float f[kPiece<T>];
#pragma unroll
        for (int e = 0; e < kPiece<T>; ++e) {
          f[e] = piece_f32<T>(yv.v[j], e) * silu_f32(piece_f32<T>(zv.v[j], e));
          if constexpr (kOwnD && decltype(first)::value) dd_own = fmaf(f[e], piece_f32<T>(xv.v[j], e), dd_own);
        }
        if constexpr (kBF) {
          uint32_t w[kPiece<T> / 2][kYP];
#pragma unroll
          for (int e = 0; e < kPiece<T> / 2; ++e) split_bf16(f[2 * e], f[2 * e + 1], w[e]);
#pragma unroll
          for (int k = 0; k < kYP; ++k) *reinterpret_cast<v4u*>(sY + k * kPartY + at) = v4u{w[0][k], w[1][k], w[2][k], w[3][k]};
        } else {
          *reinterpret_cast<v4u*>(sY + at) =
              v4u{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])};
        }
      }
    }
  };
  auto put_state = [&]() { sv.template put<kSP>(sS, kPartS, NP, tid); };
  // a 16 x 16 tile of the state (rows n, k = channel) times x or dy of `own`, whose
  // rows are in X, in as many parts; of parts' products those of 2^-16 and more
  auto state_tile = [&](int n, int kbs, const E* X, auto parts) {
    v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
    if constexpr (kBF) {
#pragma unroll
      for (int kb = 0; kb < kPB / 16; kb += 2) {
        if (kb >= kbs) continue;
        F s0[kSP], s1[kSP];
#pragma unroll
        for (int i = 0; i < kSP; ++i) {
          s0[i] = frag_down<T>(sS + i * kPartS, NP, 16 * kb, 16 * n, lr, lq);
          s1[i] = frag_down<T>(sS + i * kPartS, NP, 16 * kb + 16, 16 * n, lr, lq);
        }
#pragma unroll
        for (int j = 0; j < decltype(parts)::value; ++j) {
          const F f0 = frag_along<T>(X + j * kPartY, XP, 16 * tok, 16 * kb, lr, lq),
                  f1 = frag_along<T>(X + j * kPartY, XP, 16 * tok, 16 * kb + 16, lr, lq);
#pragma unroll
          for (int i = 0; i + j < kSP; ++i) acc = mma32(s0[i], s1[i], f0, f1, acc);
        }
      }
    } else {
#pragma unroll
      for (int kb = 0; kb < kPB / 16; ++kb)
        if (kb < kbs)
          acc = mma16<T>(frag_down<T>(sS, NP, 16 * kb, 16 * n, lr, lq), frag_along<T>(X, XP, 16 * tok, 16 * kb, lr, lq), acc);
    }
    return acc;
  };

  load_head(h0, 0);
  for (int i = 0; i < heads; ++i) {
    const int h = h0 + i;
    const TwoFloats la_s{sh.la[i][own], sh.lr[i][own]};
    const float dl_s = sh.dl[i][own];
    const float ew = decay_between(sh.la[i][kQ - 1], sh.lr[i][kQ - 1], la_s), ea = __builtin_amdgcn_exp2f(la_s.v);
    const float Dh = sh.D[i];
    v4f M[kTiles];
#pragma unroll
    for (int j = 0; j < kTiles; ++j) M[j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    float r_t = 0.0f, c_s = 0.0f, pairs = 0.0f;
    for (int p0 = 0; p0 < (kOne ? 1 : p.P); p0 += kPB) {
      const int cols = p.P - p0, kbs = (min(kPB, cols) + 15) / 16;
      if (!kOne && p0 > 0) {   // the loads of a head's first pass are under way since the head before
        __syncthreads();
        load_head(h, p0);
      }
      xv.put(sX, XP, tid);
      put_y(std::true_type{});
      put_state();
      __syncthreads();
      load_state(p.dstate, h, p0);
      // M[t][s] += dy_t . x_s
#pragma unroll
      for (int kb = 0; kb < kPB / 16; kb += kBF ? 2 : 1) {
        if (kb >= kbs) continue;
        const F x0 = frag_along<T>(sX, XP, 16 * tok, 16 * kb, lr, lq);
        [[maybe_unused]] const F x1 = kBF ? frag_along<T>(sX, XP, 16 * tok, 16 * kb + 16, lr, lq) : x0;
#pragma unroll
        for (int j = 0; j < kTiles; ++j) {
          const int tb = block_of(j);
          if (tb >= QB) continue;
          if constexpr (kBF) {
#pragma unroll
            for (int i = 0; i < kYP; ++i)
              M[j] = mma32(frag_along<T>(sY + i * kPartY, XP, 16 * tb, 16 * kb, lr, lq),
                           frag_along<T>(sY + i * kPartY, XP, 16 * tb, 16 * kb + 16, lr, lq), x0, x1, M[j]);
          } else {
            M[j] = mma16<T>(frag_along<T>(sY, XP, 16 * tb, 16 * kb, lr, lq), x0, M[j]);
          }
        }
      }
      if (kOne || p0 + kPB >= p.P) {
        // M is complete: K, its sums, and the operands of dx; only the diagonal's tile
        // (half 0, its first) has elements above it
        float below = 0.0f;
        auto tile = [&](int j, auto on_diagonal) {
          constexpr bool kDiag = decltype(on_diagonal)::value;
          const int tb = block_of(j);
          const v4f la_t = *reinterpret_cast<const v4f*>(&sh.la[i][16 * tb + 4 * lq]), lr_t = *reinterpret_cast<const v4f*>(&sh.lr[i][16 * tb + 4 * lq]);
          float w[4], in_col = 0.0f, m0 = 0.0f;
          v4f rows;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int over = 4 * lq + e - lr;   // t - s on the diagonal's tile
            float L = decay_between(la_t[e], lr_t[e], la_s), m = M[j][e];
            if constexpr (kDiag) {
              L = over >= 0 ? L : 0.0f;
              m = over >= 0 ? m : 0.0f;
            }
            w[e] = G[j][e] * L;
            if constexpr (kDiag) w[e] = over >= 0 ? w[e] : 0.0f;
            sum[j][e] = fmaf(m * L, dl_s, sum[j][e]);
            float K = w[e] * m;
            (kDiag ? in_col : below) += K;
            if constexpr (kDiag) {
              m0 += over == 0 ? m : 0.0f;
              K = over > 0 ? K : 0.0f;
            }
            rows[e] = K * dl_s;
          }
          *reinterpret_cast<F*>(sGl + own * GP + 16 * tb + 4 * lq) = tofrag<T>(w[0], w[1], w[2], w[3]);
          if constexpr (kDiag) {   // down the column from t on, then along the row up to t
#pragma unroll
            for (int e = 2; e >= 0; --e) rows[e] += rows[e + 1];
            const RowPair near = row_pair<16>(rows[0]);
            const float pair = row_pair<32>(near.first + near.second).second;
            const float under = (lq & 1 ? 0.0f : near.second) + (lq & 2 ? 0.0f : pair);
#pragma unroll
            for (int e = 0; e < 4; ++e) rows[e] = lr < 4 * lq + e ? rows[e] + under : 0.0f;
          }
          const float s = row_sums(rows, lane);
          const int t = 16 * tb + anew(4 * lq + lr);
          if (lr < 4) (kDiag ? sh.in_block[t] : sums_row(t)[tok]) = s;
          if constexpr (kDiag) {
            in_col = quarter_sum(in_col);
            if (lq == 0) sh.col[own] = in_col;
            if constexpr (!(kGate && kBF)) {
              m0 = quarter_sum(m0);
              if (lq == 0) sh.m[own] = m0;
            }
          }
        };
        if (half == 0) tile(0, std::true_type{});
        else if (block_of(0) < QB) tile(0, std::false_type{});
#pragma unroll
        for (int j = 1; j < kTiles; ++j)
          if (block_of(j) < QB) tile(j, std::false_type{});
        below = quarter_sum(below);
        if (lq == 0) sh.below[half][own] = below;
      }
      // S_in^T dy_t: lane holds states 16 n + 4 lq + e
#pragma unroll
      for (int n = 0; n < NH; ++n) {
        if (n0 + n >= nt) continue;
        const F f = half_c(n);
        const v4f v = state_tile(n0 + n, kbs, sY, std::integral_constant<int, kYP>{});
#pragma unroll
        for (int e = 0; e < 4; ++e) r_t = fmaf(elem<T>(f, e), v[e], r_t);
        dC[n] += v * ea;
      }
      __syncthreads();
      // dS_out in the place of S_in, which it meets on the way
#pragma unroll
      for (int j = 0; j < States::kN; ++j) {
        const int at = (tid / States::kPer + j * States::kStep) * NP + tid % States::kPer * 4;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float s = 0.0f;   // the parts' sum is exact
#pragma unroll
          for (int i = kSP - 1; i >= 0; --i) s += Lds<T>::f(sS[i * kPartS + at + e]);
          pairs = fmaf(s, __uint_as_float(sv.v[j][e]), pairs);
        }
      }
      put_state();
      __syncthreads();
      if (kOne && i + 1 < heads) load_head(h + 1, 0);
#pragma unroll
      for (int n = 0; n < NH; ++n) {
        if (n0 + n >= nt) continue;
        const F f = half_b(n);
        const v4f v = state_tile(n0 + n, kbs, sX, std::integral_constant<int, 1>{});
#pragma unroll
        for (int e = 0; e < 4; ++e) c_s = fmaf(elem<T>(f, e), v[e], c_s);
        dB[n] += v * (ew * dl_s);
      }
    }
    r_t = quarter_sum(r_t) * ea;
    c_s = quarter_sum(c_s) * ew;
    pairs = wave_sum(pairs);
    if (lq == 0) {
      float* const to = sums_rc(anew(own)) + half;
      to[0] = r_t;
      to[2] = c_s;
    }
    if (lane == 0) sh.pairs[wave] = pairs * __builtin_amdgcn_exp2f(sh.la[i][kQ - 1]);
    if constexpr (kOwnD) {
      const float s = wave_sum(dd_own);
      dd_own = 0.0f;
      if (lane == 0) sh.dd[wave] = s;
    }
    // dx, every other 16 channels
    for (int p0 = 0; p0 < (kOne ? 1 : p.P); p0 += kPB) {
      const int cols = p.P - p0;
      if (!kOne) {   // what is in LDS is the last pass's
        __syncthreads();
        load_y(h, p0);
        load_state(p.dstate, h, p0);
        put_y(std::false_type{});
        put_state();
        __syncthreads();
        if (p0 + kPB >= p.P && i + 1 < heads) load_head(h + 1, 0);
      }
      // the chunk's rows of dx, from the head's channel p0 on
      const __amdgpu_buffer_rsrc_t dx = __builtin_amdgcn_make_buffer_rsrc(
          static_cast<T*>(q.dx) + ((k.b * p.L + k.t0) * p.H + h) * p.P + p0, 0,
          static_cast<int>(((k.len - 1) * p.H * p.P + cols) * sizeof(T)), kRsrcWord3);
#pragma unroll
      for (int j = 0; j < kPB / 32; ++j) {
        const int pt = 2 * j + half, c0 = 16 * pt + 4 * lq;
        if (16 * pt >= cols) continue;
        v4f acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int n = 0; n < NT; n += kBF ? 2 : 1) {
          if (n >= nt) continue;
          const F s0 = frag_along<T>(sS, NP, 16 * pt, 16 * n, lr, lq);
          if constexpr (kBF) acc = mma32(s0, frag_along<T>(sS, NP, 16 * pt, 16 * n + 16, lr, lq), own_b(n), own_b(n + 1), acc);
          else acc = mma16<T>(s0, own_b(n), acc);
        }
        acc *= ew;
        // (G L)^T rows: blocks of t before the wavefront's own are not written, nor read
#pragma unroll
        for (int tb = 0; tb < QB; tb += kBF ? 2 : 1) {
          if (tb + (kBF ? 1 : 0) < tok) continue;
          const F y0 = frag_down<T>(sY, XP, 16 * tb, 16 * pt, lr, lq);
          const F w0 = tb >= tok ? frag_along<T>(sGl, GP, 16 * tok, 16 * tb, lr, lq) : tofrag<T>(0.0f, 0.0f, 0.0f, 0.0f);
          if constexpr (kBF) {
            const F w1 = frag_along<T>(sGl, GP, 16 * tok, 16 * tb + 16, lr, lq);
            acc = mma32(y0, frag_down<T>(sY, XP, 16 * tb + 16, 16 * pt, lr, lq), w0, w1, acc);
            if constexpr (kGate)
              acc = mma32(frag_down<T>(sY + kPartY, XP, 16 * tb, 16 * pt, lr, lq), frag_down<T>(sY + kPartY, XP, 16 * tb + 16, 16 * pt, lr, lq),
                          w0, w1, acc);
          } else {
            acc = mma16<T>(y0, w0, acc);
          }
        }
        if (own >= k.len || c0 >= cols) continue;
        float d[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float dy = Lds<T>::f(sY[own * XP + c0 + e]);
          if constexpr (kYP > 1) dy += Lds<T>::f(sY[kPartY + own * XP + c0 + e]);
          d[e] = fmaf(dl_s, acc[e], Dh * dy);
        }
        const uint32_t off = (own * p.H * p.P + c0) * static_cast<uint32_t>(sizeof(T));
        if constexpr (kVec && kBF) {
          __builtin_amdgcn_raw_buffer_store_b64(v2u{pack_bf16x2(d[0], d[1]), pack_bf16x2(d[2], d[3])}, dx, off, 0, 0);
        } else if constexpr (kVec) {
          __builtin_amdgcn_raw_buffer_store_b128(v4u{__float_as_uint(d[0]), __float_as_uint(d[1]), __float_as_uint(d[2]), __float_as_uint(d[3])},
                                                 dx, off, 0, 0);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (c0 + e < cols) Elem<T>::store(dx, off + e * static_cast<uint32_t>(sizeof(T)), d[e]);
        }
      }
    }
    __syncthreads();   // the sums are there, and LDS is free
    if (wave == i) {   // the steps' gradients; written over after the next barrier
      const int me = anew(lane);
      const float dl = sh.dl[i][me];
      float g0 = 0.0f;
#pragma unroll
      for (int w = 0; w < kGradThreads / 64; ++w) g0 += sh.pairs[w];
      // from the lane's token on: sums over its block, and the totals of later blocks
      const int block = me / 16;
      const float* const of_block = sums_row(me);
      const float r = row_suffix_sum(sums_rc(me)[0] + sums_rc(me)[1]);
      const float u0 = row_suffix_sum(block > 0 ? of_block[0] : 0.0f), u1 = row_suffix_sum(block > 1 ? of_block[1] : 0.0f),
                  u2 = row_suffix_sum(block > 2 ? of_block[2] : 0.0f);
      const float r3 = lane_value(r, 48), r23 = lane_value(r, 32) + r3, u03 = lane_value(u0, 48);
      const float later = block == 0   ? lane_value(r, 16) + r23
                          : block == 1 ? r23 + (lane_value(u0, 32) + u03)
                          : block == 2 ? r3 + (u03 + lane_value(u1, 48))
                                       : 0.0f;
      const float after = (r + u0) + (u1 + u2) + sh.in_block[me] + later;
      // and of the tokens before the lane's
      auto c_of = [&](int u) { return sums_rc(u)[2] + sums_rc(u)[3]; };
      auto below_of = [&](int u) { return sh.below[0][u] + sh.below[1][u]; };
      const int u = max(me - 1, 0);
      const float dl_u = me ? sh.dl[i][u] : 0.0f;
      const float flow = after + wave_prefix_sum(me ? c_of(u) * dl_u : 0.0f) +
                         row_prefix_sum(me % 16 ? below_of(u) * dl_u : 0.0f) + g0;
      float d = sh.col[me] + below_of(me) + c_of(me) + sh.A[i] * flow;
      d = me < k.len ? d * (p.softplus ? slope_of(dl) : 1.0f) : 0.0f;
      if (me < k.len) io<T>::store(static_cast<T*>(q.ddt) + (k.b * p.L + k.t0 + me) * p.H + h, d);
      const float da = wave_sum(dl * flow), db = wave_sum(d);
      float dd = 0.0f;
      if constexpr (kOwnD) {
#pragma unroll
        for (int w = 0; w < kGradThreads / 64; ++w) dd += sh.dd[w];
      } else {
        dd = wave_sum(sh.m[me]);
      }
      if (me < 3) q.parts[(static_cast<int64_t>(me) * p.H + h) * p.nc + c] = me == 0 ? da : me == 1 ? db : dd;
    }
  }

  __syncthreads();   // the last head's sums lie in the tiles' rows

  // dB and dC of the chunk: the products with C and B, over the sum of the heads
  E* const sG = lds + kG;   // [t][s]
  E* const sGt = sGl;       // [s][t]
  static_assert(kKeep ? kGl >= kQ * GP : kGl >= kEnds, "the two lie apart, and past B and C");
  if constexpr (!kKeep) stage_bc();
#pragma unroll
  for (int j = 0; j < kTiles; ++j) {
    const int tb = block_of(j);
    if (tb >= QB) continue;
    *reinterpret_cast<F*>(sGt + own * GP + 16 * tb + 4 * lq) = tofrag<T>(sum[j][0], sum[j][1], sum[j][2], sum[j][3]);
#pragma unroll
    for (int e = 0; e < 4; ++e) sG[(16 * tb + 4 * lq + e) * GP + own] = Lds<T>::from(sum[j][e]);
  }
  __syncthreads();
  typename SumOf<T>::V to_b[NH], to_c[NH];
#pragma unroll
  for (int n = 0; n < NH; ++n) {
    to_b[n] = go_on_16<T>(dB[n]);
    to_c[n] = go_on_16<T>(dC[n]);
  }
#pragma unroll
  for (int tb = 0; tb < QB; ++tb) {
    if (tb >= tok) {
      const F gf = frag_along<T>(sGt, GP, 16 * tok, 16 * tb, lr, lq);
#pragma unroll
      for (int n = 0; n < NH; ++n)
        if (n0 + n < nt) to_b[n] = mma16<T>(frag_down<T>(sC, NP, 16 * tb, 16 * (n0 + n), lr, lq), gf, to_b[n]);
    }
    if (tb <= tok) {
      const F gf = frag_along<T>(sG, GP, 16 * tok, 16 * tb, lr, lq);
#pragma unroll
      for (int n = 0; n < NH; ++n)
        if (n0 + n < nt) to_c[n] = mma16<T>(frag_down<T>(sB, NP, 16 * tb, 16 * (n0 + n), lr, lq), gf, to_c[n]);
    }
  }
  if (own >= k.len) return;
  const int64_t token = k.b * p.L + k.t0 + own, at = (token * p.G + g) * p.N;
#pragma unroll
  for (int n = 0; n < NH; ++n) {
    const int s0 = 16 * (n0 + n) + 4 * lq;
    if (s0 >= p.N) continue;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      v4f v;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = value_of(which ? to_c[n] : to_b[n], e);
      if (p.blocks > 1) {
        float* const to = (which ? q.dCparts : q.dBparts) + block * q.tokens * p.G * p.N + at + s0;
        if constexpr (kVec) {
          *reinterpret_cast<v4f*>(to) = v;
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (s0 + e < p.N) to[e] = v[e];
        }
      } else {
        T* const to = static_cast<T*>(which ? q.dC : q.dB) + at + s0;
        if constexpr (kVec) {
          if constexpr (kBF) *reinterpret_cast<uint2*>(to) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
          else *reinterpret_cast<v4f*>(to) = v;
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (s0 + e < p.N) io<T>::store(to + e, v[e]);
        }
      }
    }
  }
}

// What the workgroups left in parts, each sum in a fixed order.  The first workgroups:
// dA, ddt_bias and dD of a head, over its chunks; the others, where a group's heads
// were several workgroups': dB and dC (packed: only for tokens of a sequence; the
// others' rows are cleared elsewhere).  One launch for both: each would take 4 us
// however little it does.
struct SumParams {
  const float* parts;      // [3][H][nc]
  const float* bc;         // [2][blocks][n]
  const int32_t* cu;
  int64_t nseq, L, n, row; // elements of dB (and of dC), and of a token of theirs
  int nc, H, blocks;
  int of_heads;            // workgroups for the 3 H sums over chunks
  float *dA, *dbias, *dD;
  void *dB, *dC;
};
// kV: values of a lane, 4 where rows allow it.
template <typename T, int kV>
__global__ __launch_bounds__(kThreads) void ssd_sum_parts_kernel(SumParams p) {
  struct alignas(kV * 4) Part { float e[kV]; };
  struct alignas(kV * sizeof(T)) Out { T e[kV]; };
  if (static_cast<int>(blockIdx.x) < p.of_heads) {
    __shared__ float sums[kWaves];
    for (int i = blockIdx.x; i < 3 * p.H; i += p.of_heads) {
      const int h = i / 3, which = i % 3;
      const float* const from = p.parts + (static_cast<int64_t>(which) * p.H + h) * p.nc;
      float s = 0.0f;
      for (int c = threadIdx.x; c < p.nc; c += kThreads) s += from[c];
      s = wave_sum(s);
      if (threadIdx.x % 64 == 0) sums[threadIdx.x / 64] = s;
      __syncthreads();
      float* const to = which == 0 ? p.dA : which == 1 ? p.dbias : p.dD;
      if (threadIdx.x == 0 && to) to[h] = (sums[0] + sums[1]) + (sums[2] + sums[3]);
      __syncthreads();
    }
    return;
  }
  int64_t lo = 0, hi = p.n;
  if (p.cu) {
    lo = min(max(int64_t{p.cu[0]}, int64_t{0}), p.L) * p.row;
    hi = min(max(int64_t{p.cu[p.nseq]}, int64_t{0}), p.L) * p.row;
  }
  const int id = blockIdx.x - p.of_heads, step = (gridDim.x - p.of_heads) / 2;
  const float* const from = p.bc + (id & 1) * p.blocks * p.n;
  T* const to = static_cast<T*>(id & 1 ? p.dC : p.dB);
  for (int64_t i = (static_cast<int64_t>(id >> 1) * kThreads + threadIdx.x) * kV; i < p.n; i += static_cast<int64_t>(step) * kThreads * kV) {
    if (i < lo || i >= hi) continue;
    float s[kV] = {};
    for (int b = 0; b < p.blocks; ++b) {
      const Part v = *reinterpret_cast<const Part*>(from + b * p.n + i);
#pragma unroll
      for (int e = 0; e < kV; ++e) s[e] += v.e[e];
    }
    Out o;
#pragma unroll
    for (int e = 0; e < kV; ++e) io<T>::store(&o.e[e], s[e]);
    *reinterpret_cast<Out*>(to + i) = o;
  }
}

size_t align_up(size_t n) { return (n + 255) / 256 * 256; }

// Where the parts of a workspace lie (bytes).
struct Layout {
  size_t table, seq_chunk, lam, state, dstate, parts, bc, size;
};
Layout layout_of(const ChunkPlan& q, bool packed, bool backward, int64_t nseq, int64_t H, int64_t P, int64_t N, int64_t G, int64_t tokens) {
  Layout l;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += align_up(bytes);
    return here;
  };
  const size_t states = static_cast<size_t>(q.nc) * H * P * N * 4;
  l.table = take(packed ? static_cast<size_t>(q.nc) * sizeof(ChunkEntry) : 0);
  l.seq_chunk = take(packed ? static_cast<size_t>(nseq + 1) * 4 : 0);
  l.lam = take(static_cast<size_t>(q.nc) * H * 4);
  l.state = take(states);
  l.dstate = take(backward ? states : 0);
  l.parts = take(backward ? static_cast<size_t>(3) * H * q.nc * 4 : 0);
  l.bc = take(backward && q.blocks > 1 ? static_cast<size_t>(2) * q.blocks * tokens * G * N * 4 : 0);
  l.size = at;
  return l;
}

TokenTensor tensor(const void* ptr, int64_t sb, int64_t ss, int64_t sh, int64_t inner, bool bf16) {
  const int64_t piece = bf16 ? 8 : 4;
  const bool vec = inner % piece == 0 && reinterpret_cast<uintptr_t>(ptr) % 16 == 0 && sb % piece == 0 && ss % piece == 0 &&
                   sh % piece == 0;
  return TokenTensor{ptr, sb, ss, sh, vec};
}

template <typename T, int NMAX>
void launch_grad(const ChunkParams& p, const GradParams& q, hipStream_t stream) {
  const int grid = p.nc * p.G * p.blocks;
  auto go = [&](auto gate, auto vec) {
    if (p.P <= kPB) ssd_grad_kernel<T, NMAX, gate.value, vec.value, true><<<grid, kGradThreads, 0, stream>>>(p, q, grid);
    else ssd_grad_kernel<T, NMAX, gate.value, vec.value, false><<<grid, kGradThreads, 0, stream>>>(p, q, grid);
  };
  if (p.z.p && p.vec) go(std::true_type{}, std::true_type{});
  else if (p.z.p) go(std::true_type{}, std::false_type{});
  else if (p.vec) go(std::false_type{}, std::true_type{});
  else go(std::false_type{}, std::false_type{});
}

// The parameters that both calls have.
template <typename Args>
ChunkParams params_of(const Args& a, const ChunkPlan& q, const Layout& l, bool packed) {
  char* const ws = static_cast<char*>(a.workspace);
  ChunkParams p{};
  p.A = a.A;
  p.D = a.D;
  p.bias = a.dt_bias;
  p.L = static_cast<int>(a.seqlen);
  p.H = static_cast<int>(a.nheads);
  p.P = static_cast<int>(a.headdim);
  p.G = static_cast<int>(groups_of(a.ngroups));
  p.N = static_cast<int>(a.dstate);
  p.per_group = p.H / p.G;
  p.softplus = a.dt_softplus != 0;
  p.nc = static_cast<int>(q.nc);
  p.per_row = static_cast<int>(q.per_row);
  p.hb = static_cast<int>(q.hb);
  p.blocks = static_cast<int>(q.blocks);
  p.table = packed ? reinterpret_cast<const ChunkEntry*>(ws + l.table) : nullptr;
  p.seq_chunk = packed ? reinterpret_cast<const int32_t*>(ws + l.seq_chunk) : nullptr;
  p.lam = reinterpret_cast<float*>(ws + l.lam);
  p.state = reinterpret_cast<float*>(ws + l.state);
  p.dstate = reinterpret_cast<float*>(ws + l.dstate);
  p.dt = a.dt;
  p.dts = a.dt_seq_stride;
  return p;
}

ChunkPlan plan_of(const ssm_ssd_packed_args& a) {
  return chunk_plan(1, a.seqlen, a.nseq, true, a.nheads, groups_of(a.ngroups));
}
ChunkPlan plan_of(const ssm_ssd_bwd_args& a) {
  return chunk_plan(a.batch, a.seqlen, a.nseq, a.cu_seqlens != nullptr, a.nheads, groups_of(a.ngroups));
}
Layout layout(const ssm_ssd_packed_args& a, const ChunkPlan& q) {
  return layout_of(q, true, false, a.nseq, a.nheads, a.headdim, a.dstate, groups_of(a.ngroups), a.seqlen);
}
Layout layout(const ssm_ssd_bwd_args& a, const ChunkPlan& q) {
  return layout_of(q, a.cu_seqlens != nullptr, true, a.nseq, a.nheads, a.headdim, a.dstate, groups_of(a.ngroups),
                   a.batch * a.seqlen);
}

}  // namespace

size_t ssd_packed_workspace_bytes(const ssm_ssd_packed_args& a) { return layout(a, plan_of(a)).size; }
size_t ssd_bwd_workspace_bytes(const ssm_ssd_bwd_args& a) { return layout(a, plan_of(a)).size; }

hipError_t launch_ssd_packed_fwd(const ssm_ssd_packed_args& a, hipStream_t stream) {
  const ChunkPlan q = plan_of(a);
  const Layout l = layout(a, q);
  const bool bf16 = a.io_dtype == SSM_BF16;
  const int64_t es = bf16 ? 2 : 4;
  ChunkParams p = params_of(a, q, l, true);
  const int64_t Bg = p.G > 1 ? a.B_group_stride : 0, Cg = p.G > 1 ? a.C_group_stride : 0;
  p.x = tensor(a.x, 0, a.x_seq_stride, a.x_head_stride, p.P, bf16);
  p.z = tensor(a.z, 0, a.z_seq_stride, a.z_head_stride, p.P, bf16);
  p.B = tensor(a.B, 0, a.B_seq_stride, Bg, p.N, bf16);
  p.C = tensor(a.C, 0, a.C_seq_stride, Cg, p.N, bf16);
  p.bc_vec = p.B.vec && p.C.vec;
  p.vec = p.x.vec && p.N % 4 == 0 && tensor(a.out, 0, a.out_seq_stride, a.out_head_stride, p.P, bf16).vec &&
          (!a.z || p.z.vec);
  OutsideRows rows;
  if (a.zero_outside && a.seqlen > 0) {
    const bool whole = a.out_head_stride == a.headdim;   // the heads side by side
    rows.add(a.out, (whole ? a.nheads : 1) * a.headdim * es, a.out_seq_stride * es, whole ? 1 : a.nheads, a.out_head_stride * es);
  }
  hipError_t e = launch_chunk_table(a.cu_seqlens, a.seqlen, a.nseq, q.nc, reinterpret_cast<ChunkEntry*>(static_cast<char*>(a.workspace) + l.table),
                                    reinterpret_cast<int32_t*>(static_cast<char*>(a.workspace) + l.seq_chunk), rows, stream);
  if (e != hipSuccess) return e;
  e = launch_chunk_states(p, bf16, false, a.nseq, a.h0, a.last_state, nullptr, nullptr, stream);
  if (e != hipSuccess) return e;
  const ChunkOut o{a.out, 0, a.out_seq_stride, a.out_head_stride, nullptr};
  return launch_chunk_outputs(p, o, bf16, stream);
}

hipError_t launch_ssd_bwd(const ssm_ssd_bwd_args& a, hipStream_t stream) {
  const ChunkPlan q = plan_of(a);
  const Layout l = layout(a, q);
  const bool bf16 = a.io_dtype == SSM_BF16, packed = a.cu_seqlens != nullptr;
  const int64_t es = bf16 ? 2 : 4;
  char* const ws = static_cast<char*>(a.workspace);
  ChunkParams p = params_of(a, q, l, packed);
  const int64_t Bg = p.G > 1 ? a.B_group_stride : 0, Cg = p.G > 1 ? a.C_group_stride : 0;
  p.dtb = a.dt_batch_stride;
  p.x = tensor(a.x, a.x_batch_stride, a.x_seq_stride, a.x_head_stride, p.P, bf16);
  p.z = tensor(a.z, a.z_batch_stride, a.z_seq_stride, a.z_head_stride, p.P, bf16);
  p.B = tensor(a.B, a.B_batch_stride, a.B_seq_stride, Bg, p.N, bf16);
  p.C = tensor(a.C, a.C_batch_stride, a.C_seq_stride, Cg, p.N, bf16);
  p.bc_vec = p.B.vec && p.C.vec;
  p.dout = tensor(a.dout, a.dout_batch_stride, a.dout_seq_stride, a.dout_head_stride, p.P, bf16);
  auto aligned = [](const void* ptr) { return reinterpret_cast<uintptr_t>(ptr) % 16 == 0; };
  p.vec = p.x.vec && p.N % 4 == 0 && p.dout.vec && aligned(a.dx) && aligned(a.dB) && aligned(a.dC) &&
          (!a.z || (p.z.vec && aligned(a.dz)));
  const int64_t HP = a.nheads * a.headdim, GN = static_cast<int64_t>(p.G) * p.N;
  hipError_t e = hipSuccess;
  if (packed) {
    OutsideRows rows;
    if (a.seqlen > 0) {
      rows.add(a.dx, HP * es, HP * es);
      rows.add(a.ddt, a.nheads * es, a.nheads * es);
      rows.add(a.dB, GN * es, GN * es);
      rows.add(a.dC, GN * es, GN * es);
      if (a.z) rows.add(a.dz, HP * es, HP * es);
    }
    e = launch_chunk_table(a.cu_seqlens, a.seqlen, a.nseq, q.nc, reinterpret_cast<ChunkEntry*>(ws + l.table),
                           reinterpret_cast<int32_t*>(ws + l.seq_chunk), rows, stream);
    if (e != hipSuccess) return e;
  }
  e = launch_chunk_states(p, bf16, true, packed ? a.nseq : a.batch, a.h0, nullptr, a.dlast, a.dh0, stream);
  if (e != hipSuccess) return e;
  if (q.nc > 0) {
    if (a.z) {
      const ChunkOut o{nullptr, a.seqlen * HP, HP, a.headdim, a.dz};
      e = launch_chunk_outputs(p, o, bf16, stream);
      if (e != hipSuccess) return e;
    }
    GradParams g{a.dx, a.ddt, a.dB, a.dC, reinterpret_cast<float*>(ws + l.parts), reinterpret_cast<float*>(ws + l.bc), nullptr,
                 a.batch * a.seqlen};
    g.dCparts = g.dBparts + q.blocks * g.tokens * GN;
    if (!bf16) launch_grad<float, 64>(p, g, stream);
    else if (p.N > 64) launch_grad<uint16_t, 128>(p, g, stream);
    else launch_grad<uint16_t, 64>(p, g, stream);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  SumParams m{reinterpret_cast<float*>(ws + l.parts), reinterpret_cast<float*>(ws + l.bc), a.cu_seqlens, a.nseq, a.seqlen,
              a.batch * a.seqlen * GN, GN, p.nc, p.H, p.blocks, std::min(3 * p.H, 1 << 20), a.dA, a.ddt_bias, a.dD, a.dB, a.dC};
  const bool four = GN % 4 == 0 && aligned(a.dB) && aligned(a.dC);
  const int64_t per = kThreads * (four ? 4 : 1);
  const int64_t more = q.nc > 0 && q.blocks > 1 ? 2 * std::min<int64_t>((m.n + per - 1) / per, 4096) : 0;
  const unsigned grid = static_cast<unsigned>(m.of_heads + more);
  if (bf16 && four) ssd_sum_parts_kernel<uint16_t, 4><<<grid, kThreads, 0, stream>>>(m);
  else if (bf16) ssd_sum_parts_kernel<uint16_t, 1><<<grid, kThreads, 0, stream>>>(m);
  else if (four) ssd_sum_parts_kernel<float, 4><<<grid, kThreads, 0, stream>>>(m);
  else ssd_sum_parts_kernel<float, 1><<<grid, kThreads, 0, stream>>>(m);
  return hipGetLastError();
}

}  // namespace ssm
