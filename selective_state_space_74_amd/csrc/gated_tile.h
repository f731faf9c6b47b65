// Tiles, packed-sequence marks and the carry between tiles, shared by the
// gated recurrence's forward and backward kernels.
//
// A workgroup takes kWaveTokens tokens per wavefront of a group of channels,
// with its inputs kept in registers, so that the data is read once: the
// recurrence over a tile is h_out = P h_in + H, and only (P, H) of each tile
// has to travel to the tiles after it.
//
// The carry.  Tiles are numbered along the scan (backwards in time for the
// adjoint) and every chain_group() of them form a group.  A tile publishes its
// (P, H) as soon as it has them, without waiting for anything.  It then takes
// the state that left the group before, and folds the (P, H) of its
// predecessors within the group into it; the last tile of a group
// publishes the state that leaves the group.  The order of the products and
// sums is fixed, so results do not depend on which tile came first.
//
// Every wait ends.  A workgroup takes its tile from a counter (a ticket), so
// the tiles before it are held by workgroups that already run (or have run),
// whatever order the hardware dispatches in and whatever else shares the GPU.
// The running workgroup with the lowest ticket only waits for words that
// finished workgroups have written; hence it finishes, and so on upwards.
// (Without tickets two such kernels on two streams could hold each other's
// places: each resident on the compute units that the other's next tile
// needs.)
//
// Words.  A pair travels as one 64-bit word, written and read by relaxed
// atomics of device scope, so that no other memory needs ordering; the words
// are filled with kNoWord before the kernel, which no published pair equals:
// its low half would be one particular NaN, and NaNs are published as another.
// Bound by memory traffic (8 bytes a value forward in bf16, 16 in fp32; 14 and
// 28 backward) with the vector units about two thirds busy, where there are many
// groups of channels and rows begin on cache lines: a call of 262,144 x 1536 bf16
// takes 576 us forward (5.6 TB/s), one of 4 x 4096 x 5120 bf16 366 us forward and
// backward (5.0 TB/s).  Few groups of channels are bound by the hops of the carry
// (2,052,244 x 31 bf16 forward 241 us for 0.5 GB), rows off the lines by lines that
// two workgroups share (9 x 1386 x 1796 bf16 forward and backward 153 us for 0.5 GB).
#pragma once

#include "gated_math.h"

namespace ssm {

constexpr int kWaveTokens = 16;   // tokens of a wavefront (the backward with two channels a lane: 8)
constexpr int kMaxWaves = 8;
// Tiles of a group.  A call of few channels is one chain, which the way from
// group to group bounds, so narrow calls have longer ones: 2,052,244 x 31 bf16
// takes 249 us forward with 32 tiles and 355 with 16 (64: 225, but from 8 packed
// sequences 265 as with 32, and the backward 431 against 388).  Elsewhere the
// words to fetch count: 16 / 32 / 64 tiles 372 / 403 / 572 us at 4 x 4096 x 5120
// bf16 training.
constexpr int chain_group(bool narrow) { return narrow ? 32 : 16; }
// Words of predecessors that a thread fetches at most: the workgroup has 8 / V
// threads a channel, 16 or more in a narrow call.
constexpr int chain_mine(bool narrow, int V) {
  const int parts = narrow ? 2 * kMaxWaves : kMaxWaves / V;
  return (chain_group(narrow) - 1 + parts - 1) / parts;
}
constexpr uint64_t kNoWord = ~uint64_t{0};

__device__ __forceinline__ uint64_t chain_word(float p, float h) {
  const uint32_t lo = p != p ? 0x7fc00000u : __float_as_uint(p);
  return lo | static_cast<uint64_t>(__float_as_uint(h)) << 32;
}
__device__ __forceinline__ float word_p(uint64_t w) { return __uint_as_float(static_cast<uint32_t>(w)); }
__device__ __forceinline__ float word_h(uint64_t w) { return __uint_as_float(static_cast<uint32_t>(w >> 32)); }

__device__ __forceinline__ void chain_store(uint64_t* p, uint64_t w) {
  __hip_atomic_store(p, w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint64_t chain_load(uint64_t* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// A word that is awaited.  By the argument above it comes within microseconds; a
// workspace that another call overwrites meanwhile, which the interface forbids,
// could take it away, and then the wait is given up after some seconds with
// kNoWord itself, whose halves are NaNs: wrong use shows as NaN outputs and not
// as a GPU that hangs.
constexpr int kPolls = 1 << 22;
__device__ __forceinline__ uint64_t chain_wait(uint64_t* p, uint64_t w) {
  for (int i = 0; w == kNoWord && i < kPolls; ++i) {
    __builtin_amdgcn_s_sleep(1);
    w = chain_load(p);
  }
  return w;
}

// A stretch of packed tokens in which a sequence begins passes nothing on.
// That is not P = 0, which would turn an infinity or a NaN of the sequence
// before into a NaN: it is marked by a negative P, which no product of decays
// is.
constexpr float kCut = -1.0f;
template <bool PACKED>
__device__ __forceinline__ float chain_apply(float p, float h, float in) {
  const float r = fmaf(p, in, h);
  return PACKED && p < 0.0f ? h : r;
}
// P of a stretch (p) followed by another (q).
template <bool PACKED>
__device__ __forceinline__ float chain_product(float p, float q) {
  return PACKED && (p < 0.0f || q < 0.0f) ? kCut : p * q;
}

// Where one group of `width` channels of one batch row keeps its words: tile
// k's pair at tiles[k * width], the state leaving group j at groups[j * width].
struct Chain {
  uint64_t* tiles;
  uint64_t* groups;
  int64_t width;
};

// What a workgroup keeps of the tiles before it, and the state entering it.
template <int W, int GROUP>
struct ChainShared {
  float2 tiles[GROUP - 1][W];
  float entering[W];
};

// Called by all threads of a tile once its wavefronts' pairs are in LDS, `order`
// giving the wavefront that the scan passes w-th; `first` is the state entering
// tile 0, for channel threadIdx.x of the first 2^shift threads.  On return
// sh.entering holds the state entering tile k.
//
// The tile's pair goes out before anything is waited for.  The predecessors'
// words are brought into LDS by all wavefronts, at most MINE a thread, so that
// their latencies run side by side and none holds them all in registers.  They
// are folded into one pair, and the tile's own wavefronts into another, before
// the state that left the group before is asked for: from group to group the
// carry costs one product, one read and one write.
template <bool PACKED, int W, int GROUP, int MINE, typename Order>
__device__ __forceinline__ void chain_carry(const Chain& c, int64_t k, int64_t ntiles, float2 (&pairs)[kMaxWaves][W],
                                            ChainShared<W, GROUP>& sh, int shift, float first, Order order) {
  const int parts = (64 * kMaxWaves) >> shift;
  const int ch = threadIdx.x & ((1 << shift) - 1), part = threadIdx.x >> shift;
  const int in_group = static_cast<int>(k % GROUP);
  const int64_t group = k / GROUP;
  uint64_t* const mine = c.tiles + k * c.width + ch;
  float2 own = make_float2(1.0f, 0.0f);
  if (part == 0) {
#pragma unroll
    for (int w = 0; w < kMaxWaves; ++w) {
      const float2 q = pairs[order(w)][ch];
      own = make_float2(chain_product<PACKED>(own.x, q.x), chain_apply<PACKED>(q.x, q.y, own.y));
    }
    if (in_group != GROUP - 1) chain_store(mine, chain_word(own.x, own.y));
  }
  uint64_t w[MINE];
#pragma unroll
  for (int i = 0; i < MINE; ++i)
    if (part + i * parts < in_group) w[i] = chain_load(mine - (in_group - part - i * parts) * c.width);
#pragma unroll
  for (int i = 0; i < MINE; ++i) {
    const int j = part + i * parts;
    if (j < in_group) {
      w[i] = chain_wait(mine - (in_group - j) * c.width, w[i]);
      sh.tiles[j][ch] = make_float2(word_p(w[i]), word_h(w[i]));
    }
  }
  __syncthreads();
  if (part == 0) {
    float2 q = make_float2(1.0f, 0.0f);   // of the group's tiles before this one
#pragma unroll
    for (int j = 0; j < GROUP - 1; ++j) {
      if (j < in_group) {
        const float2 t = sh.tiles[j][ch];
        q = make_float2(chain_product<PACKED>(q.x, t.x), chain_apply<PACKED>(t.x, t.y, q.y));
      }
    }
    uint64_t* const left = c.groups + (group - 1) * c.width + ch;
    const float h = chain_apply<PACKED>(q.x, q.y, group > 0 ? word_h(chain_wait(left, chain_load(left))) : first);
    if (in_group == GROUP - 1 && k + 1 < ntiles)
      chain_store(c.groups + group * c.width + ch, chain_word(0.0f, chain_apply<PACKED>(own.x, own.y, h)));
    sh.entering[ch] = h;
  }
  __syncthreads();
}

// Narrow calls: a wavefront's lanes hold 64 >> shift stretches of 2^shift
// channels, in the scan's order (from the last stretch to the first for REV).
// Turns each lane's pair into that of the stretches before its own, and returns
// the whole wavefront's in the lanes of the stretch that the scan reaches last.
template <bool PACKED, bool REV>
__device__ __forceinline__ float2 wave_stretches(int shift, float& p, float& h) {
  const int lane = threadIdx.x & 63, rank = REV ? 63 - lane : lane;
  float ip = p, ih = h;
  for (int k = 1 << shift; k < 64; k <<= 1) {
    const float pp = REV ? __shfl_down(ip, k) : __shfl_up(ip, k), hh = REV ? __shfl_down(ih, k) : __shfl_up(ih, k);
    if (rank >= k) {
      ih = chain_apply<PACKED>(ip, ih, hh);
      ip = chain_product<PACKED>(pp, ip);
    }
  }
  const int one = 1 << shift;
  const float pp = REV ? __shfl_down(ip, one) : __shfl_up(ip, one), hh = REV ? __shfl_down(ih, one) : __shfl_up(ih, one);
  p = rank >= one ? pp : 1.0f;
  h = rank >= one ? hh : 0.0f;
  return make_float2(ip, ih);
}

// Marks of a packed token: the sequence it belongs to and whether it is its
// first or last token; kOutside: in no sequence.
constexpr int32_t kOutside = -1;   // its lowest bit, too, says that no state comes in
__device__ __forceinline__ int32_t mark_of(int32_t seq, bool first, bool last) {
  return seq << 2 | (first ? 1 : 0) | (last ? 2 : 0);
}

// Before the scan: chain words to kNoWord, the ticket counter to 0, and with
// cu_seqlens the token marks and the last states of empty sequences.
// `empty_out` receives, for each empty sequence, the row of `empty_in` (or
// zeros).
struct PrepParams {
  uint32_t* ticket;
  uint64_t* words;
  int64_t nwords;
  const int32_t* cu;
  int32_t* marks;
  const float* empty_in;
  float* empty_out;
  int64_t L, nseq, D;
};
hipError_t launch_gated_prep(const PrepParams& p, hipStream_t stream);

// V consecutive channels of a token as they are stored, at most 4 bytes: one
// fp32, one or two bf16.
template <typename T, int V>
__device__ __forceinline__ float widen(uint32_t raw, int v) {
  if constexpr (sizeof(T) == 4) return __uint_as_float(raw);
  else return __uint_as_float(v == 0 ? raw << 16 : raw & 0xffff0000u);
}
template <typename T, int V>
__device__ __forceinline__ uint32_t narrow(const float (&h)[V]) {
  if constexpr (sizeof(T) == 4) {
    return __float_as_uint(h[0]);
  } else if constexpr (V == 1) {
    return f32_to_bf16(h[0]);
  } else {
    typedef float f2 __attribute__((ext_vector_type(2)));
    typedef __bf16 b2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f2{h[0], h[1]}, b2));   // one v_cvt_pk_bf16_f32
  }
}

// Cache policy of the token rows.  Where every row begins on a cache line each
// byte passes once, and the nontemporal bit helps (2 x 8587 x 2304 bf16 forward
// and backward: 195 us, and 205 us without).
// Otherwise two wavefronts share the lines at their border, which have to stay
// until both have had them: 2 x 8587 x 2306 bf16 training takes 251 us with the
// plain policy and 278 us with the nontemporal one.
constexpr int kPlain = 0, kStream = 2;
constexpr int64_t kLine = 128;
inline bool on_lines(const void* p, int64_t batch_stride, int64_t seq_stride, int64_t esz) {
  return reinterpret_cast<uintptr_t>(p) % kLine == 0 && batch_stride * esz % kLine == 0 && seq_stride * esz % kLine == 0;
}

// One tensor's rows from a wavefront's first token on.  A row is reached
// through a buffer descriptor of its own: the descriptor is scalar work, the
// lane's offset the same for every row, and lanes past the channels read zeros
// and write nothing.  `subs` rows of 16 tokens apart are reached through one
// descriptor (narrow calls); a lane without a token there has offset kNowhere.
// The _within forms also read zeros and write nothing past `left` tokens: their
// descriptors end behind the last row, that is there.
constexpr uint32_t kNowhere = ~0u;
struct TokenRows {
  char* first;
  int64_t stride;     // bytes
  uint32_t bytes, row_bytes;
  int left;
  template <typename T>
  __device__ __forceinline__ void set(const void* p, int64_t elements, int64_t row_stride, int64_t D, int subs,
                                      int64_t tokens, T) {
    first = static_cast<char*>(const_cast<void*>(p)) + elements * static_cast<int64_t>(sizeof(T));
    stride = row_stride * static_cast<int64_t>(sizeof(T));
    row_bytes = static_cast<uint32_t>(D * static_cast<int64_t>(sizeof(T)));
    bytes = static_cast<uint32_t>((subs - 1) * kWaveTokens * stride) + row_bytes;
    left = static_cast<int>(min(tokens, static_cast<int64_t>(subs * kWaveTokens)));
  }
  __device__ __forceinline__ __amdgpu_buffer_rsrc_t row(int j, uint32_t n) const {
    return __builtin_amdgcn_make_buffer_rsrc(first + j * stride, 0, static_cast<int>(n), kRsrcWord3);
  }
  // bytes of the rows j, j + 16, ... that are there
  __device__ __forceinline__ uint32_t within(int j) const {
    return left <= j ? 0u : static_cast<uint32_t>((left - j - 1) / kWaveTokens * kWaveTokens * stride) + row_bytes;
  }
  template <int BYTES, int CACHE>
  static __device__ __forceinline__ uint32_t load(__amdgpu_buffer_rsrc_t r, uint32_t at) {
    if constexpr (BYTES == 4) return __builtin_amdgcn_raw_buffer_load_b32(r, at, 0, CACHE);
    else return __builtin_amdgcn_raw_buffer_load_b16(r, at, 0, CACHE);
  }
  template <int BYTES, int CACHE>
  static __device__ __forceinline__ void store(__amdgpu_buffer_rsrc_t r, uint32_t at, uint32_t v) {
    if constexpr (BYTES == 4) __builtin_amdgcn_raw_buffer_store_b32(v, r, at, 0, CACHE);
    else __builtin_amdgcn_raw_buffer_store_b16(static_cast<uint16_t>(v), r, at, 0, CACHE);
  }
  template <int BYTES, int CACHE>
  __device__ __forceinline__ uint32_t load(int j, uint32_t at) const { return load<BYTES, CACHE>(row(j, bytes), at); }
  template <int BYTES, int CACHE>
  __device__ __forceinline__ void store(int j, uint32_t at, uint32_t v) const {
    store<BYTES, CACHE>(row(j, bytes), at, v);
  }
  template <int BYTES, int CACHE>
  __device__ __forceinline__ uint32_t load_within(int j, uint32_t at) const {
    return load<BYTES, CACHE>(row(j, within(j)), at);
  }
  template <int BYTES, int CACHE>
  __device__ __forceinline__ void store_within(int j, uint32_t at, uint32_t v) const {
    store<BYTES, CACHE>(row(j, within(j)), at, v);
  }
};
template <typename T>
__device__ __forceinline__ TokenRows token_rows(const void* p, int64_t elements, int64_t row_stride, int64_t D,
                                                int subs = 1, int64_t left = 0) {
  TokenRows r;
  r.set(p, elements, row_stride, D, subs, left, T{});
  return r;
}

// How a call is cut into workgroups, and the parts of its workspace (bytes
// from its start, each 256-byte aligned).
struct GatedPlan {
  int waves;            // wavefronts a workgroup
  int shift;            // see gated_plan
  int64_t tiles, cols;  // along the sequence, along the channels
  int64_t words;        // 0: one tile a sequence, no chain
  int64_t marks_at, words_at, parts_at, bytes;
};

// shift: 0, or log2 of the channels that a wavefront of a narrow call takes for
// each of its 64 >> shift blocks of tokens.
inline GatedPlan gated_plan(int64_t batch, int64_t L, int64_t D, bool packed, int V, int tokens, int shift,
                            int64_t part_rows_per_tile) {
  auto round256 = [](int64_t v) { return (v + 255) / 256 * 256; };
  GatedPlan q{};
  const int64_t width = shift ? int64_t{1} << shift : 64 * V, subs = shift ? 64 >> shift : 1;
  const int64_t blocks = (L + tokens - 1) / tokens, wave_blocks = (blocks + subs - 1) / subs;
  q.shift = shift;
  q.waves = static_cast<int>(wave_blocks < 1 ? 1 : wave_blocks < kMaxWaves ? wave_blocks : kMaxWaves);
  q.tiles = (wave_blocks + q.waves - 1) / q.waves;
  q.cols = (D + width - 1) / width;
  const int64_t group = chain_group(shift != 0);
  q.words = q.tiles > 1 ? batch * q.cols * (q.tiles + (q.tiles + group - 1) / group) * width : 0;
  q.marks_at = q.words ? 256 : 0;   // the ticket counter
  q.words_at = q.marks_at + (packed ? round256((L + kWaveTokens - 1) / kWaveTokens * kWaveTokens * 4) : 0);
  q.parts_at = q.words_at + round256(q.words * 8);
  q.bytes = q.parts_at + part_rows_per_tile * q.tiles * batch * D * 4;
  return q;
}

// Channels of up to 32 leave half of a wavefront's lanes or more without work,
// and the carry through its tiles, one after another, then bounds long
// sequences (337,272 packed x 13 fp32: 214 us for 70 MB): there a wavefront
// takes several blocks of 16 tokens side by side.
inline int narrow_shift(int64_t D) { return D > 32 ? 0 : D > 16 ? 5 : D > 8 ? 4 : 3; }
// Its rows are 16 tokens apart behind one descriptor, of less than 4 GB.
inline bool narrow_fits(int64_t D, int64_t row_stride, int64_t esz) {
  const int64_t subs = 64 >> narrow_shift(D);
  return row_stride < (int64_t{1} << 31) / (subs * kWaveTokens * esz);
}

// Workspace for whichever form runs; it depends on no address.  Of a narrow call
// (shift) whose strides are not known yet, for the wide forms too: it may turn out
// not to fit.  plan_of(V, shift) is a form's plan.
template <typename PlanOf>
size_t gated_bytes(int shift, bool strides_known, PlanOf plan_of) {
  int64_t bytes = shift ? plan_of(1, shift).bytes : 0;
  if (!shift || !strides_known) bytes = max(bytes, max(plan_of(1, 0).bytes, plan_of(2, 0).bytes));
  return static_cast<size_t>(bytes);
}

}  // namespace ssm
