// gated_prep.hip -- what the gated recurrence's kernels find ready in their
// workspace (see PrepParams), in one launch: a few bytes a token and channel
// group, a percent or two of the scan's own traffic.
#include "gated_tile.h"

namespace ssm {
namespace {

constexpr int kThreads = 256;

// Two chain words, stored at once: the workspace is 8-byte aligned, no more.
struct alignas(8) WordPair { uint64_t w[2]; };

__global__ __launch_bounds__(kThreads) void gated_prep_kernel(PrepParams p) {
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads;
  if (i0 == 0 && p.ticket) *p.ticket = 0;
  // words in pairs: their number is even (8 channels a group at least)
  WordPair* const w = reinterpret_cast<WordPair*>(p.words);
  for (int64_t i = i0; i < p.nwords / 2; i += step) w[i] = WordPair{{kNoWord, kNoWord}};
  if (p.marks) {
    // padded to whole wavefronts of tokens with tokens outside
    const int64_t n = (p.L + kWaveTokens - 1) / kWaveTokens * kWaveTokens;
    for (int64_t t = i0; t < n; t += step) {
      // entries not above t, by halving: the last of equal ones begins a
      // sequence that has tokens
      int64_t lo = 0, hi = p.nseq + 1;
      while (lo < hi) {
        const int64_t mid = (lo + hi) / 2;
        if (p.cu[mid] <= t) lo = mid + 1;
        else hi = mid;
      }
      const int64_t k = lo - 1;
      const bool in = k >= 0 && k < p.nseq && t < p.L;
      p.marks[t] = in ? mark_of(static_cast<int32_t>(k), p.cu[k] == t, p.cu[k + 1] == t + 1) : kOutside;
    }
  }
  if (p.empty_out)
    for (int64_t k = blockIdx.x; k < p.nseq; k += gridDim.x)
      if (p.cu ? p.cu[k + 1] <= p.cu[k] : p.L == 0)
        for (int64_t d = threadIdx.x; d < p.D; d += kThreads)
          p.empty_out[k * p.D + d] = p.empty_in ? p.empty_in[k * p.D + d] : 0.0f;
}

}  // namespace

hipError_t launch_gated_prep(const PrepParams& p, hipStream_t stream) {
  // a token's mark is a chain of dependent reads: a thread each where there
  // are not too many; words and states are plain streams
  int64_t blocks = (p.nwords / 2 + 4 * kThreads - 1) / (4 * kThreads);
  if (p.marks) blocks = max(blocks, (p.L + kThreads - 1) / kThreads);
  if (p.empty_out) blocks = max(blocks, min(p.nseq, int64_t{256}));
  blocks = max(int64_t{1}, min(blocks, int64_t{2048}));
  gated_prep_kernel<<<static_cast<unsigned>(blocks), kThreads, 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace ssm
