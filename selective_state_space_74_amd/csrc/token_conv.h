// What the token-major causal convolution and its backward share: the walk over
// sequences, and rows of channels.
#pragma once

#include "ssm_internal.h"

namespace ssm {

constexpr int kConvThreads = 256;
constexpr int kConvLanes = 16;                              // runs of channels side by side in a workgroup
constexpr int kConvRuns = kConvThreads / kConvLanes;        // runs of tokens in a workgroup
constexpr int kConvBounds = 1024;                           // sequence bounds held in LDS
constexpr int kConvV = 4;                                   // channels of a lane: 8 bytes of bf16, 16 of fp32

// V consecutive channels of a token.  kVec: the row allows one access of V elements;
// else element by element, nv of them real.
template <typename T, int V>
struct alignas(sizeof(T) * V) Channels {
  T e[V];
  __device__ __forceinline__ void widen(float (&v)[V]) const {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = io<T>::load(&e[i]);
  }
};
template <typename T, int V, bool kVec>
__device__ __forceinline__ Channels<T, V> load_channels(const T* p, int nv) {
  if constexpr (kVec) {
    return *reinterpret_cast<const Channels<T, V>*>(p);
  } else {
    Channels<T, V> q;
#pragma unroll
    for (int i = 0; i < V; ++i) q.e[i] = i < nv ? p[i] : T{0};
    return q;
  }
}
template <typename T, int V, bool kVec>
__device__ __forceinline__ void store_channels(T* p, int nv, const float (&v)[V]) {
  if constexpr (kVec) {
    Channels<T, V> q;
#pragma unroll
    for (int i = 0; i < V; ++i) io<T>::store(&q.e[i], v[i]);
    *reinterpret_cast<Channels<T, V>*>(p) = q;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < nv) io<T>::store(p + i, v[i]);
  }
}

// The sequence that a token of a row belongs to: tokens lo .. hi - 1 of the row
// are sequence k's (or, with k < 0, nobody's).  Bounds come from the device and
// are held to the row, so that whatever they say no token outside it is reached.
struct Walk {
  const int32_t* cu;
  int nseq, len;      // sequences, tokens of the row
  int k, lo, hi;

  __device__ __forceinline__ int bound(int i) const { return min(max(cu[i], 0), len); }

  // One sequence that fills the row.
  __device__ __forceinline__ void whole(int row, int length) {
    cu = nullptr;
    nseq = 0;
    len = length;
    k = row;
    lo = 0;
    hi = length;
  }

  // The sequence of token t: the last bound that is not past it, by bisection
  // among every `step`-th bound (in LDS) and then within a step.
  __device__ __forceinline__ void find(const int32_t* bounds, int n, int length, const int32_t* held, int step, int t) {
    cu = bounds;
    nseq = n;
    len = length;
    int a = -1, b = n / step + 1;   // held[a] <= t < held[b]
    while (b - a > 1) {
      const int m = (a + b) / 2;
      if (held[m] <= t) a = m; else b = m;
    }
    if (a < 0) {
      k = -1;
    } else {
      a *= step;
      b = min(a + step, n + 1);
      while (b - a > 1) {
        const int m = (a + b) / 2;
        if (cu[m] <= t) a = m; else b = m;
      }
      k = a;
    }
    settle();
  }
  __device__ __forceinline__ void settle() {
    if (k < 0) {
      lo = 0;
      hi = nseq >= 0 ? bound(0) : len;
    } else if (k >= nseq) {
      lo = bound(nseq);
      hi = len;
    } else {
      lo = bound(k);
      hi = bound(k + 1);
    }
  }
  __device__ __forceinline__ bool inside() const { return k >= 0 && (cu == nullptr || k < nseq); }
  // To token t = hi: the next sequence that has tokens.  Says whether there was a step.
  __device__ __forceinline__ bool reach(int t) {
    if (t < hi || cu == nullptr) return false;
    while (t >= hi && k < nseq) {
      ++k;
      settle();
    }
    return true;
  }
};

// Every step-th bound into LDS, for Walk::find.
__device__ __forceinline__ int hold_bounds(const int32_t* cu, int nseq, int32_t* held) {
  const int step = nseq / kConvBounds + 1;
  for (int i = threadIdx.x; i * step <= nseq; i += kConvThreads) held[i] = cu[i * step];
  return step;
}

}  // namespace ssm
