// The gated recurrence's per-token arithmetic, shared by its forward, backward
// and single-token kernels.
#pragma once

#include "ssm_internal.h"

namespace ssm {

constexpr int kGatedCkpt = SSM_GATED_CHECKPOINT_TOKENS;

// 1 / (1 + e^-z) on the hardware exp2 and reciprocal: 0 and 1 at -inf and inf.
__device__ __forceinline__ float sigmoid_f32(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-z * kLog2e));
}

// 1 - a^2 for a = e^(-u/2), u >= 0.  Below u = 1/4 the difference would cancel
// (a layer that remembers thousands of tokens sits at u ~ 1e-3), so the series
// of 1 - e^-u is summed instead: its first omitted term, u^7 / 5040, is under
// 2^-24 of the sum there.  Above, 1 - a^2 >= 0.22 keeps full accuracy.
__device__ __forceinline__ float one_minus_square(float a, float u) {
  float s = fmaf(u, -1.0f / 720.0f, 1.0f / 120.0f);
  s = fmaf(u, s, -1.0f / 24.0f);
  s = fmaf(u, s, 1.0f / 6.0f);
  s = fmaf(u, s, -0.5f);
  s = fmaf(u, s, 1.0f);
  return u < 0.25f ? u * s : fmaf(-a, a, 1.0f);
}

// A channel's rate s = c softplus(lam), as the tokens use it: log2(a) and
// u = -2 log(a) are each one product with sigma(gate_a).
struct Rate {
  float s, log2a, u;
  __device__ __forceinline__ Rate() {}
  __device__ __forceinline__ Rate(float c, float lam) : s(c * softplus_close_f32(lam)), log2a(-s * kLog2e), u(2.0f * s) {}
};

}  // namespace ssm
