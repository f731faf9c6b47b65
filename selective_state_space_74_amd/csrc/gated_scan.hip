// gated_scan.hip -- the gated linear recurrence for gfx950: prefill and the
// single-token step.
//   a_t = exp(-s sigma(gate_a_t)), s = c softplus(lam)
//   h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigma(gate_x_t) x_t
#include "gated_math.h"

namespace ssm {
namespace {

constexpr int kThreads = 64;

struct FwdParams {
  const void* x; const void* ga; const void* gx;
  const float* lam; const int32_t* cu; const float* h0;
  float* last; void* out; float* ck;
  int64_t xb, xs, gab, gas, gxb, gxs, ob, os;
  int64_t batch, L, D, nseq, nck;
  float c;
  int zero_outside;
};

// One thread walks one sequence of one channel.
template <typename T>
__global__ __launch_bounds__(kThreads) void gated_fwd_kernel(FwdParams p) {
  const int64_t d = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (d >= p.D) return;
  const float s = p.c * softplus_f32(p.lam[d]);
  const int64_t n = p.cu ? p.nseq : p.batch;
  for (int64_t k = blockIdx.y; k < n; k += gridDim.y) {
    const int64_t b = p.cu ? 0 : k;
    int64_t lo = 0, hi = p.L;
    if (p.cu) {
      lo = min(max(static_cast<int64_t>(p.cu[k]), int64_t{0}), p.L);
      hi = min(max(static_cast<int64_t>(p.cu[k + 1]), lo), p.L);
    }
    float h = p.h0 ? p.h0[k * p.D + d] : 0.0f;
    for (int64_t t = lo; t < hi; ++t) {
      if (p.ck && t % kCkpt == 0) p.ck[(b * p.nck + t / kCkpt) * p.D + d] = h;
      const float x = io<T>::load(static_cast<const T*>(p.x) + b * p.xb + t * p.xs + d);
      const float ga = io<T>::load(static_cast<const T*>(p.ga) + b * p.gab + t * p.gas + d);
      const float gx = io<T>::load(static_cast<const T*>(p.gx) + b * p.gxb + t * p.gxs + d);
      const float v = s * sigmoid_f32(ga);
      const float a = __builtin_amdgcn_exp2f(-v * kLog2e);
      h = fmaf(a, h, sqrtf(one_minus_square(a, v)) * (sigmoid_f32(gx) * x));
      io<T>::store(static_cast<T*>(p.out) + b * p.ob + t * p.os + d, h);
    }
    if (p.last) p.last[k * p.D + d] = h;
  }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void zero_outside_kernel(FwdParams p) {
  const int64_t d = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (d >= p.D) return;
  const int64_t lo = p.nseq > 0 ? p.cu[0] : p.L, hi = p.nseq > 0 ? p.cu[p.nseq] : p.L;
  for (int64_t t = blockIdx.y; t < p.L; t += gridDim.y)
    if (t < lo || t >= hi) io<T>::store(static_cast<T*>(p.out) + t * p.os + d, 0.0f);
}

struct StepParams {
  float* state; const void* x; const void* ga; const void* gx;
  const float* lam; const int32_t* slots; void* out;
  int64_t ss, xb, gab, gxb, ob, batch, nslots, D;
  float c;
};

template <typename T>
__global__ __launch_bounds__(kThreads) void gated_step_kernel(StepParams p) {
  const int64_t d = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t b0 = blockIdx.y;
  if (d >= p.D) return;
  const int64_t slot = p.slots ? p.slots[b0] : b0;
  if (slot < 0 || slot >= p.nslots) {
    io<T>::store(static_cast<T*>(p.out) + b0 * p.ob + d, 0.0f);
    return;
  }
  // the first row of a slot takes every row of it, in order
  if (p.slots)
    for (int64_t i = 0; i < b0; ++i)
      if (p.slots[i] == slot) return;
  const float s = p.c * softplus_f32(p.lam[d]);
  float h = p.state[slot * p.ss + d];
  for (int64_t b = b0; b < p.batch; ++b) {
    if (b > b0 && (!p.slots || p.slots[b] != slot)) {
      if (!p.slots) break;
      continue;
    }
    const float x = io<T>::load(static_cast<const T*>(p.x) + b * p.xb + d);
    const float v = s * sigmoid_f32(io<T>::load(static_cast<const T*>(p.ga) + b * p.gab + d));
    const float g = sigmoid_f32(io<T>::load(static_cast<const T*>(p.gx) + b * p.gxb + d));
    const float a = __builtin_amdgcn_exp2f(-v * kLog2e);
    h = fmaf(a, h, sqrtf(one_minus_square(a, v)) * (g * x));
    io<T>::store(static_cast<T*>(p.out) + b * p.ob + d, h);
  }
  p.state[slot * p.ss + d] = h;
}

}  // namespace

size_t gated_workspace_bytes(const ssm_gated_args&) { return 0; }

hipError_t launch_gated_fwd(const ssm_gated_args& a, hipStream_t stream) {
  FwdParams p{a.x, a.gate_a, a.gate_x, a.lam, a.cu_seqlens, a.h0, a.last_state, a.out, a.checkpoints,
              a.x_batch_stride, a.x_seq_stride, a.gate_a_batch_stride, a.gate_a_seq_stride,
              a.gate_x_batch_stride, a.gate_x_seq_stride, a.out_batch_stride, a.out_seq_stride,
              a.batch, a.seqlen, a.dim, a.nseq, (a.seqlen + kCkpt - 1) / kCkpt, a.c, a.zero_outside};
  const int64_t n = a.cu_seqlens ? a.nseq : a.batch;
  const unsigned gx = static_cast<unsigned>((a.dim + kThreads - 1) / kThreads);
  if (n > 0) {
    const dim3 grid(gx, static_cast<unsigned>(n < 65535 ? n : 65535));
    if (a.io_dtype == SSM_BF16) gated_fwd_kernel<uint16_t><<<grid, kThreads, 0, stream>>>(p);
    else gated_fwd_kernel<float><<<grid, kThreads, 0, stream>>>(p);
  }
  if (a.cu_seqlens && a.zero_outside && a.seqlen > 0) {
    const dim3 grid(gx, static_cast<unsigned>(a.seqlen < 1024 ? a.seqlen : 1024));
    if (a.io_dtype == SSM_BF16) zero_outside_kernel<uint16_t><<<grid, kThreads, 0, stream>>>(p);
    else zero_outside_kernel<float><<<grid, kThreads, 0, stream>>>(p);
  }
  return hipGetLastError();
}

hipError_t launch_gated_step(const ssm_gated_update_args& a, hipStream_t stream) {
  StepParams p{a.state, a.x, a.gate_a, a.gate_x, a.lam, a.slots, a.out, a.state_slot_stride,
               a.x_batch_stride, a.gate_a_batch_stride, a.gate_x_batch_stride, a.out_batch_stride,
               a.batch, a.nslots, a.dim, a.c};
  const dim3 grid(static_cast<unsigned>((a.dim + kThreads - 1) / kThreads), static_cast<unsigned>(a.batch));
  if (a.io_dtype == SSM_BF16) gated_step_kernel<uint16_t><<<grid, kThreads, 0, stream>>>(p);
  else gated_step_kernel<float><<<grid, kThreads, 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace ssm
