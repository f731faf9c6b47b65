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
#include "gated_math.h"

namespace ssm {
namespace {

constexpr int kThreads = 64;

struct BwdParams {
  const void* x; const void* ga; const void* gx; const void* dout;
  const float* lam; const int32_t* cu; const float* h0; const float* ck; const float* dlast;
  void* dx; void* dga; void* dgx; float* dlam; float* dh0; float* part;
  int64_t xb, xs, gab, gas, gxb, gxs, dob, dos, dxb, dxs, dgab, dgas, dgxb, dgxs;
  int64_t batch, L, D, nseq, nck;
  float c;
};

// One thread walks one sequence of one channel backwards, 16 tokens at a time:
// h forward from the checkpoint, then the adjoint backward.
template <typename T>
__global__ __launch_bounds__(kThreads) void gated_bwd_kernel(BwdParams p) {
  const int64_t d = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (d >= p.D) return;
  const float s = p.c * softplus_f32(p.lam[d]);
  const int64_t n = p.cu ? p.nseq : p.batch;
  float acc = 0.0f;
  for (int64_t k = blockIdx.y; k < n; k += gridDim.y) {
    const int64_t b = p.cu ? 0 : k;
    int64_t lo = 0, hi = p.L;
    if (p.cu) {
      lo = min(max(static_cast<int64_t>(p.cu[k]), int64_t{0}), p.L);
      hi = min(max(static_cast<int64_t>(p.cu[k + 1]), lo), p.L);
    }
    float e = p.dlast ? p.dlast[k * p.D + d] : 0.0f;   // a_{t+1} e_{t+1}
    for (int64_t t1 = hi; t1 > lo;) {
      const int64_t blk = (t1 - 1) / kCkpt * kCkpt, t0 = max(blk, lo);
      float hp[kCkpt];
      float h = t0 == lo ? (p.h0 ? p.h0[k * p.D + d] : 0.0f) : p.ck[(b * p.nck + t0 / kCkpt) * p.D + d];
      for (int64_t t = t0; t < t1; ++t) {
        hp[t - t0] = h;
        const float x = io<T>::load(static_cast<const T*>(p.x) + b * p.xb + t * p.xs + d);
        const float v = s * sigmoid_f32(io<T>::load(static_cast<const T*>(p.ga) + b * p.gab + t * p.gas + d));
        const float g = sigmoid_f32(io<T>::load(static_cast<const T*>(p.gx) + b * p.gxb + t * p.gxs + d));
        const float a = __builtin_amdgcn_exp2f(-v * kLog2e);
        h = fmaf(a, h, sqrtf(one_minus_square(a, v)) * (g * x));
      }
      for (int64_t t = t1 - 1; t >= t0; --t) {
        const float x = io<T>::load(static_cast<const T*>(p.x) + b * p.xb + t * p.xs + d);
        const float sa = sigmoid_f32(io<T>::load(static_cast<const T*>(p.ga) + b * p.gab + t * p.gas + d));
        const float g = sigmoid_f32(io<T>::load(static_cast<const T*>(p.gx) + b * p.gxb + t * p.gxs + d));
        const float v = s * sa;
        const float a = __builtin_amdgcn_exp2f(-v * kLog2e);
        const float q = one_minus_square(a, v);
        const float beta = sqrtf(q);
        const float inv = q > 0.0f ? 1.0f / beta : 0.0f;
        e += io<T>::load(static_cast<const T*>(p.dout) + b * p.dob + t * p.dos + d);
        const float dx = e * beta * g;
        const float dv = e * (g * x * (a * a * inv) - a * hp[t - t0]);
        io<T>::store(static_cast<T*>(p.dx) + b * p.dxb + t * p.dxs + d, dx);
        io<T>::store(static_cast<T*>(p.dgx) + b * p.dgxb + t * p.dgxs + d, dx * x * (1.0f - g));
        io<T>::store(static_cast<T*>(p.dga) + b * p.dgab + t * p.dgas + d, dv * v * (1.0f - sa));
        acc = fmaf(dv, sa, acc);
        e *= a;
      }
      t1 = t0;
    }
    if (p.dh0) p.dh0[k * p.D + d] = e;
  }
  p.part[blockIdx.y * p.D + d] = acc;
}

template <typename T>
__global__ __launch_bounds__(kThreads) void zero_outside_kernel(BwdParams p) {
  const int64_t d = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (d >= p.D) return;
  const int64_t lo = p.nseq > 0 ? p.cu[0] : p.L, hi = p.nseq > 0 ? p.cu[p.nseq] : p.L;
  for (int64_t t = blockIdx.y; t < p.L; t += gridDim.y)
    if (t < lo || t >= hi) {
      io<T>::store(static_cast<T*>(p.dx) + t * p.dxs + d, 0.0f);
      io<T>::store(static_cast<T*>(p.dga) + t * p.dgas + d, 0.0f);
      io<T>::store(static_cast<T*>(p.dgx) + t * p.dgxs + d, 0.0f);
    }
}

__global__ __launch_bounds__(kThreads) void dlam_kernel(const float* part, int64_t n, int64_t D,
                                                        const float* lam, float c, float* dlam) {
  const int64_t d = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (d >= D) return;
  float acc = 0.0f;
  for (int64_t i = 0; i < n; ++i) acc += part[i * D + d];
  dlam[d] = c * sigmoid_f32(lam[d]) * acc;
}

int64_t rows_of(const ssm_gated_bwd_args& a) {
  const int64_t n = a.cu_seqlens ? a.nseq : a.batch;
  return n < 1 ? 1 : n < 65535 ? n : 65535;
}

}  // namespace

size_t gated_bwd_workspace_bytes(const ssm_gated_bwd_args& a) {
  return static_cast<size_t>(rows_of(a) * a.dim * 4);
}

hipError_t launch_gated_bwd(const ssm_gated_bwd_args& a, hipStream_t stream) {
  BwdParams p{a.x, a.gate_a, a.gate_x, a.dout, a.lam, a.cu_seqlens, a.h0, a.checkpoints, a.dlast,
              a.dx, a.dgate_a, a.dgate_x, a.dlam, a.dh0, static_cast<float*>(a.workspace),
              a.x_batch_stride, a.x_seq_stride, a.gate_a_batch_stride, a.gate_a_seq_stride,
              a.gate_x_batch_stride, a.gate_x_seq_stride, a.dout_batch_stride, a.dout_seq_stride,
              a.dx_batch_stride, a.dx_seq_stride, a.dgate_a_batch_stride, a.dgate_a_seq_stride,
              a.dgate_x_batch_stride, a.dgate_x_seq_stride,
              a.batch, a.seqlen, a.dim, a.nseq, (a.seqlen + kCkpt - 1) / kCkpt, a.c};
  const unsigned gx = static_cast<unsigned>((a.dim + kThreads - 1) / kThreads);
  const dim3 grid(gx, static_cast<unsigned>(rows_of(a)));
  const bool bf = a.io_dtype == SSM_BF16;
  if (bf) gated_bwd_kernel<uint16_t><<<grid, kThreads, 0, stream>>>(p);
  else gated_bwd_kernel<float><<<grid, kThreads, 0, stream>>>(p);
  if (a.cu_seqlens && a.seqlen > 0) {
    const dim3 zg(gx, static_cast<unsigned>(a.seqlen < 1024 ? a.seqlen : 1024));
    if (bf) zero_outside_kernel<uint16_t><<<zg, kThreads, 0, stream>>>(p);
    else zero_outside_kernel<float><<<zg, kThreads, 0, stream>>>(p);
  }
  dlam_kernel<<<gx, kThreads, 0, stream>>>(p.part, rows_of(a), a.dim, a.lam, a.c, a.dlam);
  return hipGetLastError();
}

}  // namespace ssm
