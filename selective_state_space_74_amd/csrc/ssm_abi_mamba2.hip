// ssm_abi_mamba2.hip -- the extern "C" surface of the token convolution and of
// the Mamba-2 SSM's packed prefill, gradients and step: host-side validation
// (pure host code, no HIP call) and dispatch.
#include <stdint.h>

#include "abi_checks.h"
#include "ssm_internal.h"

using namespace ssm;

namespace {

bool bad_dtype(int32_t dt) { return dt != SSM_F32 && dt != SSM_BF16; }

constexpr int64_t kMaxDim = int64_t{1} << 26;
constexpr int64_t kMaxPacked = int64_t{1} << 29;

// A (batch, L, dim) tensor with its strides.
struct Tokens {
  const void* p;
  int64_t sb, ss;
};

int check_tokens(const Tokens& t, int64_t esz) {
  if (!t.p) return SSM_ERR_NULL;
  if (t.sb < 0 || t.ss < 0) return SSM_ERR_STRIDE;
  return misaligned(t.p, esz) ? SSM_ERR_ALIGN : SSM_OK;
}

// Whether rows of one output can share bytes; batch rows may interleave along
// the sequence (a (L, batch, dim) layout).
bool collide(const Tokens& t, int64_t batch, int64_t L, int64_t D) {
  if (batch > 1 && L > 1 && t.ss >= batch * t.sb) return t.sb < D;
  return rows_collide(batch, t.sb, L, t.ss, D);
}

// What the convolution and its backward check alike: sizes, and the limits on them.
template <typename Args>
int check_conv(const Args* a) {
  if (a->batch < 0 || a->dim < 0 || a->seqlen < 0 || a->nseq < 0) return SSM_ERR_SHAPE;
  if (a->cu_seqlens && a->batch != 1) return SSM_ERR_SHAPE;
  if (a->d_conv < 1) return SSM_ERR_SHAPE;
  if (bad_dtype(a->io_dtype)) return SSM_ERR_DTYPE;
  if (a->d_conv > SSM_MAX_CONV || a->seqlen > kMaxSeqlen || a->dim > kMaxDim) return SSM_ERR_UNSUPPORTED;
  if (a->cu_seqlens && a->nseq >= kMaxPacked) return SSM_ERR_UNSUPPORTED;
  // a launch has less than 2^32 threads: 2^24 - 1 workgroups, 256 of them for sequences
  // without tokens at most, the others of 16 runs (of 16 tokens or more where there are
  // many) by 64 channels
  const int64_t per_row = max((a->seqlen + 15) / 16, int64_t{1}), cols = max((a->dim + 63) / 64, int64_t{1});
  if (a->batch > (int64_t{1} << 28) / per_row) return SSM_ERR_UNSUPPORTED;
  return (a->batch * per_row + 15) / 16 > ((int64_t{1} << 24) - 257) / cols ? SSM_ERR_UNSUPPORTED : SSM_OK;
}

// No output may share bytes with an input or with another output.
template <size_t NI, size_t NO>
int check_apart(const Rows (&inputs)[NI], const Rows (&outputs)[NO]) {
  for (const Rows& o : outputs) {
    for (const Rows& i : inputs)
      if (overlap(o, i)) return SSM_ERR_ALIAS;
    for (const Rows& o2 : outputs)
      if (&o2 != &o && overlap(o, o2)) return SSM_ERR_ALIAS;
  }
  return SSM_OK;
}

Rows flat(const void* p, int64_t n, int64_t esz) { return Rows{span1(p, n, esz)}; }

// ---- the SSD scans -------------------------------------------------------------------

// A (batch, token, head or group, inner) tensor.
struct Heads {
  const void* p;
  int64_t sb, ss, sh, heads, inner;
};
Rows rows_of(const Heads& t, int64_t batch, int64_t L, int64_t esz) {
  return Rows{span4(t.p, batch, t.sb, L, t.ss, t.heads, t.sh, t.inner, esz)};
}
int check_heads(const Heads& t, int64_t batch, int64_t esz) {
  if (!t.p) return SSM_ERR_NULL;
  if ((batch > 1 && t.sb < 0) || t.ss < 0 || (t.heads > 1 && t.sh < 0)) return SSM_ERR_STRIDE;
  if (misaligned(t.p, esz)) return SSM_ERR_ALIGN;
  // a chunk of 64 tokens is reached through a 31-bit byte window
  return t.ss >= (int64_t{1} << 31) || (63 * t.ss + t.inner) * esz >= (int64_t{1} << 31) ? SSM_ERR_UNSUPPORTED : SSM_OK;
}

// Sizes of the packed scan and of the gradients, and the limits on them.
int check_ssd(int64_t batch, int64_t L, int64_t H, int64_t P, int64_t ngroups, int64_t N, int64_t nseq, bool packed,
              int32_t dtype) {
  if (batch < 0 || L < 0 || nseq < 0 || H < 1 || P < 1 || N < 1 || bad_groups(ngroups, H) || (packed && batch != 1))
    return SSM_ERR_SHAPE;
  if (bad_dtype(dtype)) return SSM_ERR_DTYPE;
  // a grid has 2^32 threads, 512 to a chunk's head
  const int64_t most = (int64_t{1} << 31) - 1, chunks = (int64_t{1} << 23) - 1;
  if (N > (dtype == SSM_BF16 ? 128 : 64) || L > kMaxSeqlen || H > most / P || H * P > most / N) return SSM_ERR_UNSUPPORTED;
  if (packed && nseq >= kMaxPacked) return SSM_ERR_UNSUPPORTED;
  const int64_t of_row = packed ? L / 64 + min(nseq, L) : (L + 63) / 64;
  if (H > chunks || batch > most || (of_row > 0 && (of_row > chunks / H || batch > chunks / H / of_row)))
    return SSM_ERR_UNSUPPORTED;
  return SSM_OK;
}
int check_ssd(const ssm_ssd_packed_args* a) {
  return check_ssd(1, a->seqlen, a->nheads, a->headdim, a->ngroups, a->dstate, a->nseq, true, a->io_dtype);
}
int check_ssd(const ssm_ssd_bwd_args* a) {
  return check_ssd(a->batch, a->seqlen, a->nheads, a->headdim, a->ngroups, a->dstate, a->nseq, a->cu_seqlens != nullptr,
                   a->io_dtype);
}
// The size functions read sizes alone; those of fp32 pass the limits of bf16.
template <typename Args>
bool sizes_pass(const Args* a) {
  Args s = *a;
  s.io_dtype = SSM_BF16;
  return check_ssd(&s) == SSM_OK;
}

}  // namespace

extern "C" {

size_t ssm_token_conv_args_size(void) { return sizeof(ssm_token_conv_args); }
size_t ssm_token_conv_bwd_args_size(void) { return sizeof(ssm_token_conv_bwd_args); }
size_t ssm_token_conv_update_args_size(void) { return sizeof(ssm_token_conv_update_args); }
size_t ssm_ssd_update_args_size(void) { return sizeof(ssm_ssd_update_args); }

size_t ssm_token_conv_bwd_workspace_size(const ssm_token_conv_bwd_args* a) {
  if (!a) return 0;
  ssm_token_conv_bwd_args s = *a;   // the size is that of either type
  if (bad_dtype(s.io_dtype)) s.io_dtype = SSM_F32;
  if (check_conv(&s) != SSM_OK || s.dim == 0) return 0;
  return token_conv_bwd_workspace_bytes(s);
}

size_t ssm_ssd_packed_args_size(void) { return sizeof(ssm_ssd_packed_args); }
size_t ssm_ssd_bwd_args_size(void) { return sizeof(ssm_ssd_bwd_args); }

size_t ssm_ssd_packed_workspace_size(const ssm_ssd_packed_args* a) {
  return a && sizes_pass(a) ? ssd_packed_workspace_bytes(*a) : 0;
}
size_t ssm_ssd_bwd_workspace_size(const ssm_ssd_bwd_args* a) {
  return a && sizes_pass(a) ? ssd_bwd_workspace_bytes(*a) : 0;
}

int ssm_validate_ssd_packed(const ssm_ssd_packed_args* a) {
  if (!a) return SSM_ERR_NULL;
  if (const int st = check_ssd(a)) return st;
  const int64_t L = a->seqlen, H = a->nheads, P = a->headdim, N = a->dstate, G = groups_of(a->ngroups), S = a->nseq;
  const int64_t esz = io_size(a->io_dtype);
  if (!a->cu_seqlens || !a->A) return SSM_ERR_NULL;
  const Heads x{a->x, 0, a->x_seq_stride, a->x_head_stride, H, P}, z{a->z, 0, a->z_seq_stride, a->z_head_stride, H, P},
      B{a->B, 0, a->B_seq_stride, a->B_group_stride, G, N}, C{a->C, 0, a->C_seq_stride, a->C_group_stride, G, N},
      out{a->out, 0, a->out_seq_stride, a->out_head_stride, H, P};
  if (L > 0) {
    for (const Heads& t : {x, B, C, out})
      if (const int st = check_heads(t, 1, esz)) return st;
    if (a->z)
      if (const int st = check_heads(z, 1, esz)) return st;
    if (!a->dt) return SSM_ERR_NULL;
    if (a->dt_seq_stride < 0) return SSM_ERR_STRIDE;
    if (misaligned(a->dt, esz)) return SSM_ERR_ALIGN;
    // rows of out in either order of tokens and heads
    if (rows_collide(L, out.ss, H, out.sh, P) && rows_collide(H, out.sh, L, out.ss, P)) return SSM_ERR_ALIAS;
  }
  if (misaligned(a->A, 4) || misaligned(a->D, 4) || misaligned(a->dt_bias, 4) || misaligned(a->cu_seqlens, 4) ||
      misaligned(a->h0, 4) || misaligned(a->last_state, 4) || misaligned(a->workspace, 16))
    return SSM_ERR_ALIGN;
  const size_t need = ssd_packed_workspace_bytes(*a);
  if (need && (!a->workspace || a->workspace_bytes < need)) return SSM_ERR_SCRATCH;
  const int64_t states = S * H * P * N;
  const Rows inputs[] = {rows_of(x, 1, L, esz), rows3(a->dt, 1, 0, L, a->dt_seq_stride, H, esz), rows_of(z, 1, L, esz),
                         rows_of(B, 1, L, esz), rows_of(C, 1, L, esz), flat(a->A, H, 4), flat(a->D, H, 4),
                         flat(a->dt_bias, H, 4), flat(a->cu_seqlens, S + 1, 4), flat(a->h0, states, 4)};
  const Rows outputs[] = {rows_of(out, 1, L, esz), flat(a->last_state, states, 4),
                          flat(a->workspace, static_cast<int64_t>(a->workspace_bytes), 1)};
  for (const Rows& o : outputs) {
    for (const Rows& i : inputs) {
      // last_state may be exactly h0 (the state carried in place)
      if (&o == &outputs[1] && &i == &inputs[9] && a->last_state == a->h0) continue;
      if (overlap(o, i)) return SSM_ERR_ALIAS;
    }
    for (const Rows& o2 : outputs)
      if (&o2 != &o && overlap(o, o2)) return SSM_ERR_ALIAS;
  }
  return SSM_OK;
}

int ssm_validate_ssd_bwd(const ssm_ssd_bwd_args* a) {
  if (!a) return SSM_ERR_NULL;
  if (const int st = check_ssd(a)) return st;
  const int64_t Bt = a->batch, L = a->seqlen, H = a->nheads, P = a->headdim, N = a->dstate, G = groups_of(a->ngroups);
  const int64_t S = a->cu_seqlens ? a->nseq : Bt, esz = io_size(a->io_dtype);
  if (!a->A || !a->dA) return SSM_ERR_NULL;   // dA is set (to zero) without any token too
  const Heads x{a->x, a->x_batch_stride, a->x_seq_stride, a->x_head_stride, H, P},
      z{a->z, a->z_batch_stride, a->z_seq_stride, a->z_head_stride, H, P},
      B{a->B, a->B_batch_stride, a->B_seq_stride, a->B_group_stride, G, N},
      C{a->C, a->C_batch_stride, a->C_seq_stride, a->C_group_stride, G, N},
      dout{a->dout, a->dout_batch_stride, a->dout_seq_stride, a->dout_head_stride, H, P};
  const int64_t T = Bt * L;
  if (T > 0) {
    // dx, contiguous, is written through such windows too
    if (H * P * esz >= (int64_t{1} << 25)) return SSM_ERR_UNSUPPORTED;
    for (const Heads& t : {x, B, C, dout})
      if (const int st = check_heads(t, Bt, esz)) return st;
    if (a->z) {
      if (const int st = check_heads(z, Bt, esz)) return st;
      if (!a->dz) return SSM_ERR_NULL;
    }
    if (!a->dt || !a->dx || !a->ddt || !a->dB || !a->dC) return SSM_ERR_NULL;
    if (a->dt_seq_stride < 0 || (Bt > 1 && a->dt_batch_stride < 0)) return SSM_ERR_STRIDE;
    for (const void* p : {a->dt, static_cast<const void*>(a->dx), static_cast<const void*>(a->ddt),
                          static_cast<const void*>(a->dz), static_cast<const void*>(a->dB), static_cast<const void*>(a->dC)})
      if (misaligned(p, esz)) return SSM_ERR_ALIGN;
  }
  if (misaligned(a->A, 4) || misaligned(a->D, 4) || misaligned(a->dt_bias, 4) || misaligned(a->cu_seqlens, 4) ||
      misaligned(a->h0, 4) || misaligned(a->dlast, 4) || misaligned(a->dA, 4) || misaligned(a->dD, 4) ||
      misaligned(a->ddt_bias, 4) || misaligned(a->dh0, 4) || misaligned(a->workspace, 16))
    return SSM_ERR_ALIGN;
  const size_t need = ssd_bwd_workspace_bytes(*a);
  if (need && (!a->workspace || a->workspace_bytes < need)) return SSM_ERR_SCRATCH;
  const int64_t states = S * H * P * N;
  const Rows inputs[] = {rows_of(x, Bt, L, esz), rows3(a->dt, Bt, a->dt_batch_stride, L, a->dt_seq_stride, H, esz),
                         rows_of(z, Bt, L, esz), rows_of(B, Bt, L, esz), rows_of(C, Bt, L, esz), rows_of(dout, Bt, L, esz),
                         flat(a->A, H, 4), flat(a->D, H, 4), flat(a->dt_bias, H, 4),
                         flat(a->cu_seqlens, S + 1, 4), flat(a->h0, states, 4), flat(a->dlast, states, 4)};
  const Rows outputs[] = {flat(a->dx, T * H * P, esz), flat(a->ddt, T * H, esz), flat(a->z ? a->dz : nullptr, T * H * P, esz),
                          flat(a->dB, T * G * N, esz), flat(a->dC, T * G * N, esz), flat(a->dA, H, 4), flat(a->dD, H, 4),
                          flat(a->ddt_bias, H, 4), flat(a->dh0, states, 4),
                          flat(a->workspace, static_cast<int64_t>(a->workspace_bytes), 1)};
  return check_apart(inputs, outputs);
}

int ssm_ssd_packed_fwd(const ssm_ssd_packed_args* a, void* stream) {
  if (const int st = ssm_validate_ssd_packed(a)) return st;
  return launch_ssd_packed_fwd(*a, static_cast<hipStream_t>(stream)) == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

int ssm_ssd_scan_bwd(const ssm_ssd_bwd_args* a, void* stream) {
  if (const int st = ssm_validate_ssd_bwd(a)) return st;
  return launch_ssd_bwd(*a, static_cast<hipStream_t>(stream)) == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

int ssm_validate_token_conv(const ssm_token_conv_args* a) {
  if (!a) return SSM_ERR_NULL;
  if (const int st = check_conv(a)) return st;
  if (a->batch == 0 || a->dim == 0) return SSM_OK;
  const int64_t B = a->batch, L = a->seqlen, D = a->dim, S = a->cu_seqlens ? a->nseq : B, K = a->d_conv;
  const int64_t esz = io_size(a->io_dtype);
  const Tokens x{a->x, a->x_batch_stride, a->x_seq_stride}, out{a->out, a->out_batch_stride, a->out_seq_stride};
  if (L > 0) {
    if (!a->weight) return SSM_ERR_NULL;
    if (const int st = check_tokens(x, esz)) return st;
    if (const int st = check_tokens(out, esz)) return st;
    if (collide(out, B, L, D)) return SSM_ERR_ALIAS;
  }
  if (misaligned(a->weight, 4) || misaligned(a->bias, 4) || misaligned(a->cu_seqlens, 4) || misaligned(a->state_in, 4) ||
      misaligned(a->state_out, 4))
    return SSM_ERR_ALIGN;
  auto rows = [&](const Tokens& t) { return rows3(L > 0 ? t.p : nullptr, B, t.sb, L, t.ss, D, esz); };
  const Rows inputs[] = {rows(x), flat(a->weight, D * K, 4), flat(a->bias, D, 4), flat(a->cu_seqlens, S + 1, 4),
                         flat(a->state_in, S * D * K, 4)};
  const Rows outputs[] = {rows(out), flat(a->state_out, S * D * K, 4)};
  return check_apart(inputs, outputs);
}

int ssm_validate_token_conv_bwd(const ssm_token_conv_bwd_args* a) {
  if (!a) return SSM_ERR_NULL;
  if (const int st = check_conv(a)) return st;
  if (a->dim == 0) return SSM_OK;
  if (!a->weight || !a->dweight) return SSM_ERR_NULL;   // dweight is set (to zero) without any token too
  const int64_t B = a->batch, L = a->seqlen, D = a->dim, S = a->cu_seqlens ? a->nseq : B, K = a->d_conv;
  const int64_t esz = io_size(a->io_dtype);
  const Tokens x{a->x, a->x_batch_stride, a->x_seq_stride}, dout{a->dout, a->dout_batch_stride, a->dout_seq_stride},
      dx{a->dx, a->dx_batch_stride, a->dx_seq_stride};
  if (L > 0 && B > 0) {
    for (const Tokens& t : {x, dout, dx})
      if (const int st = check_tokens(t, esz)) return st;
    if (collide(dx, B, L, D)) return SSM_ERR_ALIAS;
  }
  if (misaligned(a->weight, 4) || misaligned(a->bias, 4) || misaligned(a->cu_seqlens, 4) || misaligned(a->state_in, 4) ||
      misaligned(a->dstate_out, 4) || misaligned(a->dweight, 4) || misaligned(a->dbias, 4) ||
      misaligned(a->dstate_in, 4) || misaligned(a->workspace, 4))
    return SSM_ERR_ALIGN;
  const size_t need = token_conv_bwd_workspace_bytes(*a);
  if (need && (!a->workspace || a->workspace_bytes < need)) return SSM_ERR_SCRATCH;
  auto rows = [&](const Tokens& t) { return rows3(L > 0 ? t.p : nullptr, B, t.sb, L, t.ss, D, esz); };
  const Rows inputs[] = {rows(x), rows(dout), flat(a->weight, D * K, 4), flat(a->bias, D, 4),
                         flat(a->cu_seqlens, S + 1, 4), flat(a->state_in, S * D * K, 4), flat(a->dstate_out, S * D * K, 4)};
  const Rows outputs[] = {rows(dx), flat(a->dweight, D * K, 4), flat(a->dbias, D, 4), flat(a->dstate_in, S * D * K, 4),
                          flat(a->workspace, static_cast<int64_t>(a->workspace_bytes), 1)};
  return check_apart(inputs, outputs);
}

int ssm_validate_token_conv_update(const ssm_token_conv_update_args* a) {
  if (!a) return SSM_ERR_NULL;
  if (a->batch < 0 || a->dim < 0 || a->nslots < 0 || a->d_conv < 1 || (!a->slots && a->batch > a->nslots))
    return SSM_ERR_SHAPE;
  if (bad_dtype(a->io_dtype)) return SSM_ERR_DTYPE;
  if (a->d_conv > SSM_MAX_CONV || a->batch > 65535 || a->dim > kMaxDim) return SSM_ERR_UNSUPPORTED;
  if (a->batch == 0 || a->dim == 0) return SSM_OK;
  if ((!a->state && a->nslots > 0) || !a->weight) return SSM_ERR_NULL;
  const int64_t esz = io_size(a->io_dtype), B = a->batch, D = a->dim, S = a->nslots, K = a->d_conv;
  const Tokens x{a->x, 0, a->x_batch_stride}, out{a->out, 0, a->out_batch_stride};
  if (const int st = check_tokens(x, esz)) return st;
  if (const int st = check_tokens(out, esz)) return st;
  if (a->state_slot_stride < 0) return SSM_ERR_STRIDE;
  if (misaligned(a->state, 4) || misaligned(a->weight, 4) || misaligned(a->bias, 4) || misaligned(a->slots, 4))
    return SSM_ERR_ALIGN;
  if (rows_collide(1, 0, B, a->out_batch_stride, D) || rows_collide(1, 0, S, a->state_slot_stride, D * K))
    return SSM_ERR_ALIAS;
  auto rows = [&](const Tokens& t) { return rows3(t.p, 1, 0, B, t.ss, D, esz); };
  const Rows inputs[] = {rows(x), flat(a->weight, D * K, 4), flat(a->bias, D, 4), flat(a->slots, B, 4)};
  const Rows outputs[] = {rows(out), rows3(a->state, 1, 0, S, a->state_slot_stride, D * K, 4)};
  return check_apart(inputs, outputs);
}

int ssm_validate_ssd_update(const ssm_ssd_update_args* a) {
  if (!a) return SSM_ERR_NULL;
  if (a->batch < 0 || a->nslots < 0 || a->nheads < 1 || a->headdim < 1 || a->dstate < 1 ||
      (!a->slots && a->batch > a->nslots) || bad_groups(a->ngroups, a->nheads))
    return SSM_ERR_SHAPE;
  if (bad_dtype(a->io_dtype)) return SSM_ERR_DTYPE;
  const int64_t most = (int64_t{1} << 31) - 1;
  // headdim: the kernel counts rows in 32 bits, up to a wavefront's share past the last
  if (a->dstate > SSM_MAX_SSD_STEP_DSTATE || a->batch > 65535 || a->headdim > int64_t{1} << 30 || a->nheads > most / a->headdim ||
      a->nheads * a->headdim > most / a->dstate)
    return SSM_ERR_UNSUPPORTED;
  // a launch has less than 2^32 threads, a wavefront for up to 64 channels of a head
  if (a->nheads * ((a->headdim + 63) / 64) > (int64_t{1} << 26) - 4) return SSM_ERR_UNSUPPORTED;
  if (a->batch == 0) return SSM_OK;
  const int64_t esz = io_size(a->io_dtype), Bt = a->batch, H = a->nheads, P = a->headdim, N = a->dstate, S = a->nslots;
  const int64_t G = groups_of(a->ngroups);
  if ((!a->state && S > 0) || !a->x || !a->dt || !a->B || !a->C || !a->A || !a->out) return SSM_ERR_NULL;
  const int64_t strides[] = {a->state_slot_stride, a->x_batch_stride, a->x_head_stride, a->dt_batch_stride,
                             a->z ? a->z_batch_stride : 0, a->z ? a->z_head_stride : 0, a->B_batch_stride,
                             a->C_batch_stride, G > 1 ? a->B_group_stride : 0, G > 1 ? a->C_group_stride : 0,
                             a->out_batch_stride, a->out_head_stride};
  for (int64_t s : strides)
    if (s < 0) return SSM_ERR_STRIDE;
  if (misaligned(a->x, esz) || misaligned(a->dt, esz) || misaligned(a->z, esz) || misaligned(a->B, esz) ||
      misaligned(a->C, esz) || misaligned(a->out, esz) || misaligned(a->state, 4) || misaligned(a->A, 4) ||
      misaligned(a->D, 4) || misaligned(a->dt_bias, 4) || misaligned(a->slots, 4))
    return SSM_ERR_ALIGN;
  if (rows_collide(Bt, a->out_batch_stride, H, a->out_head_stride, P) ||
      rows_collide(1, 0, S, a->state_slot_stride, H * P * N))
    return SSM_ERR_ALIAS;
  const Rows inputs[] = {rows3(a->x, Bt, a->x_batch_stride, H, a->x_head_stride, P, esz),
                         rows3(a->dt, 1, 0, Bt, a->dt_batch_stride, H, esz),
                         rows3(a->z, Bt, a->z_batch_stride, H, a->z_head_stride, P, esz),
                         rows3(a->B, Bt, a->B_batch_stride, G, a->B_group_stride, N, esz),
                         rows3(a->C, Bt, a->C_batch_stride, G, a->C_group_stride, N, esz),
                         flat(a->A, H, 4), flat(a->D, H, 4), flat(a->dt_bias, H, 4), flat(a->slots, Bt, 4)};
  const Rows outputs[] = {rows3(a->out, Bt, a->out_batch_stride, H, a->out_head_stride, P, esz),
                          rows3(a->state, 1, 0, S, a->state_slot_stride, H * P * N, 4)};
  return check_apart(inputs, outputs);
}

int ssm_token_conv_fwd(const ssm_token_conv_args* a, void* stream) {
  if (const int st = ssm_validate_token_conv(a)) return st;
  if (a->batch == 0 || a->dim == 0) return SSM_OK;
  return launch_token_conv_fwd(*a, static_cast<hipStream_t>(stream)) == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

int ssm_token_conv_bwd(const ssm_token_conv_bwd_args* a, void* stream) {
  if (const int st = ssm_validate_token_conv_bwd(a)) return st;
  if (a->dim == 0) return SSM_OK;
  return launch_token_conv_bwd(*a, static_cast<hipStream_t>(stream)) == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

int ssm_token_conv_update(const ssm_token_conv_update_args* a, void* stream) {
  if (const int st = ssm_validate_token_conv_update(a)) return st;
  if (a->batch == 0 || a->dim == 0) return SSM_OK;
  return launch_token_conv_update(*a, static_cast<hipStream_t>(stream)) == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

int ssm_ssd_state_update(const ssm_ssd_update_args* a, void* stream) {
  if (const int st = ssm_validate_ssd_update(a)) return st;
  if (a->batch == 0) return SSM_OK;
  return launch_ssd_step(*a, static_cast<hipStream_t>(stream)) == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

}  // extern "C"
