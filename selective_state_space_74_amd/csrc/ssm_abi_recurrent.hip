// ssm_abi_recurrent.hip -- the extern "C" surface of the gated recurrence and
// of the quantised state cache: host-side validation (pure host code, no HIP
// call) and dispatch.
#include <math.h>
#include <stdint.h>

#include "abi_checks.h"
#include "ssm_internal.h"

using namespace ssm;

namespace {

bool bad_dtype(int32_t dt) { return dt != SSM_F32 && dt != SSM_BF16; }

// A (batch, L, dim) tensor of the gated scan with its strides.
struct Tokens {
  const void* p;
  int64_t sb, ss;
};

// Output rows may interleave with another tensor's (slices of one wider
// tensor), but the batch stride of such a slice spans whole rows.
bool collide(const Tokens& t, int64_t batch, int64_t L, int64_t D) {
  // batch rows that interleave along the sequence (a (L, batch, D) layout)
  if (batch > 1 && L > 1 && t.ss >= batch * t.sb) return t.sb < D;
  return rows_collide(batch, t.sb, L, t.ss, D);
}

constexpr int64_t kMaxGroups = int64_t{1} << 31;
constexpr int64_t kGatedTokens = SSM_GATED_CHECKPOINT_TOKENS;
constexpr int64_t kMaxDim = int64_t{1} << 26;
constexpr int64_t kMaxPacked = int64_t{1} << 29;   // sequence numbers and two marks share 32 bits
// A launch has less than 2^32 threads.  Blocks of 16 tokens and 64 channels, a
// wavefront each: workgroups of 8 wavefronts and the backward's blocks of 8
// tokens make it up to 2.7 times as many wavefronts.
constexpr int64_t kMaxBlocks = int64_t{1} << 24;
bool too_many_blocks(int64_t batch, int64_t L, int64_t D) {
  const int64_t blocks = max((L + 15) / 16, int64_t{1}) * max((D + 63) / 64, int64_t{1});
  return batch > (kMaxBlocks - 1) / blocks;
}

// What the gated scan and its backward check alike: sizes, and the limits on them.
template <typename Args>
int check_shape(const Args* a) {
  if (a->batch < 0 || a->dim < 0 || a->seqlen < 0 || a->nseq < 0) return SSM_ERR_SHAPE;
  return a->cu_seqlens && a->batch != 1 ? SSM_ERR_SHAPE : SSM_OK;
}
template <typename Args>
int check_limits(const Args* a) {
  if (a->seqlen > kMaxSeqlen) return SSM_ERR_UNSUPPORTED;
  // rows are addressed by 32-bit byte offsets
  if (a->dim > kMaxDim || too_many_blocks(a->batch, a->seqlen, a->dim)) return SSM_ERR_UNSUPPORTED;
  if (a->cu_seqlens && a->nseq >= kMaxPacked) return SSM_ERR_UNSUPPORTED;
  return SSM_OK;
}
template <typename Args>
int check_gated(const Args* a) {
  if (const int st = check_shape(a)) return st;
  if (!(a->c > 0.0f) || !isfinite(a->c)) return SSM_ERR_SHAPE;
  if (bad_dtype(a->io_dtype)) return SSM_ERR_DTYPE;
  return check_limits(a);
}

int check_tokens(const Tokens* t, int n, int64_t esz) {
  for (int i = 0; i < n; ++i) {
    if (!t[i].p) return SSM_ERR_NULL;
    if (t[i].sb < 0 || t[i].ss < 0) return SSM_ERR_STRIDE;
    if (misaligned(t[i].p, esz)) return SSM_ERR_ALIGN;
  }
  return SSM_OK;
}

}  // namespace

extern "C" {

size_t ssm_gated_args_size(void) { return sizeof(ssm_gated_args); }
size_t ssm_gated_bwd_args_size(void) { return sizeof(ssm_gated_bwd_args); }
size_t ssm_gated_update_args_size(void) { return sizeof(ssm_gated_update_args); }
size_t ssm_state_cache_args_size(void) { return sizeof(ssm_state_cache_args); }
size_t ssm_cached_update_args_size(void) { return sizeof(ssm_cached_update_args); }

size_t ssm_gated_scan_workspace_size(const ssm_gated_args* a) {
  if (!a || check_shape(a) != SSM_OK || check_limits(a) != SSM_OK || a->batch == 0 || a->dim == 0) return 0;
  return gated_workspace_bytes(*a);
}

size_t ssm_gated_scan_bwd_workspace_size(const ssm_gated_bwd_args* a) {
  if (!a || check_shape(a) != SSM_OK || check_limits(a) != SSM_OK || a->dim == 0) return 0;
  return gated_bwd_workspace_bytes(*a);
}

int ssm_validate_gated(const ssm_gated_args* a) {
  if (!a) return SSM_ERR_NULL;
  if (const int st = check_gated(a)) return st;
  if (a->batch == 0 || a->dim == 0) return SSM_OK;
  const int64_t B = a->batch, L = a->seqlen, D = a->dim, S = a->cu_seqlens ? a->nseq : B;
  const int64_t esz = io_size(a->io_dtype);
  const Tokens in[] = {{a->x, a->x_batch_stride, a->x_seq_stride},
                       {a->gate_a, a->gate_a_batch_stride, a->gate_a_seq_stride},
                       {a->gate_x, a->gate_x_batch_stride, a->gate_x_seq_stride}};
  const Tokens out{a->out, a->out_batch_stride, a->out_seq_stride};
  if (L > 0) {
    if (!a->lam) return SSM_ERR_NULL;
    if (const int st = check_tokens(in, 3, esz)) return st;
    if (const int st = check_tokens(&out, 1, esz)) return st;
    if (collide(out, B, L, D)) return SSM_ERR_ALIAS;
  }
  if (misaligned(a->lam, 4) || misaligned(a->cu_seqlens, 4) || misaligned(a->h0, 4) ||
      misaligned(a->last_state, 4) || misaligned(a->checkpoints, 4) || misaligned(a->workspace, 8))
    return SSM_ERR_ALIGN;
  const size_t need = gated_workspace_bytes(*a);
  if (need && (!a->workspace || a->workspace_bytes < need)) return SSM_ERR_SCRATCH;
  auto rows = [&](const Tokens& t) { return rows3(L > 0 ? t.p : nullptr, B, t.sb, L, t.ss, D, esz); };
  auto flat = [&](const void* p, int64_t n, int64_t e) { return Rows{span1(p, n, e)}; };
  const Rows inputs[] = {rows(in[0]), rows(in[1]), rows(in[2]), flat(a->lam, D, 4),
                         flat(a->cu_seqlens, S + 1, 4), flat(a->h0, S * D, 4)};
  const Rows outputs[] = {rows(out), flat(a->last_state, S * D, 4),
                          flat(a->checkpoints, B * ((L + kGatedTokens - 1) / kGatedTokens) * D, 4),
                          flat(a->workspace, static_cast<int64_t>(a->workspace_bytes), 1)};
  for (const Rows& o : outputs) {
    for (const Rows& i : inputs) {
      // last_state may be exactly h0 (the state carried in place)
      if (&o == &outputs[1] && &i == &inputs[5] && a->last_state == a->h0) continue;
      if (overlap(o, i)) return SSM_ERR_ALIAS;
    }
    for (const Rows& o2 : outputs)
      if (&o2 != &o && overlap(o, o2)) return SSM_ERR_ALIAS;
  }
  return SSM_OK;
}

int ssm_validate_gated_bwd(const ssm_gated_bwd_args* a) {
  if (!a) return SSM_ERR_NULL;
  if (const int st = check_gated(a)) return st;
  if (a->dim == 0) return SSM_OK;
  if (!a->lam || !a->dlam) return SSM_ERR_NULL;   // dlam is set (to zero) without any token too
  const int64_t B = a->batch, L = a->seqlen, D = a->dim, S = a->cu_seqlens ? a->nseq : B;
  const int64_t esz = io_size(a->io_dtype);
  const Tokens in[] = {{a->x, a->x_batch_stride, a->x_seq_stride},
                       {a->gate_a, a->gate_a_batch_stride, a->gate_a_seq_stride},
                       {a->gate_x, a->gate_x_batch_stride, a->gate_x_seq_stride},
                       {a->dout, a->dout_batch_stride, a->dout_seq_stride}};
  const Tokens out[] = {{a->dx, a->dx_batch_stride, a->dx_seq_stride},
                        {a->dgate_a, a->dgate_a_batch_stride, a->dgate_a_seq_stride},
                        {a->dgate_x, a->dgate_x_batch_stride, a->dgate_x_seq_stride}};
  if (L > 0 && B > 0) {
    if (!a->checkpoints) return SSM_ERR_NULL;
    if (const int st = check_tokens(in, 4, esz)) return st;
    if (const int st = check_tokens(out, 3, esz)) return st;
    for (const Tokens& t : out)
      if (collide(t, B, L, D)) return SSM_ERR_ALIAS;
  }
  if (misaligned(a->lam, 4) || misaligned(a->cu_seqlens, 4) || misaligned(a->h0, 4) ||
      misaligned(a->checkpoints, 4) || misaligned(a->dlast, 4) || misaligned(a->dlam, 4) ||
      misaligned(a->dh0, 4) || misaligned(a->workspace, 8))
    return SSM_ERR_ALIGN;
  const size_t need = gated_bwd_workspace_bytes(*a);
  if (need && (!a->workspace || a->workspace_bytes < need)) return SSM_ERR_SCRATCH;
  auto rows = [&](const Tokens& t) { return rows3(L > 0 ? t.p : nullptr, B, t.sb, L, t.ss, D, esz); };
  auto flat = [&](const void* p, int64_t n, int64_t e) { return Rows{span1(p, n, e)}; };
  const Rows inputs[] = {rows(in[0]), rows(in[1]), rows(in[2]), rows(in[3]), flat(a->lam, D, 4),
                         flat(a->cu_seqlens, S + 1, 4), flat(a->h0, S * D, 4), flat(a->dlast, S * D, 4),
                         flat(a->checkpoints, B * ((L + kGatedTokens - 1) / kGatedTokens) * D, 4)};
  const Rows outputs[] = {rows(out[0]), rows(out[1]), rows(out[2]), flat(a->dlam, D, 4), flat(a->dh0, S * D, 4),
                          flat(a->workspace, static_cast<int64_t>(a->workspace_bytes), 1)};
  for (const Rows& o : outputs) {
    for (const Rows& i : inputs)
      if (overlap(o, i)) return SSM_ERR_ALIAS;
    for (const Rows& o2 : outputs)
      if (&o2 != &o && overlap(o, o2)) return SSM_ERR_ALIAS;
  }
  return SSM_OK;
}

int ssm_validate_gated_update(const ssm_gated_update_args* a) {
  if (!a) return SSM_ERR_NULL;
  if (a->batch < 0 || a->dim < 0 || a->nslots < 0 || (!a->slots && a->batch > a->nslots)) return SSM_ERR_SHAPE;
  if (!(a->c > 0.0f) || !isfinite(a->c)) return SSM_ERR_SHAPE;
  if (bad_dtype(a->io_dtype)) return SSM_ERR_DTYPE;
  if (a->batch > 65535 || a->dim >= kMaxGroups) return SSM_ERR_UNSUPPORTED;
  if (a->batch == 0 || a->dim == 0) return SSM_OK;
  const int64_t esz = io_size(a->io_dtype), B = a->batch, D = a->dim, S = a->nslots;
  if ((!a->state && S > 0) || !a->lam) return SSM_ERR_NULL;
  const Tokens io[] = {{a->x, 0, a->x_batch_stride}, {a->gate_a, 0, a->gate_a_batch_stride},
                       {a->gate_x, 0, a->gate_x_batch_stride}, {a->out, 0, a->out_batch_stride}};
  if (const int st = check_tokens(io, 4, esz)) return st;
  if (a->state_slot_stride < 0) return SSM_ERR_STRIDE;
  if (misaligned(a->state, 4) || misaligned(a->lam, 4) || misaligned(a->slots, 4)) return SSM_ERR_ALIGN;
  if (rows_collide(1, 0, B, a->out_batch_stride, D) || rows_collide(1, 0, S, a->state_slot_stride, D))
    return SSM_ERR_ALIAS;
  auto rows = [&](const Tokens& t) { return rows3(t.p, 1, 0, B, t.ss, D, esz); };
  const Rows inputs[] = {rows(io[0]), rows(io[1]), rows(io[2]), Rows{span1(a->lam, D, 4)},
                         Rows{span1(a->slots, B, 4)}};
  const Rows out = rows(io[3]), state = rows3(a->state, 1, 0, S, a->state_slot_stride, D, 4);
  for (const Rows& i : inputs)
    if (overlap(out, i) || overlap(state, i)) return SSM_ERR_ALIAS;
  return overlap(out, state) ? SSM_ERR_ALIAS : SSM_OK;
}

}  // extern "C"

namespace {

int check_cache(const ssm_state_cache_args* a, bool write) {
  if (!a) return SSM_ERR_NULL;
  if (a->batch < 0 || a->nslots < 0 || a->outer < 0 || a->inner < 0 || (!a->slots && a->batch > a->nslots))
    return SSM_ERR_SHAPE;
  if (bad_dtype(a->io_dtype)) return SSM_ERR_DTYPE;
  if (a->format != SSM_CACHE_INT8 && a->format != SSM_CACHE_FP8 && a->format != SSM_CACHE_FP4) return SSM_ERR_DTYPE;
  if (a->format == SSM_CACHE_FP4 && a->inner % 2) return SSM_ERR_SHAPE;
  const int64_t limit = int64_t{1} << 28;   // 8 lanes a block, numbered in 32 bits
  if (a->batch > 65535 || a->inner >= (int64_t{1} << 31)) return SSM_ERR_UNSUPPORTED;
  const int64_t nblk = (a->inner + SSM_CACHE_BLOCK - 1) / SSM_CACHE_BLOCK;
  if (nblk && a->outer > limit / nblk) return SSM_ERR_UNSUPPORTED;
  if (a->batch == 0 || a->outer == 0 || a->inner == 0) return SSM_OK;
  if (((!a->codes || !a->scales) && a->nslots > 0) || !a->states) return SSM_ERR_NULL;
  if (a->codes_slot_stride < 0 || a->scales_slot_stride < 0 || a->states_batch_stride < 0) return SSM_ERR_STRIDE;
  const int64_t esz = io_size(a->io_dtype), n = a->outer * a->inner;
  if (misaligned(a->states, esz) || misaligned(a->slots, 4)) return SSM_ERR_ALIGN;
  const int64_t held = a->format == SSM_CACHE_FP4 ? n / 2 : n;
  const Rows codes = rows3(a->codes, 1, 0, a->nslots, a->codes_slot_stride, held, 1);
  const Rows scales = rows3(a->scales, 1, 0, a->nslots, a->scales_slot_stride, a->outer * nblk, 1);
  const Rows states = rows3(a->states, 1, 0, a->batch, a->states_batch_stride, n, esz);
  const Rows slots{span1(a->slots, a->batch, 4)};
  if (overlap(codes, states) || overlap(scales, states)) return SSM_ERR_ALIAS;
  if (write) {
    if (rows_collide(1, 0, a->nslots, a->codes_slot_stride, held) ||
        rows_collide(1, 0, a->nslots, a->scales_slot_stride, a->outer * nblk) || overlap(codes, scales) ||
        overlap(codes, slots) || overlap(scales, slots))
      return SSM_ERR_ALIAS;
  } else if (rows_collide(1, 0, a->batch, a->states_batch_stride, n) || overlap(states, slots)) {
    return SSM_ERR_ALIAS;
  }
  return SSM_OK;
}

}  // namespace

extern "C" {

int ssm_validate_state_cache_write(const ssm_state_cache_args* a) { return check_cache(a, true); }
int ssm_validate_state_cache_read(const ssm_state_cache_args* a) { return check_cache(a, false); }

int ssm_validate_cached_update(const ssm_cached_update_args* a) {
  if (!a) return SSM_ERR_NULL;
  if (a->batch < 0 || a->dim < 0 || a->nslots < 0 || a->dstate < 1 || (!a->slots && a->batch > a->nslots))
    return SSM_ERR_SHAPE;
  if (bad_groups(a->ngroups, a->dim)) return SSM_ERR_SHAPE;
  if (bad_dtype(a->io_dtype)) return SSM_ERR_DTYPE;
  if (a->dstate > SSM_MAX_DSTATE || a->batch > 65535 || a->dim >= kMaxGroups) return SSM_ERR_UNSUPPORTED;
  if (a->batch == 0 || a->dim == 0) return SSM_OK;
  if (((!a->codes || !a->scales) && a->nslots > 0) || !a->x || !a->dt || !a->B || !a->C || !a->A || !a->out)
    return SSM_ERR_NULL;
  const int64_t G = groups_of(a->ngroups);
  const int64_t strides[] = {a->codes_slot_stride, a->scales_slot_stride, a->x_batch_stride, a->dt_batch_stride,
                             a->z ? a->z_batch_stride : 0, a->B_batch_stride, a->C_batch_stride,
                             G > 1 ? a->B_group_stride : 0, G > 1 ? a->C_group_stride : 0, a->A_dim_stride,
                             a->out_batch_stride};
  for (int64_t s : strides)
    if (s < 0) return SSM_ERR_STRIDE;
  const int64_t esz = io_size(a->io_dtype), B = a->batch, D = a->dim, N = a->dstate, S = a->nslots;
  if (misaligned(a->x, esz) || misaligned(a->dt, esz) || misaligned(a->z, esz) || misaligned(a->B, esz) ||
      misaligned(a->C, esz) || misaligned(a->out, esz) || misaligned(a->A, 4) || misaligned(a->D, 4) ||
      misaligned(a->dt_bias, 4) || misaligned(a->slots, 4) || misaligned(a->seed, 8))
    return SSM_ERR_ALIGN;
  const int64_t nblk = (N + SSM_CACHE_BLOCK - 1) / SSM_CACHE_BLOCK;
  if (rows_collide(1, 0, B, a->out_batch_stride, D) || rows_collide(1, 0, S, a->codes_slot_stride, D * N) ||
      rows_collide(1, 0, S, a->scales_slot_stride, D * nblk))
    return SSM_ERR_ALIAS;
  auto rows = [&](const void* p, int64_t s) { return rows3(p, 1, 0, B, s, D, esz); };
  const Rows inputs[] = {rows(a->x, a->x_batch_stride), rows(a->dt, a->dt_batch_stride), rows(a->z, a->z_batch_stride),
                         Rows{span3(a->B, B, a->B_batch_stride, G, a->B_group_stride, N, esz)},
                         Rows{span3(a->C, B, a->C_batch_stride, G, a->C_group_stride, N, esz)},
                         Rows{span3(a->A, 1, 0, D, a->A_dim_stride, N, 4)}, Rows{span1(a->D, D, 4)},
                         Rows{span1(a->dt_bias, D, 4)}, Rows{span1(a->slots, B, 4)}, Rows{span1(a->seed, 1, 8)}};
  const Rows outputs[] = {rows(a->out, a->out_batch_stride), rows3(a->codes, 1, 0, S, a->codes_slot_stride, D * N, 1),
                          rows3(a->scales, 1, 0, S, a->scales_slot_stride, D * nblk, 1)};
  for (const Rows& o : outputs) {
    for (const Rows& i : inputs)
      if (overlap(o, i)) return SSM_ERR_ALIAS;
    for (const Rows& o2 : outputs)
      if (&o2 != &o && overlap(o, o2)) return SSM_ERR_ALIAS;
  }
  return SSM_OK;
}

int ssm_gated_scan_fwd(const ssm_gated_args* a, void* stream) {
  if (const int st = ssm_validate_gated(a)) return st;
  if (a->batch == 0 || a->dim == 0) return SSM_OK;
  return launch_gated_fwd(*a, static_cast<hipStream_t>(stream)) == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

int ssm_gated_scan_bwd(const ssm_gated_bwd_args* a, void* stream) {
  if (const int st = ssm_validate_gated_bwd(a)) return st;
  if (a->dim == 0) return SSM_OK;
  return launch_gated_bwd(*a, static_cast<hipStream_t>(stream)) == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

int ssm_gated_state_update(const ssm_gated_update_args* a, void* stream) {
  if (const int st = ssm_validate_gated_update(a)) return st;
  if (a->batch == 0 || a->dim == 0) return SSM_OK;
  return launch_gated_step(*a, static_cast<hipStream_t>(stream)) == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

int ssm_state_cache_write(const ssm_state_cache_args* a, void* stream) {
  if (const int st = check_cache(a, true)) return st;
  if (a->batch == 0 || a->outer == 0 || a->inner == 0 || a->nslots == 0) return SSM_OK;
  return launch_cache_write(*a, static_cast<hipStream_t>(stream)) == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

int ssm_state_cache_read(const ssm_state_cache_args* a, void* stream) {
  if (const int st = check_cache(a, false)) return st;
  if (a->batch == 0 || a->outer == 0 || a->inner == 0) return SSM_OK;
  return launch_cache_read(*a, static_cast<hipStream_t>(stream)) == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

int ssm_selective_state_update_cached(const ssm_cached_update_args* a, void* stream) {
  if (const int st = ssm_validate_cached_update(a)) return st;
  if (a->batch == 0 || a->dim == 0) return SSM_OK;
  return launch_cached_update(*a, static_cast<hipStream_t>(stream)) == hipSuccess ? SSM_OK : SSM_ERR_HIP;
}

}  // extern "C"
