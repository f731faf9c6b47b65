// Rows of a batch that name the same slot of a pool.  They are taken in the
// order of the rows: the workgroup of the first such row takes them all, and
// the others leave theirs to it, so no two workgroups touch one slot.
#pragma once

#include "ssm_internal.h"

namespace ssm {

constexpr int kNames = 4;   // slots a lane compares at a time

// For rows first .. first + ROWS - 1 with slots slot[]: bit r of `before` says
// whether an earlier row names slot[r]; next[r] is the next row that does, or
// batch.  Rows with slot -1 are of no account.  Without slots every row has its
// own.
template <int ROWS>
__device__ __forceinline__ void slot_order(const int32_t* slots, int first, int batch, const int (&slot)[ROWS], int lane,
                                           uint32_t& before, int (&next)[ROWS]) {
  before = 0;
#pragma unroll
  for (int r = 0; r < ROWS; ++r) next[r] = batch;
  if (!slots) return;
  // hardly ever does any: look for that first
  bool shared = false;
  for (int base = 0; base < batch; base += 64 * kNames) {
    int named[kNames];
#pragma unroll
    for (int k = 0; k < kNames; ++k) {
      const int i = base + 64 * k + lane;
      named[k] = i < batch ? slots[i] : -2;
    }
#pragma unroll
    for (int k = 0; k < kNames; ++k)
#pragma unroll
      for (int r = 0; r < ROWS; ++r) shared |= named[k] == slot[r] && base + 64 * k + lane != first + r;
  }
  if (!__any(shared)) return;
  for (int base = 0; base < batch; base += 64) {
    const int i = base + lane;
    const int named = i < batch ? slots[i] : -2;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      const bool hit = named == slot[r];
      if (__any(hit && i < first + r)) before |= 1u << r;
      const uint64_t later = __ballot(hit && i > first + r);
      if (later && next[r] == batch) next[r] = base + __builtin_ctzll(later);
    }
  }
}

// The next row of the batch after row `from` that names this slot, or batch.
__device__ __forceinline__ int named_next(const int32_t* slots, int from, int batch, int slot, int lane) {
  for (int base = from + 1; base < batch; base += 64) {
    const int i = base + lane;
    const uint64_t hits = __ballot(i < batch && slots[i] == slot);
    if (hits) return base + __builtin_ctzll(hits);
  }
  return batch;
}

}  // namespace ssm
