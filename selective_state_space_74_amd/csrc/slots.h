// Rows of a batch that name the same slot of a pool.  They are taken in the
// order of the rows: the workgroup of the first such row takes them all, and
// the others leave theirs to it, so no two workgroups touch one slot.
#pragma once

#include "ssm_internal.h"

namespace ssm {

constexpr int kNames = 4;   // slots a lane compares at a time

// Whether an earlier row than `row` names its slot, and the next row that does,
// or batch.  Without slots every row has its own.
__device__ __forceinline__ void slot_order(const int32_t* slots, int row, int batch, int slot, int lane, bool& before,
                                           int& next) {
  before = false;
  next = batch;
  if (!slots) return;
  // hardly ever does any: look for that first
  bool shared = false;
  for (int base = 0; base < batch; base += 64 * kNames) {
    int named[kNames];
#pragma unroll
    for (int k = 0; k < kNames; ++k) {
      const int i = base + 64 * k + lane;
      named[k] = i < batch && i != row ? slots[i] : -1;
    }
#pragma unroll
    for (int k = 0; k < kNames; ++k) shared |= named[k] == slot;
  }
  if (!__any(shared)) return;
  for (int base = 0; base < batch; base += 64) {
    const int i = base + lane;
    const bool hit = i < batch && slots[i] == slot;
    if (__any(hit && i < row)) before = true;
    const uint64_t later = __ballot(hit && i > row);
    if (later && next == batch) next = base + __builtin_ctzll(later);
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
