#pragma once
// What the operators on packed prompts and on pools of state slots share: the reading of
// cu_seqlens and of slot indices, which live on the device and so are checked there.
#include <cstdint>

namespace ssm {

// What a slot index says about its row or sequence.
//   kSlotLive   0 <= slot < n_slots
//   kSlotPad    slot < 0: padding; nothing is read or written for it
//   kSlotBad    slot >= n_slots: no state is touched and the outputs are NaN
enum SlotKind { kSlotLive, kSlotPad, kSlotBad };

__device__ __forceinline__ SlotKind slot_kind(int slot, int64_t n_slots) {
    return slot < 0 ? kSlotPad : slot < n_slots ? kSlotLive : kSlotBad;
}

// Tokens [lo, hi) of sequence i in a packed buffer of `total` tokens.  Bounds that lie outside
// the buffer or run backwards are clamped, so no value in cu_seqlens makes an access outside it.
struct TokenRange {
    int64_t lo, hi;
};
__device__ __forceinline__ TokenRange token_range(const int* cu, int64_t i, int64_t total) {
    int64_t lo = __ldg(cu + i), hi = __ldg(cu + i + 1);
    lo = lo < 0 ? 0 : lo > total ? total : lo;
    hi = hi < lo ? lo : hi > total ? total : hi;
    return {lo, hi};
}

}  // namespace ssm
