#pragma once
// What the operators on packed prompts and on pools of state slots share: the reading of
// cu_seqlens and of slot indices, which live on the device and so are checked there, and index
// arithmetic that a test on the CPU walks through.
#include <cstdint>
#include <initializer_list>

namespace ssm {

// Whether each of the pointers (a null one too) lies on a boundary of n bytes, a power of two.
inline bool all_aligned(uintptr_t n, std::initializer_list<const void*> pointers) {
    for (const void* p : pointers)
        if (reinterpret_cast<uintptr_t>(p) & (n - 1)) return false;
    return true;
}
inline bool aligned_to(const void* p, uintptr_t n) { return all_aligned(n, {p}); }

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

// A CTA of the packed convolution works on `rows` channels from d0 on, in steps of ty, the channels of
// two steps as one pair: the channel whose taps row `row` of it keeps, or -1.  Where the channels end
// between the two, the second is the first once more; a first row behind the last channel has none.
__host__ __device__ __forceinline__ int64_t tap_channel(int64_t d0, int row, int ty, int64_t dim) {
    const int64_t d = d0 + row;
    if (d < dim) return d;
    return (row / ty & 1) && d - ty < dim ? d - ty : -1;
}

}  // namespace ssm
