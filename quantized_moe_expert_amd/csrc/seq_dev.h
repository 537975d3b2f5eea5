// Packed sequences on the device: which sequence a row belongs to, and where
// a token of a sequence lies in the paged cache.
#pragma once

#include "backbone.h"

namespace moeq4 {

// The last sequence that starts at or before row t (t >= 0), by the whole wave:
// 64 starts are looked at in each step.  -1: none.  With ascending starts the
// row belongs to it, or to none if it ends at or before t.
__device__ __forceinline__ int find_sequence(const int32_t *seq_start, int n_seq, int64_t t) {
    int lo = 0, n = n_seq;  // the answer is lo - 1 or among [lo, lo + n)
    const int lane = threadIdx.x & (WAVE - 1);
    while (n > 0) {
        const int step = (n + WAVE - 1) / WAVE;
        const int64_t at = (int64_t)(lane + 1) * step - 1;  // the last of the lane's step
        const bool in = at < n && seq_start[lo + at] <= t;
        const int full = __popcll(__ballot(in));            // steps that start at or before t
        if (step == 1) return lo + full - 1;
        lo += full * step;
        n = min(step - 1, n - full * step);                 // the next step, but for its last, which is behind t
        if (n <= 0) break;
    }
    return lo - 1;
}

}  // namespace moeq4
