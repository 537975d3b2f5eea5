// Rows on the device: eight bf16 values at a time, and which of the packed
// sequences a row belongs to.
#pragma once

#include "backbone.h"

namespace moeq4 {

// Two floats rounded to bf16 (nearest even), a in the low half.
__device__ __forceinline__ uint32_t pack_bf16x2(float a, float b) {
    const bf16x2_t v = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, v);
}
__device__ __forceinline__ u32x4_t pack8(const float *f) {
    return u32x4_t{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])};
}
__device__ __forceinline__ void unpack8(u32x4_t w, float *f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

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
