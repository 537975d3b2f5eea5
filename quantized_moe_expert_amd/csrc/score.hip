// Log probabilities of given tokens, entropy and the largest logits of rows.
#include "backbone.h"

namespace moeq4 {

namespace {

// Order-preserving image of a float: a larger value gives a larger key, equal
// values equal keys (-0 as +0); a NaN counts as -inf.
__device__ __forceinline__ float clean(float f) { return f == f ? f : -INFINITY; }
__device__ __forceinline__ uint32_t f32_order(float f) {
    const uint32_t b = __float_as_uint(clean(f) + 0.0f);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float f32_from_order(uint32_t o) {
    return __uint_as_float((o & 0x80000000u) ? (o ^ 0x80000000u) : ~o);
}

__device__ __forceinline__ float load_logit(const LogprobsArgs &a, int64_t at) {
    return a.f32 ? static_cast<const float *>(a.logits)[at]
                 : bf16_to_f32(static_cast<const uint16_t *>(a.logits)[at]);
}

__device__ __forceinline__ uint64_t wave_max_u64(uint64_t v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
        const uint64_t w = __shfl_xor((unsigned long long)v, o);
        v = v > w ? v : w;
    }
    return v;
}

// One workgroup per row: the maximum, the sums, then the largest keys one
// after another, a pass over the row each.
__global__ __launch_bounds__(256) void logprobs_row_kernel(LogprobsArgs a) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t t = blockIdx.x, base = t * a.ld;
    __shared__ uint64_t s_key[4];
    __shared__ float s_sum[4][2];
    auto largest_below = [&](uint64_t limit) {
        uint64_t best = 0;
        for (int64_t v = tid; v < a.V; v += 256) {
            const uint64_t key = ((uint64_t)f32_order(load_logit(a, base + v)) << 32) | (0xffffffffu - (uint32_t)v);
            if (key < limit && key > best) best = key;
        }
        best = wave_max_u64(best);
        __syncthreads();
        if (lane == 0) s_key[wave] = best;
        __syncthreads();
        best = s_key[0];
        for (int i = 1; i < 4; ++i) best = s_key[i] > best ? s_key[i] : best;
        return best;
    };
    uint64_t key = largest_below(~0ull);
    const float m = f32_from_order((uint32_t)(key >> 32));
    const bool empty = m == -INFINITY;
    // d = 0 where the logit is the maximum, so that an infinite maximum works
    auto below_max = [&](float l) { return l == m ? 0.0f : l - m; };
    float z = 0.f, sd = 0.f;
    for (int64_t v = tid; v < a.V; v += 256) {
        const float l = clean(load_logit(a, base + v));
        const float d = below_max(l), e = expf(d);
        z += e;
        if (e > 0.f) sd += e * d;
    }
    z = seg_sum<64>(z);
    sd = seg_sum<64>(sd);
    if (lane == 0) s_sum[wave][0] = z, s_sum[wave][1] = sd;
    __syncthreads();
    z = s_sum[0][0] + s_sum[1][0] + s_sum[2][0] + s_sum[3][0];
    sd = s_sum[0][1] + s_sum[1][1] + s_sum[2][1] + s_sum[3][1];
    const float lz = logf(z);
    if (tid == 0) {
        if (a.tokens) {
            const int tok = a.tokens[t];
            float lp = 0.f;
            if (tok >= 0 && tok < a.V)
                lp = empty ? -INFINITY : below_max(clean(load_logit(a, base + tok))) - lz;
            a.logprob[t] = lp;
        }
        if (a.entropy) a.entropy[t] = empty ? 0.f : lz - sd / z;
    }
    for (int i = 0; i < a.n_top; ++i) {
        if (i) key = largest_below(key);
        if (tid == 0) {
            a.top_idx[t * a.n_top + i] = (int32_t)(0xffffffffu - (uint32_t)key);
            const float l = f32_from_order((uint32_t)(key >> 32));
            a.top_logprob[t * a.n_top + i] = empty ? -INFINITY : below_max(l) - lz;
        }
    }
}

}  // namespace

hipError_t launch_logprobs(const LogprobsArgs &a, hipStream_t s) {
    hipLaunchKernelGGL(logprobs_row_kernel, dim3((unsigned)a.T), dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace moeq4
