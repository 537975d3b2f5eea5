// Attention over the paged cache.
//
// A simple form: one wave for each query row and head, the keys one after
// another, running maximum and sum of the softmax in fp32.
#include "seq_dev.h"

namespace moeq4 {

namespace {

constexpr int THREADS = 256;

template <int D>
__global__ __launch_bounds__(THREADS) void attention_kernel(AttentionArgs a) {
    constexpr int E = D / WAVE;  // entries of a lane
    const int64_t w = (int64_t)blockIdx.x * (THREADS / WAVE) + threadIdx.x / WAVE;
    if (w >= a.T * a.hq) return;
    const int64_t t = w / a.hq;
    const int h = (int)(w % a.hq), hk = h / (a.hq / a.cache.hkv), lane = threadIdx.x & (WAVE - 1);
    const int b = find_sequence(a.seq_start, a.n_seq, t);
    if (b < 0) return;
    const int64_t start = max(a.seq_start[b], 0), end = min((int64_t)a.seq_start[b + 1], a.T);
    if (t >= end) return;
    const int64_t kv = max(a.cache.kv_len[b], 0), n = end - start;
    const int64_t len = min(kv, (int64_t)a.cache.max_pages * a.cache.page), before = kv - n, row = t - start;
    const int64_t prefix = a.prefix ? a.prefix[b] : 0;
    const uint64_t mask = a.tree ? a.tree[t] : 0;
    const int64_t pos = a.tree ? before + __popcll(row < 64 ? mask & ~(1ull << row) : mask) : before + row;
    const float slope = a.slopes ? a.slopes[h] : 0.0f;
    float q[E], o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        q[e] = bf16_to_f32(a.q[t * a.ldq + (int64_t)h * D + lane * E + e]);
        o[e] = 0.0f;
    }
    float top = -INFINITY, sum = 0.0f;
    for (int64_t i = 0; i < len; ++i) {
        int64_t at = i;
        bool seen;
        if (a.tree && i >= before) {
            const int64_t j = i - before;
            seen = j < 64 && (mask >> j & 1);
            if (!seen) continue;
            at = before + __popcll(a.tree[start + j] & ~(1ull << j));
            seen = !a.window || pos - at < a.window;
        } else {
            seen = (a.tree || i <= pos) && (!a.window || pos - i < a.window);
        }
        if (!seen && i >= prefix) continue;
        const int page = a.cache.table[(int64_t)b * a.cache.max_pages + i / a.cache.page];
        if (page < 0 || page >= a.cache.n_pages) continue;
        const int64_t from = (((int64_t)page * a.cache.hkv + hk) * a.cache.page + i % a.cache.page) * D + lane * E;
        float s = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) s = fmaf(q[e], bf16_to_f32(a.cache.k[from + e]), s);
        s = seg_sum<WAVE>(s) * a.scale;
        if (a.cap > 0.0f) s = a.cap * tanhf(s / a.cap);
        s -= slope * (float)(pos > at ? pos - at : at - pos);
        const float m = fmaxf(top, s), keep = expf(top - m), p = expf(s - m);
        top = m;
        sum = sum * keep + p;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(p, bf16_to_f32(a.cache.v[from + e]), o[e] * keep);
    }
#pragma unroll
    for (int e = 0; e < E; ++e)
        a.o[t * a.ldo + (int64_t)h * D + lane * E + e] = f32_to_bf16_rne(sum == 0.0f ? 0.0f : o[e] / sum);
}

}  // namespace

size_t attention_workspace_bytes(int64_t, int, int, const Cache &) { return 0; }

hipError_t launch_attention(const AttentionArgs &a, void *, hipStream_t s) {
    const dim3 grid((unsigned)((a.T * a.hq + THREADS / WAVE - 1) / (THREADS / WAVE)));
    if (a.cache.d == 64)
        attention_kernel<64><<<grid, THREADS, 0, s>>>(a);
    else if (a.cache.d == 128)
        attention_kernel<128><<<grid, THREADS, 0, s>>>(a);
    else
        attention_kernel<256><<<grid, THREADS, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace moeq4
