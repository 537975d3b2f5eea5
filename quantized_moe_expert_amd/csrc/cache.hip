// Keys and values into the paged cache, queries and keys normed and turned on
// the way: per head
//   x <- x / sqrt(mean x^2 + eps) * norm,   (a, b) <- (a cos - b sin, b cos + a sin).
//
// Bound by the bytes of the rows, read and written once, and for few tokens by
// one chain of loads.  One workgroup per token: its rot / 2 angles are computed
// once, in 64 bits, and kept in LDS for all heads.
#include "seq_dev.h"

namespace moeq4 {

namespace {

constexpr int THREADS = 256;
constexpr int MAX_HALF = 128;  // pairs of a head of 256

__device__ __forceinline__ void unpack8(u32x4_t w, float *f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ u32x4_t pack8(const float *f) {
    u32x4_t w;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = (uint32_t)f32_to_bf16_rne(f[2 * i]) | ((uint32_t)f32_to_bf16_rne(f[2 * i + 1]) << 16);
    return w;
}

// Each lane has 8 entries of a head, D / 8 lanes a head.  The partner's entries
// (half pairs) are loaded beside its own: the second reading is the cache's.
template <int D>
__global__ __launch_bounds__(THREADS) void kv_append_kernel(AppendArgs a) {
    constexpr int LPH = D / 8, HPW = WAVE / LPH;  // lanes a head, heads a wave
    __shared__ float cs[MAX_HALF], sn[MAX_HALF];
    const int64_t t = blockIdx.x;
    const int b = find_sequence(a.seq_start, a.n_seq, t);
    if (b < 0) return;
    const int64_t end = min((int64_t)a.seq_start[b + 1], a.T);
    if (t >= end) return;  // a row behind the last sequence
    const int64_t index = (int64_t)a.cache.kv_len[b] - (end - t);
    const int64_t capacity = (int64_t)a.cache.max_pages * a.cache.page;
    // A token's place: negative when it is not stored.
    int64_t page = -1;
    int off = 0;
    if (index >= 0 && index < capacity) {
        const int p = (int)((uint32_t)index / (uint32_t)a.cache.page);
        off = (int)((uint32_t)index - (uint32_t)p * (uint32_t)a.cache.page);
        const int id = a.cache.table[(int64_t)b * a.cache.max_pages + p];
        if (id >= 0 && id < a.cache.n_pages) page = id;
    }
    const int half = a.rot / 2;
    if (half) {
        const int tid = threadIdx.x;
        if (tid < half) {
            const double pos = a.positions ? (double)a.positions[t] : (double)index;
            // In turns: what lies beyond whole ones is exact to 2^-52 of the product.
            const double turns = pos * (double)a.inv_freq[tid] * 0.15915494309189533577;
            const double rest = turns - rint(turns);
            float s, c;
            sincospif((float)(2.0 * rest), &s, &c);
            cs[tid] = c;
            sn[tid] = s;
        }
        __syncthreads();
    }
    const int lane = threadIdx.x & (WAVE - 1), wave = threadIdx.x / WAVE;
    const int c = lane % LPH;  // 8 entries from 8 c on
    const int heads = a.hq + 2 * a.cache.hkv;
    for (int h0 = wave * HPW; h0 < heads; h0 += THREADS / WAVE * HPW) {
        const int h = h0 + lane / LPH;
        if (h >= heads) break;
        const bool is_q = h < a.hq, is_v = h >= a.hq + a.cache.hkv;
        const int hh = is_q ? h : (h - a.hq) % a.cache.hkv;
        const uint16_t *src = is_q ? a.q + t * a.ldq : is_v ? a.v + t * a.ldv : a.k + t * a.ldk;
        src += (int64_t)hh * D;
        uint16_t *dst = nullptr;
        if (is_q)
            dst = a.q_out + t * a.ldqo + (int64_t)hh * D;
        else if (page >= 0)
            dst = (is_v ? a.cache.v : a.cache.k) + ((page * a.cache.hkv + hh) * a.cache.page + off) * D;
        const u32x4_t raw = *reinterpret_cast<const u32x4_t *>(src + 8 * c);
        u32x4_t res = raw;
        if (!is_v) {
            const float *w = is_q ? a.q_norm : a.k_norm;
            const bool turned = 8 * c < a.rot;
            int mate = c;  // the chunk of the other halves of the lane's pairs
            if (turned && !a.interleaved) mate = 16 * c < a.rot ? c + a.rot / 16 : c - a.rot / 16;
            float x[8], m[8];
            unpack8(raw, x);
            unpack8(mate == c ? raw : *reinterpret_cast<const u32x4_t *>(src + 8 * mate), m);
            if (w) {
                float sum = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) sum = fmaf(x[i], x[i], sum);
                // (The lanes of a head are in one wave and leave the loop together.)
                sum = seg_sum<LPH>(sum);
                const float inv = 1.0f / sqrtf(sum * (1.0f / D) + a.eps);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    x[i] *= inv * w[8 * c + i];
                    m[i] *= inv * w[8 * mate + i];
                }
            }
            if (turned) {
                float y[8];
                if (a.interleaved) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float co = cs[4 * c + i], si = sn[4 * c + i];
                        y[2 * i] = x[2 * i] * co - x[2 * i + 1] * si;
                        y[2 * i + 1] = x[2 * i + 1] * co + x[2 * i] * si;
                    }
                } else {
                    const bool second = 16 * c >= a.rot;
                    const int j = 8 * (second ? mate : c);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float si = second ? sn[j + i] : -sn[j + i];
                        y[i] = fmaf(m[i], si, x[i] * cs[j + i]);
                    }
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = y[i];
            }
            if (w || turned) res = pack8(x);
        }
        if (dst) *reinterpret_cast<u32x4_t *>(dst + 8 * c) = res;
    }
}

}  // namespace

hipError_t launch_kv_append(const AppendArgs &a, hipStream_t s) {
    const dim3 grid((unsigned)a.T);
    if (a.cache.d == 64)
        kv_append_kernel<64><<<grid, THREADS, 0, s>>>(a);
    else if (a.cache.d == 128)
        kv_append_kernel<128><<<grid, THREADS, 0, s>>>(a);
    else
        kv_append_kernel<256><<<grid, THREADS, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace moeq4
