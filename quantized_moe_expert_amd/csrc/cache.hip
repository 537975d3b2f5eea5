// Keys and values into the paged cache, queries and keys normed and turned on
// the way: per head
//   x <- x / sqrt(mean x^2 + eps) * norm,   (a, b) <- (a cos - b sin, b cos + a sin).
//
// Bound by the bytes of the rows, read and written once, and for few tokens by
// one chain of loads.  One workgroup per token: its rot / 2 angles are computed
// once, in 64 bits, and kept in LDS for all heads.  Measured: 8000 tokens of 48
// heads of 128 41 us, 4.8 TB/s (a copy's rate); 16 tokens 6 us.  It lives on
// occupancy: a wave to a token takes 64 us, four heads a lane at once (85 registers) 61.
#include "rows_dev.h"

namespace moeq4 {

namespace {

constexpr int THREADS = 256;
constexpr int MAX_HALF = 128;  // pairs of a head of 256

__device__ __forceinline__ void turn(float a, float b, float co, float si, float &y0, float &y1) {
    y0 = fmaf(-b, si, a * co);
    y1 = fmaf(a, si, b * co);
}

struct __attribute__((packed, aligned(4))) Eight {
    float v[8];
};

// Each lane has 8 entries of a head, D / 8 lanes a head; the partner's entries
// (half pairs) come from its lane.  The first GROUP heads of a lane are loaded before the token's sequence is
// looked up: neither waits for the other.
template <int D>
__global__ __launch_bounds__(THREADS, 8) void kv_append_kernel(AppendArgs a) {
    constexpr int LPH = D / 8, HPW = WAVE / LPH;  // lanes a head, heads a wave
    constexpr int STEP = THREADS / WAVE * HPW, GROUP = 2;  // (1: 47 us, 3: 42, 4: 48 for 8000 tokens)
    __shared__ __attribute__((aligned(16))) float cs[MAX_HALF], sn[MAX_HALF];
    const int64_t t = blockIdx.x;
    const int tid = threadIdx.x, lane = tid & (WAVE - 1), wave = tid / WAVE;
    const int c = lane % LPH;  // 8 entries from 8 c on
    const int heads = a.hq + 2 * a.cache.hkv, half = a.rot / 2;
    const bool turned = 8 * c < a.rot;
    int mate = c;  // the chunk of the other halves of the lane's pairs
    if (turned && !a.interleaved) mate = 16 * c < a.rot ? c + a.rot / 16 : c - a.rot / 16;
    u32x4_t own[GROUP];
    auto load = [&](int h0) {
#pragma unroll
        for (int u = 0; u < GROUP; ++u) {
            const int h = h0 + u * STEP;
            if (h >= heads) continue;
            const bool is_q = h < a.hq, is_v = h >= a.hq + a.cache.hkv;
            const int hh = is_q ? h : is_v ? h - a.hq - a.cache.hkv : h - a.hq;
            const uint16_t *src = (is_q ? a.q + t * a.ldq : is_v ? a.v + t * a.ldv : a.k + t * a.ldk) + hh * D;
            own[u] = *reinterpret_cast<const u32x4_t *>(src + 8 * c);
        }
    };
    int h0 = wave * HPW + lane / LPH;
    load(h0);
    const float freq = tid < half ? a.inv_freq[tid] : 0.0f;

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
    if (half) {
        if (tid < half) {
            const double pos = a.positions ? (double)a.positions[t] : (double)index;
            // In turns: what lies beyond whole ones is exact to 2^-52 of the product.
            const double turns = pos * (double)freq * 0.15915494309189533577;
            float si, co;
            sincospif((float)(2.0 * (turns - rint(turns))), &si, &co);
            cs[tid] = co;
            sn[tid] = si;
        }
        __syncthreads();
    }
    for (; h0 < heads; h0 += GROUP * STEP) {
#pragma unroll
        for (int u = 0; u < GROUP; ++u) {
            const int h = h0 + u * STEP;
            if (h >= heads) continue;  // (for all lanes of a head)
            const bool is_q = h < a.hq, is_v = h >= a.hq + a.cache.hkv;
            const int hh = is_q ? h : is_v ? h - a.hq - a.cache.hkv : h - a.hq;
            uint16_t *dst = nullptr;
            if (is_q)
                dst = a.q_out + t * a.ldqo + hh * D;
            else if (page >= 0)
                dst = (is_v ? a.cache.v : a.cache.k) + ((page * a.cache.hkv + hh) * a.cache.page + off) * D;
            const float *w = is_v ? nullptr : is_q ? a.q_norm : a.k_norm;
            u32x4_t res = own[u];
            if (!is_v && (w || a.rot)) {
                float x[8], m[8];
                unpack8(own[u], x);
                u32x4_t other = own[u];
                if (a.rot && !a.interleaved)
#pragma unroll
                    for (int i = 0; i < 4; ++i) other[i] = __shfl(own[u][i], lane - c + mate, WAVE);
                unpack8(other, m);
                if (w) {
                    float sum = 0.0f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) sum = fmaf(x[i], x[i], sum);
                    sum = seg_sum<LPH>(sum);
                    const float inv = 1.0f / sqrtf(sum * (1.0f / D) + a.eps);
                    const Eight wx = *reinterpret_cast<const Eight *>(w + 8 * c);
                    const Eight wm = *reinterpret_cast<const Eight *>(w + 8 * mate);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        x[i] *= inv * wx.v[i];
                        m[i] *= inv * wm.v[i];
                    }
                }
                if (turned) {
                    float y[8];
                    if (a.interleaved) {
                        const float4 co = *reinterpret_cast<const float4 *>(cs + 4 * c);
                        const float4 si = *reinterpret_cast<const float4 *>(sn + 4 * c);
                        turn(x[0], x[1], co.x, si.x, y[0], y[1]);
                        turn(x[2], x[3], co.y, si.y, y[2], y[3]);
                        turn(x[4], x[5], co.z, si.z, y[4], y[5]);
                        turn(x[6], x[7], co.w, si.w, y[6], y[7]);
                    } else {
                        const bool second = 16 * c >= a.rot;
                        const int j = 8 * (second ? mate : c);
#pragma unroll
                        for (int i = 0; i < 8; i += 4) {
                            const float4 co = *reinterpret_cast<const float4 *>(cs + j + i);
                            const float4 si = *reinterpret_cast<const float4 *>(sn + j + i);
                            const float sign = second ? 1.0f : -1.0f;
                            y[i] = fmaf(m[i], sign * si.x, x[i] * co.x);
                            y[i + 1] = fmaf(m[i + 1], sign * si.y, x[i + 1] * co.y);
                            y[i + 2] = fmaf(m[i + 2], sign * si.z, x[i + 2] * co.z);
                            y[i + 3] = fmaf(m[i + 3], sign * si.w, x[i + 3] * co.w);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i] = y[i];
                }
                res = pack8(x);
            }
            if (dst) *reinterpret_cast<u32x4_t *>(dst + 8 * c) = res;
        }
        if (h0 + GROUP * STEP < heads) load(h0 + GROUP * STEP);
    }
}

template <int D>
hipError_t launch(const AppendArgs &a, hipStream_t s) {
    kv_append_kernel<D><<<dim3((unsigned)a.T), THREADS, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_append(const AppendArgs &a, hipStream_t s) {
    return a.cache.d == 64 ? launch<64>(a, s) : a.cache.d == 128 ? launch<128>(a, s) : launch<256>(a, s);
}

}  // namespace moeq4
