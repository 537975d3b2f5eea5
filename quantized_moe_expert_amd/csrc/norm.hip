// Between two blocks: norm of a block's output, gate, residual, norm before the
// next block, in one pass:
//   r = u [/ rms(u) * post] [* act(gate)],  x_out = bf16(x + scale r),  y = x_out / rms(x_out) * pre.
//
// Bound by the bytes of the rows, each read and written once: a row stays in
// registers between the two sums of squares.  For few rows: one chain of loads
// and two sums.  Measured: 8192 rows of 4096 with every input 69 to 71 us, 4.8 TB/s (a
// copy's rate); 16 rows of 2048 3.1 us; as many values in rows of 8192 91 us, of 16384 110, of
// 32768 92, of 65536 132 (the kernel for more than 32768 has 152 bytes of scratch a lane).
#include "rows_dev.h"
#include "../../include/moe_q4_backbone.h"

namespace moeq4 {

namespace {

// Sum over the LANES lanes of a row (a part of a wave, or several waves; part:
// an array for this sum alone).
template <int LANES>
__device__ __forceinline__ float row_sum(float v, float *part) {
    v = seg_sum<(LANES < WAVE ? LANES : WAVE)>(v);
    if constexpr (LANES > WAVE) {
        const int wave = threadIdx.x / WAVE;
        if ((threadIdx.x & (WAVE - 1)) == 0) part[wave] = v;
        __syncthreads();
        v = part[0];
#pragma unroll
        for (int i = 1; i < LANES / WAVE; ++i) v += part[i];
    }
    return v;
}

// LANES lanes a row, each with N times 8 values at a distance of LANES * 8.  All
// of a row's loads are issued before the first sum.
template <int LANES, int N>
__global__ __launch_bounds__(LANES < 256 ? 256 : LANES, N == 1 ? 8 : 4) void add_norm_kernel(AddNormArgs a) {
    constexpr int THREADS = LANES < 256 ? 256 : LANES, ROWS = THREADS / LANES;
    static_assert(ROWS == 1 || LANES <= WAVE, "a barrier needs all threads");
    __shared__ float part[2][THREADS / WAVE];
    const int lane = threadIdx.x % LANES;
    const int64_t t = (int64_t)blockIdx.x * ROWS + threadIdx.x / LANES;
    const float inv_h = 1.0f / (float)a.H;
    float r[N][8];
    u32x4_t xr[N], gr[N];
    bool in[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int at = 8 * (n * LANES + lane);
        in[n] = t < a.T && at < a.H;
        xr[n] = gr[n] = u32x4_t{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < 8; ++i) r[n][i] = 0.0f;
        if (!in[n]) continue;
        if (a.u) {
            if (a.u_f32) {
                const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(a.u) + t * a.ldu + at);
                const float4 p0 = p[0], p1 = p[1];
                r[n][0] = p0.x, r[n][1] = p0.y, r[n][2] = p0.z, r[n][3] = p0.w;
                r[n][4] = p1.x, r[n][5] = p1.y, r[n][6] = p1.z, r[n][7] = p1.w;
            } else {
                unpack8(*reinterpret_cast<const u32x4_t *>(static_cast<const uint16_t *>(a.u) + t * a.ldu + at), r[n]);
            }
        }
        if (a.gate) gr[n] = *reinterpret_cast<const u32x4_t *>(a.gate + t * a.ldg + at);
        if (a.x) xr[n] = *reinterpret_cast<const u32x4_t *>(a.x + t * a.ldx + at);
    }
    float inv = 1.0f;
    if (a.post) {
        float sum = 0.0f;
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int i = 0; i < 8; ++i) sum = fmaf(r[n][i], r[n][i], sum);
        inv = 1.0f / sqrtf(row_sum<LANES>(sum, part[0]) * inv_h + a.eps);
    }
    float sum = 0.0f;
#pragma unroll
    for (int n = 0; n < N; ++n) {
        const int at = 8 * (n * LANES + lane);
        float x[8];
        unpack8(xr[n], x);
        if (in[n] && a.u) {
            if (a.post)
#pragma unroll
                for (int i = 0; i < 8; ++i) r[n][i] *= inv * a.post[at + i];
            if (a.gate) {
                float g[8];
                unpack8(gr[n], g);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    if (a.act == MOE_Q4_ACT_SILU)
                        g[i] = g[i] / (1.0f + expf(-g[i]));
                    else if (a.act == MOE_Q4_ACT_SIGMOID)
                        g[i] = 1.0f / (1.0f + expf(-g[i]));
                    r[n][i] *= g[i];
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = fmaf(a.scale, r[n][i], x[i]);
        }
        const u32x4_t w = pack8(x);
        if (in[n] && a.x_out) *reinterpret_cast<u32x4_t *>(a.x_out + t * a.ldxo + at) = w;
        unpack8(w, r[n]);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum = fmaf(r[n][i], r[n][i], sum);
    }
    if (!a.pre) return;
    inv = 1.0f / sqrtf(row_sum<LANES>(sum, part[1]) * inv_h + a.eps);
#pragma unroll
    for (int n = 0; n < N; ++n) {
        if (!in[n]) continue;
        const int at = 8 * (n * LANES + lane);
#pragma unroll
        for (int i = 0; i < 8; ++i) r[n][i] *= inv * a.pre[at + i];
        *reinterpret_cast<u32x4_t *>(a.y + t * a.ldy + at) = pack8(r[n]);
    }
}

template <int LANES, int N>
hipError_t launch(const AddNormArgs &a, hipStream_t s) {
    constexpr int THREADS = LANES < 256 ? 256 : LANES, ROWS = THREADS / LANES;
    add_norm_kernel<LANES, N><<<dim3((unsigned)((a.T + ROWS - 1) / ROWS)), THREADS, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_add_norm(const AddNormArgs &a, hipStream_t s) {
    const int chunks = a.H / 8;
    // Eight values a lane and as many lanes as that takes, up to rows of 4096: 8192
    // rows of 4096 take 71 us so, 79 with 16 values a lane, 124 with a wave to a row
    // (what counts is rows in flight).  Longer rows, by what a workgroup holds.
    if (chunks <= 8) return launch<8, 1>(a, s);
    if (chunks <= 16) return launch<16, 1>(a, s);
    if (chunks <= 32) return launch<32, 1>(a, s);
    if (chunks <= 64) return launch<64, 1>(a, s);
    if (chunks <= 256) return launch<256, 1>(a, s);
    if (chunks <= 512) return launch<512, 1>(a, s);
    if (chunks <= 1024) return launch<256, 4>(a, s);
    if (chunks <= 2048) return launch<512, 4>(a, s);
    if (chunks <= 4096) return launch<1024, 4>(a, s);
    return launch<1024, 8>(a, s);
}

}  // namespace moeq4
