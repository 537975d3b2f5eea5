// Gated delta rule, token by token.
//
// With a = exp(g), per value head:  S' = a S,  u = beta (v - S'^T k),
// S = S' + k u^T,  o = scale S^T q.  Since S^T q = a S_old^T q + (k.q) u, the
// two products with the old state, S_old^T k and S_old^T q, are one pass over
// it and one reduction per token.
//
// The columns of the state (v_dim) do not mix, so a workgroup takes 32 of
// them of one (sequence, head): 8 threads of 4 columns side by side, k_dim
// spread over the rest, the state in registers from the first token to the
// last.  Bound by the state's bytes (8 per element): each row's 32 columns
// are one 128-byte line.
#include "backbone.h"

namespace moeq4 {

namespace {

constexpr int DNB = 32;  // columns per workgroup

template <int DK, int DV>
__global__ __launch_bounds__(256) void delta_decode_kernel(DeltaArgs a) {
    constexpr int R = DK / 32;  // rows per thread
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int blk = blockIdx.x % (DV / DNB);
    const int h = (blockIdx.x / (DV / DNB)) % a.hv;
    const int b = blockIdx.x / (DV / DNB) / a.hv;
    const int hk = h / (a.hv / a.hk);
    const int cg = tid & 7, rg = tid >> 3;  // columns 4 cg.., rows R rg..
    int t0 = a.seq_start[b], t1 = a.seq_start[b + 1];
    t0 = t0 < 0 ? 0 : (t0 > a.T ? (int)a.T : t0);
    t1 = t1 < t0 ? t0 : (t1 > a.T ? (int)a.T : t1);
    const int slot = a.state_idx ? a.state_idx[b] : b;
    const bool kept = slot >= 0 && slot < a.n_states;
    const int64_t soff = (((int64_t)(kept ? slot : 0) * a.hv + h) * DK + R * rg) * DV + blk * DNB + 4 * cg;
    float4 S[R];
#pragma unroll
    for (int i = 0; i < R; ++i)
        S[i] = kept && a.s_in ? *reinterpret_cast<const float4 *>(a.s_in + soff + i * DV)
                              : make_float4(0.f, 0.f, 0.f, 0.f);

    __shared__ float s_red[2][4][8][8];
    for (int t = t0; t < t1; ++t) {
        // k and q of this thread's rows; sums over the head in every wave
        float kr[R], qr[R];
        const uint16_t *kp = a.k + (int64_t)t * a.ldk + hk * DK, *qp = a.q + (int64_t)t * a.ldq + hk * DK;
#pragma unroll
        for (int i = 0; i < R; ++i) {
            kr[i] = bf16_to_f32(kp[R * rg + i]);
            qr[i] = bf16_to_f32(qp[R * rg + i]);
        }
        float kk = 0.f, qq = 0.f, kq = 0.f;
#pragma unroll
        for (int i = 0; i < DK / 64; ++i) {
            const float kv = bf16_to_f32(kp[lane + 64 * i]), qv = bf16_to_f32(qp[lane + 64 * i]);
            kk += kv * kv;
            qq += qv * qv;
            kq += kv * qv;
        }
        kk = seg_sum<64>(kk);
        qq = seg_sum<64>(qq);
        kq = seg_sum<64>(kq);
        const float rk = a.norm ? 1.0f / sqrtf(kk + 1e-6f) : 1.0f;
        const float rq = (a.norm ? 1.0f / sqrtf(qq + 1e-6f) : 1.0f) * a.scale;
        const float decay = expf(a.g[(int64_t)t * a.hv + h]), beta = a.beta[(int64_t)t * a.hv + h];
        const uint2 vv =
            *reinterpret_cast<const uint2 *>(a.v + (int64_t)t * a.ldv + (int64_t)h * DV + blk * DNB + 4 * cg);
        const float v[4] = {bf16_to_f32(vv.x & 0xffffu), bf16_to_f32(vv.x >> 16), bf16_to_f32(vv.y & 0xffffu),
                            bf16_to_f32(vv.y >> 16)};
        // partial S^T k (0..3) and S^T q (4..7) of the thread's columns
        float p[8] = {};
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const float s[4] = {S[i].x, S[i].y, S[i].z, S[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                p[j] += s[j] * kr[i];
                p[4 + j] += s[j] * qr[i];
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            p[j] += __shfl_xor(p[j], 8);
            p[j] += __shfl_xor(p[j], 16);
            p[j] += __shfl_xor(p[j], 32);
        }
        const int buf = t & 1;
        if (lane < 8) {
#pragma unroll
            for (int j = 0; j < 8; ++j) s_red[buf][wave][cg][j] = p[j];
        }
        __syncthreads();
        float u[4], o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float sk = s_red[buf][0][cg][j] + s_red[buf][1][cg][j] + s_red[buf][2][cg][j] + s_red[buf][3][cg][j];
            const float sq = s_red[buf][0][cg][4 + j] + s_red[buf][1][cg][4 + j] + s_red[buf][2][cg][4 + j] +
                             s_red[buf][3][cg][4 + j];
            u[j] = beta * (v[j] - decay * rk * sk);
            o[j] = rq * (decay * sq + kq * rk * u[j]);
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const float kn = kr[i] * rk;
            S[i].x = decay * S[i].x + kn * u[0];
            S[i].y = decay * S[i].y + kn * u[1];
            S[i].z = decay * S[i].z + kn * u[2];
            S[i].w = decay * S[i].w + kn * u[3];
        }
        if (tid < 8) {
            uint2 w;
            w.x = f32_to_bf16_rne(o[0]) | ((uint32_t)f32_to_bf16_rne(o[1]) << 16);
            w.y = f32_to_bf16_rne(o[2]) | ((uint32_t)f32_to_bf16_rne(o[3]) << 16);
            *reinterpret_cast<uint2 *>(a.o + (int64_t)t * a.ldo + (int64_t)h * DV + blk * DNB + 4 * cg) = w;
        }
    }
    if (kept && a.s_out && !(t1 == t0 && a.s_in == a.s_out)) {
#pragma unroll
        for (int i = 0; i < R; ++i) *reinterpret_cast<float4 *>(a.s_out + soff + i * DV) = S[i];
    }
}

template <int DK, int DV>
hipError_t launch_decode(const DeltaArgs &a, hipStream_t s) {
    const int64_t blocks = (int64_t)a.n_seq * a.hv * (DV / DNB);
    if (blocks >= (int64_t)1 << 31) return hipErrorInvalidValue;
    hipLaunchKernelGGL((delta_decode_kernel<DK, DV>), dim3((unsigned)blocks), dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_decode(const DeltaArgs &a, hipStream_t s) {
    if (a.dk == 64) return a.dv == 64 ? launch_decode<64, 64>(a, s) : launch_decode<64, 128>(a, s);
    return a.dv == 64 ? launch_decode<128, 64>(a, s) : launch_decode<128, 128>(a, s);
}

}  // namespace moeq4
