// Gated delta rule: token by token, and in chunks of 64 tokens (below).
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
// are one 128-byte line.  Measured: 64 sequences of one token, 32 heads of
// 128 x 128 (268 MB of states): 43 us, 6.2 TB/s (a part of the states comes
// from the last-level cache; a large copy moves 5.1 TB/s); one sequence: 5.0 us,
// the latency of one load, reduction and store.
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
    hipLaunchKernelGGL((delta_decode_kernel<DK, DV>), dim3((unsigned)blocks), dim3(256), 0, s, a);
    return hipGetLastError();
}

// ------------------------------------------------------- chunks of 64 tokens
//
// Within a chunk, with G the running sum of g, the updates u_i solve
//   u_i + sum_{j<i} A_ij u_j = beta_i (v_i - e^{G_i} S0^T k_i),
//   A_ij = beta_i e^{G_i - G_j} k_i.k_j,
// so U = T' (V - diag(e^G) K S0) with T' = (I + A)^-1 diag(beta), and
//   O  = scale (diag(e^G) Q S0 + P U),  P_ij = e^{G_i - G_j} q_i.k_j (j <= i),
//   S1 = e^{G_63} S0 + sum_j e^{G_63 - G_j} k_j u_j^T.
// T' and P do not depend on the state: delta_prep_kernel computes them for
// every chunk and head at once; delta_scan_kernel walks the chunks of a
// sequence with what is left, products of the matrix cores.
//
// Operands are f16: k, q rows, T', P rows and the columns of S, X, U are
// scaled by a power of two each, taken off again in fp32 (so f16's range
// limits none of them).  All but k and q, whose 8 bits fit, have a second f16
// with the remainder (22 bits; the product of two remainders is left out).
// With one f16 the error of o was 2^-13 of the state, 1.1e-3 of o's norm in bf16
// roundings that fell to the other side.  Sums are fp32.  G is
// summed in double: e^{G_i - G_j} of neighbours is then right behind a strong
// decay.
//
// The 16x16x32 product reads its right operand 8 rows per lane and leaves its
// result 4 rows per lane (row 4 g + e, column lane % 16, g = lane / 16).  The
// order of the inner index is free, so everything that meets such a result is
// stored in the order "4 g + e of one tile, then of the next": a result goes
// into the next product straight from its registers.
typedef __attribute__((__vector_size__(4 * sizeof(float)))) float f32x4_t;
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));

constexpr int CH = 64;
// Per (chunk, head): 24 operands of 1 KB (T' first f16: 6, remainder: 6, P the
// same; row tile 0: inner tiles 0-1; 1: 0-1; 2: 0-1, 2-3; 3: 0-1, 2-3), then
// vectors of 64 floats, then e^{G_63}.
constexpr int OPS = 24;
constexpr int UNIT = 26624, UNIT_VEC = OPS * 1024;
enum { V_A, V_B, V_C, V_T, V_P, V_SK, V_SQ, V_COUNT };
constexpr int UNIT_GAMMA = UNIT_VEC + V_COUNT * CH * 4;
__device__ __forceinline__ constexpr int frag_index(int it, int ks) { return it < 2 ? it : 2 * it - 2 + ks; }

__device__ __forceinline__ f32x4_t mfma_f16(u32x4_t a, u32x4_t b, f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c, 0,
                                                  0, 0);
}
__device__ __forceinline__ uint32_t f16_pair(float a, float b) {
    return __builtin_bit_cast(uint32_t, f16x2_t{(_Float16)a, (_Float16)b});
}
// a pair's remainders after rounding to f16, as f16
__device__ __forceinline__ uint32_t f16_rest(float a, float b, uint32_t first) {
    const f16x2_t h = __builtin_bit_cast(f16x2_t, first);
    return f16_pair(a - (float)h[0], b - (float)h[1]);
}
// The power of two 2^s that puts values whose largest magnitude is m in
// [2^14, 2^15) (as row_scale, over almost all of fp32's range: m from 2^-112).
__device__ __forceinline__ RowScale unit_scale(float m) {
    int be = (int)((__float_as_uint(m) >> 23) & 0xffu);
    be = be < 15 ? 15 : (be > 254 ? 254 : be);
    return RowScale{__uint_as_float((uint32_t)(268 - be) << 23), 141 - be};
}
// v sc as f16 and its remainder, half `which` of a right operand.
__device__ __forceinline__ void split(f32x4_t v, float sc, u32x4_t &first, u32x4_t &rest, int which) {
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
        const f16x2_t h = {(_Float16)(v[e] * sc), (_Float16)(v[e + 1] * sc)};
        const f16x2_t r = {(_Float16)fmaf(v[e], sc, -(float)h[0]), (_Float16)fmaf(v[e + 1], sc, -(float)h[1])};
        first[2 * which + e / 2] = __builtin_bit_cast(uint32_t, h);
        rest[2 * which + e / 2] = __builtin_bit_cast(uint32_t, r);
    }
}
// Largest over the four lane groups (lanes l, l ^ 16, l ^ 32, l ^ 48).
__device__ __forceinline__ float groups_max(float v) {
    typedef unsigned int u32x2_t __attribute__((ext_vector_type(2)));
    const uint32_t a = __float_as_uint(v);
    const u32x2_t p = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_permlane16_swap(a, a, false, false));
    const uint32_t b = __float_as_uint(fmaxf(__uint_as_float(p.x), __uint_as_float(p.y)));
    const u32x2_t q = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_permlane32_swap(b, b, false, false));
    return fmaxf(__uint_as_float(q.x), __uint_as_float(q.y));
}
__device__ __forceinline__ float max_abs(f32x4_t v, float m) {
    return fmaxf(fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3]))), m);
}

// Barrier that orders LDS only: loads of the next chunk and stores of outputs
// stay in flight over it.
__device__ __forceinline__ void lds_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

// Rows [t0, t1) of sequence b, inside [0, T].
__device__ __forceinline__ void seq_rows(const DeltaArgs &a, int b, int &t0, int &t1) {
    t0 = a.seq_start[b];
    t1 = a.seq_start[b + 1];
    t0 = t0 < 0 ? 0 : (t0 > a.T ? (int)a.T : t0);
    t1 = t1 < t0 ? t0 : (t1 > a.T ? (int)a.T : t1);
}
// First chunk number of a sequence: t0 / 64 + b leaves every sequence the
// numbers it needs (the next one's start is at least t1 / 64 + b + 1) without
// a prefix sum, and stays below T / 64 + n_seq.
__device__ __forceinline__ int first_chunk(int t0, int b) { return t0 / CH + b; }

// e^d (d rounded to fp32 only after the factor log2 e).
__device__ __forceinline__ float exp_diff(double d) {
    return __builtin_amdgcn_exp2f((float)(d * 1.4426950408889634));
}

// T', P and the row factors of one chunk and HP heads of one key head (k and q,
// and their products, are read and formed once for them).  Bound by the vector
// work: about 1500 instructions a wave and chunk with one head, 80% of the
// vector units' time.  Measured: 16384 tokens, 32 heads of 128 x 128 on 16 key
// heads: 108 to 114 us with two heads (2.0 TB/s of the 216 MB it writes).  Without P's
// remainders 103 us, and then 122 us with one head, 128 us with the tiles of A and
// P on one wave each (up to eight a wave), 171 us with a row's load waiting for the
// one before it.
template <int DK, int HP>
__global__ __launch_bounds__(256) void delta_prep_kernel(DeltaArgs a, uint8_t *__restrict__ ws) {
    constexpr int LDA = 68, PL = DK / 16;  // elements per lane of a row's 16 lanes
    constexpr int KQ = 2 * CH * DK * 2, TB = CH * LDA * 4;
    __shared__ __align__(16) uint8_t s_kq[KQ > TB ? KQ : TB];  // k, q as f16; then T
    __shared__ __align__(16) float s_A[CH * LDA];
    __shared__ __align__(16) float s_f[2][CH];   // k and q: sums of squares, then row factors
    __shared__ float s_sc[2][CH];  // and the scales
    __shared__ __align__(16) float s_beta[HP][CH];
    __shared__ double s_G[HP][CH];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, m = lane & 15, g4 = lane >> 4;
    const int h0 = blockIdx.x % (a.hv / HP) * HP, id = blockIdx.x / (a.hv / HP);
    // the sequence: the last whose first chunk is at most id
    int lo = 0, hi = a.n_seq - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        int t0, t1;
        seq_rows(a, mid, t0, t1);
        if (first_chunk(t0, mid) <= id) lo = mid;
        else hi = mid - 1;
    }
    int t0, t1;
    seq_rows(a, lo, t0, t1);
    const int c = id - first_chunk(t0, lo);
    if (c < 0 || t0 + (int64_t)c * CH >= t1) return;
    t0 += c * CH;
    const int len = t1 - t0 < CH ? t1 - t0 : CH;
    const int hk = h0 / (a.hv / a.hk);

    // rows of k and q to f16: every load first (rows behind the last read the
    // last one's and are cleared)
    constexpr int MASK = DK / 8 - 1;
    auto place = [](int which, int row, int chunk) { return ((which * CH + row) * (DK / 8) + (chunk ^ (row & MASK))) * 16; };
    const int64_t gate_at = (int64_t)(t0 + (lane < len ? lane : len - 1)) * a.hv + h0 + (w < HP ? w : 0);
    const float g_raw = a.g[gate_at], beta_raw = a.beta[gate_at];
    uint2 raw[2][4][PL / 4];
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        const uint8_t *base = reinterpret_cast<const uint8_t *>((which ? a.q + (int64_t)t0 * a.ldq : a.k + (int64_t)t0 * a.ldk) + hk * DK);
        const uint32_t ld = (uint32_t)(which ? a.ldq : a.ldk) * 2;
#pragma unroll
        for (int r4 = 0; r4 < 4; ++r4) {
            const int row = 16 * w + 4 * r4 + g4;
            const uint32_t at = (uint32_t)(row < len ? row : len - 1) * ld + m * PL * 2;
#pragma unroll
            for (int e = 0; e < PL / 4; ++e) raw[which][r4][e] = *reinterpret_cast<const uint2 *>(base + (at + 8 * e));
        }
    }
    {
        const float gl = lane < len ? g_raw : 0.f;
        double G = gl < -1000.f ? -1000.0 : (double)gl;  // e^-1000 is 0 too, and -inf - -inf is not
        if (w < HP) {  // wave w: head h0 + w
#pragma unroll
            for (int o = 1; o < 64; o <<= 1) {
                const double up = __shfl_up(G, o);
                if (lane >= o) G += up;
            }
            s_G[w][lane] = G;
            s_beta[w][lane] = lane < len ? beta_raw : 0.f;
        }
    }
#pragma unroll
    for (int which = 0; which < 2; ++which) {
#pragma unroll
        for (int r4 = 0; r4 < 4; ++r4) {
            const int row = 16 * w + 4 * r4 + g4;
            const uint32_t keep = row < len ? ~0u : 0u;
            float x[PL];
#pragma unroll
            for (int e = 0; e < PL; e += 4) {
                const uint32_t dx = raw[which][r4][e / 4].x & keep, dy = raw[which][r4][e / 4].y & keep;
                x[e] = __uint_as_float(dx << 16);
                x[e + 1] = __uint_as_float(dx & 0xffff0000u);
                x[e + 2] = __uint_as_float(dy << 16);
                x[e + 3] = __uint_as_float(dy & 0xffff0000u);
            }
            float mx = 0.f, ss = 0.f;
#pragma unroll
            for (int e = 0; e < PL; ++e) {
                mx = fmaxf(mx, fabsf(x[e]));
                ss += x[e] * x[e];
            }
            mx = row16_max(mx);
            ss = seg_sum_dpp<16>(ss);
            const RowScale sc = unit_scale(mx);
#pragma unroll
            for (int e = 0; e < PL; e += 4) {
                uint2 d;
                d.x = f16_pair(x[e] * sc.sc, x[e + 1] * sc.sc);
                d.y = f16_pair(x[e + 2] * sc.sc, x[e + 3] * sc.sc);
                const int at = m * PL + e;
                *reinterpret_cast<uint2 *>(s_kq + place(which, row, at / 8) + at % 8 * 2) = d;
            }
            if (m == 0) {
                s_f[which][row] = ss;
                s_sc[which][row] = sc.sc;
            }
        }
    }
    __syncthreads();
    if (tid < 2 * CH) {
        // what takes a row's scale off and normalises it (1 / sc: a power of two)
        const int which = tid >> 6, row = lane;
        const float off = __uint_as_float((uint32_t)(254 - (__float_as_uint(s_sc[which][row]) >> 23)) << 23);
        s_f[which][row] = (a.norm ? off / sqrtf(s_f[which][row] + 1e-6f) : off) * (which ? a.scale : 1.0f);
    }
    __syncthreads();

    // k_j.k_i and k_j.q_i, row j = 16 jt + 4 g4 + e, column i; wave w takes the
    // columns 16 w.. of P and 16 (3 - w).. of A, so that each has five tiles
    const int i = 16 * w + m, wa = 3 - w, ia = 16 * wa + m;
    f32x4_t kk[4], kq[4];
    {
        u32x4_t bk[DK / 32], bq[DK / 32];
#pragma unroll
        for (int ks = 0; ks < DK / 32; ++ks) {
            bk[ks] = *reinterpret_cast<const u32x4_t *>(s_kq + place(0, ia, 4 * ks + g4));
            bq[ks] = *reinterpret_cast<const u32x4_t *>(s_kq + place(1, i, 4 * ks + g4));
        }
#pragma unroll
        for (int jt = 0; jt < 4; ++jt) {
            kk[jt] = kq[jt] = f32x4_t{0.f, 0.f, 0.f, 0.f};
            u32x4_t ak[DK / 32];
#pragma unroll
            for (int ks = 0; ks < DK / 32; ++ks)
                ak[ks] = *reinterpret_cast<const u32x4_t *>(s_kq + place(0, 16 * jt + m, 4 * ks + g4));
#pragma unroll
            for (int ks = 0; ks < DK / 32; ++ks) {
                if (jt <= w) kq[jt] = mfma_f16(ak[ks], bq[ks], kq[jt]);
                if (jt <= wa) kk[jt] = mfma_f16(ak[ks], bk[ks], kk[jt]);
            }
            const f32x4_t f = *reinterpret_cast<const f32x4_t *>(&s_f[0][16 * jt + 4 * g4]);
            kq[jt] *= f * s_f[1][i];
            kk[jt] *= f * s_f[0][ia];
        }
    }
#pragma unroll 1
    for (int hh = 0; hh < HP; ++hh) {
        uint8_t *unit = ws + ((int64_t)id * a.hv + h0 + hh) * UNIT;
        float *vec = reinterpret_cast<float *>(unit + UNIT_VEC);
        const double *sG = s_G[hh];
        f32x4_t P[4];
        {
            const double Gi = sG[i], Ga = sG[ia];
            const float ba = s_beta[hh][ia];
#pragma unroll
            for (int jt = 0; jt < 4; ++jt) {
                P[jt] = f32x4_t{0.f, 0.f, 0.f, 0.f};
                if (jt <= w) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int j = 16 * jt + 4 * g4 + e;
                        P[jt][e] = j <= i ? kq[jt][e] * exp_diff(Gi - sG[j]) : 0.f;
                    }
                }
                if (jt <= wa) {
                    f32x4_t A;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int j = 16 * jt + 4 * g4 + e;
                        A[e] = j < ia ? kk[jt][e] * (ba * exp_diff(Ga - sG[j])) : 0.f;
                    }
                    *reinterpret_cast<f32x4_t *>(&s_A[ia * LDA + 16 * jt + 4 * g4]) = A;
                }
            }
        }
        {
            float mx = 0.f;
#pragma unroll
            for (int jt = 0; jt < 4; ++jt) mx = max_abs(P[jt], mx);
            const RowScale sc = unit_scale(groups_max(mx));
            if (g4 == 0) vec[V_P * CH + i] = exp2i(-sc.s);
#pragma unroll
            for (int ks = 0; ks < 2; ++ks)
                if (ks <= w / 2) {
                    u32x4_t f, r;
                    split(P[2 * ks], sc.sc, f, r, 0);
                    split(P[2 * ks + 1], sc.sc, f, r, 1);
                    const int at = w < 2 ? w : 2 * w - 2 + ks;
                    *reinterpret_cast<u32x4_t *>(unit + (12 + at) * 1024 + lane * 16) = f;
                    *reinterpret_cast<u32x4_t *>(unit + (18 + at) * 1024 + lane * 16) = r;
                }
        }
        __syncthreads();  // s_A is whole, k and q are used up

        // T = (I + A)^-1 by 16 x 16 tiles: the diagonal ones by substitution (a
        // lane a column), then T_ij = -T_ii sum_k A_ik T_kj, one distance from the
        // diagonal after another
        float *T = reinterpret_cast<float *>(s_kq);
        {
            float col[16];
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                float t = r == m ? 1.f : 0.f;
#pragma unroll
                for (int q = 0; q < (r + 3) / 4; ++q) {
                    const f32x4_t A = *reinterpret_cast<const f32x4_t *>(&s_A[(16 * w + r) * LDA + 16 * w + 4 * q]);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (4 * q + e < r) t = fmaf(-A[e], col[4 * q + e], t);
                }
                col[r] = t;
            }
            if (g4 == 0) {
#pragma unroll
                for (int r = 0; r < 16; ++r) T[(16 * w + r) * LDA + 16 * w + m] = col[r];
            }
        }
        __syncthreads();
#pragma unroll
        for (int d = 1; d < 4; ++d) {
            if (w >= d) {
                const int j = w - d;
                f32x4_t M = {0.f, 0.f, 0.f, 0.f}, R = {0.f, 0.f, 0.f, 0.f};
                for (int k = j; k < w; ++k) {
                    const f32x4_t A = *reinterpret_cast<const f32x4_t *>(&s_A[i * LDA + 16 * k + 4 * g4]);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        M = __builtin_amdgcn_mfma_f32_16x16x4f32(A[e], T[(16 * k + 4 * g4 + e) * LDA + 16 * j + m], M, 0, 0, 0);
                }
                const f32x4_t D = *reinterpret_cast<const f32x4_t *>(&T[i * LDA + 16 * w + 4 * g4]);
#pragma unroll
                for (int e = 0; e < 4; ++e) R = __builtin_amdgcn_mfma_f32_16x16x4f32(-D[e], M[e], R, 0, 0, 0);
#pragma unroll
                for (int e = 0; e < 4; ++e) T[(16 * w + 4 * g4 + e) * LDA + 16 * j + m] = R[e];
            }
            __syncthreads();
        }
        {
            f32x4_t t[4];
            float mx = 0.f;
#pragma unroll
            for (int jt = 0; jt < 4; ++jt) {
                t[jt] = f32x4_t{0.f, 0.f, 0.f, 0.f};
                if (jt <= w) {
                    const f32x4_t x = *reinterpret_cast<const f32x4_t *>(&T[i * LDA + 16 * jt + 4 * g4]);
                    const f32x4_t be = *reinterpret_cast<const f32x4_t *>(&s_beta[hh][16 * jt + 4 * g4]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) t[jt][e] = x[e] * be[e];
                }
                mx = max_abs(t[jt], mx);
            }
            const RowScale sc = unit_scale(groups_max(mx));
            if (g4 == 0) vec[V_T * CH + i] = exp2i(-sc.s);
#pragma unroll
            for (int ks = 0; ks < 2; ++ks)
                if (ks <= w / 2) {
                    u32x4_t f, r;
#pragma unroll
                    for (int q = 0; q < 2; ++q)
#pragma unroll
                        for (int e = 0; e < 4; e += 2) {
                            const float x = t[2 * ks + q][e] * sc.sc, y = t[2 * ks + q][e + 1] * sc.sc;
                            f[2 * q + e / 2] = f16_pair(x, y);
                            r[2 * q + e / 2] = f16_rest(x, y, f[2 * q + e / 2]);
                        }
                    const int at = w < 2 ? w : 2 * w - 2 + ks;
                    *reinterpret_cast<u32x4_t *>(unit + at * 1024 + lane * 16) = f;
                    *reinterpret_cast<u32x4_t *>(unit + (6 + at) * 1024 + lane * 16) = r;
                }
        }
        if (tid < CH) {
            const double G = sG[tid], last = sG[CH - 1];
            const float f = s_f[0][tid], eg = exp_diff(G);
            vec[V_A * CH + tid] = eg * f;
            vec[V_B * CH + tid] = eg * s_f[1][tid];
            vec[V_C * CH + tid] = exp_diff(last - G) * f;
            vec[V_SK * CH + tid] = s_sc[0][tid];
            vec[V_SQ * CH + tid] = s_sc[1][tid];
            if (tid == 0) *reinterpret_cast<float *>(unit + UNIT_GAMMA) = exp_diff(last);
        }
        if (hh + 1 < HP) __syncthreads();  // T and s_A are used
    }
}

// The chunks of one sequence and head, one after another.  Waves 0-3 hold the
// state in registers from the first chunk to the last, waves 4-7 bring the next
// chunk to LDS meanwhile: k and q as f16 rows, k transposed, and the operands
// of delta_prep_kernel.
//   SPLIT false: 64 columns per workgroup, each state wave has 16 of them and
//     works alone.  A chunk of a 128 x 128 head takes 4.6 us: about 600 vector
//     instructions on each of the 8 waves (half of the vector units' time) and
//     the products (a fifth of the matrix units').
//   SPLIT true: 16 columns per workgroup, the state waves share their rows (of
//     the state and of the chunk) and hand each other S, X and U through LDS:
//     a shorter chain (3.2 us a chunk, a third of it the last stage), more LDS
//     traffic per column.  For few columns in all.
// Measured: one prompt of 8192 tokens, 32 heads of 128 x 128: 410 us with SPLIT;
// 8 prompts of 2048: 296 to 302 us without.  (With one f16 for what only o sees 385 and
// 284 us, and then 540 us for the first without SPLIT, 440 us with one state wave
// of 512 registers and three others.)
template <int DK, bool SPLIT>
__global__ __launch_bounds__(512) void delta_scan_kernel(DeltaArgs a, const uint8_t *__restrict__ ws) {
    constexpr int COLS = SPLIT ? 16 : 64;
    constexpr int NT = DK / 16, NQ = DK / 32;
    constexpr int ROWS = CH * DK * 2;                              // bytes of k, of q, of k transposed
    constexpr int FR = 3 * ROWS, VEC = FR + OPS * 1024, BUF = VEC + V_COUNT * CH * 4 + 16;
    __shared__ __align__(16) uint8_t s_buf[2][BUF];
    // SPLIT: S as right operands (f16 and remainders; their place takes the U
    // tiles, which are written behind the barrier after S's last read and read
    // before the one that the next S is written behind), X tiles, largest
    // magnitude of each column of S in each wave's rows
    __shared__ __align__(16) uint8_t s_S[SPLIT ? 2 * NQ * 1024 : 16];
    __shared__ f32x4_t s_X[SPLIT ? 4 * 64 : 1];
    f32x4_t *const s_U = reinterpret_cast<f32x4_t *>(s_S);
    __shared__ float s_max[SPLIT ? 64 : 1];
    const int tid = threadIdx.x, lane = tid & 63, m = lane & 15, g4 = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    // the workgroups that read the same k and q on one XCD (they are dealt to
    // the 8 XCDs in turn)
    const int rep = a.hv / a.hk, blocks = a.dv / COLS, per = rep * blocks;
    const int group = blockIdx.x / (8 * per) * 8 + blockIdx.x % 8, in = blockIdx.x / 8 % per;
    if (group >= a.n_seq * a.hk) return;
    const int b = group / a.hk, hk = group % a.hk, h = hk * rep + in / blocks;
    const int col0 = in % blocks * COLS;
    int t0, t1;
    seq_rows(a, b, t0, t1);
    const int chunks = (t1 - t0 + CH - 1) / CH;
    const uint8_t *units = ws + ((int64_t)first_chunk(t0, b) * a.hv + h) * UNIT;
    const int64_t unit_step = (int64_t)a.hv * UNIT;
    constexpr int MASK = DK / 8 - 1;
    // chunk `at` (8 f16) of row `row` of k (which 0) or q (1)
    auto row_at = [](int which, int row, int at) { return which * ROWS + (row * (DK / 8) + (at ^ (row & MASK))) * 16; };
    // and of row d of k transposed
    auto col_at = [](int d, int at) { return 2 * ROWS + (d * (CH / 8) + (at ^ ((d ^ d >> 3) & 7))) * 16; };

    if (wave >= 4) {
        // ---- bringing chunks to LDS.  Items of a thread: KI pairs of rows x 8
        // of k, QN rows x 8 of q, FN 16-byte pieces of operands, VN floats
        const int p = tid - 256;
        constexpr int KI = 32 * (DK / 8) / 256, QN = CH * (DK / 8) / 256, FN = OPS * 64 / 256, VN = 2;
        u32x4_t k_reg[KI][2], q_reg[QN], f_reg[FN];
        float v_reg[VN], k_sc[KI][2], q_sc[QN];
        // byte offsets from the chunk's first row (64 rows of at most 2^22
        // elements)
        uint32_t k_off[KI], q_off[QN];
#pragma unroll
        for (int it = 0; it < KI; ++it) {
            const int x = it * 256 + p;
            k_off[it] = (uint32_t)(2 * (x / (DK / 8))) * (uint32_t)a.ldk * 2 + x % (DK / 8) * 16;
        }
#pragma unroll
        for (int it = 0; it < QN; ++it) {
            const int x = it * 256 + p;
            q_off[it] = (uint32_t)(x / (DK / 8)) * (uint32_t)a.ldq * 2 + x % (DK / 8) * 16;
        }
        const u32x4_t zero = {0, 0, 0, 0};
        auto rows_of = [&](int c) { return t1 - t0 - c * CH < CH ? t1 - t0 - c * CH : CH; };
        auto load_k = [&](int c, int it) {
            const int len = rows_of(c);
            const uint8_t *unit = units + c * unit_step;
            const uint8_t *kb = reinterpret_cast<const uint8_t *>(a.k + (t0 + (int64_t)c * CH) * a.ldk + hk * DK);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = 2 * ((it * 256 + p) / (DK / 8)) + e;
                k_sc[it][e] = *reinterpret_cast<const float *>(unit + (uint32_t)(UNIT_VEC + (V_SK * CH + row) * 4));
                k_reg[it][e] = len == CH || row < len
                                   ? *reinterpret_cast<const u32x4_t *>(kb + (k_off[it] + e * (uint32_t)a.ldk * 2))
                                   : zero;
            }
        };
        auto load_q = [&](int c) {
            const int len = rows_of(c);
            const uint8_t *unit = units + c * unit_step;
            const uint8_t *qb = reinterpret_cast<const uint8_t *>(a.q + (t0 + (int64_t)c * CH) * a.ldq + hk * DK);
#pragma unroll
            for (int it = 0; it < QN; ++it) {
                const int row = (it * 256 + p) / (DK / 8);
                q_sc[it] = *reinterpret_cast<const float *>(unit + (uint32_t)(UNIT_VEC + (V_SQ * CH + row) * 4));
                q_reg[it] = len == CH || row < len ? *reinterpret_cast<const u32x4_t *>(qb + q_off[it]) : zero;
            }
        };
        auto load_f = [&](int c) {
            const uint8_t *unit = units + c * unit_step;
#pragma unroll
            for (int it = 0; it < FN; ++it)
                f_reg[it] = *reinterpret_cast<const u32x4_t *>(unit + (uint32_t)((it * 256 + p) * 16));
#pragma unroll
            for (int it = 0; it < VN; ++it)
                if (it * 256 + p <= V_COUNT * CH)
                    v_reg[it] = *reinterpret_cast<const float *>(unit + (uint32_t)(UNIT_VEC + (it * 256 + p) * 4));
        };
        // 8 bf16 times f as f16
        auto halves = [](u32x4_t x, float f) {
            u32x4_t r;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                r[e] = f16_pair(__uint_as_float(x[e] << 16) * f, __uint_as_float(x[e] & 0xffff0000u) * f);
            return r;
        };
        // inner order of the products: elements 0-3 of an 8-chunk u of a block
        // of 32 to chunk 2 (u % 2), 4-7 to the next, half u / 2
        auto store_row = [&](uint8_t *buf, int which, int row, int at, u32x4_t x) {
            const int blk = at / 4, u = at % 4;
            uint8_t *d = buf + (u / 2) * 8;
            *reinterpret_cast<uint2 *>(d + row_at(which, row, 4 * blk + 2 * (u & 1))) = make_uint2(x[0], x[1]);
            *reinterpret_cast<uint2 *>(d + row_at(which, row, 4 * blk + 2 * (u & 1) + 1)) = make_uint2(x[2], x[3]);
        };
        auto store_k = [&](int c, int it) {
            uint8_t *buf = s_buf[c & 1];
            const int x = it * 256 + p, pair = x / (DK / 8), at = x % (DK / 8);
            const u32x4_t r0 = halves(k_reg[it][0], k_sc[it][0]), r1 = halves(k_reg[it][1], k_sc[it][1]);
            store_row(buf, 0, 2 * pair, at, r0);
            store_row(buf, 0, 2 * pair + 1, at, r1);
            const int o = 2 * pair % 32, slot = 4 * (pair / 16) + o % 16 / 4, in8 = (o / 16) * 4 + o % 4;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t two = __builtin_amdgcn_perm(r1[e / 2], r0[e / 2], e & 1 ? 0x07060302u : 0x05040100u);
                *reinterpret_cast<uint32_t *>(buf + col_at(8 * at + e, slot) + in8 * 2) = two;
            }
        };
        auto store_q = [&](int c) {
            uint8_t *buf = s_buf[c & 1];
#pragma unroll
            for (int it = 0; it < QN; ++it) {
                const int x = it * 256 + p;
                store_row(buf, 1, x / (DK / 8), x % (DK / 8), halves(q_reg[it], q_sc[it]));
            }
        };
        auto store_f = [&](int c) {
            uint8_t *buf = s_buf[c & 1];
#pragma unroll
            for (int it = 0; it < FN; ++it)
                *reinterpret_cast<u32x4_t *>(buf + FR + (it * 256 + p) * 16) = f_reg[it];
#pragma unroll
            for (int it = 0; it < VN; ++it)
                if (it * 256 + p <= V_COUNT * CH) *reinterpret_cast<float *>(buf + VEC + (it * 256 + p) * 4) = v_reg[it];
        };
        // chunk c to LDS, and the loads of the one after it, in the four parts
        // between the state waves' barriers (one part when they have one)
        auto part = [&](int c, int i) {
            if (c >= chunks) return;
            const bool more = c + 1 < chunks;
            if (i < KI) {
                store_k(c, i);
                if (more) load_k(c + 1, i);
            }
            if (i == 2) {
                store_q(c);
                if (more) load_q(c + 1);
            }
            if (i == 3) {
                store_f(c);
                if (more) load_f(c + 1);
            }
        };
        if (chunks > 0) {
#pragma unroll
            for (int it = 0; it < KI; ++it) load_k(0, it);
            load_q(0);
            load_f(0);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) part(0, i);
        lds_barrier();
        for (int c = 0; c < chunks; ++c) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                part(c + 1, i);
                if (SPLIT || i == 3) lds_barrier();
            }
        }
        return;
    }

    // ---- the state's waves
    const int slot = a.state_idx ? a.state_idx[b] : b;
    const bool kept = slot >= 0 && slot < a.n_states;
    const f32x4_t zero4 = {0.f, 0.f, 0.f, 0.f};
    if constexpr (SPLIT) {
        constexpr int NTW = NT / 4;  // row tiles of the state per wave
        const int w = wave, col = col0 + m;
        const int64_t soff = ((int64_t)(kept ? slot : 0) * a.hv + h) * DK * a.dv + col;
        f32x4_t S[NTW];
        auto publish_max = [&] {
            float mx = 0.f;
#pragma unroll
            for (int i = 0; i < NTW; ++i) mx = max_abs(S[i], mx);
            mx = groups_max(mx);
            if (g4 == 0) s_max[16 * w + m] = mx;
        };
#pragma unroll
        for (int i = 0; i < NTW; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                S[i][e] = kept && a.s_in ? a.s_in[soff + (int64_t)(16 * (NTW * w + i) + 4 * g4 + e) * a.dv] : 0.f;
        publish_max();
        const int64_t head_col = (int64_t)h * a.dv + col;
        uint16_t v_next[4];
        auto load_v = [&](int c) {
            const int64_t r0 = t0 + (int64_t)c * CH;
            const int len = t1 - r0 < CH ? (int)(t1 - r0) : CH;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int row = 16 * w + 4 * g4 + e;
                v_next[e] = a.v[(r0 + (row < len ? row : len - 1)) * a.ldv + head_col];
            }
        };
        if (chunks > 0) load_v(0);
        const int last_x = w / 2;  // inner blocks of 32 tokens up to this wave's own
        lds_barrier();
        for (int c = 0; c < chunks; ++c) {
            const uint8_t *buf = s_buf[c & 1];
            auto frag = [&](int at) { return *reinterpret_cast<const u32x4_t *>(buf + at); };
            auto vec4 = [&](int which, int t) {
                return *reinterpret_cast<const f32x4_t *>(buf + VEC + (which * CH + 16 * t + 4 * g4) * 4);
            };
            const int op0 = FR + (w < 2 ? w : 2 * w - 2) * 1024 + lane * 16;
            // S as right operand, each wave its rows; and what this wave needs
            // of the chunk
            float mx = s_max[m];
#pragma unroll
            for (int i = 1; i < 4; ++i) mx = fmaxf(mx, s_max[16 * i + m]);
            u32x4_t fk[NQ], fq[NQ];
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
                fk[q] = frag(row_at(0, 16 * w + m, 4 * q + g4));
                fq[q] = frag(row_at(1, 16 * w + m, 4 * q + g4));
            }
            const f32x4_t fa = vec4(V_A, w), ft = vec4(V_T, w), fb = vec4(V_B, w), fp = vec4(V_P, w);
            const float gamma = *reinterpret_cast<const float *>(buf + VEC + V_COUNT * CH * 4);
            const RowScale ss = unit_scale(mx);
            const float s_off = exp2i(-ss.s);
#pragma unroll
            for (int i = 0; i < NTW; ++i) {
                const int t = NTW * w + i;
                u32x4_t f, r;
                split(S[i], ss.sc, f, r, 0);
                uint8_t *d = s_S + (t / 2) * 1024 + lane * 16 + (t & 1) * 8;
                *reinterpret_cast<uint2 *>(d) = make_uint2(f[0], f[1]);
                *reinterpret_cast<uint2 *>(d + NQ * 1024) = make_uint2(r[0], r[1]);
            }
            float v[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = bf16_to_f32(v_next[e]);
            load_v(c + 1 < chunks ? c + 1 : c);
            lds_barrier();
            // K S and Q S of the wave's tokens, X = V - diag(e^G) K S
            u32x4_t sh[NQ], sl[NQ];
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
                sh[q] = *reinterpret_cast<const u32x4_t *>(s_S + q * 1024 + lane * 16);
                sl[q] = *reinterpret_cast<const u32x4_t *>(s_S + (NQ + q) * 1024 + lane * 16);
            }
            f32x4_t kh = zero4, kl = zero4, QS = zero4, ql = zero4;
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
                kh = mfma_f16(fk[q], sh[q], kh);
                kl = mfma_f16(fk[q], sl[q], kl);
                QS = mfma_f16(fq[q], sh[q], QS);
                ql = mfma_f16(fq[q], sl[q], ql);
            }
            QS += ql;
            f32x4_t X[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) X[0][e] = fmaf(-(kh[e] + kl[e]), fa[e] * s_off, v[e]);
            s_X[64 * w + lane] = X[0];
            u32x4_t th[2], tl[2], tp[2], tr[2];
#pragma unroll
            for (int x = 0; x < 2; ++x)
                if (x <= last_x) {
                    th[x] = frag(op0 + x * 1024);
                    tl[x] = frag(op0 + (6 + x) * 1024);
                    tp[x] = frag(op0 + (12 + x) * 1024);
                    tr[x] = frag(op0 + (18 + x) * 1024);
                }
            lds_barrier();
            // U = T' X of the wave's tokens
#pragma unroll
            for (int t = 0; t < 4; ++t)
                if (t / 2 <= last_x) X[t] = s_X[64 * t + lane];
            mx = 0.f;
#pragma unroll
            for (int t = 0; t < 4; ++t)
                if (t / 2 <= last_x) mx = max_abs(X[t], mx);
            const RowScale xs = unit_scale(groups_max(mx));
            const float x_off = exp2i(-xs.s);
            f32x4_t uh = zero4, ul = zero4, um = zero4;
#pragma unroll
            for (int x = 0; x < 2; ++x)
                if (x <= last_x) {
                    u32x4_t xh, xl;
                    split(X[2 * x], xs.sc, xh, xl, 0);
                    split(X[2 * x + 1], xs.sc, xh, xl, 1);
                    um = mfma_f16(tl[x], xh, um);
                    ul = mfma_f16(th[x], xl, ul);
                    uh = mfma_f16(th[x], xh, uh);
                }
            f32x4_t U[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) U[0][e] = (uh[e] + (ul[e] + um[e])) * (ft[e] * x_off);
            s_U[64 * w + lane] = U[0];
            u32x4_t kt[NTW][2];
#pragma unroll
            for (int i = 0; i < NTW; ++i)
#pragma unroll
                for (int x = 0; x < 2; ++x) kt[i][x] = frag(col_at(16 * (NTW * w + i) + m, 4 * x + g4));
            f32x4_t fc[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) fc[t] = vec4(V_C, t);
            lds_barrier();
            // S = e^{G_63} S + K^T diag(c) U, each wave its rows
            f32x4_t W[4];
            mx = 0.f;
            float mw = 0.f;
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                U[t] = s_U[64 * t + lane];
                W[t] = U[t] * fc[t];
                mw = max_abs(W[t], mw);
                if (t / 2 <= last_x) mx = max_abs(U[t], mx);
            }
            const RowScale wsc = unit_scale(groups_max(mw));
            const float w_off = exp2i(-wsc.s);
            f32x4_t dh[NTW], dl[NTW];
#pragma unroll
            for (int i = 0; i < NTW; ++i) dh[i] = dl[i] = zero4;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                u32x4_t wh, wl;
                split(W[2 * x], wsc.sc, wh, wl, 0);
                split(W[2 * x + 1], wsc.sc, wh, wl, 1);
#pragma unroll
                for (int i = 0; i < NTW; ++i) {
                    dh[i] = mfma_f16(kt[i][x], wh, dh[i]);
                    dl[i] = mfma_f16(kt[i][x], wl, dl[i]);
                }
            }
#pragma unroll
            for (int i = 0; i < NTW; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) S[i][e] = fmaf(dh[i][e] + dl[i][e], w_off, gamma * S[i][e]);
            publish_max();
            // O = diag(b) Q S + P U of the wave's tokens
            const RowScale us = unit_scale(groups_max(mx));
            const float u_off = exp2i(-us.s);
            f32x4_t o = zero4, ol = zero4, om = zero4;
#pragma unroll
            for (int x = 0; x < 2; ++x)
                if (x <= last_x) {
                    u32x4_t f, r;
                    split(U[2 * x], us.sc, f, r, 0);
                    split(U[2 * x + 1], us.sc, f, r, 1);
                    om = mfma_f16(tr[x], f, om);
                    ol = mfma_f16(tp[x], r, ol);
                    o = mfma_f16(tp[x], f, o);
                }
            o += ol + om;
            const int64_t r0 = t0 + (int64_t)c * CH;
            const int len = t1 - r0 < CH ? (int)(t1 - r0) : CH;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int row = 16 * w + 4 * g4 + e;
                const float z = fmaf(QS[e], fb[e] * s_off, o[e] * (fp[e] * u_off));
                if (row < len) *reinterpret_cast<__bf16 *>(a.o + (r0 + row) * a.ldo + head_col) = (__bf16)z;
            }
            lds_barrier();
        }
        if (kept && a.s_out && !(chunks == 0 && a.s_in == a.s_out)) {
#pragma unroll
            for (int i = 0; i < NTW; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) a.s_out[soff + (int64_t)(16 * (NTW * w + i) + 4 * g4 + e) * a.dv] = S[i][e];
        }
    } else {
        const int col = col0 + 16 * wave + m;
        const int64_t soff = ((int64_t)(kept ? slot : 0) * a.hv + h) * DK * a.dv + col;
        f32x4_t S[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                S[t][e] = kept && a.s_in ? a.s_in[soff + (int64_t)(16 * t + 4 * g4 + e) * a.dv] : 0.f;
        // rows 16 t + 4 g4 + e of v and o: a uniform base and the lane's offset
        uint16_t v_next[16];
        const uint32_t v_lane = ((uint32_t)(4 * g4) * (uint32_t)a.ldv + m) * 2;
        const uint32_t o_lane = ((uint32_t)(4 * g4) * (uint32_t)a.ldo + m) * 2;
        const int64_t head_col = (int64_t)h * a.dv + col0 + 16 * wave;
        auto load_v = [&](int c) {
            const int64_t r0 = t0 + (int64_t)c * CH;
            const int len = t1 - r0 < CH ? (int)(t1 - r0) : CH;
            const uint16_t *base = a.v + r0 * a.ldv + head_col;
            if (len == CH) {
#pragma unroll
                for (int x = 0; x < 16; ++x)
                    v_next[x] = *reinterpret_cast<const uint16_t *>(
                        reinterpret_cast<const uint8_t *>(base + (int64_t)(16 * (x / 4) + x % 4) * a.ldv) + v_lane);
            } else {
#pragma unroll
                for (int x = 0; x < 16; ++x) {
                    const int row = 16 * (x / 4) + 4 * g4 + x % 4;
                    v_next[x] = base[(int64_t)(row < len ? row : len - 1) * a.ldv + m];
                }
            }
        };
        if (chunks > 0) load_v(0);
        lds_barrier();
        for (int c = 0; c < chunks; ++c) {
            const uint8_t *buf = s_buf[c & 1];
            auto frag = [&](int at) { return *reinterpret_cast<const u32x4_t *>(buf + at); };
            auto vec4 = [&](int which, int t) {
                return *reinterpret_cast<const f32x4_t *>(buf + VEC + (which * CH + 16 * t + 4 * g4) * 4);
            };
            float v[16];
#pragma unroll
            for (int x = 0; x < 16; ++x) v[x] = bf16_to_f32(v_next[x]);
            load_v(c + 1 < chunks ? c + 1 : c);
            const float gamma = *reinterpret_cast<const float *>(buf + VEC + V_COUNT * CH * 4);

            auto k_frag = [&](int t, int q) { return frag(row_at(0, 16 * t + m, 4 * q + g4)); };
            auto q_frag = [&](int t, int q) { return frag(row_at(1, 16 * t + m, 4 * q + g4)); };
            auto kt_frag = [&](int t, int x) { return frag(col_at(16 * t + m, 4 * x + g4)); };
            auto op = [&](int which, int t, int x) { return frag(FR + (6 * which + frag_index(t, x)) * 1024 + lane * 16); };
            // the state as right operand
            u32x4_t sh[NQ], sl[NQ];
            float mx = 0.f;
#pragma unroll
            for (int t = 0; t < NT; ++t) mx = max_abs(S[t], mx);
            const RowScale ss = unit_scale(groups_max(mx));
            const float s_off = exp2i(-ss.s);
#pragma unroll
            for (int t = 0; t < NT; ++t) split(S[t], ss.sc, sh[t / 2], sl[t / 2], t & 1);
            // K S, X = V - diag(e^G) K S (the remainders' products go into the same
            // sums).  Here and below the inner index is the outer loop, so that
            // products into one sum are four or more apart: one after another they
            // wait for each other's result.
            f32x4_t QS[4], X[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) X[t] = QS[t] = zero4;
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
                u32x4_t fk[4];
#pragma unroll
                for (int t = 0; t < 4; ++t) fk[t] = k_frag(t, q);
#pragma unroll
                for (int t = 0; t < 4; ++t) X[t] = mfma_f16(fk[t], sl[q], X[t]);
#pragma unroll
                for (int t = 0; t < 4; ++t) X[t] = mfma_f16(fk[t], sh[q], X[t]);
#pragma unroll
                for (int t = 0; t < 4; ++t) QS[t] = mfma_f16(q_frag(t, q), sl[q], QS[t]);
#pragma unroll
                for (int t = 0; t < 4; ++t) QS[t] = mfma_f16(q_frag(t, q), sh[q], QS[t]);
            }
            mx = 0.f;
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const f32x4_t fa = vec4(V_A, t);
#pragma unroll
                for (int e = 0; e < 4; ++e) X[t][e] = fmaf(-X[t][e], fa[e] * s_off, v[4 * t + e]);
                mx = max_abs(X[t], mx);
            }
            // U = T' X (in units of 2^-xs.s), W = diag(c) U
            const RowScale xs = unit_scale(groups_max(mx));
            const float x_off = exp2i(-xs.s);
            u32x4_t xh[2], xl[2];
#pragma unroll
            for (int t = 0; t < 4; ++t) split(X[t], xs.sc, xh[t / 2], xl[t / 2], t & 1);
            f32x4_t U[4], W[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) U[t] = zero4;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
#pragma unroll
                for (int t = 2 * x; t < 4; ++t)
                    U[t] = mfma_f16(op(1, t, x), xh[x], U[t]);
#pragma unroll
                for (int t = 2 * x; t < 4; ++t) U[t] = mfma_f16(op(0, t, x), xl[x], U[t]);
#pragma unroll
                for (int t = 2 * x; t < 4; ++t) U[t] = mfma_f16(op(0, t, x), xh[x], U[t]);
            }
            mx = 0.f;
            float mw = 0.f;
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const f32x4_t ft = vec4(V_T, t), fc = vec4(V_C, t);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    U[t][e] *= ft[e];
                    W[t][e] = U[t][e] * fc[e];
                }
                mx = max_abs(U[t], mx);
                mw = max_abs(W[t], mw);
            }
            // S = e^{G_63} S + K^T W first: the next chunk waits for it.  (Nothing is
            // moved over this line: else 8 registers are spilled in the loop.)
            __builtin_amdgcn_sched_barrier(0);
            const RowScale wsc = unit_scale(groups_max(mw));
            const float w_off = exp2i(-wsc.s) * x_off;
            u32x4_t wh[2], wl[2];
#pragma unroll
            for (int t = 0; t < 4; ++t) split(W[t], wsc.sc, wh[t / 2], wl[t / 2], t & 1);
            f32x4_t D[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) D[t] = zero4;
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int t4 = 0; t4 < NT; t4 += 4) {
                    u32x4_t fk[4];
#pragma unroll
                    for (int t = 0; t < 4; ++t) fk[t] = kt_frag(t4 + t, x);
#pragma unroll
                    for (int t = 0; t < 4; ++t) D[t4 + t] = mfma_f16(fk[t], wl[x], D[t4 + t]);
#pragma unroll
                    for (int t = 0; t < 4; ++t) D[t4 + t] = mfma_f16(fk[t], wh[x], D[t4 + t]);
                }
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) S[t][e] = fmaf(D[t][e], w_off, gamma * S[t][e]);
            // O = diag(b) Q S + P U
            const RowScale us = unit_scale(groups_max(mx));
            const float u_off = exp2i(-us.s) * x_off;
            u32x4_t uh[2], ul[2];
#pragma unroll
            for (int t = 0; t < 4; ++t) split(U[t], us.sc, uh[t / 2], ul[t / 2], t & 1);
            f32x4_t O[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) O[t] = zero4;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
#pragma unroll
                for (int t = 2 * x; t < 4; ++t) O[t] = mfma_f16(op(3, t, x), uh[x], O[t]);
#pragma unroll
                for (int t = 2 * x; t < 4; ++t) O[t] = mfma_f16(op(2, t, x), ul[x], O[t]);
#pragma unroll
                for (int t = 2 * x; t < 4; ++t) O[t] = mfma_f16(op(2, t, x), uh[x], O[t]);
            }
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const f32x4_t fb = vec4(V_B, t), fp = vec4(V_P, t);
#pragma unroll
                for (int e = 0; e < 4; ++e) O[t][e] = fmaf(QS[t][e], fb[e] * s_off, O[t][e] * (fp[e] * u_off));
            }
            const int64_t r0 = t0 + (int64_t)c * CH;
            const int len = t1 - r0 < CH ? (int)(t1 - r0) : CH;
            uint16_t *ob = a.o + r0 * a.ldo + head_col;
            if (len == CH) {
#pragma unroll
                for (int x = 0; x < 16; ++x)
                    *reinterpret_cast<__bf16 *>(reinterpret_cast<uint8_t *>(ob + (int64_t)(16 * (x / 4) + x % 4) * a.ldo) +
                                                o_lane) = (__bf16)O[x / 4][x % 4];
            } else {
#pragma unroll
                for (int x = 0; x < 16; ++x) {
                    const int row = 16 * (x / 4) + 4 * g4 + x % 4;
                    if (row < len) *reinterpret_cast<__bf16 *>(ob + (int64_t)row * a.ldo + m) = (__bf16)O[x / 4][x % 4];
                }
            }
            lds_barrier();
        }
        if (kept && a.s_out && !(chunks == 0 && a.s_in == a.s_out)) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) a.s_out[soff + (int64_t)(16 * t + 4 * g4 + e) * a.dv] = S[t][e];
        }
    }
}

constexpr int SPLIT_TILES = 256;

template <int DK>
hipError_t launch_chunks(const DeltaArgs &a, void *ws, hipStream_t s) {
    if (a.T > 0) {
        const int64_t chunks = a.T / CH + a.n_seq;
        uint8_t *units = static_cast<uint8_t *>(ws);
        // Two heads of a key head together where that leaves enough workgroups.
        // Measured (whole calls, us, one head / two, 32 heads): k_dim 128, 768 chunks
        // and heads 94 / 96, 832 56.6 / 58.7, 1056 121 / 118, 8448 427 / 404; k_dim 64
        // (less to share): 2112 78 / 78, 4160 334 / 335, 8448 of eight prompts
        // 212 / 208, of one (its chain of chunks is the time) 704 / 715.
        if (a.hv / a.hk % 2 == 0 && chunks * a.hv >= (DK == 128 ? 1024 : 4096))
            hipLaunchKernelGGL((delta_prep_kernel<DK, 2>), dim3((unsigned)(chunks * (a.hv / 2))), dim3(256), 0, s, a, units);
        else
            hipLaunchKernelGGL((delta_prep_kernel<DK, 1>), dim3((unsigned)(chunks * a.hv)), dim3(256), 0, s, a, units);
    }
    // Workgroups of 16 columns while there are no more than compute units (a unit
    // holds one); else of 64.  Measured (whole calls, us, 16 / 64): 256 tiles of 16
    // columns, k_dim 128: 4096 tokens 225 / 260; 512: 2 x 1024 119 / 87; k_dim 64,
    // 256: 8 x 256 28.2 / 30.3; 512: 16 x 256 44.7 / 36.3.  (The count is of all
    // units.  The kernel keeps the workgroups of a sequence and key head on one XCD
    // of 32 units, so with few such pairs and many columns for each they take turns
    // there while other XCDs have none: 4096 tokens of 32 value heads on 16, 4, 2
    // and 1 key heads take 223, 399, 758 and 1474 us.  Nothing here avoids that.)
    const int64_t tiles = (int64_t)a.n_seq * a.hv * (a.dv / 16);
    const bool split_rows = tiles <= SPLIT_TILES;
    const int64_t groups = (int64_t)a.n_seq * a.hk, per = a.hv / a.hk * (a.dv / (split_rows ? 16 : 64));
    const dim3 grid((unsigned)((groups + 7) / 8 * 8 * per));
    const uint8_t *units = static_cast<const uint8_t *>(ws);
    if (split_rows)
        hipLaunchKernelGGL((delta_scan_kernel<DK, true>), grid, dim3(512), 0, s, a, units);
    else
        hipLaunchKernelGGL((delta_scan_kernel<DK, false>), grid, dim3(512), 0, s, a, units);
    return hipGetLastError();
}

}  // namespace

size_t delta_workspace_bytes(int64_t T, int n_seq, int hv) { return (size_t)(T / CH + n_seq) * hv * UNIT; }

hipError_t launch_delta_prefill(const DeltaArgs &a, void *ws, hipStream_t s) {
    return a.dk == 64 ? launch_chunks<64>(a, ws, s) : launch_chunks<128>(a, ws, s);
}

hipError_t launch_delta_decode(const DeltaArgs &a, hipStream_t s) {
    if (a.dk == 64) return a.dv == 64 ? launch_decode<64, 64>(a, s) : launch_decode<64, 128>(a, s);
    return a.dv == 64 ? launch_decode<128, 64>(a, s) : launch_decode<128, 128>(a, s);
}

}  // namespace moeq4
