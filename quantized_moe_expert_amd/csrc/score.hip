// Log probabilities of given tokens, entropy and the largest logits of rows.
//
// With m the largest logit of a row, d = l - m, z = sum e^d and s = sum d e^d:
//   log p = d - log z,   entropy = log z - s / z.
// A row is cut into segments of 8192 logits, one workgroup each, 32 logits per
// thread held in registers: the row is read once, and the maximum, the sums
// and the selection are passes over registers.  A segment's sums are relative
// to its own maximum; a row of several segments has them joined by a second
// launch, in segment order, so that the same input gives the same bits.
//
// The largest n of a segment (n <= 32): the n-th largest of the 64 lanes'
// maxima of a wave bounds the n-th largest logit from below (found bit by bit
// with ballots; where many lanes share it, the logit's index, inverted, decides
// ties).  Logits at or above the largest of the four waves' bounds, a few n of
// them, are collected in LDS, and each one's rank is the number of larger ones
// (keys of value and index are unique, so the order of collecting, by an LDS
// counter, does not matter).
#include "backbone.h"

namespace moeq4 {

namespace {

constexpr int THREADS = 256;
constexpr int PER = 32;                  // logits per thread
constexpr int SEG = THREADS * PER;       // logits per workgroup
constexpr int CAND = 1024;               // candidates held in LDS
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

// Sums of part of a row: largest logit, sum e^(l - m), sum (l - m) e^(l - m).
struct Sums {
    float m, z, s;
};

// Order-preserving image of a float without NaNs: a larger value gives a
// larger key, equal values equal keys (-0 as +0).
__device__ __forceinline__ uint32_t f32_order(float f) {
    const uint32_t b = __float_as_uint(f + 0.0f);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float f32_from_order(uint32_t o) {
    return __uint_as_float((o & 0x80000000u) ? (o ^ 0x80000000u) : ~o);
}
// 64-bit key: value, then the lower index first.
__device__ __forceinline__ uint64_t make_key(float l, uint32_t index) {
    return ((uint64_t)f32_order(l) << 32) | (0xffffffffu - index);
}

// A NaN counts as -inf.
__device__ __forceinline__ float clean(float f) { return fmaxf(f, -INFINITY); }

template <bool F32>
__device__ __forceinline__ float load_logit(const void *logits, int64_t at) {
    if (F32) return clean(static_cast<const float *>(logits)[at]);
    return clean(bf16_to_f32(static_cast<const uint16_t *>(logits)[at]));
}

// l - m; 0 where l is the maximum, so that an infinite maximum works.
__device__ __forceinline__ float below(float l, float m) { return l == m ? 0.0f : l - m; }

__device__ __forceinline__ Sums join(Sums a, Sums b) {
    if (a.m == -INFINITY) return b;
    if (b.m == -INFINITY) return a;
    Sums r;
    r.m = fmaxf(a.m, b.m);
    const float da = below(a.m, r.m), db = below(b.m, r.m);
    const float ea = expf(da), eb = expf(db);
    r.z = ea * a.z + eb * b.z;
    r.s = (ea > 0.f ? ea * (a.s + da * a.z) : 0.f) + (eb > 0.f ? eb * (b.s + db * b.z) : 0.f);
    return r;
}

__device__ __forceinline__ uint64_t wave_max_u64(uint64_t v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
        const uint64_t w = __shfl_xor((unsigned long long)v, o);
        v = v > w ? v : w;
    }
    return v;
}

// 16 bytes at any element address (rows may start anywhere).
struct __attribute__((packed, aligned(2))) Vec16b2 {
    uint32_t v[4];
};
struct __attribute__((packed, aligned(4))) Vec16b4 {
    uint32_t v[4];
};

// The row's outputs from its sums, its largest keys (tid < n_top) and the
// token's logit; called by one workgroup.
template <bool F32>
__device__ __forceinline__ void finish_row(const LogprobsArgs &a, int64_t t, const Sums &r, const uint64_t *top) {
    const int tid = threadIdx.x;
    const bool empty = r.m == -INFINITY;
    const float lz = empty ? 0.f : logf(r.z);
    if (tid == 64) {
        if (a.tokens) {
            const int tok = a.tokens[t];
            float lp = 0.f;
            if (tok >= 0 && tok < a.V) lp = empty ? -INFINITY : below(load_logit<F32>(a.logits, t * a.ld + tok), r.m) - lz;
            a.logprob[t] = lp;
        }
        if (a.entropy) a.entropy[t] = empty ? 0.f : lz - r.s / r.z;
    }
    if (tid < a.n_top) {
        const uint64_t key = top[tid];
        a.top_idx[t * a.n_top + tid] = (int32_t)(0xffffffffu - (uint32_t)key);
        a.top_logprob[t * a.n_top + tid] = empty ? -INFINITY : below(f32_from_order((uint32_t)(key >> 32)), r.m) - lz;
    }
}

// Ranks `count` unique keys (LDS, followed by room for 31 more, which are
// cleared here) into top[0 .. n), largest first: the four lanes of a quad
// compare a key with eight others at a time each.
__device__ __forceinline__ void rank_keys(uint64_t *cand, int count, int n, uint64_t *top) {
    if (threadIdx.x < 31) cand[count + threadIdx.x] = 0;
    __syncthreads();
    for (int i = threadIdx.x >> 2; i < count; i += THREADS / 4) {
        const uint64_t key = cand[i];
        int rank = 0;
        for (int j = (threadIdx.x & 3) * 8; j < count; j += 32) {
#pragma unroll
            for (int e = 0; e < 8; ++e) rank += cand[j + e] > key;
        }
        rank += (int)dpp_u32<0xb1>((uint32_t)rank);  // lane ^ 1
        rank += (int)dpp_u32<0x4e>((uint32_t)rank);  // lane ^ 2
        if (rank < n) top[rank] = key;
    }
}

// Lower bound of a wave's n-th largest key, from its lanes' largest keys
// hi:lo (unique, or 0 for a lane without one): the n-th largest of those,
// found bit by bit with ballots; 0 with fewer than n.  hi differs between
// lanes in its bits from HI_BIT up only, lo in its lower LO_BITS bits.  When
// up to 16 lanes more share the n-th largest hi the bound is that hi alone (a
// few more keys reach it); when more do, lo (from lo_of) tells them apart.
template <int HI_BIT, int LO_BITS, typename F>
__device__ __forceinline__ uint64_t wave_bound(uint32_t hi, int n, F lo_of) {
    uint32_t v = 0;
#pragma unroll
    for (int bit = 31; bit >= HI_BIT; --bit) {
        const uint32_t w = v | (1u << bit);
        if (__popcll(__ballot(hi >= w)) >= n) v = w;
    }
    const uint32_t top = hi & (~0u << HI_BIT);
    const int above = __popcll(__ballot(top > v)), level = __popcll(__ballot(top == v));
    uint32_t w = 0;
    if (above + level > n + 16) {
        const uint32_t lo = lo_of();
        for (int bit = LO_BITS - 1; bit >= 0; --bit) {
            const uint32_t u = w | (1u << bit);
            if (above + __popcll(__ballot(top == v && lo >= u)) >= n) w = u;
        }
    }
    return ((uint64_t)v << 32) | w;
}

// Bit 31 - i: l[i] < limit, for a finite limit: the sign of the difference,
// shifted in (two instructions a logit; a compare and a select would wait for
// each other).
__device__ __forceinline__ uint32_t below_bits(const float (&l)[PER], float limit) {
    uint32_t bits = 0;
    // +0 for a zero limit: -0 is not below 0 (opaque, or l - limit is formed)
    float minus = limit == 0.f ? 0.f : -limit;
    asm("" : "+v"(minus));
#pragma unroll
    for (int i = 0; i < PER; ++i) bits = __builtin_amdgcn_alignbit(bits, __float_as_uint(l[i] + minus), 31);
    return bits;
}
// The same of l[i] > limit.
__device__ __forceinline__ uint32_t above_bits(const float (&l)[PER], float limit) {
    uint32_t bits = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) bits = __builtin_amdgcn_alignbit(bits, __float_as_uint(limit - l[i]), 31);
    return bits;
}
__device__ __forceinline__ int first_equal(const float (&l)[PER], float value) {
    int at = 0;
#pragma unroll
    for (int i = PER - 1; i >= 0; --i) at = l[i] == value ? i : at;
    return at;
}

// Bits (31 - i for logit i) of the thread's logits whose place in the segment
// is below `end`.
__device__ __forceinline__ uint32_t places_below(int end, int tid) {
    uint32_t bits = 0;
#pragma unroll
    for (int j = 0; j < PER / 8; ++j) {
        int c = end - (j * THREADS + tid) * 8;
        c = c < 0 ? 0 : (c > 8 ? 8 : c);
        bits |= (0xff00u >> c & 0xffu) << (24 - 8 * j);
    }
    return bits;
}

// The largest of three floats, none of them NaN.
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
    return r;
}

// One segment per workgroup.  DIRECT: the row has one segment and the outputs
// are written here; otherwise its sums and keys go to part / part_top.
// Bound by the vector work (620 instructions a wave with a top list, 32 of them
// exponentials of four times the cost; without a list by the bytes).  Measured,
// 512 rows of 151939 bf16 (156 MB): 62 us with n = 20 (2.5 TB/s) and 7 us for the
// join, 34.5 us in all with n = 0 (4.5 TB/s).  Before the candidates were found
// by the sign of a difference and reloaded by place: 82 us; ranked by one lane
// each with one key after another: 128 us.  One row of 4097, n = 8: 4.9 us.
template <bool F32, bool TOP, bool DIRECT>
__global__ __launch_bounds__(THREADS) void logprobs_segment_kernel(LogprobsArgs a, int segs,
                                                                   Sums *__restrict__ part,
                                                                   uint64_t *__restrict__ part_top) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t t = DIRECT ? blockIdx.x : blockIdx.x / segs;
    const int64_t v0 = DIRECT ? 0 : (int64_t)(blockIdx.x % segs) * SEG;
    const int64_t row = t * a.ld + v0;
    const int len = a.V - v0 < SEG ? (int)(a.V - v0) : SEG;  // logits of this segment

    // logit e of vector j: index (j * 256 + tid) * 8 + e of the segment
    float l[PER];
    typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
    uint32_t big = 0;     // largest magnitude bits (float)
    u16x2_t big2 = {0, 0};  // the same of bf16 pairs
#pragma unroll
    for (int j = 0; j < PER / 8; ++j) {
        const int i0 = (j * THREADS + tid) * 8;
        if (i0 + 8 <= len) {
            if (F32) {
                const Vec16b4 *p = reinterpret_cast<const Vec16b4 *>(static_cast<const float *>(a.logits) + row + i0);
                const Vec16b4 x = p[0], y = p[1];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    l[8 * j + e] = __uint_as_float(x.v[e]);
                    l[8 * j + 4 + e] = __uint_as_float(y.v[e]);
                    const uint32_t bx = x.v[e] & 0x7fffffffu, by = y.v[e] & 0x7fffffffu;
                    big = big > bx ? big : bx;
                    big = big > by ? big : by;
                }
            } else {
                const Vec16b2 x =
                    *reinterpret_cast<const Vec16b2 *>(static_cast<const uint16_t *>(a.logits) + row + i0);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    l[8 * j + 2 * e] = __uint_as_float(x.v[e] << 16);
                    l[8 * j + 2 * e + 1] = __uint_as_float(x.v[e] & 0xffff0000u);
                    big2 = __builtin_elementwise_max(big2, __builtin_bit_cast(u16x2_t, x.v[e] & 0x7fff7fffu));
                }
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                l[8 * j + e] = i0 + e < len ? load_logit<F32>(a.logits, row + i0 + e) : -INFINITY;
        }
    }
    // maximum of the segment, and each lane's first largest logit
    if (__any(big > 0x7f800000u || big2[0] > 0x7f80u || big2[1] > 0x7f80u)) {
#pragma unroll
        for (int i = 0; i < PER; ++i) l[i] = clean(l[i]);
    }
    float lmax = l[0];
#pragma unroll
    for (int i = 1; i + 1 < PER; i += 2) lmax = max3(lmax, l[i], l[i + 1]);
    lmax = max3(lmax, l[PER - 1], l[PER - 1]);
    __shared__ float s_m[4], s_z[4], s_s[4];
    const uint32_t lane_hi = f32_order(lmax);
    const float wmax = f32_from_order(wave_max_u32(lane_hi));
    if (lane == 0) s_m[wave] = wmax;

    __shared__ uint64_t s_bound[TOP ? 4 : 1];
    __shared__ int s_count;
    if (TOP) {
        // keys of bf16 logits differ in their upper 16 bits; the place of a
        // logit is below SEG = 2^13
        const uint64_t bound = wave_bound<F32 ? 0 : 16, 13>(tid * 8 < len ? lane_hi : 0u, a.n_top, [&] {
            // the first of the thread's largest logits
            const int at = lmax - lmax == 0.f ? __clz((int)~below_bits(l, lmax)) : first_equal(l, lmax);
            return tid * 8 < len ? (uint32_t)(SEG - 1 - (((at >> 3) * THREADS + tid) * 8 + (at & 7))) : 0u;
        });
        if (lane == 0) s_bound[wave] = bound;
        if (tid == 0) s_count = 0;
    }
    __syncthreads();
    const float m = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3]));
    float z = 0.f, s = 0.f;
    if (m == INFINITY) {
#pragma unroll
        for (int i = 0; i < PER; ++i) z += l[i] == m ? 1.f : 0.f;
    } else if (fabsf(m) < 1048576.f) {
        // d / log 2 = l LOG2E - mc - c, with mc + c = m LOG2E: one fma a
        // logit, c (below 1/8) taken off the sums.  The clamp keeps 0 * -inf
        // out (2^-200 is 0).
        const float mc = m * LOG2E, c = fmaf(m, LOG2E, -mc);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const float d = fmaxf(fmaf(l[i], LOG2E, -mc), -200.f);
            const float e = __builtin_amdgcn_exp2f(d);
            z += e;
            s = fmaf(e, d, s);
        }
        const float scale = __builtin_amdgcn_exp2f(-c);
        s = scale * fmaf(-c, z, s) * LN2;
        z *= scale;
    } else if (m != -INFINITY) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const float d = fmaxf((l[i] - m) * LOG2E, -200.f);
            const float e = __builtin_amdgcn_exp2f(d);
            z += e;
            s = fmaf(e, d, s);
        }
        s *= LN2;
    }
    z = seg_sum_dpp<64>(z);
    s = seg_sum_dpp<64>(s);
    if (lane == 63) s_z[wave] = z, s_s[wave] = s;

    __shared__ uint64_t s_cand[TOP ? CAND + 32 : 1], s_top[TOP ? 32 : 1];
    if (TOP) {
        if (tid < 32) s_top[tid] = 0;
        uint64_t bound = s_bound[0];
#pragma unroll
        for (int i = 1; i < 4; ++i) bound = s_bound[i] > bound ? s_bound[i] : bound;
        const uint32_t bv = (uint32_t)(bound >> 32), bi = (uint32_t)bound;
        // value of the bound (-inf when it is 0); ties only up to its place,
        // and no places behind the row
        const float bf = bv ? f32_from_order(F32 ? bv : (bv & 0x80000000u) ? bv : bv | 0xffffu) : -INFINITY;
        uint32_t mask;
        if (bf - bf == 0.f) {
            mask = ~below_bits(l, bf);
            if (bi) mask &= above_bits(l, bf) | places_below(SEG - (int)bi, tid);
        } else {
            const uint32_t in = places_below(SEG - (int)bi, tid);
            mask = 0;
#pragma unroll
            for (int i = 0; i < PER; ++i)
                mask |= l[i] > bf || (l[i] == bf && in << i >> 31) ? 0x80000000u >> i : 0u;
        }
        mask &= places_below(len, tid);
        const int mine = __popc(mask), upto = wave_inclusive_scan_i32(mine);
        int base = 0;
        if (lane == 63 && upto) base = atomicAdd(&s_count, upto);
        int c = __builtin_amdgcn_readlane(base, 63) + upto - mine;
        if (c + mine > CAND) mask = 0;  // counted, not stored
        while (mask) {
            const int i = __clz((int)mask);
            const int at = ((i >> 3) * THREADS + tid) * 8 + (i & 7);
            s_cand[c++] = make_key(load_logit<F32>(a.logits, row + at), (uint32_t)(v0 + at));
            mask &= ~(0x80000000u >> i);
        }
        __syncthreads();
        const int count = s_count;
        if (count <= CAND) {
            rank_keys(s_cand, count, a.n_top, s_top);
        } else {
            // many logits in few lanes: the largest below the last, one by one
            uint64_t last = ~0ull;
            for (int k = 0; k < a.n_top; ++k) {
                uint64_t best = 0;
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    const int at = ((i >> 3) * THREADS + tid) * 8 + (i & 7);
                    const uint64_t key = at < len ? make_key(l[i], (uint32_t)(v0 + at)) : 0;
                    if (key < last && key > best) best = key;
                }
                best = wave_max_u64(best);
                if (lane == 0) s_cand[wave] = best;
                __syncthreads();
                last = s_cand[0];
#pragma unroll
                for (int i = 1; i < 4; ++i) last = s_cand[i] > last ? s_cand[i] : last;
                if (tid == 0) s_top[k] = last;
                __syncthreads();
            }
        }
    }
    __syncthreads();
    const Sums r{m, s_z[0] + s_z[1] + s_z[2] + s_z[3], s_s[0] + s_s[1] + s_s[2] + s_s[3]};
    if (DIRECT) {
        finish_row<F32>(a, t, r, s_top);
    } else {
        if (tid == 0) part[blockIdx.x] = r;
        if (TOP && tid < a.n_top) part_top[(int64_t)blockIdx.x * a.n_top + tid] = s_top[tid];
    }
}

// Joins the segments of a row, one workgroup per row.  Sums: each thread its
// segments in order, then the threads in a tree of fixed shape.  Keys: the
// best so far and the next segments' lists, ranked batch by batch.
template <bool F32>
__global__ __launch_bounds__(THREADS) void logprobs_join_kernel(LogprobsArgs a, int segs,
                                                                const Sums *__restrict__ part,
                                                                const uint64_t *__restrict__ part_top) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int64_t t = blockIdx.x;
    Sums r{-INFINITY, 0.f, 0.f};
    for (int p = tid; p < segs; p += THREADS) r = join(r, part[t * segs + p]);
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
        const Sums b{__shfl_xor(r.m, o), __shfl_xor(r.z, o), __shfl_xor(r.s, o)};
        r = (lane & o) ? join(b, r) : join(r, b);
    }
    __shared__ Sums s_sums[4];
    if (lane == 0) s_sums[wave] = r;
    __shared__ uint64_t s_cand[CAND + 32], s_top[32], s_bound[4];
    __shared__ int s_count;
    if (tid < 32) s_top[tid] = 0;
    __syncthreads();
    r = join(join(s_sums[0], s_sums[1]), join(s_sums[2], s_sums[3]));
    const int64_t total = (int64_t)segs * a.n_top;
    for (int64_t at = 0; at < total; at += CAND - 32) {
        const int next = total - at < CAND - 32 ? (int)(total - at) : CAND - 32;
        const int kept = at ? a.n_top : 0;
        uint64_t key[CAND / THREADS], best = 0;
#pragma unroll
        for (int e = 0; e < CAND / THREADS; ++e) {
            const int i = e * THREADS + tid;
            key[e] = i < kept ? s_top[i] : i < kept + next ? part_top[t * total + at + i - kept] : 0;
            best = key[e] > best ? key[e] : best;
        }
        const uint64_t wb = wave_bound<0, 32>((uint32_t)(best >> 32), a.n_top, [&] { return (uint32_t)best; });
        if (lane == 0) s_bound[wave] = wb;
        if (tid == 0) s_count = 0;
        __syncthreads();
        uint64_t bound = s_bound[0] ? s_bound[0] : 1;
#pragma unroll
        for (int i = 1; i < 4; ++i) bound = s_bound[i] > bound ? s_bound[i] : bound;
#pragma unroll
        for (int e = 0; e < CAND / THREADS; ++e)
            if (key[e] >= bound) s_cand[atomicAdd(&s_count, 1)] = key[e];
        __syncthreads();
        rank_keys(s_cand, s_count, a.n_top, s_top);
        __syncthreads();
    }
    finish_row<F32>(a, t, r, s_top);
}

template <bool F32>
hipError_t launch(const LogprobsArgs &a, void *ws, hipStream_t s) {
    const int segs = logprobs_segments(a.V);
    const int64_t blocks = a.T * segs;
    const dim3 grid((unsigned)blocks), block(THREADS);
    Sums *part = nullptr;
    uint64_t *part_top = static_cast<uint64_t *>(ws);
    if (segs == 1) {
        if (a.n_top)
            hipLaunchKernelGGL((logprobs_segment_kernel<F32, true, true>), grid, block, 0, s, a, segs, part, part_top);
        else
            hipLaunchKernelGGL((logprobs_segment_kernel<F32, false, true>), grid, block, 0, s, a, segs, part, part_top);
        return hipGetLastError();
    }
    part = reinterpret_cast<Sums *>(part_top + blocks * a.n_top);
    if (a.n_top)
        hipLaunchKernelGGL((logprobs_segment_kernel<F32, true, false>), grid, block, 0, s, a, segs, part, part_top);
    else
        hipLaunchKernelGGL((logprobs_segment_kernel<F32, false, false>), grid, block, 0, s, a, segs, part, part_top);
    hipLaunchKernelGGL((logprobs_join_kernel<F32>), dim3((unsigned)a.T), block, 0, s, a, segs, part, part_top);
    return hipGetLastError();
}

}  // namespace

int logprobs_segments(int64_t V) { return (int)((V + SEG - 1) / SEG); }
size_t logprobs_part_bytes(int n_top) { return sizeof(Sums) + (size_t)n_top * sizeof(uint64_t); }

hipError_t launch_logprobs(const LogprobsArgs &a, void *ws, hipStream_t s) {
    return a.f32 ? launch<true>(a, ws, s) : launch<false>(a, ws, s);
}

}  // namespace moeq4
