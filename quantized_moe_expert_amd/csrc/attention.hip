// Attention over the paged cache:
//   o = sum_j p_j v_j / sum_j p_j,  p_j = exp(s_j - max s),  s = cap tanh(scale q.k / cap) - slope |distance|.
//
// The rows of a sequence that read one head of the cache (its tokens times the
// query heads that share it, token by token) are cut into blocks, the keys that
// a block sees into tiles.  Both kernels compute S^T = K Q^T and O^T = V^T P^T,
// so that a lane has scores of one query and its weights are the second
// product's operand where they are: they never leave the lane's registers.
// Running maximum and sum of a row are fp32.
//
//   attention_rows_kernel  few rows in a sequence (single tokens): blocks of 16
//       rows, every wave with key tiles of its own, K and V straight from memory
//       into the operands.  Bound by the cache's bytes.
//   attention_tile_kernel  more rows: blocks of 128 rows, 32 to a wave, tiles of
//       keys shared through LDS.  Bound by the matrix products and the
//       exponentials beside them.
//   attention_join_kernel  joins the parts of blocks whose keys were split.
//
// How many workgroups share the keys of a block is decided on the device from
// the sequences' lengths (plan_find), so that a captured call goes with them.
#include "rows_dev.h"

namespace moeq4 {

namespace {

typedef __attribute__((__vector_size__(4 * sizeof(float)))) float f32x4_t;
typedef __bf16 bf16v8_t __attribute__((ext_vector_type(8)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2_t __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) void lds_void;

constexpr int THREADS = 256, WAVES = THREADS / WAVE;
// Scores as they are; capped by a quotient (caps up to QUOTIENT_CAP); by more; less a
// bias (and capped by either, or not).
enum { PLAIN, QUOTIENT, CAPPED, BIASED };
constexpr float LOG2E = 1.44269504088896340736f;
// Rows are scaled to a new maximum when it is more than 2^RISE times the old
// one: weights stay below 2^RISE, whose sums fp32 holds as well.
constexpr float RISE = 8.0f;
// The least maximum of a row that sees a key, whatever its scores: NaN, which a
// maximum passes over, or -inf.  -inf itself says that a row sees none (and has o = 0).
constexpr float LEAST = -3.402823466e38f;

__device__ __forceinline__ f32x4_t mfma16(u32x4_t a, u32x4_t b, f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16v8_t, a), __builtin_bit_cast(bf16v8_t, b),
                                                   c, 0, 0, 0);
}
__device__ __forceinline__ f32x16_t mfma32(u32x4_t a, u32x4_t b, f32x16_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16v8_t, a), __builtin_bit_cast(bf16v8_t, b),
                                                   c, 0, 0, 0);
}
// Finite, so that a product or a distance of 0 stays one.
__device__ __forceinline__ float finite(float v) { return fminf(fmaxf(v, -3e38f), 3e38f); }

// A score's cap, cap2 tanh(w / cap2) with all in powers of two (cap2 = cap log2(e)).
//
// Up to QUOTIENT_CAP: the quotient rest = 1 / (1 + e^2x), x = w / cap2, of v = 2 x log2(e),
// and from it cap2 - 2 cap2 rest.  Off by at most 10 half steps of the *cap* (2^-14.7 at 64;
// a weight is then rounded to 2^-16 of itself in the rows kernel, 2^-8 in the tile kernel).
//
// Beyond: score(), off by at most 12 half steps of the score.  Up to |x| = 1/2 a
// polynomial, w p(x^2) (coefficients: least largest relative error, 2^-26), then cap2
// (1 - 2 / (1 + e^2|x|)) with the sign of x.
//
// Measured, no cap / quotient / score(): pieces of long prompts, heads of 256, 1.35 / 1.56 /
// 2.05 ms; prompt of 8192, heads of 128, 553 / 665 / 907 us; 64 streams over 790 k keys
// 572 us in all three.
constexpr float QUOTIENT_CAP = 64.0f;
__device__ __forceinline__ float cap_rest(float v) { return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(v)); }
struct Cap {
    float cap2, inverse;
    __device__ __forceinline__ explicit Cap(float cap)
        : cap2(finite(cap * LOG2E)), inverse(finite(1.0f / cap2)) {}
    // Whether the quotient caps, and what a product is multiplied by: to v then, to w otherwise.
    static __device__ __forceinline__ bool quotient(const AttentionArgs &a) { return a.cap > 0.0f && a.cap <= QUOTIENT_CAP; }
    static __device__ __forceinline__ float scale(const AttentionArgs &a) {
        return finite(quotient(a) ? a.scale / a.cap * (2.0f * LOG2E) : a.scale * LOG2E);
    }
    __device__ __forceinline__ float of_rest(float rest) const { return fmaf(-2.0f * cap2, rest, cap2); }
    __device__ __forceinline__ float score(float w) const {
        const float x = w * inverse, y = x * x;
        const float p = fmaf(y, fmaf(y, fmaf(y, fmaf(y, 0.01724149f, -0.05304549f), 0.13325879f), -0.33333144f), 1.0f);
        const float far = cap2 * fmaf(-2.0f, cap_rest(fabsf(x) * (2.0f * LOG2E)), 1.0f);
        return fabsf(x) < 0.5f ? w * p : copysignf(far, x);
    }
};
// Largest value and sum over the lanes that hold one query: l, l ^ 32 and, of
// 16 queries, l ^ 16 and l ^ 48.
template <bool OF16>
__device__ __forceinline__ float query_max(float v) {
    if (OF16) {
        const uint32_t a = __float_as_uint(v);
        const u32x2_t p = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_permlane16_swap(a, a, false, false));
        v = fmaxf(__uint_as_float(p.x), __uint_as_float(p.y));
    }
    const uint32_t b = __float_as_uint(v);
    const u32x2_t q = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_permlane32_swap(b, b, false, false));
    return fmaxf(__uint_as_float(q.x), __uint_as_float(q.y));
}
template <bool OF16>
__device__ __forceinline__ float query_sum(float v) {
    if (OF16) v += __shfl_xor(v, 16, WAVE);
    return v + __shfl_xor(v, 32, WAVE);
}
__device__ __forceinline__ bool not_finite(u32x4_t w) {
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) bad |= (w[i] & 0x7f80u) == 0x7f80u || (w[i] & 0x7f800000u) == 0x7f800000u;
    return bad;
}

// ------------------------------------------------------------- sequences

struct Seq {
    int start, n;      // rows
    int kv, len;       // tokens; those that the table has room for
    int before, prefix;
};
__device__ __forceinline__ Seq load_seq(const AttentionArgs &a, int b) {
    Seq s;
    const int T = (int)a.T;
    s.start = min(max(a.seq_start[b], 0), T);
    s.n = min(max(a.seq_start[b + 1], s.start), T) - s.start;
    s.kv = min(max(a.cache.kv_len[b], 0), 0x7fff0000);
    s.len = min(s.kv, a.cache.max_pages * a.cache.page);
    s.before = s.kv - s.n;
    s.prefix = a.prefix ? min(max(a.prefix[b], 0), s.len) : 0;
    return s;
}

// Tiles of n keys that rows i0 to i1 of a sequence see some of: those of the
// prefix, [0, n1), and from lo on; tile j of them is j < n1 ? j : j - n1 + lo.
struct Range {
    int n1, lo, count;
    __device__ __forceinline__ int tile(int j) const { return j < n1 ? j : j - n1 + lo; }
};
template <int N>
__device__ __forceinline__ Range tiles_of(const AttentionArgs &a, const Seq &s, int i0, int i1) {
    // A drafted token's position is from `before` on, and it may see all of the draft.
    const int first = s.before + (a.tree ? 0 : i0);
    const int hi = a.tree ? s.len : min(s.len, s.before + i1 + 1);
    const int lo = a.window ? (int)max((int64_t)0, (int64_t)first - a.window + 1) : 0;
    Range r;
    const int end = hi > lo ? (hi + N - 1) / N : 0, begin = min(lo / N, end);
    r.n1 = (s.prefix + N - 1) / N;
    if (r.n1 >= begin) {
        r.lo = r.n1;
        r.count = max(end, r.n1);
    } else {
        r.lo = begin;
        r.count = r.n1 + end - begin;
    }
    return r;
}
// Whether rows i0 to i1 see every key of [k0, k0 + n).
template <int N>
__device__ __forceinline__ bool sees_all(const AttentionArgs &a, const Seq &s, int i0, int i1, int k0) {
    if (k0 + N > s.len) return false;
    if (a.tree) return k0 + N <= s.before && (!a.window || s.before + WAVE - k0 < a.window);
    return k0 + N <= s.prefix || (k0 + N - 1 <= s.before + i0 && (!a.window || s.before + i1 - k0 < a.window));
}

// What one query sees: keys lo to hi of all (tree: of the cached ones), and of
// the draft's rows those in mask.
struct Query {
    int pos, lo, hi;
    uint64_t mask;
};
// depth: of the draft's rows (load_depths).
__device__ __forceinline__ Query load_query(const AttentionArgs &a, const Seq &s, const int *depth, int i) {
    Query q;
    q.mask = 0;
    q.pos = s.before + i;
    if (a.tree) {
        q.mask = a.tree[s.start + i];
        q.pos = s.before + __popcll(i < WAVE ? q.mask & ~(1ull << i) : q.mask);
    }
    q.hi = (a.tree ? min(s.before, s.len) : min(s.len, q.pos + 1)) - 1;
    q.lo = a.window ? (int)max((int64_t)0, (int64_t)q.pos - a.window + 1) : 0;
    if (a.tree && a.window)
        for (int c = 0; c < WAVE; ++c)
            if (q.pos - (s.before + depth[c]) >= a.window) q.mask &= ~(1ull << c);
    return q;
}
// Bits 0 to n - 1 of 64.
__device__ __forceinline__ uint64_t below(int n) { return n >= 64 ? ~0ull : (1ull << max(n, 0)) - 1; }
// Which of the 64 keys from k0 on the query sees.
__device__ __forceinline__ uint64_t seen(const AttentionArgs &a, const Seq &s, const Query &q, int k0) {
    uint64_t bits = (below(q.hi + 1 - k0) & ~below(q.lo - k0)) | below(s.prefix - k0);
    if (a.tree) {
        const int up = s.before - k0;
        const uint64_t drafted = up >= 0 ? (up < 64 ? q.mask << up : 0) : (up > -64 ? q.mask >> -up : 0);
        bits |= drafted & below(s.len - k0);
    }
    return bits;
}
// Position of a key.
__device__ __forceinline__ int key_pos(const AttentionArgs &a, const Seq &s, const int *depth, int key) {
    const int c = key - s.before;
    return a.tree && c >= 0 ? s.before + depth[min(c, WAVE - 1)] : key;
}
__device__ __forceinline__ void load_depths(const AttentionArgs &a, const Seq &s, int *depth) {
    const int c = threadIdx.x;
    if (c < WAVE) depth[c] = c < s.n ? __popcll(a.tree[s.start + c] & ~(1ull << c)) : 0;
    __syncthreads();
}

// ------------------------------------------------------------------ plan

// A sequence of n rows has R = ceil(n r / rows) blocks (r query heads to a head
// of the cache), each with at most m tiles of keys.  With C = max(cmin,
// ceil(sum R m / target)) tiles to a part, a block has S = ceil(m / C) parts: at
// most target + sum R parts in all, for each head of the cache, and at most
// 2 target of blocks with more than one (m > C: S <= 2 m / C), whose sums go
// through the workspace.
struct Plan {
    int rows, row_shift;    // of a block, a power of two
    int key_shift;          // keys of a tile, a power of two
    int cmin, target_shift;
    int join_groups;        // workgroups that share the rows of a split block (share_parts)
    int items, joins, slots;  // most parts; most split blocks; most of their parts (each per head of the cache)
};

struct Found {
    int b, block, part, parts, slot;
    Seq seq;
};

__device__ __forceinline__ void blocks_of(const AttentionArgs &a, const Plan &p, const Seq &s, int &R, int &m) {
    const int r = a.hq / a.cache.hkv, up = (1 << p.key_shift) - 1;
    R = (s.n * r + p.rows - 1) >> p.row_shift;
    m = (s.len + up) >> p.key_shift;
    if (a.window) {
        // Keys that some row of a block sees: the window and the block's tokens before it.
        const int64_t span = (int64_t)a.window + (a.tree ? WAVE : p.rows / r + 1);
        m = (int)min((int64_t)m, ((s.prefix + up) >> p.key_shift) + (span >> p.key_shift) + 2);
    }
    m = max(m, 1);
}
// Tiles to a part. (No sequence has 2^30.)
__device__ __forceinline__ int tiles_to_a_part(const Plan &p, uint64_t work) {
    const uint64_t c = (work + (1u << p.target_shift) - 1) >> p.target_shift;
    return max(p.cmin, (int)min(c, (uint64_t)1 << 30));
}

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

__device__ __forceinline__ Seq uniform(const Seq &s) {
    return Seq{uniform(s.start), uniform(s.n), uniform(s.kv), uniform(s.len), uniform(s.before), uniform(s.prefix)};
}

// Finds the part (JOIN: the split block) with this number; false: there are
// fewer.  All threads of the workgroup call it.
//
// Each workgroup goes over all sequences: up to 64 in a few instructions, more in
// steps of 256.  Single tokens over 100 keys, 8 heads on 2 of 64: 64 sequences 7.2 us, 65
// 7.5, 256 9.1, 1024 27.5, 4096 187, 16384 2009: from about a thousand on it is
// what the call takes, and grows with their square.
template <bool JOIN>
__device__ __forceinline__ bool plan_find(const AttentionArgs &a, const Plan &p, int64_t item, Found &f) {
    if (a.n_seq <= WAVE) {
        // Each wave for itself, a sequence to a lane: no barrier.
        const int lane = threadIdx.x & (WAVE - 1);
        Seq s = {0, 0, 0, 0, 0, 0};
        int R = 0, m = 1;
        if (lane < a.n_seq) {
            s = load_seq(a, lane);
            blocks_of(a, p, s, R, m);
        }
        uint64_t work = (uint64_t)R * m;
        if (a.n_seq > 1)
#pragma unroll
            for (int o = 1; o < WAVE; o <<= 1) work += __shfl_xor(work, o, WAVE);
        else
            work = (uint64_t)uniform((int)(work >> 32)) << 32 | (uint32_t)uniform((int)work);
        const int C = tiles_to_a_part(p, work), S = (m + C - 1) / C;
        const int all = R * S, split = S > 1 ? all : 0, mine = JOIN ? (S > 1 ? R : 0) : all;
        // (At most items and slots of the plan: they fit in 32 bits.)
        int before = wave_inclusive_scan_i32(mine) - mine;
        if (!JOIN && p.row_shift > 4 && a.n_seq > 1) {
            // The longest parts first.
            const int size = mine ? (m + S - 1) / S : 0;
            before = 0;
            for (int i = 0; i < a.n_seq; ++i) {
                const int other = __builtin_amdgcn_readlane(size, i);
                if (other > size || (other == size && i < lane)) before += __builtin_amdgcn_readlane(mine, i);
            }
        }
        const int at = (int)item - before;
        const uint64_t hit = __ballot(at >= 0 && at < mine);
        if (!hit) return false;
        const int b = __builtin_ctzll(hit);
        f.b = b;
        f.parts = __builtin_amdgcn_readlane(S, b);
        const int j = __builtin_amdgcn_readlane(at, b);
        const int blocks = __builtin_amdgcn_readlane(R, b);
        // (The blocks of one part read the same keys; the last blocks have the most.)
        f.block = JOIN ? j : blocks - 1 - j % blocks;
        f.part = JOIN ? 0 : j / blocks;
        f.slot = __builtin_amdgcn_readlane(wave_inclusive_scan_i32(split) - split, b) + f.block * f.parts;
        f.seq = Seq{__builtin_amdgcn_readlane(s.start, b), __builtin_amdgcn_readlane(s.n, b),
                    __builtin_amdgcn_readlane(s.kv, b), __builtin_amdgcn_readlane(s.len, b),
                    __builtin_amdgcn_readlane(s.before, b), __builtin_amdgcn_readlane(s.prefix, b)};
        return true;
    }
    __shared__ uint64_t part_sum[WAVES + 1];
    __shared__ int found[5];
    const int tid = threadIdx.x, lane = tid & (WAVE - 1), wave = tid / WAVE;
    int R = 0, m = 0;
    uint64_t work = 0;
    for (int b = tid; b < a.n_seq; b += THREADS) {
        blocks_of(a, p, load_seq(a, b), R, m);
        work += (uint64_t)R * m;
    }
#pragma unroll
    for (int o = WAVE / 2; o > 0; o >>= 1) work += __shfl_xor(work, o, WAVE);
    if (lane == 0) part_sum[wave] = work;
    if (tid == 0) found[0] = -1;
    __syncthreads();
    work = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) work += part_sum[w];
    const int C = tiles_to_a_part(p, work);
    uint64_t carry = 0;  // parts (or split blocks) before, in the upper half; slots before, in the lower
    for (int b0 = 0; b0 < a.n_seq; b0 += THREADS) {
        const int b = b0 + tid;
        int S = 0;
        uint64_t mine = 0;
        if (b < a.n_seq) {
            blocks_of(a, p, load_seq(a, b), R, m);
            S = (m + C - 1) / C;
            const uint32_t all = (uint32_t)R * S, split = S > 1 ? all : 0;
            mine = (uint64_t)(JOIN ? (S > 1 ? R : 0) : all) << 32 | split;
        }
        uint64_t sum = mine;
#pragma unroll
        for (int o = 1; o < WAVE; o <<= 1) {
            const uint64_t v = __shfl_up(sum, o, WAVE);
            if (lane >= o) sum += v;
        }
        __syncthreads();
        if (lane == WAVE - 1) part_sum[wave] = sum;
        __syncthreads();
        uint64_t before = carry + sum - mine;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            if (w < wave) before += part_sum[w];
            carry += part_sum[w];
        }
        const int64_t at = item - (int64_t)(before >> 32);
        if (at >= 0 && at < (int64_t)(mine >> 32)) {
            const int block = JOIN ? (int)at : R - 1 - (int)at % R;
            found[0] = b;
            found[1] = block;
            found[2] = JOIN ? 0 : (int)at / R;
            found[3] = S;
            found[4] = (int)(uint32_t)before + block * S;
        }
        __syncthreads();
        if (uniform(found[0]) >= 0) break;
    }
    f.b = uniform(found[0]);
    if (f.b < 0) return false;
    f.block = uniform(found[1]);
    f.part = uniform(found[2]);
    f.parts = uniform(found[3]);
    f.slot = uniform(found[4]);
    f.seq = load_seq(a, f.b);
    return true;
}

// A slot of the workspace: O [rows][d] over the part's own maximum, then the rows'
// maxima (in powers of two) and sums.
template <int D>
__device__ __forceinline__ float *slot_of(float *ws, const Plan &p, int hkv, int64_t slot, int h) {
    return ws + (slot * hkv + h) * ((int64_t)p.rows * (D + 2));
}

// --------------------------------------------------------------- few rows

constexpr int ROWS_KEYS = 32;  // of a tile

// K: A operand, row l % 16 a token, 8 entries from 8 (l / 16) on: 16 bytes from
// memory.  Scores: lane l has query l % 16 and tokens 4 (l / 16) + 0..3 of each
// 16.  V: the same four tokens, VE entries each; four byte permutes turn two
// times four tokens of one entry into an operand, whose 16 rows are the entries
// VE apart.  No LDS before the waves' sums are joined, no barrier: each wave keeps
// K and V of a tile (D / 2 KB) in flight while it works on the other.
//
// Measured: 64 streams of 32 heads on 8 of 128, 790 k keys: 572 us, 5.7 TB/s of the
// cache; one stream over 4097 keys, 16 heads on 2 of 256: 14.2 us with the join,
// which is launches and chains of loads (a call over one key takes 7 us).  Heads of
// 256 have 256 registers and 44 to 76 bytes of scratch a lane.
//
// The weights enter the second product as two bf16, value and remainder (16
// bits): the matrix cores have time to spare here.
template <int D, int MODE>
__global__ __launch_bounds__(THREADS, 2) void attention_rows_kernel(AttentionArgs a, Plan p, float *ws) {
    constexpr int N = ROWS_KEYS, NB = N / 16, ROWS = 16;
    constexpr int KS = D / 32;                       // steps of the first product
    constexpr int VE = D >= 128 ? 8 : 4, VU = D / (16 * VE);
    constexpr int PITCH = D + 4;
    __shared__ float o_part[WAVES][ROWS][PITCH];
    __shared__ float m_part[WAVES][ROWS], l_part[WAVES][ROWS];
    __shared__ int depth[WAVE];
    const int hk = blockIdx.x % a.cache.hkv;
    Found f;
    if (!plan_find<false>(a, p, blockIdx.x / a.cache.hkv, f)) return;
    const Seq s = uniform(f.seq);
    if (a.tree) load_depths(a, s, depth);
    const int lane = threadIdx.x & (WAVE - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / WAVE);
    const int c = lane % 16, g = lane / 16;
    const int r = a.hq / a.cache.hkv;
    const int rows = s.n * r, row0 = f.block * ROWS;  // (T * hq < 2^26)
    const int row = min(row0 + c, rows - 1);
    const int i = row / r, head = hk * r + row % r;
    const int i0 = uniform(row0 / r), i1 = uniform((min(row0 + ROWS, rows) - 1) / r);
    const Range range = tiles_of<N>(a, s, i0, i1);
    const int per = uniform((range.count + f.parts - 1) / f.parts);
    const int j_end = min(range.count, (f.part + 1) * per);
    const Query query = load_query(a, s, depth, i);
    const Cap cap(a.cap);
    const float scale2 = Cap::scale(a);
    const float slope2 = MODE == BIASED ? finite(a.slopes[head] * LOG2E) : 0.0f;

    u32x4_t q[KS];
    {
        const uint16_t *src = a.q + (int64_t)(s.start + i) * a.ldq + (int64_t)head * D + 8 * g;
#pragma unroll
        for (int k = 0; k < KS; ++k) q[k] = *reinterpret_cast<const u32x4_t *>(src + 32 * k);
    }
    f32x4_t o[VU * VE];
#pragma unroll
    for (int n = 0; n < VU * VE; ++n) o[n] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    float m_ref = -INFINITY, l_sum = 0.0f;

    // Where the blocks of 16 tokens of this wave's next 64 tiles lie: lane l has
    // the l-th tile's, as heads' tokens from the pool's start on (the memory's size keeps them below 2^32).
    const int32_t *table = a.cache.table + (int64_t)f.b * a.cache.max_pages;
    const int last16 = max(s.len - 1, 0) / 16;
    uint32_t block_at[NB];
    uint64_t page_ok[NB];
    auto load_pages = [&](int j) {
        const int k16 = NB * range.tile(min(j + WAVES * lane, range.count - 1));
#pragma unroll
        for (int t = 0; t < NB; ++t) {
            const int k = 16 * min(k16 + t, last16), page = k / a.cache.page;
            const int id = table[page];
            const bool ok = id >= 0 && id < a.cache.n_pages;
            page_ok[t] = __ballot(ok);
            block_at[t] = (uint32_t)((ok ? id : 0) * a.cache.hkv + hk) * a.cache.page + (k - page * a.cache.page);
        }
    };
    typedef __attribute__((ext_vector_type(VE / 2))) uint32_t vload_t;
    u32x4_t kr[NB][KS];
    vload_t vr[NB][4][VU];
    auto block = [&](int u, int t) { return (int64_t)(uint32_t)__builtin_amdgcn_readlane(block_at[t], u) * D; };
    auto load_k = [&](int at) {
#pragma unroll
        for (int t = 0; t < NB; ++t) {
            const uint16_t *src = a.cache.k + block(at, t) + c * D + 8 * g;
#pragma unroll
            for (int k = 0; k < KS; ++k) kr[t][k] = *reinterpret_cast<const u32x4_t *>(src + 32 * k);
        }
    };
    auto load_v = [&](int at) {
#pragma unroll
        for (int t = 0; t < NB; ++t) {
            const uint16_t *src = a.cache.v + block(at, t) + 4 * g * D + VE * c;
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int u = 0; u < VU; ++u)
                    vr[t][x][u] = *reinterpret_cast<const vload_t *>(src + x * D + 16 * VE * u);
        }
    };
    int j = f.part * per + wave, at = 0;
    if (j < j_end) {
        load_pages(j);
        load_k(0);
        load_v(0);
    }
    for (; j < j_end; j += WAVES) {
        const int k0 = N * range.tile(j);
        uint32_t there = 0;
#pragma unroll
        for (int t = 0; t < NB; ++t) there |= (uint32_t)(page_ok[t] >> at & 1) << t;
        f32x4_t acc[NB];
#pragma unroll
        for (int t = 0; t < NB; ++t) {
            acc[t] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int k = 0; k < KS; ++k) acc[t] = mfma16(kr[t][k], q[k], acc[t]);
        }
        // The next tile's keys (past the end the same ones again).
        const int next = j + WAVES < j_end ? j + WAVES : j;
        if (next != j && ++at == WAVE) {
            load_pages(next);
            at = 0;
        }
        load_k(at);

        const bool whole = there == (1u << NB) - 1 && sees_all<N>(a, s, i0, i1, k0);
        float sc[4 * NB];
        auto scores = [&](auto score) {
#pragma unroll
            for (int x = 0; x < 4 * NB; ++x) sc[x] = score(acc[x / 4][x % 4] * scale2);
        };
        // (Loops of their own: in one, all three ways are computed.)
        if (MODE == QUOTIENT || (MODE == BIASED && Cap::quotient(a)))
            scores([&](float v) { return cap.of_rest(cap_rest(v)); });
        else if (MODE == CAPPED || (MODE == BIASED && a.cap > 0.0f))
            scores([&](float w) { return cap.score(w); });
        else
            scores([&](float w) { return w; });
        if (MODE == BIASED)
#pragma unroll
            for (int x = 0; x < 4 * NB; ++x)
                sc[x] -= slope2 * fabsf((float)(query.pos - key_pos(a, s, depth, k0 + 16 * (x / 4) + 4 * g + x % 4)));
        uint32_t all = ~0u;  // keys of the tile that the lane's query sees
        if (!whole) {
            all = (uint32_t)seen(a, s, query, k0);
#pragma unroll
            for (int t = 0; t < NB; ++t)
                if (!(there >> t & 1)) all &= ~(0xffffu << (16 * t));
            const uint32_t bits = all >> (4 * g);
#pragma unroll
            for (int t = 0; t < NB; ++t)
#pragma unroll
                for (int x = 0; x < 4; ++x) sc[4 * t + x] = bits >> (16 * t + x) & 1 ? sc[4 * t + x] : -INFINITY;
        }
        float top = sc[0];
#pragma unroll
        for (int x = 1; x < 4 * NB; ++x) top = fmaxf(top, sc[x]);
        top = query_max<true>(top);
        top = all != 0 ? fmaxf(top, LEAST) : -INFINITY;
        const bool rise = top > m_ref + RISE;
        if (__any(rise)) {
            // (Each row by its own scores: its bits do not depend on the rows beside it.)
            const float m_new = rise ? top : m_ref;
            const float keep = rise ? __builtin_amdgcn_exp2f(m_ref - m_new) : 1.0f;
            l_sum *= keep;
#pragma unroll
            for (int n = 0; n < VU * VE; ++n) o[n] *= keep;
            m_ref = m_new;
        }
        const float m_use = m_ref == -INFINITY ? 0.0f : m_ref;
        float w[4 * NB];
#pragma unroll
        for (int x = 0; x < 4 * NB; ++x) {
            w[x] = __builtin_amdgcn_exp2f(sc[x] - m_use);
            l_sum += w[x];
        }
        if (!whole) {
            // 0 times NaN or infinity: values of keys that some row does not see are
            // cleared, and the rows that see one get NaN for it.
#pragma unroll
            for (int t = 0; t < NB; ++t)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    bool bad = false;
#pragma unroll
                    for (int u = 0; u < VU; ++u) {
                        bool b = false;
#pragma unroll
                        for (int e = 0; e < VE / 2; ++e)
                            b |= (vr[t][x][u][e] & 0x7f80u) == 0x7f80u || (vr[t][x][u][e] & 0x7f800000u) == 0x7f800000u;
                        if (b) vr[t][x][u] = vload_t(0u);
                        bad |= b;
                    }
                    // (The lanes with the same four tokens are 16 neighbours.)
                    if ((__ballot(bad) >> (16 * g) & 0xffffu) && (all >> (4 * g) >> (16 * t + x) & 1)) w[4 * t + x] = NAN;
                }
        }
#pragma unroll
        for (int y = 0; y < NB / 2; ++y) {  // 32 keys
            u32x4_t hi, lo;
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const float w0 = w[8 * y + 2 * x], w1 = w[8 * y + 2 * x + 1];
                hi[x] = pack_bf16x2(w0, w1);
                lo[x] = pack_bf16x2(w0 - __uint_as_float(hi[x] << 16), w1 - __uint_as_float(hi[x] & 0xffff0000u));
            }
#pragma unroll
            for (int u = 0; u < VU; ++u)
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    const uint32_t sel = e & 1 ? 0x07060302u : 0x05040100u;
                    u32x4_t v;
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        v[x] = __builtin_amdgcn_perm(vr[2 * y + x / 2][2 * (x & 1) + 1][u][e / 2],
                                                     vr[2 * y + x / 2][2 * (x & 1)][u][e / 2], sel);
                    o[VE * u + e] = mfma16(v, hi, o[VE * u + e]);
                    o[VE * u + e] = mfma16(v, lo, o[VE * u + e]);
                }
        }
        load_v(at);
    }

    // The waves' parts over their common maximum.
    l_sum = query_sum<true>(l_sum);
    if (g == 0) {
        m_part[wave][c] = m_ref;
        l_part[wave][c] = l_sum;
    }
#pragma unroll
    for (int u = 0; u < VU; ++u)
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int e = 0; e < VE; e += 4) {
                const float4 v = {o[VE * u + e][x], o[VE * u + e + 1][x], o[VE * u + e + 2][x], o[VE * u + e + 3][x]};
                *reinterpret_cast<float4 *>(&o_part[wave][c][16 * VE * u + VE * (4 * g + x) + e]) = v;
            }
    __syncthreads();
    const int live = min(ROWS, rows - row0);
    const bool direct = f.parts == 1;
    const int64_t slot = (int64_t)f.slot + f.part;
    if (!direct && (uint64_t)slot >= (uint64_t)p.slots) return;  // (starts that do not ascend)
    float *out = direct ? nullptr : slot_of<D>(ws, p, a.cache.hkv, slot, hk);
    for (int x = threadIdx.x; x < live * (D / 4); x += THREADS) {
        const int rr = x / (D / 4), d = 4 * (x % (D / 4));
        float top = m_part[0][rr];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) top = fmaxf(top, m_part[w][rr]);
        float sum = 0.0f;
        float4 v = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            const float mw = m_part[w][rr];
            const float k = mw == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(mw - top);
            const float4 y = *reinterpret_cast<const float4 *>(&o_part[w][rr][d]);
            sum = fmaf(k, l_part[w][rr], sum);
            v.x = fmaf(k, y.x, v.x), v.y = fmaf(k, y.y, v.y), v.z = fmaf(k, y.z, v.z), v.w = fmaf(k, y.w, v.w);
        }
        if (direct) {
            const float inv = top == -INFINITY ? 0.0f : 1.0f / sum;
            const int rw = row0 + rr;
            uint16_t *dst = a.o + (int64_t)(s.start + rw / r) * a.ldo + (int64_t)(hk * r + rw % r) * D + d;
            *reinterpret_cast<uint2 *>(dst) = uint2{pack_bf16x2(v.x * inv, v.y * inv), pack_bf16x2(v.z * inv, v.w * inv)};
        } else {
            *reinterpret_cast<float4 *>(out + rr * D + d) = v;
            if (d == 0) {
                out[ROWS * D + rr] = top;
                out[ROWS * D + ROWS + rr] = sum;
            }
        }
    }
}

// ------------------------------------------------------------------- join

// Rows of split blocks: four entries to a thread, G groups of threads share the
// parts of a row.  Bound by the latency of the parts' loads (single tokens: 64
// parts and more, G as large as a workgroup allows) or by their bytes.
template <int D, int G>
__global__ __launch_bounds__(THREADS) void attention_join_kernel(AttentionArgs a, Plan p, float *ws) {
    constexpr int TD = D / 4, ROWS = THREADS / (TD * G);
    __shared__ float4 v_part[G > 1 ? G * ROWS : 1][TD];
    __shared__ float m_part[G * ROWS], l_part[G * ROWS];
    const int groups = G > 1 ? p.join_groups : p.rows / ROWS;
    const int64_t x = blockIdx.x / a.cache.hkv;
    const int hk = blockIdx.x % a.cache.hkv;
    Found f;
    if (!plan_find<true>(a, p, x / groups, f)) return;
    const Seq s = uniform(f.seq);
    const int r = a.hq / a.cache.hkv;
    if (f.slot < 0 || (int64_t)f.slot + f.parts > p.slots) return;  // (starts that do not ascend)
    const int sub = threadIdx.x / TD, g = sub / ROWS, d = 4 * (threadIdx.x % TD);
    const int64_t stride = (int64_t)a.cache.hkv * p.rows * (D + 2);
    const float *part = slot_of<D>(ws, p, a.cache.hkv, f.slot, hk);
    const int live = min(p.rows, s.n * r - f.block * p.rows);
    for (int row0 = (int)(x % groups) * ROWS; row0 < live; row0 += groups * ROWS) {
        // (Rows behind the sequence's last are in the slots too, as whatever is there; they are not stored.)
        const int rr = row0 + sub % ROWS, row = f.block * p.rows + rr;
        const float *ms = part + p.rows * D + rr, *ls = ms + p.rows;
        float top = -INFINITY, sum = 0.0f;
        float4 v = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int i0 = g; i0 < f.parts; i0 += 8 * G) {
            // Eight parts at once (past the end the last one again, with weight 0).
            float mi[8], li[8];
            float4 y[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int i = min(i0 + u * G, f.parts - 1);
                mi[u] = ms[i * stride];
                li[u] = ls[i * stride];
                y[u] = *reinterpret_cast<const float4 *>(part + i * stride + rr * D + d);
            }
            float now = top;
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                if (i0 + u * G >= f.parts) mi[u] = -INFINITY;
                now = fmaxf(now, mi[u]);
            }
            const float keep = top == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(top - now);
            top = now;
            sum *= keep;
            v.x *= keep, v.y *= keep, v.z *= keep, v.w *= keep;
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                if (mi[u] == -INFINITY) continue;
                const float k = __builtin_amdgcn_exp2f(mi[u] - top);
                sum = fmaf(k, li[u], sum);
                v.x = fmaf(k, y[u].x, v.x), v.y = fmaf(k, y[u].y, v.y);
                v.z = fmaf(k, y[u].z, v.z), v.w = fmaf(k, y[u].w, v.w);
            }
        }
        if (G > 1) {
            __syncthreads();
            if (d == 0) {
                m_part[sub] = top;
                l_part[sub] = sum;
            }
            v_part[sub][d / 4] = v;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < G; ++i) top = fmaxf(top, m_part[sub % ROWS + i * ROWS]);
            sum = 0.0f;
            v = float4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < G; ++i) {
                const float mi = m_part[sub % ROWS + i * ROWS];
                const float k = mi == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(mi - top);
                const float4 y = v_part[sub % ROWS + i * ROWS][d / 4];
                sum = fmaf(k, l_part[sub % ROWS + i * ROWS], sum);
                v.x = fmaf(k, y.x, v.x), v.y = fmaf(k, y.y, v.y), v.z = fmaf(k, y.z, v.z), v.w = fmaf(k, y.w, v.w);
            }
        }
        if (g > 0 || rr >= live) continue;
        const float inv = top == -INFINITY ? 0.0f : 1.0f / sum;
        uint16_t *dst = a.o + (int64_t)(s.start + row / r) * a.ldo + (int64_t)(hk * r + row % r) * D + d;
        *reinterpret_cast<uint2 *>(dst) = uint2{pack_bf16x2(v.x * inv, v.y * inv), pack_bf16x2(v.z * inv, v.w * inv)};
    }
}

// -------------------------------------------------------------- more rows

constexpr int TILE_ROWS = 128;
__host__ __device__ constexpr int tile_keys(int d) { return d <= 128 ? 64 : 32; }

// This wave's vector-memory (LDS) operations are done; the fences keep memory
// operations from moving over the waits.
#define FENCE() asm volatile("" ::: "memory")
__device__ __forceinline__ void wait_loads() {
    FENCE();
    __builtin_amdgcn_s_waitcnt((0x7 << 4) | (0xf << 8));  // vmcnt(0)
    FENCE();
}
__device__ __forceinline__ void wait_lds() {
    FENCE();
    __builtin_amdgcn_s_waitcnt(0xf | (0x3 << 14) | (0x7 << 4));  // lgkmcnt(0)
    FENCE();
}
__device__ __forceinline__ void lds_barrier() {
    FENCE();
    __builtin_amdgcn_s_barrier();
    FENCE();
}

// Four 16-bit entries at p and those of the 15 lanes beside it as a 16 x 4 block,
// transposed: lane l % 16 gets column l % 16 of four rows.
__device__ __forceinline__ u32x2_t read_transposed(const u32x4_t *lds, int byte) {
    typedef __attribute__((address_space(3))) s16x4_t lds_s16x4;
    const auto *p = reinterpret_cast<const char *>(lds) + byte;
    return __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(lds_void *)p));
}

// K: A operand of 32 x 32 x 16, row l % 32 a key.  Scores: lane l has query l % 32
// and of each 8 keys 4 (l / 32) + 0..3.  V: transposed reads bring those four keys
// of one entry to a lane.
//
// Tiles come by direct loads to LDS, two buffers, each an array of its own (so
// that the compiler sees that loads into one and reads of another do not meet);
// one barrier a tile: behind it the tile is there and the other buffer is free.
// 16-byte chunks of a row are permuted by the row number (the source address
// carries it), so that reads spread over the banks.
//
// Measured: a prompt of 8192, 32 heads on 8 of 128: 560 us, 980 TFLOP/s of what is
// seen, the matrix units busy 51 % of the time (64 keys a tile or 32, and priority for
// the products, change 3 %); with a window of 1024 184 us, with slopes 789 us (144
// bytes of scratch a lane: the three ways to a score have loops of their own).
//
// Of heads of 256 a workgroup has half of the entries of o (and reads that half of
// V): with all of them a wave has 512 registers, is alone on its SIMD and waits
// for LDS (pieces of long prompts 2.05 ms; so 1.57 ms, 590 TFLOP/s with a cap of 50, and
// 1.35 ms without one); the first product, cap and exponentials are done twice.
//
// The weights are rounded to bf16 for the second product (half a step, 2^-8 of a
// weight, random over the keys); their sum is that of the unrounded ones.
template <int D, int MODE>
__global__ __launch_bounds__(THREADS, 2) void attention_tile_kernel(AttentionArgs a, Plan p, float *ws) {
    constexpr int DO = D < 128 ? D : 128, HALVES = D / DO;
    constexpr int N = tile_keys(D), CH = D / 8, CV = DO / 8, KT = N / 32, DS = D / 16, DT = DO / 32, NB = N / 16;
    constexpr int LOADS = N * CH / THREADS, V_LOADS = N * CV / THREADS;
    __shared__ u32x4_t k_a[N * CH], k_b[N * CH], v_a[N * CV], v_b[N * CV];
    __shared__ uint32_t bad_a[2], bad_b[2];
    __shared__ int depth[WAVE];
    const int hk = blockIdx.x % a.cache.hkv;
    const int d0 = HALVES == 1 ? 0 : (int)(blockIdx.x / a.cache.hkv) % HALVES * DO;  // the first of its entries of o
    Found f;
    if (!plan_find<false>(a, p, blockIdx.x / a.cache.hkv / HALVES, f)) return;
    const Seq s = uniform(f.seq);
    if (a.tree) load_depths(a, s, depth);
    const int tid = threadIdx.x, lane = tid & (WAVE - 1), wave = __builtin_amdgcn_readfirstlane(tid / WAVE);
    const int c = lane % 32, hh = lane / 32;
    const int r = a.hq / a.cache.hkv;
    const int rows = s.n * r, row0 = f.block * TILE_ROWS;
    const int my_row = row0 + wave * 32 + c, row = min(my_row, rows - 1);
    const int i = row / r, head = hk * r + row % r;
    const int i0 = uniform(row0 / r), i1 = uniform((min(row0 + TILE_ROWS, rows) - 1) / r);
    const Range range = tiles_of<N>(a, s, i0, i1);
    const int per = uniform((range.count + f.parts - 1) / f.parts);
    const int j0 = f.part * per, j_end = min(range.count, j0 + per);
    const Query query = load_query(a, s, depth, i);
    const bool idle = row0 + wave * 32 >= rows;  // a wave without rows brings keys for the others
    const Cap cap(a.cap);
    // (A negative scale goes to the queries' signs, so that the largest product has the largest
    // score; above 0, so that -inf stays.)
    const float scale2 = fmaxf(fabsf(Cap::scale(a)), 1e-37f);
    const float slope2 = MODE == BIASED ? finite(a.slopes[head] * LOG2E) : 0.0f;

    u32x4_t q[DS];
    {
        const uint16_t *src = a.q + (int64_t)(s.start + i) * a.ldq + (int64_t)head * D + 8 * hh;
#pragma unroll
        for (int k = 0; k < DS; ++k) {
            q[k] = *reinterpret_cast<const u32x4_t *>(src + 16 * k);
            if (a.scale < 0.0f) q[k] ^= u32x4_t{0x80008000u, 0x80008000u, 0x80008000u, 0x80008000u};
        }
    }
    f32x16_t o[DT];
#pragma unroll
    for (int n = 0; n < DT; ++n)
#pragma unroll
        for (int x = 0; x < 16; ++x) o[n][x] = 0.0f;
    float m_ref = -INFINITY, l_sum = 0.0f;

    // Where this thread's chunks of a tile come from: bytes from the first of 16 tokens on.
    uint32_t k_from[LOADS], v_from[V_LOADS];
    auto k_swizzle = [](int row) { return D == 64 ? row >> 1 & 7 : row & 15; };
    auto v_swizzle = [](int row) { return D == 64 ? (row >> 1 & 1) << 2 : (row & 3) << 2; };
#pragma unroll
    for (int x = 0; x < LOADS; ++x) {
        const int at = (wave * LOADS + x) * WAVE + lane, key = at / CH, pos = at % CH;
        k_from[x] = key % 16 * (2 * D) + 16 * (pos ^ k_swizzle(key));
    }
#pragma unroll
    for (int x = 0; x < V_LOADS; ++x) {
        const int at = (wave * V_LOADS + x) * WAVE + lane, key = at / CV, pos = at % CV;
        v_from[x] = key % 16 * (2 * D) + 16 * (pos ^ v_swizzle(key)) + 2 * d0;
    }
    // Where a lane's operands lie in a tile: K (chunks), V (bytes).
    const int k_read = c * CH;
    const int v_key = 4 * hh + lane % 16 / 4;
    const int v_read = (v_key * CV + (lane / 16 % 2) * 2 + lane % 4 / 2) * 16 + lane % 2 * 8;
    // A wave loads keys of one block of 16.  Where it lies in the next 64 tiles
    // (attention_rows_kernel), and which blocks of them are there.
    const int my_block = wave * (N / WAVES) / 16;
    const int32_t *table = a.cache.table + (int64_t)f.b * a.cache.max_pages;
    const int last16 = max(s.len - 1, 0) / 16;
    int from_tile = j0;
    uint32_t block_at = 0;
    uint64_t page_ok[NB];
    auto load_pages = [&](int j) {
        const int k16 = NB * range.tile(min(j + lane, range.count - 1));
#pragma unroll
        for (int t = 0; t < NB; ++t) {
            const int k = 16 * min(k16 + t, last16), page = k / a.cache.page;
            const int id = table[page];
            const bool ok = id >= 0 && id < a.cache.n_pages;
            page_ok[t] = __ballot(ok);
            if (t == my_block)
                block_at = (uint32_t)((ok ? id : 0) * a.cache.hkv + hk) * a.cache.page + (k - page * a.cache.page);
        }
        from_tile = j;
    };
    auto load = [&](int j, u32x4_t *kd, u32x4_t *vd) {
        const int64_t block = (int64_t)(uint32_t)__builtin_amdgcn_readlane(block_at, j - from_tile) * (2 * D);
        const char *ks = reinterpret_cast<const char *>(a.cache.k) + block;
        const char *vs = reinterpret_cast<const char *>(a.cache.v) + block;
#pragma unroll
        for (int x = 0; x < LOADS; ++x)
            __builtin_amdgcn_global_load_lds((const void *)(ks + k_from[x]),
                                             (lds_void *)(kd + (wave * LOADS + x) * WAVE), 16, 0, 0);
#pragma unroll
        for (int x = 0; x < V_LOADS; ++x)
            __builtin_amdgcn_global_load_lds((const void *)(vs + v_from[x]),
                                             (lds_void *)(vd + (wave * V_LOADS + x) * WAVE), 16, 0, 0);
    };
    auto step = [&](int j, u32x4_t *kb, u32x4_t *vb, u32x4_t *kn, u32x4_t *vn, uint32_t *bad) {
        const int k0 = N * range.tile(j);
        uint32_t there = 0;
#pragma unroll
        for (int t = 0; t < NB; ++t) there |= (uint32_t)(page_ok[t] >> (j - from_tile) & 1) << t;
        const bool whole = there == (1u << NB) - 1 && sees_all<N>(a, s, i0, i1, k0);
        if (!whole) {
            if (tid < 2) bad[tid] = 0;
            wait_lds();
        }
        wait_loads();
        lds_barrier();
        // (Past the end the last tile again, never used.)
        const int next = min(j + 1, j_end - 1);
        if (next - from_tile == WAVE) load_pages(next);
        load(next, kn, vn);
        if (!whole) {
            // 0 times NaN or infinity: values of keys that some row does not see are
            // cleared, and the rows that see one get NaN for it.
#pragma unroll
            for (int x = 0; x < V_LOADS; ++x) {
                const int at = (wave * V_LOADS + x) * WAVE + lane, key = at / CV;
                if (not_finite(vb[at])) {
                    vb[at] = u32x4_t{0, 0, 0, 0};
                    atomicOr(&bad[key / 32], 1u << key % 32);
                }
            }
            wait_lds();
            lds_barrier();
        }
        uint64_t all = ~0ull;  // keys of the tile that the lane's query sees
        if (!whole) {
            all = seen(a, s, query, k0) & below(N);
#pragma unroll
            for (int t = 0; t < NB; ++t)
                if (!(there >> t & 1)) all &= ~(0xffffull << (16 * t));
        }
        if (idle || !__any(all != 0)) return;
        // Products before the other workgroup's exponentials (3 % of a prompt's time).
        __builtin_amdgcn_s_setprio(2);
        f32x16_t sc[KT];
#pragma unroll
        for (int t = 0; t < KT; ++t) {
#pragma unroll
            for (int x = 0; x < 16; ++x) sc[t][x] = 0.0f;
            // (The upper bits of a chunk's number are not permuted: one address for all k % 8.)
#pragma unroll
            for (int k = 0; k < DS; ++k)
                sc[t] = mfma32(kb[k_read + ((2 * (k % 8) + hh) ^ k_swizzle(c)) + 16 * (k / 8) + 32 * t * CH], q[k], sc[t]);
        }
        __builtin_amdgcn_s_setprio(1);
        if (MODE == BIASED) {
            auto scores = [&](auto score) {
#pragma unroll
                for (int t = 0; t < KT; ++t)
#pragma unroll
                    for (int x = 0; x < 16; ++x) sc[t][x] = score(sc[t][x] * scale2);
            };
            if (Cap::quotient(a))  // (as in attention_rows_kernel)
                scores([&](float v) { return cap.of_rest(cap_rest(v)); });
            else if (a.cap > 0.0f)
                scores([&](float w) { return cap.score(w); });
            else
                scores([&](float w) { return w; });
            const bool drafted = a.tree && k0 + N > s.before;
            const float gap0 = (float)(query.pos - k0 - 4 * hh);
#pragma unroll
            for (int t = 0; t < KT; ++t)
#pragma unroll
                for (int x = 0; x < 16; ++x) {
                    const int key = 32 * t + 8 * (x / 4) + x % 4;
                    const float gap = drafted ? (float)(query.pos - key_pos(a, s, depth, k0 + 4 * hh + key)) : gap0 - (float)key;
                    sc[t][x] -= slope2 * fabsf(gap);
                }
        }
        if (!whole) {
#pragma unroll
            for (int t = 0; t < KT; ++t) {
                const uint32_t bits = (uint32_t)(all >> (32 * t)) >> (4 * hh), spoiled = bad[t] >> (4 * hh);
#pragma unroll
                for (int x = 0; x < 16; ++x) {
                    const int at = 8 * (x / 4) + x % 4;
                    sc[t][x] = bits >> at & 1 ? (spoiled >> at & 1 ? NAN : sc[t][x]) : -INFINITY;
                }
            }
        }
        float top = -INFINITY;
#pragma unroll
        for (int t = 0; t < KT; ++t)
#pragma unroll
            for (int x = 0; x < 16; ++x) top = fmaxf(top, sc[t][x]);
        top = query_max<false>(top);
        if (MODE == PLAIN) top *= scale2;
        // (A product of -inf that is seen is a score of -cap.)
        if (MODE == CAPPED) top = cap.score(top * scale2);
        if (MODE == QUOTIENT) top = cap.of_rest(cap_rest(top * scale2));
        top = all != 0 ? fmaxf(top, LEAST) : -INFINITY;
        const bool rise = top > m_ref + RISE;
        if (__any(rise)) {
            // (Each row by its own scores: its bits do not depend on the rows beside it.)
            const float m_new = rise ? top : m_ref;
            const float keep = rise ? __builtin_amdgcn_exp2f(m_ref - m_new) : 1.0f;
            l_sum *= keep;
#pragma unroll
            for (int n = 0; n < DT; ++n)
#pragma unroll
                for (int x = 0; x < 16; ++x) o[n][x] *= keep;
            m_ref = m_new;
        }
        const float m_use = m_ref == -INFINITY ? 0.0f : m_ref;
        if (MODE == CAPPED || MODE == QUOTIENT) {
#pragma unroll
            for (int t = 0; t < KT; ++t)
#pragma unroll
                for (int x = 0; x < 16; ++x) {
                    const float v = sc[t][x] * scale2;
                    sc[t][x] = MODE == CAPPED ? cap.score(v) : cap_rest(v);
                }
            if (!whole) {
                const float none = MODE == CAPPED ? -INFINITY : INFINITY;  // whose weight is 0
#pragma unroll
                for (int t = 0; t < KT; ++t) {
                    const uint32_t bits = (uint32_t)(all >> (32 * t)) >> (4 * hh);
#pragma unroll
                    for (int x = 0; x < 16; ++x) sc[t][x] = bits >> (8 * (x / 4) + x % 4) & 1 ? sc[t][x] : none;
                }
            }
        }
        __builtin_amdgcn_s_setprio(0);
#pragma unroll
        for (int t = 0; t < KT; ++t) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                float e[8];
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    const float v = sc[t][8 * u + x];
                    e[x] = __builtin_amdgcn_exp2f(MODE == PLAIN      ? fmaf(v, scale2, -m_use)
                                                  : MODE == QUOTIENT ? fmaf(v, -2.0f * cap.cap2, cap.cap2 - m_use)
                                                                     : v - m_use);
                    l_sum += e[x];
                }
                const u32x4_t w = {pack_bf16x2(e[0], e[1]), pack_bf16x2(e[2], e[3]), pack_bf16x2(e[4], e[5]),
                                   pack_bf16x2(e[6], e[7])};
#pragma unroll
                for (int n = 0; n < DT; ++n) {
                    const int byte = v_read + ((4 * n) ^ v_swizzle(v_key)) * 16 + (32 * t + 16 * u) * CV * 16;
                    const u32x2_t x = read_transposed(vb, byte), y = read_transposed(vb, byte + 8 * CV * 16);
                    o[n] = mfma32(u32x4_t{x[0], x[1], y[0], y[1]}, w, o[n]);
                }
            }
        }
    };
    if (j0 < j_end) {
        load_pages(j0);
        load(j0, k_a, v_a);
        int j = j0;
        for (; j + 1 < j_end; j += 2) {
            step(j, k_a, v_a, k_b, v_b, bad_a);
            step(j + 1, k_b, v_b, k_a, v_a, bad_b);
        }
        if (j < j_end) step(j, k_a, v_a, k_b, v_b, bad_a);
        wait_loads();  // (nothing comes to LDS after the end)
    }
    l_sum = query_sum<false>(l_sum);
    if (my_row >= rows) return;
    if (f.parts == 1) {
        const float inv = m_ref == -INFINITY ? 0.0f : 1.0f / l_sum;
        uint16_t *dst = a.o + (int64_t)(s.start + i) * a.ldo + (int64_t)head * D + d0 + 4 * hh;
#pragma unroll
        for (int n = 0; n < DT; ++n)
#pragma unroll
            for (int x = 0; x < 4; ++x)
                *reinterpret_cast<uint2 *>(dst + 32 * n + 8 * x) =
                    uint2{pack_bf16x2(o[n][4 * x] * inv, o[n][4 * x + 1] * inv),
                          pack_bf16x2(o[n][4 * x + 2] * inv, o[n][4 * x + 3] * inv)};
        return;
    }
    const int64_t slot = (int64_t)f.slot + f.part;
    if ((uint64_t)slot >= (uint64_t)p.slots) return;  // (starts that do not ascend)
    const int rr = wave * 32 + c;
    float *out = slot_of<D>(ws, p, a.cache.hkv, slot, hk);
#pragma unroll
    for (int n = 0; n < DT; ++n)
#pragma unroll
        for (int x = 0; x < 4; ++x)
            *reinterpret_cast<float4 *>(out + rr * D + d0 + 32 * n + 8 * x + 4 * hh) =
                float4{o[n][4 * x], o[n][4 * x + 1], o[n][4 * x + 2], o[n][4 * x + 3]};
    if (hh == 0 && d0 == 0) {
        out[TILE_ROWS * D + rr] = m_ref;
        out[TILE_ROWS * D + TILE_ROWS + rr] = l_sum;
    }
}

// ------------------------------------------------------------------ launch

// Which kernel: up to 16 rows in a sequence, on average, for the rows kernel (the
// device alone knows each sequence's; both are right for any).  Measured, rows
// / tile kernel: 16 sequences over 4096 keys, 32 heads on 8 of 128: 8 rows
// 49 / 56 us, 16 rows 54 / 55, 24 rows 64 / 56, 64 rows 110 / 61; 64 over 2000, 16
// on 2 of 256: 8 rows 57 / 91, 16 rows 63 / 92, 24 rows 105 / 93.  Not the best where one
// sequence is unlike the others: 999 single tokens and a piece of 3000 in one call take
// 901 us, apart 402 and 124.
bool few_rows(int64_t T, int n_seq, int r) { return T * r <= (int64_t)16 * n_seq; }

Plan make_plan(int64_t T, int n_seq, int hq, const Cache &c) {
    const int r = hq / c.hkv;
    Plan p;
    const bool few = few_rows(T, n_seq, r);
    p.row_shift = few ? 4 : 7;
    p.rows = 1 << p.row_shift;
    p.key_shift = (few ? ROWS_KEYS : tile_keys(c.d)) == 32 ? 5 : 6;
    // A tile to a wave; two tiles, so that the second comes while the first is worked on (a
    // tree of 16 over 2016 keys: 1 tile 19.9 us, 2 16.9, 8 28).
    p.cmin = few ? WAVES : 2;
    // Parts of all heads: what is resident at once, for single tokens twice that
    // (64 streams, 790 k keys: 512 parts 610 us, 1024 571, 2048 562; 24 streams of 1 k keys
    // 27.9, 26.6, 28.0); prompts: 256 parts 542, 512 560, 1024 575 us (8192 tokens), ragged
    // prompts of 2000 34.7, 29.5, 36.3.
    p.target_shift = 0;
    while ((2 << p.target_shift) * c.hkv <= (few ? 1024 : 512)) ++p.target_shift;
    const int target = 1 << p.target_shift;
    // Of 16 rows as many as a sequence has, on average.
    p.join_groups = few ? (int)min((int64_t)16, (T * r + n_seq - 1) / n_seq) : p.rows;
    const int64_t blocks = T * r / p.rows + min(T, (int64_t)n_seq);
    const int64_t tiles = ((int64_t)c.max_pages * c.page + (1 << p.key_shift) - 1) >> p.key_shift;
    const int64_t parts = (tiles + p.cmin - 1) / p.cmin;  // of one block, at most
    p.items = (int)min(blocks * parts, blocks + target);
    p.joins = parts > 1 ? (int)min(blocks, (int64_t)target) : 0;
    p.slots = parts > 1 ? (int)min(blocks * parts, (int64_t)2 * target) : 0;
    return p;
}

// Whether a workgroup joins one row at a time, the parts shared by its threads:
// where there are few rows.  (A tree of 16 tokens, 32 parts: 4.6 us so, 7.5 us with a row to 64 threads;
// with many rows the workgroups' own time counts, not the chain of loads.)
bool share_parts(const Plan &p, int hkv) { return p.rows == 16 || (int64_t)p.joins * hkv * p.rows <= 4096; }

template <int D, int MODE>
hipError_t launch_mode(const AttentionArgs &a, const Plan &p, float *ws, hipStream_t s) {
    const dim3 grid((unsigned)((int64_t)p.items * a.cache.hkv));
    if (p.rows == 16)
        attention_rows_kernel<D, MODE><<<grid, THREADS, 0, s>>>(a, p, ws);
    else
        attention_tile_kernel<D, MODE><<<dim3(grid.x * (D > 128 ? D / 128 : 1)), THREADS, 0, s>>>(a, p, ws);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !p.joins) return e;
    const unsigned heads = (unsigned)(p.joins * a.cache.hkv);
    if (share_parts(p, a.cache.hkv))
        attention_join_kernel<D, 1024 / D><<<dim3(heads * p.join_groups), THREADS, 0, s>>>(a, p, ws);
    else
        attention_join_kernel<D, 1><<<dim3(heads * (p.rows * D / 1024)), THREADS, 0, s>>>(a, p, ws);
    return hipGetLastError();
}

template <int D>
hipError_t launch(const AttentionArgs &a, const Plan &p, float *ws, hipStream_t s) {
    if (a.slopes) return launch_mode<D, BIASED>(a, p, ws, s);
    if (a.cap > QUOTIENT_CAP) return launch_mode<D, CAPPED>(a, p, ws, s);
    return a.cap > 0.0f ? launch_mode<D, QUOTIENT>(a, p, ws, s) : launch_mode<D, PLAIN>(a, p, ws, s);
}

}  // namespace

size_t attention_workspace_bytes(int64_t T, int n_seq, int hq, const Cache &c) {
    const Plan p = make_plan(T, n_seq, hq, c);
    return (size_t)p.slots * c.hkv * p.rows * (c.d + 2) * sizeof(float);
}

hipError_t launch_attention(const AttentionArgs &a, void *ws, hipStream_t s) {
    const Plan p = make_plan(a.T, a.n_seq, a.hq, a.cache);
    float *w = static_cast<float *>(ws);
    return a.cache.d == 64 ? launch<64>(a, p, w, s) : a.cache.d == 128 ? launch<128>(a, p, w, s) : launch<256>(a, p, w, s);
}

}  // namespace moeq4
