// Linear layer: y = act(x W^T + bias) + residual, x bf16, W int8 with one f16
// scale per 128 inputs or bf16.
//
// Both kernels feed bf16 matrix instructions with exact operands: x and bf16
// weights as they are, int8 codes converted to bf16 (8 bits hold them).  Sums
// are fp32; a group's scale enters in fp32.
//
//   linear_rows_kernel  few tokens, or too few tiles for the other: no LDS in
//       the main loop.  Bound by the weights' bytes (T small) or by what the
//       caches deliver of x and W.
//   linear_tile_kernel  many tokens: tiles staged through LDS, bound by what LDS
//       delivers to the matrix cores and, with few tiles, by the chain of steps.
#include "backbone.h"

namespace moeq4 {

namespace {

typedef __attribute__((__vector_size__(4 * sizeof(float)))) float f32x4_t;
typedef __bf16 bf16v8_t __attribute__((ext_vector_type(8)));

__device__ __forceinline__ f32x4_t mfma16(u32x4_t a, u32x4_t b, f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16v8_t, a), __builtin_bit_cast(bf16v8_t, b),
                                                   c, 0, 0, 0);
}
__device__ __forceinline__ f32x16_t mfma32(u32x4_t a, u32x4_t b, f32x16_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16v8_t, a), __builtin_bit_cast(bf16v8_t, b),
                                                   c, 0, 0, 0);
}

// Upper halves of two floats as a bf16 pair, a in the low half (exact for
// values of at most 8 significant bits).
__device__ __forceinline__ uint32_t upper_pair(float a, float b) {
    return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
}
// Code j of a dword whose codes' top bits are flipped (unsigned, 128 + q),
// times f: f u - 128 f, exact for f a power of two or 0.
__device__ __forceinline__ float code(uint32_t w, int j, float f) {
    return fmaf((float)(w >> (8 * j) & 0xffu), f, -128.0f * f);
}
// The same with f = 1.
__device__ __forceinline__ float code1(uint32_t w, int j) { return (float)(int8_t)(w >> (8 * j)); }
__device__ __forceinline__ u32x4_t codes_bf16(uint32_t lo, uint32_t hi) {
    u32x4_t r;
    r.x = upper_pair(code1(lo, 0), code1(lo, 1));
    r.y = upper_pair(code1(lo, 2), code1(lo, 3));
    r.z = upper_pair(code1(hi, 0), code1(hi, 1));
    r.w = upper_pair(code1(hi, 2), code1(hi, 3));
    return r;
}
// 8 codes (two dwords) times f, a power of two or 0, as 8 bf16 (exact).
__device__ __forceinline__ u32x4_t codes_bf16(uint32_t lo, uint32_t hi, float f) {
    lo ^= 0x80808080u;
    hi ^= 0x80808080u;
    u32x4_t r;
    r.x = upper_pair(code(lo, 0, f), code(lo, 1, f));
    r.y = upper_pair(code(lo, 2, f), code(lo, 3, f));
    r.z = upper_pair(code(hi, 0, f), code(hi, 1, f));
    r.w = upper_pair(code(hi, 2, f), code(hi, 3, f));
    return r;
}

__device__ __forceinline__ float activate(float z, int act) {
    if (act == 1) return z / (1.0f + expf(-z));
    // 1 + erf(x) = erfc(-x), which keeps its digits where erf nears -1 (4096 tokens,
    // 2048 -> 8192: 220 us, 212 with erf)
    if (act == 2) return 0.5f * z * erfcf(z * -0.70710678118654752f);
    return z;
}

// bias, activation, residual and the rounding of one output.
__device__ __forceinline__ void store_output(const LinearArgs &a, int64_t t, int n, float bias, float z) {
    z = activate(z + bias, a.act);
    if (a.residual) z += bf16_to_f32(a.residual[t * a.ldr + n]);
    if (a.y_f32)
        static_cast<float *>(a.y)[t * a.ldy + n] = z;
    else
        static_cast<uint16_t *>(a.y)[t * a.ldy + n] = f32_to_bf16_rne(z);
}

// ------------------------------------------------------------- few tokens
//
// A workgroup owns 16 MT tokens x 16 NT outputs; its waves take the inputs in
// units of 128, unit u to wave u % WAVES, and their partial sums meet in LDS
// (in wave order).  A lane loads 16 bytes of a row of W and what belongs to
// them of a row of x straight into the operands of 16x16x32 products: the
// order of the inputs within a product is free as long as both operands have
// the same, so lane group g = lane / 16 takes 16 consecutive codes and two
// products the halves of them.  Measured: one token, 4097 x 2048 bf16 (17 MB):
// 5.5 us (3.1 TB/s); 16 tokens, 12288 x 2048 int8 (26 MB): 13.3 us (2.0 TB/s),
// where each workgroup reads x (64 KB) besides 32 KB of codes.
template <bool INT8, int MT, int NT, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void linear_rows_kernel(LinearArgs a, int ntiles, int ttiles) {
    constexpr int LW = INT8 ? 2 : 4;  // 16-byte loads of a row of W per unit
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, r = lane & 15, g = lane >> 4;
    const int tt = blockIdx.x % ttiles, nt = blockIdx.x / ttiles;
    const int64_t t0 = (int64_t)tt * 16 * MT;
    const int n0 = nt * 16 * NT;
    const int K = a.K, units = (K + 127) / 128;

    const uint16_t *xp[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int64_t t = t0 + 16 * i + r;
        xp[i] = a.x + (t < a.T ? t : a.T - 1) * a.ldx;
    }
    const uint8_t *wp[NT];
    const uint16_t *sp[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        int n = n0 + 16 * j + r;
        n = n < a.N ? n : a.N - 1;
        wp[j] = static_cast<const uint8_t *>(a.q) + (int64_t)n * K * (INT8 ? 1 : 2);
        sp[j] = INT8 ? a.scale + (int64_t)n * (K / 128) : nullptr;
    }

    f32x4_t acc[MT][NT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    struct Unit {
        u32x4_t w[NT][LW], x[MT][4];
        uint16_t s[NT];
    };
    const u32x4_t zero = {0, 0, 0, 0};
    auto load = [&](int u, Unit &d) {
        const int k0 = u * 128;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
#pragma unroll
            for (int l = 0; l < LW; ++l) {
                if (INT8) {
                    d.w[j][l] = *reinterpret_cast<const u32x4_t *>(wp[j] + k0 + 64 * l + 16 * g);
                } else {
                    const int k = k0 + 32 * l + 8 * g;
                    d.w[j][l] = k < K ? *reinterpret_cast<const u32x4_t *>(wp[j] + 2 * (size_t)k) : zero;
                }
            }
            if (INT8) d.s[j] = sp[j][u];
        }
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int l = 0; l < 4; ++l) {
                const int k = INT8 ? k0 + 64 * (l >> 1) + 16 * g + 8 * (l & 1) : k0 + 32 * l + 8 * g;
                d.x[i][l] = INT8 || k < K ? *reinterpret_cast<const u32x4_t *>(xp[i] + k) : zero;
            }
    };
    auto multiply = [&](const Unit &d) {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            if (INT8) {
                u32x4_t b[4];
#pragma unroll
                for (int l = 0; l < 4; ++l)
                    b[l] = (l & 1) ? codes_bf16(d.w[j][l >> 1].z, d.w[j][l >> 1].w)
                                   : codes_bf16(d.w[j][l >> 1].x, d.w[j][l >> 1].y);
                const float s = f16_to_f32(d.s[j]);
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    f32x4_t p = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int l = 0; l < 4; ++l) p = mfma16(d.x[i][l], b[l], p);
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[i][j][e] = fmaf(p[e], s, acc[i][j][e]);
                }
            } else {
#pragma unroll
                for (int l = 0; l < LW; ++l)
#pragma unroll
                    for (int i = 0; i < MT; ++i) acc[i][j] = mfma16(d.x[i][l], d.w[j][l], acc[i][j]);
            }
        }
    };
    // two units in flight
    Unit d0, d1;
    if (wave < units) load(wave, d0);
    for (int u = wave; u < units; u += 2 * WAVES) {
        if (u + WAVES < units) load(u + WAVES, d1);
        multiply(d0);
        if (u + 2 * WAVES < units) load(u + 2 * WAVES, d0);
        if (u + WAVES < units) multiply(d1);
    }

    // product of tile (i, j): token 4 g + e, output r
    constexpr int LD = 16 * NT + 1;
    __shared__ float s_part[WAVES][16 * MT * LD];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) s_part[wave][(16 * i + 4 * g + e) * LD + 16 * j + r] = acc[i][j][e];
    __syncthreads();
    for (int o = tid; o < 256 * MT * NT; o += WAVES * 64) {
        const int m = o / (16 * NT), c = o % (16 * NT), n = n0 + c;
        const int64_t t = t0 + m;
        if (t >= a.T || n >= a.N) continue;
        float z = s_part[0][m * LD + c];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) z += s_part[w][m * LD + c];
        store_output(a, t, n, a.bias ? a.bias[n] : 0.f, z);
    }
}

template <bool INT8, int MT, int NT, int WAVES>
hipError_t launch_rows(const LinearArgs &a, hipStream_t s) {
    const int ntiles = (a.N + 16 * NT - 1) / (16 * NT);
    const int64_t ttiles = (a.T + 16 * MT - 1) / (16 * MT);
    hipLaunchKernelGGL((linear_rows_kernel<INT8, MT, NT, WAVES>), dim3((unsigned)(ntiles * ttiles)), dim3(WAVES * 64),
                       0, s, a, ntiles, (int)ttiles);
    return hipGetLastError();
}

// ------------------------------------------------------------ many tokens
//
// Tiles of BM tokens x BN outputs by WM x WN x WK waves, each with a piece of
// BM / WM x BN / WN as 32x32x16 products; with WK > 1 the waves also share out
// the inputs and their sums meet in LDS at the end (small tiles: a wave with
// the whole tile needs half the LDS reads per product of a wave with a
// quarter).  A stage is 32 WK inputs: WK blocks of rows of 32 bf16 (64 bytes),
// 16-byte chunk c of row r at place c ^ (r / 2 & 3), so that the lanes of a
// read spread over the banks.  x and bf16 weights go to LDS by direct loads
// (the source address carries the swizzle); int8 codes go there the same way.
//
// Codes that several waves use are converted, LDS to LDS, once for all of
// them.  Codes that one wave uses alone (WM = 1, the small tiles) it converts
// in its registers, 1.5 instructions a code; a stage is a group then, whose
// products start from 0 and are scaled and added under the next stage's.
// Measured: 300 tokens, N = 2048, K = 4096: 23 to 25 us so, 35 us by way of LDS
// (a step costs 0.75 us however few the tiles: the chain from barrier to
// barrier, with two waves on a SIMD; bf16 19 us); its scales read by each wave
// for itself, 64 bytes a row apart, cost 6 us more.
//
// Else a group's scale s = m 2^e, 1 <= |m| < 2: 2^e goes into the converted codes
// (exact in bf16), and the sums are kept in units of the current group's m,
// i.e. multiplied by m_g / m_(g+1) between groups and by the last m at the
// end.  A zero scale has codes 0 and m = 1.
//
// A ring of four stages, each an LDS array of its own (so that the compiler
// sees that the loads into one and the reads of another do not meet): three
// stages are in flight under the products of one.  With two stages a step
// waited for a whole memory latency (128 x 128 tile, 32 steps of 64 inputs:
// 43 us).  Every step issues one stage (past the end the last one again,
// never used), so that the wait before a step is one constant count.  Past
// the row's end chunks are read from its last one and masked where they are
// used.
//
// Measured: 4096 tokens, N = 8192, K = 2048: bf16 161 us (853 TFLOP/s; torch's
// product takes 98 us), int8 195 us (705 TFLOP/s; 32% of the matrix
// units' time, half of the vector units': the conversion, 2.5 instructions a
// code, and the rescaling, one per sum and group).
constexpr int BLK = 32;   // inputs of a block
constexpr int RING = 4;
constexpr int OWN_GROUPS = 64;  // groups whose scales are in LDS at a time (OWN)

// m and 2^e of a group's scale (f16 bits).
__device__ __forceinline__ float scale_pow2(uint16_t s) {
    return __uint_as_float(__float_as_uint(f16_to_f32(s)) & 0x7f800000u);
}
__device__ __forceinline__ float scale_m(uint16_t s) {
    const uint32_t b = __float_as_uint(f16_to_f32(s));
    return (b & 0x7fffffffu) ? __uint_as_float((b & 0x807fffffu) | 0x3f800000u) : 1.0f;
}

// This wave's vector-memory operations but the n youngest, and its LDS
// operations, are done.  The fences keep loads from moving over the wait, on
// whose count it relies.
#define FENCE() asm volatile("" ::: "memory")
#define WAIT_VM(n)                                                                          \
    do {                                                                                    \
        FENCE();                                                                            \
        __builtin_amdgcn_s_waitcnt(((n) & 0xf) | (((n) >> 4) << 14) | (0x7 << 4) | (0xf << 8)); \
        FENCE();                                                                            \
    } while (0)
#define WAIT_VM_LDS(n)                                                                      \
    do {                                                                                    \
        FENCE();                                                                            \
        __builtin_amdgcn_s_waitcnt(((n) & 0xf) | (((n) >> 4) << 14) | (0x7 << 4));          \
        FENCE();                                                                            \
    } while (0)

__device__ __forceinline__ void lds_barrier() {
    FENCE();
    __builtin_amdgcn_s_barrier();
    FENCE();
}

template <bool INT8, int BM, int BN, int WM, int WN, int WK>
struct Tile {
    static constexpr int THREADS = 64 * WM * WN * WK;
    static constexpr int TM = BM / WM / 32, TN = BN / WN / 32;  // 32x32 products of a wave
    static constexpr int BK = BLK * WK;
    static constexpr int A_ITEMS = BM * 4 * WK / THREADS;  // 16-byte chunks per thread
    static constexpr int B_ITEMS = BN * (INT8 ? 2 : 4) * WK / THREADS;
    static constexpr int OPS = A_ITEMS + B_ITEMS;  // loads per stage and thread
    // codes that one wave uses alone are converted in its registers; a stage is
    // a group then
    static constexpr bool OWN = INT8 && WM == 1;
    static_assert(!OWN || WK == 4, "a stage is a group");
    static_assert(!INT8 || OWN || WK == 1, "a stage is a quarter of a group");
    static_assert(BM * 4 * WK % THREADS == 0 && BN * 2 * WK % THREADS == 0, "whole chunks");
};

template <bool INT8, int BM, int BN, int WM, int WN, int WK>
__global__ __launch_bounds__((Tile<INT8, BM, BN, WM, WN, WK>::THREADS)) void linear_tile_kernel(LinearArgs a,
                                                                                              int ntiles,
                                                                                              int ttiles) {
    using C = Tile<INT8, BM, BN, WM, WN, WK>;
    constexpr int TM = C::TM, TN = C::TN;
    constexpr bool OWN = C::OWN;
    // a slot: x, weights as bf16, codes (and, once they are converted, the m of
    // the weight rows in their place)
    constexpr int A_BYTES = WK * BM * 64, B_BYTES = OWN ? 0 : WK * BN * 64, C_BYTES = INT8 ? WK * BN * 32 : 0;
    constexpr int S_BYTES = OWN ? BN * (OWN_GROUPS / RING) * 2 : 0;
    constexpr int SLOT = A_BYTES + B_BYTES + C_BYTES + S_BYTES;
    __shared__ __align__(16) uint8_t s_0[SLOT], s_1[SLOT], s_2[SLOT], s_3[SLOT];
    // The compiler waits for all direct loads in flight before an LDS access
    // that it cannot tell to be in another array, or whose own stage's loads it
    // does not know to be done (so that the explicit waits stand before every
    // read).  It can when each stage is
    // one array (what is converted too: an array without direct loads counts
    // as any) and offsets are integers added once (no chains of pointer sums).
    auto slot_a = [&](int u) { return u == 0 ? s_0 : u == 1 ? s_1 : u == 2 ? s_2 : s_3; };
    auto slot_b = [&](int u, int at) { return slot_a(u) + (A_BYTES + at); };
    auto slot_c = [&](int u, int at) { return slot_a(u) + (A_BYTES + B_BYTES + at); };
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave % WM, wn = wave / WM % WN, wk = wave / (WM * WN);
    // neighbouring tiles on one XCD (workgroups are dealt to the 8 XCDs in
    // turn), token tiles fastest in bands of 8
    int tt, nt;
    {
        const int total = ntiles * ttiles, xcd = blockIdx.x & 7, i = blockIdx.x >> 3;
        const int big = total & 7, per = total >> 3;
        const int id = xcd * per + (xcd < big ? xcd : big) + i;
        const int band = id / (8 * ntiles), first = band * 8, rows = ttiles - first < 8 ? ttiles - first : 8;
        const int in = id - band * 8 * ntiles;
        tt = first + in % rows;
        nt = in / rows;
    }
    const int64_t t0 = (int64_t)tt * BM;
    const int n0 = nt * BN, K = a.K;
    const int steps = (K + C::BK - 1) / C::BK;

    // chunk i of this thread (i * THREADS + tid): block, row, place; byte
    // offsets of the rows from the tile's first (below 2^31: ld <= 2^22)
    const uint8_t *xb = reinterpret_cast<const uint8_t *>(a.x + t0 * a.ldx);
    uint32_t xo[C::A_ITEMS];
    int xk[C::A_ITEMS];
#pragma unroll
    for (int i = 0; i < C::A_ITEMS; ++i) {
        const int c = i * C::THREADS + tid, blk = c / (BM * 4), r = c / 4 % BM;
        xk[i] = blk * BLK + ((c & 3) ^ (r >> 1 & 3)) * 8;
        xo[i] = (uint32_t)(t0 + r < a.T ? r : (int)(a.T - 1 - t0)) * (uint32_t)a.ldx * 2;
    }
    const uint8_t *wb = static_cast<const uint8_t *>(a.q) + (int64_t)n0 * K * (INT8 ? 1 : 2);
    const uint8_t *sb = reinterpret_cast<const uint8_t *>(a.scale + (INT8 ? (int64_t)n0 * (K / 128) : 0));
    uint32_t wo[C::B_ITEMS], so[C::B_ITEMS];
    const int groups = K / 128;
    int wkk[C::B_ITEMS];
#pragma unroll
    for (int i = 0; i < C::B_ITEMS; ++i) {
        constexpr int PER_ROW = INT8 ? 2 : 4;
        const int c = i * C::THREADS + tid, blk = c / (BN * PER_ROW), r = c / PER_ROW % BN;
        const int row = n0 + r < a.N ? r : a.N - 1 - n0;
        wkk[i] = blk * BLK + (INT8 ? (c & 1) * 16 : ((c & 3) ^ (r >> 1 & 3)) * 8);
        wo[i] = (uint32_t)row * (uint32_t)K * (INT8 ? 1 : 2);
        so[i] = (uint32_t)row * (uint32_t)(K / 128) * 2;
    }
    typedef __attribute__((address_space(3))) void lds_void;
    auto load = [&](int step, int u) {
        const int k0 = (step < steps ? step : steps - 1) * C::BK;
        // (int8 rows are whole stages)
        const uint8_t *xk0 = xb + (INT8 ? 2 * (int64_t)k0 : 0), *wk0 = wb + (INT8 ? k0 : 0);
#pragma unroll
        for (int i = 0; i < C::A_ITEMS; ++i) {
            int k = INT8 ? xk[i] : k0 + xk[i];
            if (!INT8) k = k < K ? k : K - 8;
            __builtin_amdgcn_global_load_lds((const void *)(xk0 + (xo[i] + 2u * (uint32_t)k)),
                                             (lds_void *)(slot_a(u) + (i * C::THREADS + wave * 64) * 16), 16, 0,
                                             0);
        }
#pragma unroll
        for (int i = 0; i < C::B_ITEMS; ++i) {
            int k = INT8 ? wkk[i] : k0 + wkk[i];
            if (!INT8) k = k < K ? k : K - 8;
            const int at = (i * C::THREADS + wave * 64) * 16;
            __builtin_amdgcn_global_load_lds((const void *)(wk0 + (wo[i] + (INT8 ? 1u : 2u) * (uint32_t)k)),
                                             (lds_void *)(INT8 ? slot_c(u, at) : slot_b(u, at)), 16, 0, 0);
        }
    };
    // Scales of a chunk's row, eight groups at a time in registers (a load to
    // registers makes the compiler wait for every load in flight, so they come
    // once in eight groups).
    u32x4_t scale8[INT8 ? C::B_ITEMS : 1];
    auto load_scales = [&](int first) {
#pragma unroll
        for (int i = 0; i < C::B_ITEMS; ++i) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int g0 = first + 2 * j < groups ? first + 2 * j : groups - 1, g1 = g0 + 1 < groups ? g0 + 1 : g0;
                scale8[i][j] = *reinterpret_cast<const uint16_t *>(sb + (so[i] + 2u * g0)) |
                               (uint32_t)*reinterpret_cast<const uint16_t *>(sb + (so[i] + 2u * g1)) << 16;
            }
            // (waited for here, and not by every later step)
            asm volatile("" : "+v"(scale8[i]));
        }
    };
    // codes of stage `step` (each thread's own) to bf16; a stage is a quarter
    // of a group
    auto convert = [&](int step, int u) {
        int group = step >> 2;
        if ((group & 7) == 0 && (step & 3) == 0) load_scales(group);
        group = group < groups ? group : groups - 1;  // behind the row: the last scale again
        const int pair = group >> 1 & 3;
#pragma unroll
        for (int i = 0; i < C::B_ITEMS; ++i) {
            const int c = i * C::THREADS + tid, blk = c / (BN * 2), r = c / 2 % BN, p = 2 * (c & 1);
            const uint32_t lo = pair & 1 ? scale8[i].y : scale8[i].x, hi = pair & 1 ? scale8[i].w : scale8[i].z;
            const uint32_t two = pair & 2 ? hi : lo;
            const uint16_t s = (uint16_t)(group & 1 ? two >> 16 : two);
            const float f = scale_pow2(s);
            u32x4_t *own = reinterpret_cast<u32x4_t *>(slot_c(u, c * 16));
            const u32x4_t q = *own;
            const int row = (blk * BN + r) * 64, swz = r >> 1 & 3;
            *reinterpret_cast<u32x4_t *>(slot_b(u, row + (p ^ swz) * 16)) = codes_bf16(q.x, q.y, f);
            *reinterpret_cast<u32x4_t *>(slot_b(u, row + ((p + 1) ^ swz) * 16)) = codes_bf16(q.z, q.w, f);
            if (p == 0) *reinterpret_cast<float *>(own) = scale_m(s);
        }
    };

    f32x16_t acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
    const int col = lane & 31, half = lane >> 5;
    const int row_a = wm * TM * 32 + col, row_b = wn * TN * 32 + col;
    const int place = col >> 1 & 3;  // rows of a lane differ by multiples of 32
    struct Frags {
        u32x4_t a[TM], b[TN];
        uint2 c[TN];  // OWN: codes in place of b
    };
    // operands of half `kk` of the wave's block of a stage
    auto read = [&](int step, int u, int kk, Frags &f) {
        const int at = ((2 * kk + half) ^ place) * 16;
        const int oa = (wk * BM + row_a) * 64 + at, ob = (wk * BN + row_b) * 64 + at;
#pragma unroll
        for (int i = 0; i < TM; ++i) f.a[i] = *reinterpret_cast<const u32x4_t *>(slot_a(u) + (oa + i * 32 * 64));
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            if (OWN)
                f.c[j] = *reinterpret_cast<const uint2 *>(
                    slot_c(u, (wk * BN + row_b + 32 * j) * 32 + (2 * kk + half) * 8));
            else
                f.b[j] = *reinterpret_cast<const u32x4_t *>(slot_b(u, ob + j * 32 * 64));
        }
        if ((step + 1) * C::BK > K) {
            const bool in = step * C::BK + wk * BLK + (2 * kk + half) * 8 < K;
            const u32x4_t zero = {0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < TM; ++i) f.a[i] = in ? f.a[i] : zero;
#pragma unroll
            for (int j = 0; j < TN; ++j)
                if (!OWN) f.b[j] = in ? f.b[j] : zero;  // (codes are finite)
        }
    };
    auto multiply = [&](const Frags &f) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) acc[i][j] = mfma32(f.a[i], f.b[j], acc[i][j]);
    };
    // int8: the m that the sums of this lane's outputs are in units of
    float m_now[TN];
    auto read_m = [&](int u, int j) {
        return *reinterpret_cast<const float *>(slot_c(u, (wk * BN + row_b + 32 * j) * 32));
    };
    auto rescale = [&](int u) {
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            const float m = read_m(u, j), f = m_now[j] * __builtin_amdgcn_rcpf(m);  // within 1.5 ulp
            m_now[j] = m;
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int e = 0; e < 16; ++e) acc[i][j][e] *= f;
        }
    };

    // OWN: scales of groups first .. first + 63, group g in slot g % RING: a wave
    // takes one slot, 16 lanes a row
    auto store_scales = [&](int first) {
        static_assert(OWN_GROUPS / RING == 16, "lanes of a row");
        constexpr int WAVES = C::THREADS / 64;
        int l = lane;
        asm volatile("" : "+v"(l));  // (addresses formed here, not held in registers over the products)
        const int i = l & 15, r0 = wave / RING * 4 + (l >> 4);
#pragma unroll
        for (int u = 0; u < RING; ++u) {
            if (wave % RING != u) continue;
            const int g = first + i * RING + u;
#pragma unroll
            for (int it = 0; it < BN / WAVES; ++it) {
                const int r = r0 + it * WAVES, n = n0 + r < a.N ? n0 + r : a.N - 1;
                *reinterpret_cast<uint16_t *>(slot_c(u, C_BYTES + (r * 16 + i) * 2)) =
                    g < groups ? a.scale[(int64_t)n * groups + g] : 0;  // 0 for the steps behind the last
            }
        }
    };
    if constexpr (OWN) {
        // A step's products start from 0; they are scaled and summed one step
        // later, under the next products.
        f32x16_t p[2][TM][TN];
        float s_now[TN], s_last[TN];
        auto multiply_own = [&](const Frags &f, f32x16_t (&q)[TM][TN], bool first) {
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const u32x4_t b = codes_bf16(f.c[j].x, f.c[j].y);
#pragma unroll
                for (int i = 0; i < TM; ++i) {
                    f32x16_t c;
#pragma unroll
                    for (int e = 0; e < 16; ++e) c[e] = 0.f;
                    q[i][j] = mfma32(f.a[i], b, first ? c : q[i][j]);
                }
            }
        };
        auto add_last = [&](const f32x16_t (&q)[TM][TN]) {
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int i = 0; i < TM; ++i)
#pragma unroll
                    for (int e = 0; e < 16; ++e) acc[i][j][e] = fmaf(q[i][j][e], s_last[j], acc[i][j][e]);
        };
        auto read_scales = [&](int step, int u) {
#pragma unroll
            for (int j = 0; j < TN; ++j)
                s_now[j] = f16_to_f32(*reinterpret_cast<const uint16_t *>(
                    slot_c(u, C_BYTES + ((row_b + 32 * j) * 16 + step % OWN_GROUPS / RING) * 2)));
        };
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            s_last[j] = 0.f;
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int e = 0; e < 16; ++e) p[1][i][j][e] = 0.f;
        }
#pragma unroll
        for (int u = 0; u < RING; ++u) {
            load(u, u);
            FENCE();
        }
        Frags f0, f1;
        for (int base = 0; base < steps; base += RING) {
            // (every wave has read the last scales before the last barrier)
            if (base % OWN_GROUPS == 0) {
                store_scales(base);
                WAIT_VM_LDS(0);
                lds_barrier();
                if (base == 0) read(0, 0, 0, f0);
            }
#pragma unroll
            for (int u = 0; u < RING; ++u) {
                const int step = base + u;
                read(step, u, 1, f1);
                read_scales(step, u);
                multiply_own(f0, p[u & 1], true);
                add_last(p[(u + 1) & 1]);
#pragma unroll
                for (int j = 0; j < TN; ++j) s_last[j] = s_now[j];
                WAIT_VM_LDS((RING - 2) * C::OPS);
                lds_barrier();
                load(step + RING, u);
                read(step + 1, (u + 1) % RING, 0, f0);
                multiply_own(f1, p[u & 1], false);
            }
        }
        add_last(p[1]);
    } else {
        // step s: the second half's operands are read under the products of the
        // first, the next step's first half under those of the second; between
        // them stage s + 1 is waited for, and stage s + RING takes the slot that
        // every wave has read by then.  Steps behind the last one, up to a
        // multiple of RING, multiply zeros.
#pragma unroll
        for (int u = 0; u < RING; ++u) {
            load(u, u);
            FENCE();
        }
        if (INT8) {
            WAIT_VM((RING - 1) * C::OPS);
            convert(0, 0);
        }
        WAIT_VM_LDS((RING - 1) * C::OPS);
        lds_barrier();
        Frags f0, f1;
        read(0, 0, 0, f0);
        if (INT8) {
#pragma unroll
            for (int j = 0; j < TN; ++j) m_now[j] = read_m(0, j);
        }
        for (int base = 0; base < steps; base += RING) {
#pragma unroll
            for (int u = 0; u < RING; ++u) {
                const int step = base + u;
                read(step, u, 1, f1);
                if (INT8) {
                    WAIT_VM((RING - 2) * C::OPS);
                    convert(step + 1, (u + 1) % RING);
                    if (u == 0 && step > 0) rescale(u);  // a group is four stages
                }
                multiply(f0);
                WAIT_VM_LDS((RING - 2) * C::OPS);
                lds_barrier();
                load(step + RING, u);
                read(step + 1, (u + 1) % RING, 0, f0);
                multiply(f1);
            }
        }
        if (INT8) {
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int i = 0; i < TM; ++i)
#pragma unroll
                    for (int e = 0; e < 16; ++e) acc[i][j][e] *= m_now[j];
        }
    }
    WAIT_VM_LDS(0);
    lds_barrier();  // every wave is done with the slots
    // element e of a product: token 8 (e / 4) + 4 half + e % 4, output col
    if (WK == 1) {
        // through LDS, 32 tokens of the wave's outputs at a time, so that a
        // lane has one output column and a store whole rows
        constexpr int W = TN * 32, PER_SLOT = SLOT / (32 * W * 4);
        static_assert(PER_SLOT * RING >= C::THREADS / 64, "a region per wave");
        float *mine = reinterpret_cast<float *>(slot_a(wave / PER_SLOT)) + wave % PER_SLOT * 32 * W;
        constexpr int COLS = W < 64 ? W : 64;  // columns side by side in a wave
        const int c0 = lane % COLS;
#pragma unroll
        for (int i = 0; i < TM; ++i) {
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    mine[(8 * (e >> 2) + 4 * half + (e & 3)) * W + 32 * j + col] = acc[i][j][e];
            WAIT_VM_LDS(63);
            const int64_t t1 = t0 + (wm * TM + i) * 32;
            const int rows = a.T - t1 < 32 ? (int)(a.T - t1) : 32;
#pragma unroll 1
            for (int c = c0; c < W; c += COLS) {
                const int n = n0 + wn * W + c;
                if (n >= a.N) continue;
                const float bias = a.bias ? a.bias[n] : 0.f;
#pragma unroll 4
                for (int r = lane / COLS; r < rows; r += 64 / COLS) store_output(a, t1 + r, n, bias, mine[r * W + c]);
            }
            WAIT_VM_LDS(63);
        }
    } else {
        static_assert(WK == 1 || (WK == 4 && BM * BN * 4 <= A_BYTES), "one stage array holds a wave's sums");
        float *mine = reinterpret_cast<float *>(slot_a(wk));
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    mine[((wm * TM + i) * 32 + 8 * (e >> 2) + 4 * half + (e & 3)) * BN + row_b + 32 * j] = acc[i][j][e];
        WAIT_VM_LDS(0);
        lds_barrier();
        const float *p0 = reinterpret_cast<const float *>(s_0), *p1 = reinterpret_cast<const float *>(s_1),
                    *p2 = reinterpret_cast<const float *>(s_2), *p3 = reinterpret_cast<const float *>(s_3);
        for (int o = tid; o < BM * BN; o += C::THREADS) {
            const int64_t t = t0 + o / BN;
            const int n = n0 + o % BN;
            if (t < a.T && n < a.N)
                store_output(a, t, n, a.bias ? a.bias[n] : 0.f, p0[o] + p1[o] + p2[o] + p3[o]);
        }
    }
}

template <bool INT8, int BM, int BN, int WM, int WN, int WK>
hipError_t launch_tile(const LinearArgs &a, hipStream_t s) {
    const int64_t ttiles = (a.T + BM - 1) / BM, ntiles = (a.N + BN - 1) / BN;
    hipLaunchKernelGGL((linear_tile_kernel<INT8, BM, BN, WM, WN, WK>), dim3((unsigned)(ntiles * ttiles)),
                       dim3(Tile<INT8, BM, BN, WM, WN, WK>::THREADS), 0, s, a, (int)ntiles, (int)ttiles);
    return hipGetLastError();
}

// Which kernel and tile.  Measured (us, int8 / bf16, in a graph, MI355X; rows<MT,NT,WAVES>):
//   16 tokens, N = 12288, K = 2048: rows<1,1,8> 13.3 / 15.3, <1,2,8> 14.4 / 15.9, <1,4,4> 12.5 / 14.2;
//   N = 2048, K = 4096: 9.9 / 10.8, 12.6 / 14.0, 19.2 / 21.7
//   17 tokens, N = 2048, K = 4096: rows<2,1,4> 11.0 / 12.9, <2,2,4> 14.1 / 16.3, 64x32 tiles 18.6 / 12.8;
//   N = 4097, K = 2048: 9.9 / 10.4, 9.5 / 10.6, 12.6 / 9.1; N = 12288: 15.4 / 16.7, 14.5 / 16.9, 22.7 / 16.0,
//   64x64 14.6 / 13.3
//   64 tokens, N = 2048, K = 4096: rows<2,1,4> 13.6 / 16.0, <2,2,4> 17.3 / 19.3, 64x32 19.2 / 13.6;
//   N = 4097, K = 2048: 17.6 / 18.6, 15.0 / 17.1, 13.4 / 10.0; N = 12288: 34.1 / 36.3, 24.5 / 28.9, 24.8 / 18.6,
//   64x64 16.2 / 15.4
//   128 tokens, N = 2048, K = 4096: rows<2,2,4> 17.5 / 21.3, 64x32 19.5 / 13.8, 64x64 22.7 / 15.8;
//   N = 8192, K = 2048: 31.0 / 34.6, 25.0 / 18.6, 17.0 / 14.7
//   300 tokens, N = 2048, K = 4096: 64x32 35.9 / 25.3, 64x64 23.2 / 20.0, 128x128 82 / 40;
//   N = 8192, K = 2048: 64x64 43.2 / 33.2, 128x128 48.7 / 28.9
//   1000 tokens, N = 4097, K = 2048: 64x64 73 / 55, 128x128 59 / 42, 128x256 57.5 / 39.9, 256x256 85 / 64
//   4096 tokens, N = 2048, K = 4096: 128x128 117 / 88, 128x256 109 / 79, 256x256 150 / 102;
//   N = 8192, K = 2048: 248 / 184, 240 / 185, 195 / 161
// The rule: rows up to 64 tokens; then the largest tile that leaves the 256 compute
// units enough of them, and the smallest while it gives each unit one at most.  It is
// one rule for both types, by tokens and tiles alone, and not the best of the above
// everywhere: at 33 to 64 tokens tiles are 1.2 to 1.9 times as fast where N is large
// (12288: 16.2 / 15.4 against 24.5 / 28.9), and with bf16 also at N = 2048 (13.6
// against 16.0); with int8 64x64 is 11% faster at 300 tokens and N = 8192, rows 10%
// at 128 tokens and N = 2048; <1,4,4> is 6 to 7% faster at 16 tokens and N = 12288.
template <bool INT8>
hipError_t launch_any(const LinearArgs &a, hipStream_t s) {
    if (a.T <= 16) return launch_rows<INT8, 1, 1, 8>(a, s);
    if (a.T <= 64) return a.N <= 4096 ? launch_rows<INT8, 2, 1, 4>(a, s) : launch_rows<INT8, 2, 2, 4>(a, s);
    auto tiles = [&](int64_t bm, int64_t bn) { return ((a.T + bm - 1) / bm) * ((a.N + bn - 1) / bn); };
    if (tiles(256, 256) >= 400) return launch_tile<INT8, 256, 256, 2, 4, 1>(a, s);
    if (tiles(128, 256) >= 128) return launch_tile<INT8, 128, 256, 2, 4, 1>(a, s);
    if (tiles(128, 128) >= 160) return launch_tile<INT8, 128, 128, 2, 2, 1>(a, s);
    if (tiles(64, 32) <= 256) return launch_tile<INT8, 64, 32, 1, 1, 4>(a, s);
    return launch_tile<INT8, 64, 64, 1, 2, 4>(a, s);
}

}  // namespace

hipError_t launch_linear(const LinearArgs &a, hipStream_t s) {
    return a.int8 ? launch_any<true>(a, s) : launch_any<false>(a, s);
}

}  // namespace moeq4
