// C ABI of the operators beside the experts: argument checks, workspace
// layout and launches.
#include "../../include/moe_q4_backbone.h"
#include "backbone.h"

#include <cmath>

using namespace moeq4;

namespace {

// (The limits on products of sizes keep every launch below 2^32 threads.)
constexpr int64_t LD_MAX = (int64_t)1 << 22;

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int hip_status(hipError_t e) { return e == hipSuccess ? MOE_Q4_OK : MOE_Q4_ERR_HIP; }

// Rows of `width` elements at distance ld, vector loads when vec.
int check_rows(const void *p, int64_t ld, int64_t width, uintptr_t align, bool vec) {
    if (!p || !aligned(p, align) || ld < width || (vec && ld % 8)) return MOE_Q4_ERR_INVALID_ARG;
    return ld > LD_MAX ? MOE_Q4_ERR_UNSUPPORTED : MOE_Q4_OK;
}

int check_delta_shape(const moe_q4_delta_shape *sh) {
    if (!sh || sh->k_heads < 1 || sh->v_heads < 1 || sh->k_dim < 1 || sh->v_dim < 1 || sh->v_heads % sh->k_heads)
        return MOE_Q4_ERR_INVALID_ARG;
    if (sh->v_heads > 1024 || (sh->k_dim != 64 && sh->k_dim != 128) || (sh->v_dim != 64 && sh->v_dim != 128))
        return MOE_Q4_ERR_UNSUPPORTED;
    return MOE_Q4_OK;
}

// Every check of the two delta entry points but the workspace; fills a.
int delta_args(const void *q, int64_t ldq, const void *k, int64_t ldk, const void *v, int64_t ldv, const float *g,
               const float *beta, int64_t T, const int32_t *seq_start, int32_t n_seq, const int32_t *state_idx,
               int32_t n_states, const moe_q4_delta_shape *sh, float scale, int32_t norm_qk, const float *state_in,
               float *state_out, void *o, int64_t ldo, DeltaArgs &a) {
    int st = check_delta_shape(sh);
    if (st) return st;
    if (T < 0 || n_seq < 0 || n_states < 0) return MOE_Q4_ERR_INVALID_ARG;
    if (T >= (int64_t)1 << 31 || n_seq >= 1 << 20 || (int64_t)n_seq * sh->v_heads >= 1 << 21 ||
        (T / 64 + n_seq) * sh->v_heads >= 1 << 24)
        return MOE_Q4_ERR_UNSUPPORTED;
    if (n_seq == 0) return MOE_Q4_OK;
    if (!seq_start || !aligned(seq_start, 4) || !aligned(state_idx, 4) || !aligned(state_in, 16) ||
        !aligned(state_out, 16))
        return MOE_Q4_ERR_INVALID_ARG;
    if (T > 0) {
        const int64_t kw = (int64_t)sh->k_heads * sh->k_dim, vw = (int64_t)sh->v_heads * sh->v_dim;
        if ((st = check_rows(q, ldq, kw, 16, true)) || (st = check_rows(k, ldk, kw, 16, true)) ||
            (st = check_rows(v, ldv, vw, 16, true)) || (st = check_rows(o, ldo, vw, 16, true)))
            return st;
        if (!g || !beta || !aligned(g, 4) || !aligned(beta, 4)) return MOE_Q4_ERR_INVALID_ARG;
    }
    a = DeltaArgs{static_cast<const uint16_t *>(q), static_cast<const uint16_t *>(k),
                  static_cast<const uint16_t *>(v), ldq, ldk, ldv, g, beta, T, seq_start, n_seq, state_idx,
                  n_states, sh->k_heads, sh->v_heads, sh->k_dim, sh->v_dim, scale, norm_qk != 0, state_in,
                  state_out, static_cast<uint16_t *>(o), ldo};
    return MOE_Q4_OK;
}

// A cache's own fields; pointers are looked at when it is used (a size may be
// asked for before they exist).
int check_cache(const moe_q4_kv_cache *c, int32_t q_heads) {
    if (!c || c->kv_heads < 1 || c->head_dim < 1 || c->page_size < 1 || c->max_pages < 1 || c->n_pages < 1 ||
        q_heads < 1 || q_heads % c->kv_heads)
        return MOE_Q4_ERR_INVALID_ARG;
    if ((c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) || c->page_size % 16 || q_heads > 1024 ||
        c->n_pages >= (int64_t)1 << 31 || (int64_t)c->max_pages * c->page_size > (int64_t)1 << 30)
        return MOE_Q4_ERR_UNSUPPORTED;
    return MOE_Q4_OK;
}

int check_cache_pointers(const moe_q4_kv_cache *c) {
    return c->k && c->v && c->page_table && c->kv_len && aligned(c->k, 16) && aligned(c->v, 16) &&
                   aligned(c->page_table, 4) && aligned(c->kv_len, 4)
               ? MOE_Q4_OK
               : MOE_Q4_ERR_INVALID_ARG;
}

Cache cache_of(const moe_q4_kv_cache *c) {
    return Cache{c->kv_heads, c->head_dim, c->page_size, c->max_pages, c->n_pages, static_cast<uint16_t *>(c->k),
                 static_cast<uint16_t *>(c->v), c->page_table, c->kv_len};
}

bool attention_sizes(int64_t T, int32_t n_seq, int32_t q_heads, int32_t kv_heads) {
    return T < (int64_t)1 << 26 && T * q_heads < (int64_t)1 << 26 && n_seq < 1 << 20 &&
           (int64_t)n_seq * kv_heads < 1 << 22;
}

}  // namespace

extern "C" {

int moe_q4_linear(const void *x, int64_t ldx, int64_t T, const moe_q4_linear_weights *w, int32_t act,
                  const void *residual, int64_t ldr, void *y, int64_t ldy, int32_t y_dtype, moe_q4_stream stream) {
    if (!w || !w->q || !aligned(w->q, 16) || !aligned(w->bias, 4)) return MOE_Q4_ERR_INVALID_ARG;
    const int K = w->in_features, N = w->out_features;
    if (T < 0 || K < 1 || N < 1) return MOE_Q4_ERR_INVALID_ARG;
    if (w->format != MOE_Q4_LINEAR_INT8 && w->format != MOE_Q4_LINEAR_BF16) return MOE_Q4_ERR_UNSUPPORTED;
    const bool int8 = w->format == MOE_Q4_LINEAR_INT8;
    if (int8 && (!w->scale || !aligned(w->scale, 2))) return MOE_Q4_ERR_INVALID_ARG;
    if (K % (int8 ? 128 : 8) || K > 65536 || N >= 1 << 24 || T >= (int64_t)1 << 29 || T * N >= (int64_t)1 << 38)
        return MOE_Q4_ERR_UNSUPPORTED;
    if (act < MOE_Q4_ACT_NONE || act > MOE_Q4_ACT_GELU) return MOE_Q4_ERR_UNSUPPORTED;
    if (y_dtype != MOE_Q4_BF16 && y_dtype != MOE_Q4_F32) return MOE_Q4_ERR_UNSUPPORTED;
    if (T == 0) return MOE_Q4_OK;
    int st = check_rows(x, ldx, K, 16, true);
    if (!st) st = check_rows(y, ldy, N, y_dtype == MOE_Q4_F32 ? 4 : 2, false);
    if (!st && residual) st = check_rows(residual, ldr, N, 2, false);
    if (st) return st;
    if (residual == y && (y_dtype != MOE_Q4_BF16 || ldr != ldy)) return MOE_Q4_ERR_INVALID_ARG;
    const LinearArgs a{static_cast<const uint16_t *>(x), ldx, T, K, N, int8, w->q, w->scale, w->bias, act,
                       static_cast<const uint16_t *>(residual), ldr, y, ldy, y_dtype == MOE_Q4_F32};
    return hip_status(launch_linear(a, reinterpret_cast<hipStream_t>(stream)));
}

size_t moe_q4_delta_workspace_size(int64_t T, int32_t n_seq, const moe_q4_delta_shape *shape) {
    if (T <= 0 || n_seq < 1 || check_delta_shape(shape)) return 0;
    return delta_workspace_bytes(T, n_seq, shape->v_heads);
}

int moe_q4_delta_decode(const void *q, int64_t ldq, const void *k, int64_t ldk, const void *v, int64_t ldv,
                        const float *g, const float *beta, int64_t T, const int32_t *seq_start, int32_t n_seq,
                        const int32_t *state_idx, int32_t n_states, const moe_q4_delta_shape *shape, float scale,
                        int32_t norm_qk, const float *state_in, float *state_out, void *o, int64_t ldo,
                        moe_q4_stream stream) {
    DeltaArgs a;
    const int st = delta_args(q, ldq, k, ldk, v, ldv, g, beta, T, seq_start, n_seq, state_idx, n_states, shape, scale,
                              norm_qk, state_in, state_out, o, ldo, a);
    if (st || n_seq == 0) return st;
    return hip_status(launch_delta_decode(a, reinterpret_cast<hipStream_t>(stream)));
}

int moe_q4_delta_prefill(const void *q, int64_t ldq, const void *k, int64_t ldk, const void *v, int64_t ldv,
                         const float *g, const float *beta, int64_t T, const int32_t *seq_start, int32_t n_seq,
                         const int32_t *state_idx, int32_t n_states, const moe_q4_delta_shape *shape, float scale,
                         int32_t norm_qk, const float *state_in, float *state_out, void *o, int64_t ldo, void *ws,
                         size_t ws_bytes, moe_q4_stream stream) {
    DeltaArgs a;
    const int st = delta_args(q, ldq, k, ldk, v, ldv, g, beta, T, seq_start, n_seq, state_idx, n_states, shape, scale,
                              norm_qk, state_in, state_out, o, ldo, a);
    if (st || n_seq == 0) return st;
    const size_t need = moe_q4_delta_workspace_size(T, n_seq, shape);
    if (need && (!ws || ws_bytes < need)) return MOE_Q4_ERR_WORKSPACE;
    if (need && !aligned(ws, 256)) return MOE_Q4_ERR_INVALID_ARG;
    return hip_status(launch_delta_prefill(a, ws, reinterpret_cast<hipStream_t>(stream)));
}

int moe_q4_kv_append(const void *q, int64_t ldq, int32_t q_heads, const void *k, int64_t ldk, const void *v,
                     int64_t ldv, int64_t T, const int32_t *seq_start, int32_t n_seq, const moe_q4_kv_cache *cache,
                     const int32_t *positions, const float *inv_freq, int32_t rot_dim, int32_t interleaved,
                     const float *q_norm, const float *k_norm, float eps, void *q_out, int64_t ldqo,
                     moe_q4_stream stream) {
    // Without q its heads do not count.
    int st = check_cache(cache, q ? q_heads : cache ? cache->kv_heads : 0);
    if (st) return st;
    if (cache->kv_heads > 1024) return MOE_Q4_ERR_UNSUPPORTED;
    if (T < 0 || n_seq < 0 || rot_dim < 0 || rot_dim > cache->head_dim || !(eps >= 0.0f)) return MOE_Q4_ERR_INVALID_ARG;
    if (T >= 1 << 24 || n_seq >= 1 << 20 || rot_dim % 16) return MOE_Q4_ERR_UNSUPPORTED;
    if (T == 0 || n_seq == 0) return MOE_Q4_OK;
    if ((rot_dim > 0) != (inv_freq != nullptr) || !aligned(inv_freq, 4) || !aligned(positions, 4) ||
        !aligned(q_norm, 4) || !aligned(k_norm, 4) || !seq_start || !aligned(seq_start, 4))
        return MOE_Q4_ERR_INVALID_ARG;
    if ((st = check_cache_pointers(cache))) return st;
    const int64_t kw = (int64_t)cache->kv_heads * cache->head_dim, qw = (int64_t)q_heads * cache->head_dim;
    if ((st = check_rows(k, ldk, kw, 16, true)) || (st = check_rows(v, ldv, kw, 16, true))) return st;
    if (q && ((st = check_rows(q, ldq, qw, 16, true)) || (st = check_rows(q_out, ldqo, qw, 16, true)))) return st;
    if (q ? q == q_out && ldq != ldqo : q_out != nullptr || q_norm != nullptr) return MOE_Q4_ERR_INVALID_ARG;
    const AppendArgs a{static_cast<const uint16_t *>(q), static_cast<const uint16_t *>(k),
                       static_cast<const uint16_t *>(v), ldq, ldk, ldv, q ? q_heads : 0, T, seq_start, n_seq,
                       cache_of(cache), positions, inv_freq, rot_dim, interleaved != 0, q_norm, k_norm, eps,
                       static_cast<uint16_t *>(q_out), ldqo};
    return hip_status(launch_kv_append(a, reinterpret_cast<hipStream_t>(stream)));
}

size_t moe_q4_attention_workspace_size(int64_t T, int32_t n_seq, int32_t q_heads, const moe_q4_kv_cache *cache) {
    if (T <= 0 || n_seq < 1 || check_cache(cache, q_heads) || !attention_sizes(T, n_seq, q_heads, cache->kv_heads)) return 0;
    return attention_workspace_bytes(T, n_seq, q_heads, cache_of(cache));
}

int moe_q4_attention(const void *q, int64_t ldq, int32_t q_heads, int64_t T, const int32_t *seq_start, int32_t n_seq,
                     const moe_q4_kv_cache *cache, float scale, float cap, int32_t window, const float *slopes,
                     const int32_t *prefix, const uint64_t *tree, void *o, int64_t ldo, void *ws, size_t ws_bytes,
                     moe_q4_stream stream) {
    int st = check_cache(cache, q_heads);
    if (st) return st;
    if (T < 0 || n_seq < 0 || window < 0 || !(cap >= 0.0f) || !std::isfinite(cap) || !std::isfinite(scale) ||
        (tree && prefix))
        return MOE_Q4_ERR_INVALID_ARG;
    if (!attention_sizes(T, n_seq, q_heads, cache->kv_heads)) return MOE_Q4_ERR_UNSUPPORTED;
    if (T == 0 || n_seq == 0) return MOE_Q4_OK;
    if (!seq_start || !aligned(seq_start, 4) || !aligned(slopes, 4) || !aligned(prefix, 4) || !aligned(tree, 8))
        return MOE_Q4_ERR_INVALID_ARG;
    if ((st = check_cache_pointers(cache))) return st;
    const int64_t width = (int64_t)q_heads * cache->head_dim;
    if ((st = check_rows(q, ldq, width, 16, true)) || (st = check_rows(o, ldo, width, 16, true))) return st;
    if (q == o) return MOE_Q4_ERR_INVALID_ARG;
    const size_t need = moe_q4_attention_workspace_size(T, n_seq, q_heads, cache);
    if (need && (!ws || ws_bytes < need)) return MOE_Q4_ERR_WORKSPACE;
    if (need && !aligned(ws, 256)) return MOE_Q4_ERR_INVALID_ARG;
    const AttentionArgs a{static_cast<const uint16_t *>(q), ldq, q_heads, T, seq_start, n_seq, cache_of(cache), scale,
                          cap, window, slopes, prefix, tree, static_cast<uint16_t *>(o), ldo};
    return hip_status(launch_attention(a, ws, reinterpret_cast<hipStream_t>(stream)));
}

int moe_q4_add_norm(const void *x, int64_t ldx, const void *u, int64_t ldu, int32_t u_dtype, int64_t T, int32_t H,
                    const float *post_norm, const void *gate, int64_t ldg, int32_t gate_act, float scale,
                    const float *pre_norm, float eps, void *x_out, int64_t ldxo, void *y, int64_t ldy,
                    moe_q4_stream stream) {
    if (T < 0 || H < 1 || !(eps >= 0.0f) || !std::isfinite(scale)) return MOE_Q4_ERR_INVALID_ARG;
    if (H % 8 || H > 65536 || T >= 1 << 26 || T * H >= (int64_t)1 << 33) return MOE_Q4_ERR_UNSUPPORTED;
    if (u_dtype != MOE_Q4_BF16 && u_dtype != MOE_Q4_F32) return MOE_Q4_ERR_UNSUPPORTED;
    if (gate_act != MOE_Q4_ACT_NONE && gate_act != MOE_Q4_ACT_SILU && gate_act != MOE_Q4_ACT_SIGMOID)
        return MOE_Q4_ERR_UNSUPPORTED;
    if (T == 0) return MOE_Q4_OK;
    if (!x && !u) return MOE_Q4_ERR_INVALID_ARG;
    if (!u && (post_norm || gate)) return MOE_Q4_ERR_INVALID_ARG;
    if ((pre_norm != nullptr) != (y != nullptr) || (!x_out && !y)) return MOE_Q4_ERR_INVALID_ARG;
    if (!aligned(post_norm, 16) || !aligned(pre_norm, 16)) return MOE_Q4_ERR_INVALID_ARG;
    int st = MOE_Q4_OK;
    if (x) st = check_rows(x, ldx, H, 16, true);
    if (!st && u) st = check_rows(u, ldu, H, 16, true);
    if (!st && gate && ldg) st = check_rows(gate, ldg, H, 16, true);
    if (!st && gate && !ldg && !aligned(gate, 16)) st = MOE_Q4_ERR_INVALID_ARG;
    if (!st && x_out) st = check_rows(x_out, ldxo, H, 16, true);
    if (!st && y) st = check_rows(y, ldy, H, 16, true);
    if (st) return st;
    if (x_out && ((x == x_out && ldx != ldxo) || x_out == y || u == x_out || gate == x_out)) return MOE_Q4_ERR_INVALID_ARG;
    if (y && (x == y || u == y || gate == y)) return MOE_Q4_ERR_INVALID_ARG;
    const AddNormArgs a{static_cast<const uint16_t *>(x), ldx, u, ldu, u_dtype == MOE_Q4_F32, T, H, post_norm,
                        static_cast<const uint16_t *>(gate), ldg, gate_act, scale, pre_norm, eps,
                        static_cast<uint16_t *>(x_out), ldxo, static_cast<uint16_t *>(y), ldy};
    return hip_status(launch_add_norm(a, reinterpret_cast<hipStream_t>(stream)));
}

size_t moe_q4_logprobs_workspace_size(int64_t T, int64_t V, int32_t n_top) {
    if (T <= 0 || V < 1 || n_top < 0 || n_top > MOE_Q4_MAX_TOP || T >= (int64_t)1 << 31 ||
        V >= ((int64_t)1 << 31) - (1 << 16))
        return 0;
    const int segs = logprobs_segments(V);
    return segs == 1 ? 0 : (size_t)T * segs * logprobs_part_bytes(n_top);
}

int moe_q4_logprobs(const void *logits, int32_t dtype, int64_t T, int64_t V, int64_t ld, const int32_t *tokens,
                    float *logprob, float *entropy, int32_t n_top, int32_t *top_idx, float *top_logprob, void *ws,
                    size_t ws_bytes, moe_q4_stream stream) {
    if (T < 0 || V < 1 || n_top < 0 || n_top > V) return MOE_Q4_ERR_INVALID_ARG;
    if (n_top > MOE_Q4_MAX_TOP || T >= (int64_t)1 << 31 || V >= ((int64_t)1 << 31) - (1 << 16) ||
        ld >= (int64_t)1 << 40)
        return MOE_Q4_ERR_UNSUPPORTED;
    if (dtype != MOE_Q4_BF16 && dtype != MOE_Q4_F32) return MOE_Q4_ERR_UNSUPPORTED;
    if (T == 0) return MOE_Q4_OK;
    if (T * logprobs_segments(V) >= 1 << 24) return MOE_Q4_ERR_UNSUPPORTED;
    if (!logits || !aligned(logits, dtype == MOE_Q4_F32 ? 4 : 2) || ld < V) return MOE_Q4_ERR_INVALID_ARG;
    if ((tokens && !logprob) || (n_top > 0 && (!top_idx || !top_logprob))) return MOE_Q4_ERR_INVALID_ARG;
    if (!aligned(tokens, 4) || !aligned(logprob, 4) || !aligned(entropy, 4) || !aligned(top_idx, 4) ||
        !aligned(top_logprob, 4))
        return MOE_Q4_ERR_INVALID_ARG;
    const size_t need = moe_q4_logprobs_workspace_size(T, V, n_top);
    if (need && (!ws || ws_bytes < need)) return MOE_Q4_ERR_WORKSPACE;
    if (need && !aligned(ws, 16)) return MOE_Q4_ERR_INVALID_ARG;
    if (!tokens && !entropy && n_top == 0) return MOE_Q4_OK;
    const LogprobsArgs a{logits, dtype == MOE_Q4_F32, T, V, ld, tokens, logprob, entropy, n_top, top_idx, top_logprob};
    return hip_status(launch_logprobs(a, ws, reinterpret_cast<hipStream_t>(stream)));
}

}  // extern "C"
