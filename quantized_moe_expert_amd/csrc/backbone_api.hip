// C ABI of the operators beside the experts: argument checks, workspace
// layout and launches.
#include "../../include/moe_q4_backbone.h"
#include "backbone.h"

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
