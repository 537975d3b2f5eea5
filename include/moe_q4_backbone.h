/*
 * moe_q4_backbone.h -- C ABI of libmoe_q4.so, continued: the operators beside
 * the experts in a backbone layer on AMD Instinct MI355X (gfx950).
 *
 *   - moe_q4_linear: the int8 linears around the mixers (drama-q4 card,
 *     "What's quantized": attention / DeltaNet / shared expert linears int8,
 *     symmetric, group 128) and the bf16 output head, with bias, activation
 *     and residual;
 *   - moe_q4_delta_decode, moe_q4_delta_prefill: the gated delta rule, the
 *     mixer of three layers in four (drama-rs page, first paragraph and
 *     "Layout": gated DeltaNet);
 *   - moe_q4_logprobs: log probabilities of given tokens, entropy and the most
 *     likely tokens from the head's logits.
 *
 * The conventions are those of moe_q4.h: device pointers owned by the caller,
 * work enqueued on `stream` with nothing synchronised or allocated, every
 * argument checked on the host before the first launch, moe_q4_status codes.
 * Every call may be captured into a HIP graph; calls that share a workspace
 * must be ordered.  The stream must belong to the current device, and the
 * pointers to memory that this device can reach.
 *
 * Rows: a `ld*` argument is the distance between two tokens' rows in
 * elements, so that rows may be parts of wider ones (q, k and v of one
 * projection's output).  Leading dimensions are at most 2^22.
 */
#ifndef MOE_Q4_BACKBONE_H
#define MOE_Q4_BACKBONE_H

#include "moe_q4.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    MOE_Q4_BF16 = 0,
    MOE_Q4_F32 = 1
} moe_q4_dtype;

typedef enum {
    MOE_Q4_LINEAR_INT8 = 0,   /* w = scale * q, q the signed byte, one f16 scale per 128 inputs */
    MOE_Q4_LINEAR_BF16 = 1
} moe_q4_linear_format;

typedef enum {
    MOE_Q4_ACT_NONE = 0,
    MOE_Q4_ACT_SILU = 1,      /* z / (1 + exp(-z)) */
    MOE_Q4_ACT_GELU = 2       /* z (1 + erf(z / sqrt 2)) / 2 */
} moe_q4_act;

/*
 * Weights of a linear layer with K inputs and N outputs:
 *   q      int8 [N][K] or bf16 [N][K], 16-byte aligned
 *   scale  f16 bit patterns [N][K/128], 2-byte aligned (int8; NULL for bf16).
 *          Scales must be finite.
 *   bias   float [N] or NULL
 * int8 needs K % 128 == 0, bf16 K % 8 == 0; K <= 65536, N <= 2^22 (a row of y).
 */
typedef struct moe_q4_linear_weights {
    int32_t in_features;    /* K */
    int32_t out_features;   /* N */
    int32_t format;         /* moe_q4_linear_format */
    const void *q;
    const uint16_t *scale;
    const float *bias;
} moe_q4_linear_weights;

/*
 * Linear layer:
 *   y[t][n] = act(sum_k x[t][k] w[n][k] + bias[n]) + residual[t][n],
 * sums in fp32, one rounding at the end.  The products of the int8 codes (and
 * of the bf16 weights) with x are exact; a group's scale multiplies its
 * partial sum.
 *   x         bf16 [T] rows of K at distance ldx (16-byte aligned, ldx % 8 == 0)
 *   act       moe_q4_act
 *   residual  bf16 [T] rows of N at distance ldr, or NULL; may be y itself
 *             (same pointer and distance, y_dtype MOE_Q4_BF16)
 *   y         bf16 or float (y_dtype) [T] rows of N at distance ldy; must not
 *             overlap the inputs otherwise
 * T < 2^29, T * N < 2^38.
 */
MOE_Q4_API int moe_q4_linear(const void *x, int64_t ldx, int64_t T, const moe_q4_linear_weights *w, int32_t act,
                             const void *residual, int64_t ldr, void *y, int64_t ldy, int32_t y_dtype,
                             moe_q4_stream stream);

/*
 * Heads of a gated delta rule: each of the v_heads value heads has a state of
 * k_dim x v_dim floats and reads key head h * k_heads / v_heads.  k_dim and
 * v_dim: 64 or 128; v_heads a multiple of k_heads, at most 1024.
 */
typedef struct moe_q4_delta_shape {
    int32_t k_heads, v_heads, k_dim, v_dim;
} moe_q4_delta_shape;

/*
 * Gated delta rule over n_seq packed sequences.  Per value head, token by
 * token, from the sequence's initial state S (k_dim x v_dim):
 *   S <- exp(g) S
 *   u  = beta (v - S^T k)
 *   S <- S + k u^T
 *   o  = scale S^T q
 * with k and q divided by sqrt(sum of squares + 1e-6) first when norm_qk != 0.
 * States and sums are fp32, o is rounded once to bf16.
 *   q, k       bf16 [T] rows of [k_heads][k_dim] at distances ldq, ldk
 *   v          bf16 [T] rows of [v_heads][v_dim] at distance ldv
 *              (all 16-byte aligned, distances % 8 == 0)
 *   g, beta    float [T][v_heads]; g is the log decay (at most 0)
 *   seq_start  int32 [n_seq + 1]: sequence b is rows seq_start[b] ..
 *              seq_start[b + 1] - 1, ascending from 0, the last at most T
 *              (clamped, so malformed starts give undefined numbers but stay
 *              in bounds).  Rows behind the last sequence are neither read nor
 *              written.
 *   state_idx  int32 [n_seq] or NULL: sequence b's entry of the state
 *              arrays, b itself when NULL.  A sequence whose entry lies
 *              outside [0, n_states) starts from a zero state and its final
 *              state is dropped.  Two sequences must not share an entry (their
 *              numbers would be undefined).
 *   state_in   float [n_states][v_heads][k_dim][v_dim], 16-byte aligned, or
 *              NULL: every sequence starts from a zero state
 *   state_out  the same layout, or NULL: final states are dropped.  May be
 *              state_in itself; otherwise the two must not overlap.  A
 *              sequence without tokens hands its initial state on.  Entries
 *              that no sequence names are left as they were.
 *   o          bf16 [T] rows of [v_heads][v_dim] at distance ldo, 16-byte
 *              aligned, ldo % 8 == 0; must not overlap the inputs
 * n_seq = 0 returns MOE_Q4_OK without launching anything.  With T = 0 the row
 * pointers may be NULL.  T < 2^31, n_seq < 2^20, n_seq * v_heads < 2^21,
 * (T / 64 + n_seq) * v_heads < 2^24.
 *
 * moe_q4_delta_decode takes the tokens of a sequence one after another (tuned
 * for a few tokens per sequence); moe_q4_delta_prefill takes them in chunks of
 * 64 on the matrix cores (tuned for prompts) and needs
 *   ws  >= moe_q4_delta_workspace_size(T, n_seq, shape) bytes, 256-byte aligned.
 * The operands of prefill's products hold 22 bits of every value down to 2^-16 of
 * the largest beside it (in a column of the state, or of a chunk's values and
 * updates) and steps of 2^-39 of that one below; decode works in fp32.
 * A NaN or an infinity in a token's inputs makes the outputs of its sequence
 * from that token on (prefill: from its chunk on) undefined numbers.
 */
MOE_Q4_API size_t moe_q4_delta_workspace_size(int64_t T, int32_t n_seq, const moe_q4_delta_shape *shape);
MOE_Q4_API int moe_q4_delta_decode(const void *q, int64_t ldq, const void *k, int64_t ldk, const void *v,
                                   int64_t ldv, const float *g, const float *beta, int64_t T,
                                   const int32_t *seq_start, int32_t n_seq, const int32_t *state_idx,
                                   int32_t n_states, const moe_q4_delta_shape *shape, float scale, int32_t norm_qk,
                                   const float *state_in, float *state_out, void *o, int64_t ldo,
                                   moe_q4_stream stream);
MOE_Q4_API int moe_q4_delta_prefill(const void *q, int64_t ldq, const void *k, int64_t ldk, const void *v,
                                    int64_t ldv, const float *g, const float *beta, int64_t T,
                                    const int32_t *seq_start, int32_t n_seq, const int32_t *state_idx,
                                    int32_t n_states, const moe_q4_delta_shape *shape, float scale, int32_t norm_qk,
                                    const float *state_in, float *state_out, void *o, int64_t ldo, void *ws,
                                    size_t ws_bytes, moe_q4_stream stream);

#define MOE_Q4_MAX_TOP 32
/*
 * Scores of T rows of V logits, with p = softmax(row):
 *   logits       bf16 or float (dtype) [T] rows of V at distance ld, aligned
 *                to their element; any values: -inf (and NaN, which counts as
 *                -inf) has probability 0; a row whose logits are all -inf
 *                gives logprob and top_logprob -inf and entropy 0; the
 *                probability of a row with +inf is shared by its +inf entries
 *   tokens       int32 [T] or NULL
 *   logprob      float [T] out (with tokens): log p[tokens[t]]; 0 for a token
 *                outside [0, V) (a position that is not scored)
 *   entropy      float [T] out or NULL: -sum p log p
 *   n_top        0 .. MOE_Q4_MAX_TOP, at most V
 *   top_idx      int32 [T][n_top] out (n_top > 0): the n_top largest logits,
 *                descending, equal logits ordered by lower index
 *   top_logprob  float [T][n_top] out (n_top > 0): their log p
 *   ws           >= moe_q4_logprobs_workspace_size(T, V, n_top) bytes,
 *                16-byte aligned (may be NULL when that is 0)
 * T * ceil(V / 8192) < 2^24, V < 2^31 - 2^16, ld < 2^40.  Sums are fp32, each over one part of a
 * row, joined in a fixed order: the same input gives the same bits.
 */
MOE_Q4_API size_t moe_q4_logprobs_workspace_size(int64_t T, int64_t V, int32_t n_top);
MOE_Q4_API int moe_q4_logprobs(const void *logits, int32_t dtype, int64_t T, int64_t V, int64_t ld,
                               const int32_t *tokens, float *logprob, float *entropy, int32_t n_top,
                               int32_t *top_idx, float *top_logprob, void *ws, size_t ws_bytes,
                               moe_q4_stream stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_Q4_BACKBONE_H */
