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
 *   - moe_q4_kv_append, moe_q4_attention: the paged cache of the attention
 *     layers, one layer in four (drama-rs page, first paragraph: full attention
 *     every 4th layer), and the attention of prompts, single tokens and trees of
 *     drafted tokens over it;
 *   - moe_q4_add_norm: what lies between two blocks: norm of a block's output,
 *     gate, residual, norm before the next block;
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
    MOE_Q4_ACT_GELU = 2,      /* z (1 + erf(z / sqrt 2)) / 2 */
    MOE_Q4_ACT_SIGMOID = 3    /* 1 / (1 + exp(-z)): gates of moe_q4_add_norm only */
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
 *   act       moe_q4_act, but for MOE_Q4_ACT_SIGMOID
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

/*
 * Keys and values of n_seq sequences in pages of a pool.  Token i of sequence
 * b (its cache index, from 0) lies in page p = page_table[b][i / page_size],
 * at k and v [p][head][i % page_size].
 *   k, v        bf16 [n_pages][kv_heads][page_size][head_dim], 16-byte aligned
 *   page_table  int32 [n_seq][max_pages].  An entry outside [0, n_pages) is a
 *               page that is not there: its keys are seen by nobody and nothing
 *               is stored in it.  Entries behind a sequence's last token are not
 *               used.  Sequences may share pages that they only read.
 *   kv_len      int32 [n_seq]: tokens of each sequence, the call's own (the
 *               rows of seq_start) the last among them: row i of the call's n
 *               rows of sequence b has cache index kv_len[b] - n + i.  Tokens
 *               with an index below 0 or behind the table are not stored; keys
 *               behind the table are seen by nobody.
 * head_dim 64, 128 or 256; page_size a multiple of 16, max_pages * page_size
 * at most 2^30; kv_heads at most 1024.
 */
typedef struct moe_q4_kv_cache {
    int32_t kv_heads, head_dim;
    int32_t page_size;          /* tokens per page */
    int32_t max_pages;          /* entries per sequence of page_table */
    int64_t n_pages;            /* pages of the pool, below 2^31 */
    void *k, *v;
    const int32_t *page_table;
    const int32_t *kv_len;
} moe_q4_kv_cache;

/*
 * Heads of T packed tokens into the cache.  Per head of q and k, in fp32 and
 * rounded once:
 *   x <- x / sqrt(mean(x^2) + eps) * norm      (with q_norm, k_norm)
 *   the first rot_dim entries turned in pairs by position * inv_freq[j]:
 *   (a, b) <- (a cos - b sin, b cos + a sin)
 * The angle is computed in 64 bits, so that it is right for every position.
 *   q, k, v      bf16 [T] rows of [q_heads or kv_heads][head_dim] at distances
 *                ldq, ldk, ldv (16-byte aligned, distances % 8 == 0).  q may be
 *                NULL: keys and values alone.
 *   seq_start    int32 [n_seq + 1] as of moe_q4_delta_decode.  Rows behind the
 *                last sequence are not written, whatever they hold.
 *   positions    int32 [T] or NULL: a token's position is its cache index
 *   inv_freq     float [rot_dim / 2]; NULL with rot_dim = 0: no rotation.
 *                rot_dim % 16 == 0, at most head_dim.
 *   interleaved  0: pair j is entries j and j + rot_dim / 2; else 2j and 2j + 1
 *   q_norm, k_norm  float [head_dim] or NULL
 *   q_out        bf16 [T] rows of [q_heads][head_dim] at distance ldqo; may be q
 *                itself (same pointer and distance), must not overlap the inputs
 *                otherwise.
 * Two tokens of one call must not share a place in the cache (its contents would
 * be undefined).  q_heads at most 1024; T < 2^24, n_seq < 2^20.
 */
MOE_Q4_API int moe_q4_kv_append(const void *q, int64_t ldq, int32_t q_heads, const void *k, int64_t ldk,
                                const void *v, int64_t ldv, int64_t T, const int32_t *seq_start, int32_t n_seq,
                                const moe_q4_kv_cache *cache, const int32_t *positions, const float *inv_freq,
                                int32_t rot_dim, int32_t interleaved, const float *q_norm, const float *k_norm,
                                float eps, void *q_out, int64_t ldqo, moe_q4_stream stream);

/*
 * Attention of T packed query rows over the cache.  Query head h reads head
 * h * kv_heads / q_heads of the cache.  For a query and a key that it sees
 *   s = scale q . k,  then s = cap tanh(s / cap)     (cap > 0)
 *                     then s -= slopes[h] * |distance|  (with slopes)
 *   o = sum softmax(s) v
 * with scores, softmax and sums in fp32 (capping adds at most 2^-20 of the score to
 * its error, with caps up to 64 at most 2^-20 of the cap); the weights may be
 * rounded to bf16 for their products with v.  A query that sees no key gets o = 0.  The distance is
 * the query's position less the key's; positions are cache indices.  A query sees
 *   - the keys up to its own index, with window > 0 only those at a distance
 *     below window,
 *   - and the first prefix[b] keys of its sequence, wherever it stands,
 * of its own sequence alone.
 * With a tree the rows of a sequence are drafted tokens, at most 64: bit j of
 * tree[t] says that row t sees row j of its sequence (itself, as a rule, and
 * those that it follows).  Cached tokens before the rows are seen as above; a
 * row's position is the number of those plus the number of other bits of its
 * mask, and distances (window, slopes) go by it.  Rows behind the 64th of a
 * sequence are seen by nobody.  prefix must be NULL with a tree.
 *   q          bf16 [T] rows of [q_heads][head_dim] at distance ldq (as
 *              moe_q4_kv_append leaves them)
 *   seq_start  int32 [n_seq + 1] as of moe_q4_delta_decode; the keys of the rows
 *              themselves are read from the cache
 *   slopes     float [q_heads] or NULL
 *   prefix     int32 [n_seq] or NULL
 *   tree       uint64 [T], 8-byte aligned, or NULL
 *   o          bf16 [T] rows of [q_heads][head_dim] at distance ldo; must not
 *              overlap the inputs.  (q and o 16-byte aligned, distances % 8 == 0)
 *   ws         >= moe_q4_attention_workspace_size(T, n_seq, q_heads, cache)
 *              bytes, 256-byte aligned (may be NULL when that is 0)
 * scale, cap and the slopes must be finite, cap and window at least 0; q_heads a
 * multiple of kv_heads, at most 1024; T * q_heads < 2^26, n_seq < 2^20, n_seq * kv_heads < 2^22.
 * Rows behind the last sequence are neither read nor written.  Parts of a row's
 * keys are joined in a fixed order: the same input gives the same bits.  A NaN in
 * a query makes its outputs NaN; one in a key or value reaches the queries that see
 * it (some or all of a head's outputs are NaN) and no others.  Infinities go by the
 * formula: a score of inf gives NaN; one of -inf has weight 0, and where a query
 * sees no other the outputs are NaN; a capped score is cap or -cap.  An infinite
 * value makes outputs of the queries that see it infinite or NaN.
 */
MOE_Q4_API size_t moe_q4_attention_workspace_size(int64_t T, int32_t n_seq, int32_t q_heads,
                                                  const moe_q4_kv_cache *cache);
MOE_Q4_API int moe_q4_attention(const void *q, int64_t ldq, int32_t q_heads, int64_t T, const int32_t *seq_start,
                                int32_t n_seq, const moe_q4_kv_cache *cache, float scale, float cap, int32_t window,
                                const float *slopes, const int32_t *prefix, const uint64_t *tree, void *o, int64_t ldo,
                                void *ws, size_t ws_bytes, moe_q4_stream stream);

/*
 * Between two blocks, over T rows of H values, in fp32:
 *   r = u, then r = r / sqrt(mean(r^2) + eps) * post_norm   (with post_norm)
 *          then r = r * act(gate)                           (with gate)
 *   x_out = x + scale r                                     (rounded to bf16)
 *   y     = x_out / sqrt(mean(x_out^2) + eps) * pre_norm    (with pre_norm; of the rounded x_out)
 *   x          bf16 rows at distance ldx, or NULL: nothing is added (x_out = scale r)
 *   u          bf16 or float (u_dtype) rows at distance ldu (the experts' float
 *              output, a linear layer's), or NULL: a plain norm of x (x_out = x; post_norm
 *              and gate must be NULL)
 *   gate       bf16 rows at distance ldg, or NULL; ldg = 0: one row for all tokens
 *   gate_act   MOE_Q4_ACT_NONE, MOE_Q4_ACT_SILU or MOE_Q4_ACT_SIGMOID
 *   post_norm, pre_norm  float [H], 16-byte aligned, or NULL
 *   x_out      bf16 rows at distance ldxo, or NULL: not wanted (pre_norm is given);
 *              may be x itself (same pointer and distance)
 *   y          bf16 rows at distance ldy (with pre_norm)
 * Rows are 16-byte aligned with distances % 8 == 0; H % 8 == 0, H <= 65536;
 * T < 2^26, T * H < 2^33.  The outputs must not overlap each other or, but for x_out,
 * the inputs; u, gate and x may be the same memory.
 */
MOE_Q4_API int moe_q4_add_norm(const void *x, int64_t ldx, const void *u, int64_t ldu, int32_t u_dtype, int64_t T,
                               int32_t H, const float *post_norm, const void *gate, int64_t ldg, int32_t gate_act,
                               float scale, const float *pre_norm, float eps, void *x_out, int64_t ldxo, void *y,
                               int64_t ldy, moe_q4_stream stream);

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
