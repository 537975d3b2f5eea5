// Internal launch interface of the operators beside the experts
// (include/moe_q4_backbone.h): backbone_api.hip checks and calls these.
#pragma once

#include "moe_internal.h"

namespace moeq4 {

struct LinearArgs {
    const uint16_t *x;
    int64_t ldx;
    int64_t T;
    int K, N;
    bool int8;
    const void *q;
    const uint16_t *scale;
    const float *bias;
    int act;
    const uint16_t *residual;  // bf16 or null
    int64_t ldr;
    void *y;
    int64_t ldy;
    bool y_f32;
};
hipError_t launch_linear(const LinearArgs &a, hipStream_t s);

struct DeltaArgs {
    const uint16_t *q, *k, *v;
    int64_t ldq, ldk, ldv;
    const float *g, *beta;
    int64_t T;
    const int32_t *seq_start;
    int n_seq;
    const int32_t *state_idx;
    int n_states;
    int hk, hv, dk, dv;
    float scale;
    bool norm;
    const float *s_in;
    float *s_out;
    uint16_t *o;
    int64_t ldo;
};
hipError_t launch_delta_decode(const DeltaArgs &a, hipStream_t s);
size_t delta_workspace_bytes(int64_t T, int n_seq, int hv);
hipError_t launch_delta_prefill(const DeltaArgs &a, void *ws, hipStream_t s);

struct Cache {
    int hkv, d, page, max_pages;
    int64_t n_pages;
    uint16_t *k, *v;
    const int32_t *table, *kv_len;
};
struct AppendArgs {
    const uint16_t *q, *k, *v;
    int64_t ldq, ldk, ldv;
    int hq;
    int64_t T;
    const int32_t *seq_start;
    int n_seq;
    Cache cache;
    const int32_t *positions;
    const float *inv_freq;
    int rot;
    bool interleaved;
    const float *q_norm, *k_norm;
    float eps;
    uint16_t *q_out;
    int64_t ldqo;
};
hipError_t launch_kv_append(const AppendArgs &a, hipStream_t s);

struct AttentionArgs {
    const uint16_t *q;
    int64_t ldq;
    int hq;
    int64_t T;
    const int32_t *seq_start;
    int n_seq;
    Cache cache;
    float scale, cap;
    int window;
    const float *slopes;
    const int32_t *prefix;
    const uint64_t *tree;
    uint16_t *o;
    int64_t ldo;
};
size_t attention_workspace_bytes(int64_t T, int n_seq, int hq, const Cache &c);
hipError_t launch_attention(const AttentionArgs &a, void *ws, hipStream_t s);

struct AddNormArgs {
    const uint16_t *x;
    int64_t ldx;
    const void *u;
    int64_t ldu;
    bool u_f32;
    int64_t T;
    int H;
    const float *post;
    const uint16_t *gate;
    int64_t ldg;
    int act;
    float scale;
    const float *pre;
    float eps;
    uint16_t *x_out;
    int64_t ldxo;
    uint16_t *y;
    int64_t ldy;
};
hipError_t launch_add_norm(const AddNormArgs &a, hipStream_t s);

struct LogprobsArgs {
    const void *logits;
    bool f32;
    int64_t T, V, ld;
    const int32_t *tokens;
    float *logprob, *entropy;
    int n_top;
    int32_t *top_idx;
    float *top_logprob;
};
// Segments of a row; rows of more than one need ws: T * segments parts.
int logprobs_segments(int64_t V);
size_t logprobs_part_bytes(int n_top);
hipError_t launch_logprobs(const LogprobsArgs &a, void *ws, hipStream_t s);

}  // namespace moeq4
