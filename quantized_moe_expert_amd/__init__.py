"""MI355X-native routed int4 MoE expert layer (HIP kernels behind a C ABI).

The library (``libmoe_q4.so``, built from ``csrc/`` by ``build.py``) computes
router logits and top-k gates, groups token rows by expert, runs the int4
SwiGLU experts (fused-dequant GEMVs for decode, matrix-core grouped GEMMs for
prefill), the gate-weighted combine and the int8 shared expert.  This package is its thin Python
binding: ``_lib`` mirrors the C entry points, ``layer`` holds buffers;
``_backbone`` mirrors the entry points beside the experts (linear layers, the
gated delta rule, attention over a paged cache, norms between blocks, token
scores).
"""
from ._lib import (ASYM_G64, SYM_G128, FP8_B128, NVFP4, WS_DECODE, WS_GROUP, WS_PREFILL, WS_ROUTE, EXPORTS, MoeQ4Error,
                   error_string, layer_struct, lib, moe_q4_decode, moe_q4_dequant, moe_q4_group,
                   moe_q4_prefill, moe_q4_residual_bf16, moe_q4_route, workspace_size,
                   moe_q4_decode_timed, moe_q4_prefill_timed, STAGE_EVENTS, WS_FORWARD, moe_q4_forward,
                   moe_q4_forward_timed, moe_q4_workspace_init, WS_SHARED, SharedExpert, shared_struct,
                   moe_q4_shared, moe_q4_dequant_int8, moe_q4_forward_ex, moe_q4_shared_timed,
                   moe_q4_prefill_pack_size, moe_q4_prefill_pack, prefill_pack,
                   moe_q4_forward_noalloc, NOALLOC_SCRATCH_BYTES, moe_q4_forward_det, WS_FORWARD_DET,
                   FRAME_MAX_LANES, frame_workspace_size, moe_q4_frame)
from ._backbone import (ACT_GELU, ACT_NONE, ACT_SIGMOID, ACT_SILU, BACKBONE_EXPORTS, LINEAR_BF16, LINEAR_INT8, MAX_TOP,
                        DeltaShape, KVCache, LinearWeights, attention_workspace_size, delta_workspace_size,
                        kv_cache_struct, linear_struct, logprobs_workspace_size, moe_q4_add_norm, moe_q4_attention,
                        moe_q4_delta_decode, moe_q4_delta_prefill, moe_q4_kv_append, moe_q4_linear, moe_q4_logprobs)
from .layer import MoeQ4Layer
from .mixer import AttentionMixer, DeltaMixer

__all__ = ["ASYM_G64", "SYM_G128", "FP8_B128", "NVFP4", "WS_DECODE", "WS_GROUP", "WS_PREFILL", "WS_ROUTE", "EXPORTS", "MoeQ4Error",
           "error_string", "layer_struct", "lib", "moe_q4_decode", "moe_q4_dequant", "moe_q4_group",
           "moe_q4_prefill", "moe_q4_residual_bf16", "moe_q4_route", "workspace_size", "MoeQ4Layer",
           "moe_q4_decode_timed", "moe_q4_prefill_timed", "STAGE_EVENTS", "WS_FORWARD", "moe_q4_forward",
           "moe_q4_forward_timed", "moe_q4_workspace_init", "WS_SHARED", "SharedExpert", "shared_struct",
           "moe_q4_shared", "moe_q4_dequant_int8", "moe_q4_forward_ex", "moe_q4_shared_timed",
           "moe_q4_prefill_pack_size", "moe_q4_prefill_pack", "prefill_pack",
           "moe_q4_forward_noalloc", "NOALLOC_SCRATCH_BYTES", "moe_q4_forward_det", "WS_FORWARD_DET",
           "FRAME_MAX_LANES", "frame_workspace_size", "moe_q4_frame",
           "ACT_GELU", "ACT_NONE", "ACT_SILU", "BACKBONE_EXPORTS", "LINEAR_BF16", "LINEAR_INT8", "MAX_TOP", "DeltaShape",
           "LinearWeights", "delta_workspace_size", "linear_struct", "logprobs_workspace_size",
           "moe_q4_delta_decode", "moe_q4_delta_prefill", "moe_q4_linear", "moe_q4_logprobs", "DeltaMixer",
           "ACT_SIGMOID", "KVCache", "attention_workspace_size", "kv_cache_struct", "moe_q4_add_norm", "moe_q4_attention",
           "moe_q4_kv_append", "AttentionMixer"]
