"""Convenience wrappers: buffers for a plain gated delta rule mixer and a plain
attention mixer.

A fused q | k | v projection, the gated delta rule and an output projection
added to the stream, one after another.  Allocates the buffers and the
workspace once (torch device memory) and calls the C ABI; the computation
itself is the library's.

The first is the rule between its two linears and nothing else.  The backbone's own
gated DeltaNet layers have more around it, which the library does not offer:
a short causal convolution and SiLU behind the input projection, a gated norm
before the output projection, and g and beta computed from the stream.  A layer
with those makes the three calls itself, with its own steps between.
"""
from __future__ import annotations

import torch

from . import _backbone


class DeltaMixer:
    """x + W_out delta(W_in x) for batches of up to ``max_tokens`` tokens of up
    to ``max_seqs`` sequences.

    ``w_in``: linear_struct of the fused projection, outputs q [k_heads,
    k_dim] | k [k_heads, k_dim] | v [v_heads, v_dim]; ``w_out``: linear_struct
    from [v_heads, v_dim] back to the stream.  The structs' tensors are the
    caller's to keep.  q and k are normalised per head; scale 1 / sqrt(k_dim).
    ``mode``: "decode" (token by token) or "prefill" (chunks of 64 tokens).

    The buffers are the mixer's, one set for all of its calls: a call must be
    ordered after the one before, so that streams or threads that run at the
    same time need a mixer each (they may share the weights).
    """

    def __init__(self, w_in, w_out, k_heads: int, v_heads: int, k_dim: int, v_dim: int, max_tokens: int,
                 max_seqs: int = 1, mode: str = "decode", device="cuda"):
        if mode not in ("decode", "prefill"):
            raise ValueError("mode must be 'decode' or 'prefill'")
        if w_in.out_features != 2 * k_heads * k_dim + v_heads * v_dim:
            raise ValueError("w_in must have 2 k_heads k_dim + v_heads v_dim outputs")
        if w_out.in_features != v_heads * v_dim or w_out.out_features != w_in.in_features:
            raise ValueError("w_out must take v_heads v_dim inputs back to w_in's")
        self.w_in, self.w_out, self.mode = w_in, w_out, mode
        self.heads = (k_heads, v_heads, k_dim, v_dim)
        self.max_tokens, self.max_seqs = max_tokens, max_seqs
        self.rows = torch.empty((max_tokens, w_in.out_features), dtype=torch.bfloat16, device=device)
        self.o = torch.empty((max_tokens, v_heads, v_dim), dtype=torch.bfloat16, device=device)
        self.ws = None
        if mode == "prefill":
            need = _backbone.delta_workspace_size(max_tokens, max_seqs, *self.heads)
            self.ws = torch.empty(need, dtype=torch.uint8, device=device)

    def forward(self, x, g, beta, seq_start, state_in, state_out, y, state_idx=None):
        """y (bf16 [T, hidden], may be x) = x + mixer(x).  g, beta, seq_start
        and the states as moe_q4_delta_decode.  Every one of the T rows must
        belong to a sequence: one that only fills up the batch is a sequence of
        its own whose ``state_idx`` is -1 (no state is read or written)."""
        T = x.shape[0]
        if T > self.max_tokens or seq_start.numel() - 1 > self.max_seqs:
            raise ValueError(f"{T} tokens of {seq_start.numel() - 1} sequences do not fit in the buffers")
        hk, hv, dk, dv = self.heads
        rows, o = self.rows[:T], self.o[:T]
        _backbone.moe_q4_linear(x, self.w_in, rows)
        q = rows[:, :hk * dk].unflatten(1, (hk, dk))
        k = rows[:, hk * dk:2 * hk * dk].unflatten(1, (hk, dk))
        v = rows[:, 2 * hk * dk:].unflatten(1, (hv, dv))
        args = (q, k, v, g, beta, seq_start, state_idx, state_in, state_out, o, dk ** -0.5, True)
        if self.mode == "decode":
            _backbone.moe_q4_delta_decode(*args)
        else:
            _backbone.moe_q4_delta_prefill(*args, self.ws)
        _backbone.moe_q4_linear(o.flatten(1), self.w_out, y, residual=x)
        return y


class AttentionMixer:
    """residual + W_out attention(W_in x) over a paged cache, for batches of up
    to ``max_tokens`` tokens of up to ``max_seqs`` sequences.

    ``w_in``: linear_struct of the fused projection, outputs q [q_heads,
    head_dim] | k [kv_heads, head_dim] | v [kv_heads, head_dim]; ``w_out``:
    linear_struct from [q_heads, head_dim] back to the stream.  ``cache``: the
    kv_cache_struct whose keys and values are this layer's.  ``inv_freq``,
    ``q_norm``, ``k_norm``, ``interleaved``: as moe_q4_kv_append; ``cap``,
    ``window``, ``slopes``: as moe_q4_attention; scale 1 / sqrt(head_dim).  The
    tensors are the caller's to keep.  No gate on the attention's output.

    The buffers are the mixer's, one set for all of its calls: a call must be
    ordered after the one before, so that streams or threads that run at the
    same time need a mixer each (they may share the weights).
    """

    def __init__(self, w_in, w_out, q_heads: int, cache, max_tokens: int, max_seqs: int = 1, inv_freq=None, q_norm=None,
                 k_norm=None, interleaved=False, cap=0.0, window=0, slopes=None, device="cuda"):
        hkv, d = cache.kv_heads, cache.head_dim
        if w_in.out_features != (q_heads + 2 * hkv) * d:
            raise ValueError("w_in must have (q_heads + 2 kv_heads) head_dim outputs")
        if w_out.in_features != q_heads * d or w_out.out_features != w_in.in_features:
            raise ValueError("w_out must take q_heads head_dim inputs back to w_in's")
        if q_heads % hkv:
            raise ValueError("q_heads must be a multiple of the cache's heads")
        self.w_in, self.w_out, self.cache = w_in, w_out, cache
        self.heads = (q_heads, hkv, d)
        self.max_tokens, self.max_seqs = max_tokens, max_seqs
        self.turn = (inv_freq, q_norm, k_norm, interleaved)
        self.cap, self.window, self.slopes = cap, window, slopes
        self.rows = torch.empty((max_tokens, w_in.out_features), dtype=torch.bfloat16, device=device)
        self.o = torch.empty((max_tokens, q_heads, d), dtype=torch.bfloat16, device=device)
        # The size grows with the tokens, for few and for more rows in a sequence.
        few = 16 * hkv // q_heads
        need = max(_backbone.attention_workspace_size(t, n, q_heads, cache)
                   for n in range(1, max_seqs + 1) for t in (max_tokens, min(max_tokens, few * n)) if t)
        self.ws = torch.empty(need, dtype=torch.uint8, device=device)

    def forward(self, x, seq_start, y, positions=None, prefix=None, tree=None, residual=None):
        """y (bf16 [T, hidden], may be x or residual) = residual + mixer(x); None:
        x itself.  The batch's sequences are the cache's first seq_start.numel()
        - 1.  Its kv_len counts the T rows already; their keys and values are stored
        by the call.  ``positions`` are the rotation's (drafted tokens: their depth,
        not their place in the cache).  Every one of the T rows must belong to a
        sequence: one that only fills up the batch is a sequence of its own whose
        kv_len is 0."""
        T = x.shape[0]
        if T > self.max_tokens or seq_start.numel() - 1 > self.max_seqs:
            raise ValueError(f"{T} tokens of {seq_start.numel() - 1} sequences do not fit in the buffers")
        hq, hkv, d = self.heads
        rows, o = self.rows[:T], self.o[:T]
        _backbone.moe_q4_linear(x, self.w_in, rows)
        q = rows[:, :hq * d].unflatten(1, (hq, d))
        k = rows[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
        v = rows[:, (hq + hkv) * d:].unflatten(1, (hkv, d))
        inv_freq, q_norm, k_norm, interleaved = self.turn
        _backbone.moe_q4_kv_append(q, k, v, seq_start, self.cache, q, inv_freq, positions, q_norm, k_norm,
                                   interleaved=interleaved)
        _backbone.moe_q4_attention(q, seq_start, self.cache, o, d ** -0.5, self.ws, self.cap, self.window, self.slopes,
                                   prefix, tree)
        _backbone.moe_q4_linear(o.flatten(1), self.w_out, y, residual=x if residual is None else residual)
        return y
