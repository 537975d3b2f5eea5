"""Convenience wrapper: buffers for a plain gated delta rule mixer.

A fused q | k | v projection, the gated delta rule and an output projection
added to the stream, one after another.  Allocates the buffers and the
workspace once (torch device memory) and calls the C ABI; the computation
itself is the library's.

This is the rule between its two linears and nothing else.  The backbone's own
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
