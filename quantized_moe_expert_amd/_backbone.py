"""ctypes binding of include/moe_q4_backbone.h: the operators beside the experts.

Marshalling and checks only, as in ``_lib``: each call runs in the library's
HIP kernels, on torch's current HIP stream when ``stream`` is None.  Sizes and
row distances are the tensors' own, so rows may be parts of wider rows (q, k
and v of one projection's output).  bf16 tensors are torch.bfloat16, or
torch.int16 bit patterns.
"""
from __future__ import annotations

import ctypes

import torch

from . import _lib

LINEAR_INT8, LINEAR_BF16 = 0, 1
ACT_NONE, ACT_SILU, ACT_GELU = 0, 1, 2
BF16, F32 = 0, 1
MAX_TOP = 32       # MOE_Q4_MAX_TOP
LINEAR_GROUP = 128  # inputs per int8 weight scale

# every entry point declared in include/moe_q4_backbone.h
BACKBONE_EXPORTS = ("moe_q4_linear", "moe_q4_delta_workspace_size", "moe_q4_delta_decode", "moe_q4_delta_prefill",
                    "moe_q4_logprobs_workspace_size", "moe_q4_logprobs")


class LinearWeights(ctypes.Structure):
    """struct moe_q4_linear_weights"""
    _fields_ = [("in_features", ctypes.c_int32), ("out_features", ctypes.c_int32), ("format", ctypes.c_int32),
                ("q", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("bias", ctypes.c_void_p)]


class DeltaShape(ctypes.Structure):
    """struct moe_q4_delta_shape"""
    _fields_ = [("k_heads", ctypes.c_int32), ("v_heads", ctypes.c_int32), ("k_dim", ctypes.c_int32),
                ("v_dim", ctypes.c_int32)]


_ready = None


def lib() -> ctypes.CDLL:
    """The library, with this header's entry points declared."""
    global _ready
    if _ready is None:
        L = _lib.lib()
        P, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
        L.moe_q4_linear.restype = ctypes.c_int
        L.moe_q4_linear.argtypes = [P, i64, i64, ctypes.POINTER(LinearWeights), i32, P, i64, P, i64, i32, P]
        L.moe_q4_delta_workspace_size.restype = sz
        L.moe_q4_delta_workspace_size.argtypes = [i64, i32, ctypes.POINTER(DeltaShape)]
        delta = [P, i64, P, i64, P, i64, P, P, i64, P, i32, P, i32, ctypes.POINTER(DeltaShape), f32, i32, P, P, P, i64]
        L.moe_q4_delta_decode.restype = ctypes.c_int
        L.moe_q4_delta_decode.argtypes = delta + [P]
        L.moe_q4_delta_prefill.restype = ctypes.c_int
        L.moe_q4_delta_prefill.argtypes = delta + [P, sz, P]
        L.moe_q4_logprobs_workspace_size.restype = sz
        L.moe_q4_logprobs_workspace_size.argtypes = [i64, i64, i32]
        L.moe_q4_logprobs.restype = ctypes.c_int
        L.moe_q4_logprobs.argtypes = [P, i32, i64, i64, i64, P, P, P, i32, P, P, P, sz, P]
        _ready = L
    return _ready


_SIXTEEN = (torch.bfloat16, torch.int16)


_current_device = torch._C._cuda_getDevice              # torch.cuda.current_device() without its checks
_current_stream = torch._C._cuda_getCurrentRawStream    # torch.cuda.current_stream(dev).cuda_stream


def _stream(stream, dev):
    """Raw handle of a stream; None: torch's current one (read without
    building a Stream object: 0.1 us against 2.8 us, of calls of about 6 us)."""
    return _current_stream(dev) if stream is None else _lib._stream(stream)


def _device() -> int:
    if not torch.cuda.is_initialized():
        torch.cuda.init()
    return _current_device()


def _here(t, dev):
    if t.get_device() != dev:
        raise ValueError("moe_q4 takes device tensors of the current device")


def _rows(t, what, dev, shape, types=_SIXTEEN):
    """(pointer, row distance) of a tensor of shape [T, ...] whose rows are
    contiguous; the distance of a single row is its width (torch leaves that
    stride open)."""
    if t.dtype not in types or t.shape != shape:
        raise ValueError(f"{what}: expected {tuple(shape)} of {types}, got {tuple(t.shape)} of {t.dtype}")
    _here(t, dev)
    st, width = t.stride(), 1
    for d in range(len(shape) - 1, 0, -1):
        if shape[d] != 1 and st[d] != width:
            raise ValueError(f"{what}: rows must be contiguous")
        width *= shape[d]
    return t.data_ptr(), st[0] if shape[0] > 1 else width


def _flat(t, what, dev, shape, dtype):
    """Pointer of a contiguous tensor of this shape and type (None -> NULL)."""
    if t is None:
        return None
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{what}: expected contiguous {tuple(shape)} of {dtype}, got {tuple(t.shape)} of {t.dtype}")
    _here(t, dev)
    return t.data_ptr()


def _ws(ws, dev):
    if ws is None:
        return None, 0
    if not ws.is_contiguous():
        raise ValueError("workspace must be contiguous")
    _here(ws, dev)
    return ws.data_ptr(), ws.numel() * ws.element_size()


def linear_struct(q, scale=None, bias=None) -> LinearWeights:
    """struct moe_q4_linear_weights from q [N, K] (int8 with f16 scale
    [N, K / 128], or bf16) and an optional float bias [N].  The caller keeps
    the tensors alive."""
    n, k = q.shape
    int8 = q.dtype == torch.int8
    dev = q.get_device()
    if dev < 0:
        raise ValueError("moe_q4 takes device tensors")
    if not int8 and q.dtype not in _SIXTEEN:
        raise ValueError("q: expected int8 or bf16 weights")
    if int8 != (scale is not None):
        raise ValueError("scale: int8 weights need one, bf16 weights take none")
    if not q.is_contiguous():
        raise ValueError("moe_q4 takes contiguous tensors")
    sp = None
    if int8:
        if scale.dtype not in (torch.float16, torch.int16):
            raise ValueError("scale: expected f16")
        sp = _flat(scale, "scale", dev, (n, k // LINEAR_GROUP), scale.dtype)
    w = LinearWeights(k, n, LINEAR_INT8 if int8 else LINEAR_BF16, q.data_ptr(), sp,
                      _flat(bias, "bias", dev, (n,), torch.float32))
    w.device = dev
    return w


def moe_q4_linear(x, weights, y, act=ACT_NONE, residual=None, stream=None):
    """y = act(x W^T + bias) + residual: x bf16 [T, K], ``weights`` from
    linear_struct, y bf16 or float32 [T, N], residual bf16 [T, N] (may be y)."""
    dev = _device()
    T, N = x.shape[0], weights.out_features
    if getattr(weights, "device", dev) != dev:
        raise ValueError("moe_q4 takes device tensors of the current device")
    xp, ldx = _rows(x, "x", dev, (T, weights.in_features))
    f32 = y.dtype == torch.float32
    yp, ldy = _rows(y, "y", dev, (T, N), (torch.float32,) if f32 else _SIXTEEN)
    rp, ldr = (None, 0) if residual is None else _rows(residual, "residual", dev, (T, N))
    st = lib().moe_q4_linear(xp, ldx, T, weights, act, rp, ldr, yp, ldy, F32 if f32 else BF16, _stream(stream, dev))
    if st:
        raise _lib.MoeQ4Error("moe_q4_linear", st)


def delta_workspace_size(T: int, n_seq: int, k_heads: int, v_heads: int, k_dim: int, v_dim: int) -> int:
    return int(lib().moe_q4_delta_workspace_size(int(T), int(n_seq), DeltaShape(k_heads, v_heads, k_dim, v_dim)))


def _delta(name, q, k, v, g, beta, seq_start, state_idx, state_in, state_out, o, scale, norm_qk, ws, stream):
    dev = _device()
    T, hk, dk = q.shape
    _, hv, dv = v.shape
    n_seq = seq_start.numel() - 1
    if n_seq < 0:
        raise ValueError("seq_start: expected n_seq + 1 starts")
    qp, ldq = _rows(q, "q", dev, (T, hk, dk))
    kp, ldk = _rows(k, "k", dev, (T, hk, dk))
    vp, ldv = _rows(v, "v", dev, (T, hv, dv))
    op, ldo = _rows(o, "o", dev, (T, hv, dv))
    pool = state_in if state_in is not None else state_out
    n_states = 0 if pool is None else pool.shape[0]
    states = (n_states, hv, dk, dv)
    args = [qp, ldq, kp, ldk, vp, ldv, _flat(g, "g", dev, (T, hv), torch.float32),
            _flat(beta, "beta", dev, (T, hv), torch.float32), T,
            _flat(seq_start, "seq_start", dev, (n_seq + 1,), torch.int32), n_seq,
            _flat(state_idx, "state_idx", dev, (n_seq,), torch.int32), n_states, DeltaShape(hk, hv, dk, dv), scale,
            1 if norm_qk else 0, _flat(state_in, "state_in", dev, states, torch.float32),
            _flat(state_out, "state_out", dev, states, torch.float32), op, ldo]
    if ws is not False:
        args += _ws(ws, dev)
    st = getattr(lib(), name)(*args, _stream(stream, dev))
    if st:
        raise _lib.MoeQ4Error(name, st)


def moe_q4_delta_decode(q, k, v, g, beta, seq_start, state_idx, state_in, state_out, o, scale, norm_qk=False,
                        stream=None):
    """Gated delta rule, token by token: q, k bf16 [T, Hk, dk], v, o bf16
    [T, Hv, dv] (rows may lie in wider ones), g, beta float32 [T, Hv],
    seq_start int32 [n_seq + 1], state_idx int32 [n_seq] or None, state_in /
    state_out float32 [n_states, Hv, dk, dv] or None (may be the same)."""
    _delta("moe_q4_delta_decode", q, k, v, g, beta, seq_start, state_idx, state_in, state_out, o, scale, norm_qk,
           False, stream)


def moe_q4_delta_prefill(q, k, v, g, beta, seq_start, state_idx, state_in, state_out, o, scale, norm_qk=False,
                         ws=None, stream=None):
    """moe_q4_delta_decode for prompts, in chunks of tokens; ``ws``: device
    memory of delta_workspace_size bytes."""
    _delta("moe_q4_delta_prefill", q, k, v, g, beta, seq_start, state_idx, state_in, state_out, o, scale, norm_qk,
           ws, stream)


def logprobs_workspace_size(T: int, V: int, n_top: int) -> int:
    return int(lib().moe_q4_logprobs_workspace_size(int(T), int(V), int(n_top)))


def moe_q4_logprobs(logits, tokens, logprob, entropy, top_idx, top_logprob, ws, stream=None):
    """Scores of logits [T, V] (bf16 or float32, rows may lie in wider ones):
    logprob float32 [T] of tokens int32 [T] (None: not wanted), entropy float32
    [T] or None, top_idx int32 / top_logprob float32 [T, n] or None."""
    dev = _device()
    T, V = logits.shape
    f32 = logits.dtype == torch.float32
    lp, ld = _rows(logits, "logits", dev, (T, V), (torch.float32,) if f32 else _SIXTEEN)
    n = 0 if top_idx is None else top_idx.shape[1]
    wp, nb = _ws(ws, dev)
    st = lib().moe_q4_logprobs(lp, F32 if f32 else BF16, T, V, ld, _flat(tokens, "tokens", dev, (T,), torch.int32),
                               _flat(logprob, "logprob", dev, (T,), torch.float32),
                               _flat(entropy, "entropy", dev, (T,), torch.float32), n,
                               _flat(top_idx, "top_idx", dev, (T, n), torch.int32),
                               _flat(top_logprob, "top_logprob", dev, (T, n), torch.float32), wp, nb,
                               _stream(stream, dev))
    if st:
        raise _lib.MoeQ4Error("moe_q4_logprobs", st)
