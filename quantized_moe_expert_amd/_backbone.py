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
ACT_NONE, ACT_SILU, ACT_GELU, ACT_SIGMOID = 0, 1, 2, 3
BF16, F32 = 0, 1
MAX_TOP = 32       # MOE_Q4_MAX_TOP
LINEAR_GROUP = 128  # inputs per int8 weight scale

# every entry point declared in include/moe_q4_backbone.h
BACKBONE_EXPORTS = ("moe_q4_linear", "moe_q4_delta_workspace_size", "moe_q4_delta_decode", "moe_q4_delta_prefill",
                    "moe_q4_kv_append", "moe_q4_attention_workspace_size", "moe_q4_attention", "moe_q4_add_norm",
                    "moe_q4_logprobs_workspace_size", "moe_q4_logprobs")


class LinearWeights(ctypes.Structure):
    """struct moe_q4_linear_weights"""
    _fields_ = [("in_features", ctypes.c_int32), ("out_features", ctypes.c_int32), ("format", ctypes.c_int32),
                ("q", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("bias", ctypes.c_void_p)]


class DeltaShape(ctypes.Structure):
    """struct moe_q4_delta_shape"""
    _fields_ = [("k_heads", ctypes.c_int32), ("v_heads", ctypes.c_int32), ("k_dim", ctypes.c_int32),
                ("v_dim", ctypes.c_int32)]


class KVCache(ctypes.Structure):
    """struct moe_q4_kv_cache; kv_cache_struct makes those that calls take"""
    device, n_seq = None, 0
    _fields_ = [("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("n_pages", ctypes.c_int64), ("k", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("page_table", ctypes.c_void_p), ("kv_len", ctypes.c_void_p)]


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
        cache = ctypes.POINTER(KVCache)
        L.moe_q4_kv_append.restype = ctypes.c_int
        L.moe_q4_kv_append.argtypes = [P, i64, i32, P, i64, P, i64, i64, P, i32, cache, P, P, i32, i32, P, P, f32, P,
                                       i64, P]
        L.moe_q4_attention_workspace_size.restype = sz
        L.moe_q4_attention_workspace_size.argtypes = [i64, i32, i32, cache]
        L.moe_q4_attention.restype = ctypes.c_int
        L.moe_q4_attention.argtypes = [P, i64, i32, i64, P, i32, cache, f32, f32, i32, P, P, P, P, i64, P, sz, P]
        L.moe_q4_add_norm.restype = ctypes.c_int
        L.moe_q4_add_norm.argtypes = [P, i64, P, i64, i32, i64, i32, P, P, i64, i32, f32, P, f32, P, i64, P, i64, P]
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
    if t.get_device() != dev:
        raise ValueError("moe_q4 takes device tensors of the current device")
    if t.is_contiguous():
        return t.data_ptr(), shape[1] if len(shape) == 2 else shape[1] * shape[2]
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
    if t.get_device() != dev:
        raise ValueError("moe_q4 takes device tensors of the current device")
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


def kv_cache_struct(k, v, page_table, kv_len) -> KVCache:
    """struct moe_q4_kv_cache from the pool's pages k, v bf16 [n_pages,
    kv_heads, page_size, head_dim], page_table int32 [n_seq, max_pages] and
    kv_len int32 [n_seq].  A call may have the first of these sequences alone:
    the length of its seq_start says how many.  The caller keeps the tensors
    alive; their contents are read when a call runs."""
    dev = k.get_device()
    if dev < 0:
        raise ValueError("moe_q4 takes device tensors")
    if k.dim() != 4 or k.dtype not in _SIXTEEN:
        raise ValueError("k: expected bf16 pages [n_pages, kv_heads, page_size, head_dim]")
    if page_table.dim() != 2:
        raise ValueError("page_table: expected [n_seq, max_pages]")
    n_pages, heads, page, d = k.shape
    n_seq, cols = page_table.shape
    c = KVCache(heads, d, page, cols, n_pages, _flat(k, "k", dev, k.shape, k.dtype),
                _flat(v, "v", dev, k.shape, k.dtype), _flat(page_table, "page_table", dev, (n_seq, cols), torch.int32),
                _flat(kv_len, "kv_len", dev, (n_seq,), torch.int32))
    c.device, c.n_seq = dev, n_seq
    return c


def _cached(cache, seq_start, dev):
    """(pointer, n_seq) of the starts of the cache's sequences, or of the first
    of them."""
    if cache.device is None:
        raise ValueError("cache: expected one of kv_cache_struct")
    if cache.device != dev:
        raise ValueError("moe_q4 takes device tensors of the current device")
    n_seq = cache.n_seq if seq_start is None else seq_start.numel() - 1
    if n_seq != cache.n_seq and not 1 <= n_seq < cache.n_seq:
        raise ValueError(f"seq_start: expected the starts of up to {cache.n_seq} sequences and an end, got {n_seq + 1}")
    return _flat(seq_start, "seq_start", dev, (n_seq + 1,), torch.int32), n_seq


def moe_q4_kv_append(q, k, v, seq_start, cache, q_out, inv_freq=None, positions=None, q_norm=None, k_norm=None,
                     eps=1e-6, interleaved=False, stream=None):
    """q bf16 [T, Hq, d] (or None), k, v bf16 [T, Hkv, d] (rows may lie in
    wider ones): heads of q and k normed (q_norm, k_norm float32 [d]) and
    turned by position * inv_freq (float32 [rot / 2]; positions int32 [T],
    None: the cache index), q into q_out (may be q), k and v into the cache of
    kv_cache_struct behind the tokens that it has of their sequences."""
    dev = _device()
    start, n_seq = _cached(cache, seq_start, dev)
    T, d = k.shape[0], cache.head_dim
    kv = (T, cache.kv_heads, d)
    kp, ldk = _rows(k, "k", dev, kv)
    vp, ldv = _rows(v, "v", dev, kv)
    qp, ldq, op, ldo, hq = None, 0, None, 0, 0
    if q is not None:
        hq = q.shape[1]
        qp, ldq = _rows(q, "q", dev, (T, hq, d))
        op, ldo = _rows(q_out, "q_out", dev, (T, hq, d))
    elif q_out is not None:
        raise ValueError("q_out: without q there is none")
    rot = 0 if inv_freq is None else 2 * inv_freq.numel()
    st = lib().moe_q4_kv_append(qp, ldq, hq, kp, ldk, vp, ldv, T, start, n_seq, cache,
                                _flat(positions, "positions", dev, (T,), torch.int32),
                                _flat(inv_freq, "inv_freq", dev, (rot // 2,), torch.float32), rot,
                                1 if interleaved else 0, _flat(q_norm, "q_norm", dev, (d,), torch.float32),
                                _flat(k_norm, "k_norm", dev, (d,), torch.float32), eps, op, ldo, _stream(stream, dev))
    if st:
        raise _lib.MoeQ4Error("moe_q4_kv_append", st)


def attention_workspace_size(T: int, n_seq: int, q_heads: int, cache) -> int:
    return int(lib().moe_q4_attention_workspace_size(int(T), int(n_seq), int(q_heads), cache))


def moe_q4_attention(q, seq_start, cache, o, scale, ws=None, cap=0.0, window=0, slopes=None, prefix=None, tree=None,
                     stream=None):
    """Attention of q, o bf16 [T, Hq, d] (rows may lie in wider ones) over the
    cache of kv_cache_struct: scores scale q.k, capped (cap > 0), less slopes
    float32 [Hq] times the distance; causal, within ``window`` keys, and the
    first prefix int32 [n_seq] keys of a sequence for all of it; tree int64 [T]:
    bit j says that a row sees row j of its sequence's new ones.  ``ws``: device
    memory of attention_workspace_size bytes."""
    dev = _device()
    start, n_seq = _cached(cache, seq_start, dev)
    T, hq, d = q.shape
    if d != cache.head_dim:
        raise ValueError(f"q: expected heads of {cache.head_dim}, got {d}")
    if not 0 <= window < 1 << 31:
        raise ValueError(f"window: expected 0 (none) to 2^31 - 1, got {window}")
    qp, ldq = _rows(q, "q", dev, (T, hq, d))
    op, ldo = _rows(o, "o", dev, (T, hq, d))
    wp, nb = _ws(ws, dev)
    st = lib().moe_q4_attention(qp, ldq, hq, T, start, n_seq, cache, scale, cap, window,
                                _flat(slopes, "slopes", dev, (hq,), torch.float32),
                                _flat(prefix, "prefix", dev, (n_seq,), torch.int32),
                                _flat(tree, "tree", dev, (T,), torch.int64), op, ldo, wp, nb, _stream(stream, dev))
    if st:
        raise _lib.MoeQ4Error("moe_q4_attention", st)


def moe_q4_add_norm(x, u, x_out, y, pre_norm=None, post_norm=None, gate=None, gate_act=ACT_NONE, scale=1.0, eps=1e-6,
                    stream=None):
    """x_out = x + scale * u', u' = u normed (post_norm float32 [H]) and
    gated (gate bf16 [T, H], or [1, H] for all rows), y = x_out normed
    (pre_norm).  x bf16 [T, H] or None, u bf16 or float32 [T, H] or None, x_out
    (may be x) and y bf16 [T, H] or None; rows may lie in wider ones."""
    dev = _device()
    T, H = (u if x is None else x).shape
    xp, ldx = (None, 0) if x is None else _rows(x, "x", dev, (T, H))
    f32 = u is not None and u.dtype == torch.float32
    up, ldu = (None, 0) if u is None else _rows(u, "u", dev, (T, H), (torch.float32,) if f32 else _SIXTEEN)
    gp, ldg = None, 0
    if gate is not None:
        one = gate.shape[0] == 1 and T != 1
        gp, ldg = _rows(gate, "gate", dev, (1 if one else T, H))
        ldg = 0 if one else ldg
    op, ldo = (None, 0) if x_out is None else _rows(x_out, "x_out", dev, (T, H))
    yp, ldy = (None, 0) if y is None else _rows(y, "y", dev, (T, H))
    st = lib().moe_q4_add_norm(xp, ldx, up, ldu, F32 if f32 else BF16, T, H,
                               _flat(post_norm, "post_norm", dev, (H,), torch.float32), gp, ldg, gate_act, scale,
                               _flat(pre_norm, "pre_norm", dev, (H,), torch.float32), eps, op, ldo, yp, ldy,
                               _stream(stream, dev))
    if st:
        raise _lib.MoeQ4Error("moe_q4_add_norm", st)


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
