"""The C ABI of the paged cache, the attention and the norms without a GPU:
host-side argument checks.  Every call here fails validation (or has nothing to
do) and returns before anything is launched; fake pointers are never
dereferenced on those paths."""
import ctypes
import os

import pytest

import quantized_moe_expert_amd as m
from quantized_moe_expert_amd import _backbone, _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "moe_q4_backbone.h")
FAKE = 0x10000
OK, INVALID, UNSUPPORTED, WORKSPACE = _lib.OK, _lib.ERR_INVALID_ARG, _lib.ERR_UNSUPPORTED, _lib.ERR_WORKSPACE
NAN, INF = float("nan"), float("inf")


def test_constants_and_sizes(tmp_path):
    import subprocess
    src = tmp_path / "c.c"
    src.write_text(f'#include "{HEADER}"\n#include <stdio.h>\n#include <stddef.h>\nint main(void) {{ printf("%d %zu %zu %zu", '
                   "MOE_Q4_ACT_SIGMOID, sizeof(moe_q4_kv_cache), offsetof(moe_q4_kv_cache, n_pages), "
                   "offsetof(moe_q4_kv_cache, kv_len)); return 0; }\n")
    subprocess.check_call(["gcc", "-std=c11", "-Wall", "-Werror", str(src), "-o", str(tmp_path / "c")])
    out = subprocess.check_output([str(tmp_path / "c")], text=True)
    assert [int(v) for v in out.split()] == [m.ACT_SIGMOID, ctypes.sizeof(m.KVCache), m.KVCache.n_pages.offset,
                                             m.KVCache.kv_len.offset]


def test_linear_takes_no_sigmoid():
    w = m.LinearWeights(256, 100, m.LINEAR_BF16, FAKE, None, None)
    assert _backbone.lib().moe_q4_linear(FAKE, 256, 4, ctypes.byref(w), m.ACT_SIGMOID, None, 0, FAKE, 100, 0, None) == UNSUPPORTED


def cache(hkv=2, d=128, page=16, cols=8, pages=20, k=FAKE, v=FAKE, table=FAKE, kv_len=FAKE):
    return m.KVCache(hkv, d, page, cols, pages, k, v, table, kv_len)


CACHES = [
    (INVALID, dict(hkv=0)), (INVALID, dict(hkv=3)), (INVALID, dict(d=0)), (INVALID, dict(page=0)), (INVALID, dict(cols=0)),
    (INVALID, dict(pages=0)), (UNSUPPORTED, dict(d=96)), (UNSUPPORTED, dict(d=512)), (UNSUPPORTED, dict(page=24)),
    (UNSUPPORTED, dict(page=8)), (UNSUPPORTED, dict(pages=1 << 31)), (UNSUPPORTED, dict(cols=(1 << 26) + 1)),
    (INVALID, dict(k=None)), (INVALID, dict(v=None)), (INVALID, dict(table=None)), (INVALID, dict(kv_len=None)),
    (INVALID, dict(k=FAKE + 8)), (INVALID, dict(v=FAKE + 8)), (INVALID, dict(table=FAKE + 2)), (INVALID, dict(kv_len=FAKE + 1)),
]


def _append(q=FAKE, ldq=None, hq=4, k=FAKE, ldk=None, v=FAKE, ldv=None, T=4, start=FAKE, n_seq=2, c=None, pos=None,
            inv=FAKE, rot=32, qn=None, kn=None, eps=1e-6, qo=FAKE + 4096, ldqo=None):
    c = c or cache()
    kw, qw = c.kv_heads * c.head_dim, hq * c.head_dim
    ld = lambda given, width: width if given is None else given
    return _backbone.lib().moe_q4_kv_append(q, ld(ldq, qw), hq, k, ld(ldk, kw), v, ld(ldv, kw), T, start, n_seq,
                                            ctypes.byref(c), pos, inv, rot, 0, qn, kn, eps, qo, ld(ldqo, qw), None)


@pytest.mark.parametrize("status,kw", CACHES)
def test_append_cache(status, kw):
    assert _append(c=cache(**kw)) == status


@pytest.mark.parametrize("status,kw", [
    (INVALID, dict(hq=0)), (INVALID, dict(hq=3)), (UNSUPPORTED, dict(hq=1026)), (INVALID, dict(T=-1)), (INVALID, dict(n_seq=-1)),
    (UNSUPPORTED, dict(T=1 << 24)), (UNSUPPORTED, dict(n_seq=1 << 20)),
    (INVALID, dict(rot=-16)), (INVALID, dict(rot=144)), (UNSUPPORTED, dict(rot=24)), (INVALID, dict(rot=0)),
    (INVALID, dict(inv=None)), (INVALID, dict(inv=FAKE + 2)), (INVALID, dict(pos=FAKE + 2)), (INVALID, dict(qn=FAKE + 1)),
    (INVALID, dict(kn=FAKE + 1)), (INVALID, dict(eps=-1.0)), (INVALID, dict(eps=NAN)),
    (INVALID, dict(start=None)), (INVALID, dict(start=FAKE + 2)),
    (INVALID, dict(k=None)), (INVALID, dict(v=None)), (INVALID, dict(k=FAKE + 8)), (INVALID, dict(v=FAKE + 2)),
    (INVALID, dict(ldk=248)), (INVALID, dict(ldk=260)), (INVALID, dict(ldv=248)), (UNSUPPORTED, dict(ldv=(1 << 22) + 8)),
    (INVALID, dict(q=FAKE + 8)), (INVALID, dict(ldq=504)), (INVALID, dict(qo=None)), (INVALID, dict(qo=FAKE + 8)),
    (INVALID, dict(ldqo=516)), (INVALID, dict(qo=FAKE, ldq=512, ldqo=520)),
    (INVALID, dict(q=None)), (INVALID, dict(q=None, qo=None, qn=FAKE)),
    (OK, dict(T=0)), (OK, dict(n_seq=0)), (OK, dict(T=0, q=None, k=None, v=None)),
])
def test_append_validation(status, kw):
    assert _append(**kw) == status


def test_append_needs_a_cache():
    assert _backbone.lib().moe_q4_kv_append(FAKE, 512, 4, FAKE, 256, FAKE, 256, 4, FAKE, 2, None, None, None, 0, 0, None,
                                            None, 1e-6, FAKE, 512, None) == INVALID


def _attention(q=FAKE, ldq=None, hq=4, T=4, start=FAKE, n_seq=2, c=None, scale=1.0, cap=0.0, window=0, slopes=None,
               prefix=None, tree=None, o=FAKE + 4096, ldo=None, ws=FAKE, nb=1 << 40):
    c = c or cache()
    width = hq * c.head_dim
    return _backbone.lib().moe_q4_attention(q, width if ldq is None else ldq, hq, T, start, n_seq, ctypes.byref(c), scale,
                                            cap, window, slopes, prefix, tree, o, width if ldo is None else ldo, ws, nb,
                                            None)


@pytest.mark.parametrize("status,kw", CACHES)
def test_attention_cache(status, kw):
    assert _attention(c=cache(**kw)) == status


@pytest.mark.parametrize("status,kw", [
    (INVALID, dict(hq=0)), (INVALID, dict(hq=5)), (UNSUPPORTED, dict(hq=1026)), (INVALID, dict(T=-1)), (INVALID, dict(n_seq=-1)),
    (UNSUPPORTED, dict(T=1 << 24)), (UNSUPPORTED, dict(T=1 << 60)), (UNSUPPORTED, dict(n_seq=1 << 20)),
    (INVALID, dict(scale=NAN)), (INVALID, dict(scale=INF)), (INVALID, dict(cap=-1.0)), (INVALID, dict(cap=NAN)),
    (INVALID, dict(cap=INF)), (INVALID, dict(window=-1)), (INVALID, dict(tree=FAKE, prefix=FAKE)),
    (INVALID, dict(slopes=FAKE + 2)), (INVALID, dict(prefix=FAKE + 2)), (INVALID, dict(tree=FAKE + 4)),
    (INVALID, dict(start=None)), (INVALID, dict(start=FAKE + 2)), (INVALID, dict(q=None)), (INVALID, dict(o=None)),
    (INVALID, dict(q=FAKE + 8)), (INVALID, dict(o=FAKE + 8)), (INVALID, dict(ldq=504)), (INVALID, dict(ldo=516)),
    (UNSUPPORTED, dict(ldq=(1 << 22) + 8)), (INVALID, dict(o=FAKE)),  # q itself
    (OK, dict(T=0)), (OK, dict(n_seq=0)), (OK, dict(T=0, q=None, o=None, start=None)),
])
def test_attention_validation(status, kw):
    assert _attention(**kw) == status


def test_limits_on_sequences_and_heads():
    """Launches of 2^32 threads: sequences times heads of the cache."""
    assert _attention(c=cache(hkv=16), hq=16, n_seq=1 << 18, T=1 << 18) == UNSUPPORTED
    assert _attention(c=cache(hkv=16, cols=4096), hq=16, n_seq=(1 << 18) - 1, T=1 << 18, ws=None) == WORKSPACE
    assert m.attention_workspace_size(1 << 18, 1 << 18, 16, cache(hkv=16)) == 0


def test_attention_workspace():
    size = m.attention_workspace_size
    big = cache(cols=4096)
    assert size(0, 2, 4, big) == 0 and size(4, 0, 4, big) == 0 and size(4, 2, 3, big) == 0 and size(4, 2, 4, cache(d=96)) == 0
    need = size(4, 2, 4, big)
    assert need > 0  # else the calls below would be launched
    assert _attention(c=big, ws=None) == WORKSPACE
    assert _attention(c=big, nb=need - 1) == WORKSPACE
    assert _attention(c=big, ws=FAKE + 16, nb=need) == INVALID


def _norm(x=FAKE, ldx=None, u=FAKE + 256, ldu=None, udt=0, T=4, H=128, post=None, gate=None, ldg=None, act=0, scale=1.0,
          pre=FAKE, eps=1e-6, xo=FAKE + 4096, ldxo=None, y=FAKE + 8192, ldy=None):
    ld = lambda given: H if given is None else given
    return _backbone.lib().moe_q4_add_norm(x, ld(ldx), u, ld(ldu), udt, T, H, post, gate, ld(ldg), act, scale, pre, eps, xo,
                                           ld(ldxo), y, ld(ldy), None)


@pytest.mark.parametrize("status,kw", [
    (INVALID, dict(T=-1)), (INVALID, dict(H=0)), (INVALID, dict(H=-8)), (UNSUPPORTED, dict(H=100)), (UNSUPPORTED, dict(H=65544)),
    (UNSUPPORTED, dict(T=1 << 26)), (UNSUPPORTED, dict(T=1 << 25, H=256)), (UNSUPPORTED, dict(udt=2)), (UNSUPPORTED, dict(act=2)),
    (UNSUPPORTED, dict(act=4)), (UNSUPPORTED, dict(act=-1)), (INVALID, dict(eps=-1e-6)), (INVALID, dict(eps=NAN)),
    (INVALID, dict(scale=NAN)), (INVALID, dict(scale=INF)),
    (INVALID, dict(x=None, u=None)), (INVALID, dict(u=None, post=FAKE)), (INVALID, dict(u=None, gate=FAKE)),
    (INVALID, dict(pre=None)), (INVALID, dict(y=None)), (INVALID, dict(pre=None, y=None, xo=None)),
    (INVALID, dict(post=FAKE + 4)), (INVALID, dict(pre=FAKE + 4)), (INVALID, dict(x=FAKE + 8)), (INVALID, dict(u=FAKE + 8)),
    (INVALID, dict(gate=FAKE + 8)), (INVALID, dict(gate=FAKE + 8, ldg=0)), (INVALID, dict(xo=FAKE + 8)), (INVALID, dict(y=FAKE + 8)),
    (INVALID, dict(ldx=120)), (INVALID, dict(ldx=132)), (INVALID, dict(ldu=120)), (INVALID, dict(gate=FAKE, ldg=120)),
    (INVALID, dict(ldxo=120)), (INVALID, dict(ldy=132)), (UNSUPPORTED, dict(ldx=(1 << 22) + 8)),
    (INVALID, dict(xo=FAKE, ldxo=256)), (INVALID, dict(y=FAKE + 4096)), (INVALID, dict(xo=FAKE + 256)), (INVALID, dict(y=FAKE)),
    (INVALID, dict(y=FAKE + 256)), (INVALID, dict(gate=FAKE + 4096)), (INVALID, dict(gate=FAKE + 8192)),
    (OK, dict(T=0)), (OK, dict(T=0, x=None, u=None)),
])
def test_add_norm_validation(status, kw):
    assert _norm(**kw) == status
