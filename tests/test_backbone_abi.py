"""The C ABI of the operators beside the experts without a GPU: exports and
host-side argument checks.  Every call here fails validation (or has nothing
to do) and returns before anything is launched; fake pointers are never
dereferenced on those paths."""
import ctypes
import os
import re

import pytest

import quantized_moe_expert_amd as m
from quantized_moe_expert_amd import _backbone, _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "moe_q4_backbone.h")
FAKE = 0x10000
OK, INVALID, UNSUPPORTED, WORKSPACE = _lib.OK, _lib.ERR_INVALID_ARG, _lib.ERR_UNSUPPORTED, _lib.ERR_WORKSPACE


def test_every_declared_function_is_exported():
    names = re.findall(r"MOE_Q4_API\s+[\w\s\*]+?\b(moe_q4_\w+)\s*\(", open(HEADER).read())
    assert set(names) == set(m.BACKBONE_EXPORTS) and len(names) == len(set(names))
    lib = _backbone.lib()
    for n in names:
        assert hasattr(lib, n), n


def test_header_is_c(tmp_path):
    """The header compiles as C and its constants are the binding's."""
    import subprocess
    src = tmp_path / "c.c"
    src.write_text(f'#include "{HEADER}"\n#include <stdio.h>\nint main(void) {{ printf("%d %d %d %d %d %d %d %d %zu %zu", '
                   "MOE_Q4_LINEAR_INT8, MOE_Q4_LINEAR_BF16, MOE_Q4_ACT_NONE, MOE_Q4_ACT_SILU, MOE_Q4_ACT_GELU, "
                   "MOE_Q4_BF16, MOE_Q4_F32, MOE_Q4_MAX_TOP, sizeof(moe_q4_linear_weights), "
                   "sizeof(moe_q4_delta_shape)); return 0; }\n")
    subprocess.check_call(["gcc", "-std=c11", "-Wall", "-Werror", str(src), "-o", str(tmp_path / "c")])
    out = subprocess.check_output([str(tmp_path / "c")], text=True)
    want = [m.LINEAR_INT8, m.LINEAR_BF16, m.ACT_NONE, m.ACT_SILU, m.ACT_GELU, _backbone.BF16, _backbone.F32, m.MAX_TOP,
            ctypes.sizeof(m.LinearWeights), ctypes.sizeof(m.DeltaShape)]
    assert [int(v) for v in out.split()] == want


def _linear(K=256, N=100, fmt=m.LINEAR_INT8, q=FAKE, scale=FAKE, bias=None, x=FAKE, ldx=None, T=4, act=0, res=None,
            ldr=None, y=FAKE, ldy=None, ydt=0):
    w = m.LinearWeights(K, N, fmt, q, scale, bias)
    return _backbone.lib().moe_q4_linear(x, K if ldx is None else ldx, T, ctypes.byref(w), act, res,
                                         N if ldr is None else ldr, y, N if ldy is None else ldy, ydt, None)


@pytest.mark.parametrize("status,kw", [
    (INVALID, dict(x=None)), (INVALID, dict(y=None)), (INVALID, dict(q=None)), (INVALID, dict(scale=None)),
    (INVALID, dict(T=-1)), (INVALID, dict(K=0)), (INVALID, dict(N=0)),
    (UNSUPPORTED, dict(fmt=2)), (UNSUPPORTED, dict(fmt=-1)), (UNSUPPORTED, dict(act=3)), (UNSUPPORTED, dict(act=-1)),
    (UNSUPPORTED, dict(ydt=2)),
    (UNSUPPORTED, dict(K=192)), (UNSUPPORTED, dict(K=65664)), (UNSUPPORTED, dict(fmt=1, K=100)),
    (UNSUPPORTED, dict(N=1 << 24)), (UNSUPPORTED, dict(T=1 << 31)), (UNSUPPORTED, dict(T=1 << 20, N=1 << 20)),
    (UNSUPPORTED, dict(T=1 << 29, N=1)), (UNSUPPORTED, dict(T=1 << 16, N=1 << 22)),  # launches of 2^32 threads
    (INVALID, dict(ldx=248)), (INVALID, dict(ldx=260)), (UNSUPPORTED, dict(ldx=(1 << 22) + 8)),
    (INVALID, dict(ldy=99)), (UNSUPPORTED, dict(ldy=(1 << 22) + 1)),
    (INVALID, dict(res=FAKE + 64, ldr=99)), (UNSUPPORTED, dict(res=FAKE + 64, ldr=(1 << 22) + 1)),
    (INVALID, dict(x=FAKE + 8)), (INVALID, dict(q=FAKE + 8)), (INVALID, dict(scale=FAKE + 1)),
    (INVALID, dict(bias=FAKE + 2)), (INVALID, dict(y=FAKE + 1)), (INVALID, dict(y=FAKE + 2, ydt=1)),
    (INVALID, dict(res=FAKE + 65)),
    (INVALID, dict(res=FAKE, ydt=1)),              # in place needs a bf16 y
    (INVALID, dict(res=FAKE, ldr=128, ldy=100)),   # and the same rows
    (OK, dict(T=0)), (OK, dict(T=0, x=None, y=None)),
])
def test_linear_validation(status, kw):
    assert _linear(**kw) == status


def test_linear_needs_weights():
    assert _backbone.lib().moe_q4_linear(FAKE, 256, 4, None, 0, None, 0, FAKE, 100, 0, None) == INVALID


def _delta(prefill, hk=2, hv=4, dk=128, dv=128, T=10, n_seq=2, n_states=2, q=FAKE, ldq=None, k=FAKE, v=FAKE, ldv=None,
           g=FAKE, beta=FAKE, start=FAKE, idx=None, s_in=FAKE, s_out=FAKE, o=FAKE, ldo=None, ws=FAKE, nb=1 << 40,
           shape=True):
    L = _backbone.lib()
    sh = ctypes.byref(m.DeltaShape(hk, hv, dk, dv)) if shape else None
    ld = lambda given, width: width if given is None else given
    args = [q, ld(ldq, hk * dk), k, hk * dk, v, ld(ldv, hv * dv), g, beta, T, start, n_seq, idx, n_states, sh, 1.0, 0,
            s_in, s_out, o, ld(ldo, hv * dv)]
    return L.moe_q4_delta_prefill(*args, ws, nb, None) if prefill else L.moe_q4_delta_decode(*args, None)


@pytest.mark.parametrize("prefill", [False, True])
@pytest.mark.parametrize("status,kw", [
    (INVALID, dict(shape=False)), (INVALID, dict(hk=0)), (INVALID, dict(hk=3)), (INVALID, dict(dk=0)),
    (UNSUPPORTED, dict(dk=96)), (UNSUPPORTED, dict(dv=256)), (UNSUPPORTED, dict(hk=1, hv=1025)),
    (INVALID, dict(T=-1)), (INVALID, dict(n_seq=-1)), (INVALID, dict(n_states=-1)),
    (UNSUPPORTED, dict(T=1 << 31)), (UNSUPPORTED, dict(n_seq=1 << 20)),
    (UNSUPPORTED, dict(n_seq=1 << 19, hk=1, hv=512)),
    (UNSUPPORTED, dict(n_seq=1 << 19)), (UNSUPPORTED, dict(T=1 << 28)),  # launches of 2^32 threads
    (INVALID, dict(q=None)), (INVALID, dict(k=None)), (INVALID, dict(v=None)), (INVALID, dict(o=None)),
    (INVALID, dict(g=None)), (INVALID, dict(beta=None)), (INVALID, dict(start=None)),
    (INVALID, dict(q=FAKE + 8)), (INVALID, dict(o=FAKE + 8)), (INVALID, dict(g=FAKE + 2)),
    (INVALID, dict(idx=FAKE + 2)), (INVALID, dict(s_in=FAKE + 8)), (INVALID, dict(s_out=FAKE + 4)),
    (INVALID, dict(ldq=248)), (INVALID, dict(ldq=260)), (INVALID, dict(ldv=504)), (INVALID, dict(ldo=516)),
    (UNSUPPORTED, dict(ldq=(1 << 22) + 8)),
    (OK, dict(n_seq=0)), (OK, dict(n_seq=0, start=None, q=None)),
])
def test_delta_validation(prefill, status, kw):
    assert _delta(prefill, **kw) == status


def test_delta_workspace():
    size = m.delta_workspace_size
    assert size(0, 1, 2, 4, 128, 128) == 0 and size(10, 0, 2, 4, 128, 128) == 0 and size(10, 1, 3, 4, 128, 128) == 0
    need = size(1000, 3, 2, 4, 128, 128)
    if need:
        assert _delta(True, T=1000, n_seq=3, n_states=3, ws=None) == WORKSPACE
        assert _delta(True, T=1000, n_seq=3, n_states=3, nb=need - 1) == WORKSPACE
        assert _delta(True, T=1000, n_seq=3, n_states=3, ws=FAKE + 16, nb=need) == INVALID


def _scores(logits=FAKE, dtype=0, T=4, V=100, ld=100, tokens=FAKE, logprob=FAKE, entropy=FAKE, n=5, idx=FAKE, top=FAKE,
            ws=FAKE, nb=1 << 40):
    return _backbone.lib().moe_q4_logprobs(logits, dtype, T, V, ld, tokens, logprob, entropy, n, idx, top, ws, nb, None)


@pytest.mark.parametrize("status,kw", [
    (INVALID, dict(logits=None)), (INVALID, dict(T=-1)), (INVALID, dict(V=0)), (INVALID, dict(n=-1)),
    (INVALID, dict(V=4, ld=4)), (INVALID, dict(ld=99)), (INVALID, dict(logprob=None)), (INVALID, dict(idx=None)),
    (INVALID, dict(top=None)), (INVALID, dict(logits=FAKE + 1)), (INVALID, dict(logits=FAKE + 2, dtype=1)),
    (INVALID, dict(tokens=FAKE + 2)), (INVALID, dict(entropy=FAKE + 2)), (INVALID, dict(idx=FAKE + 2)),
    (UNSUPPORTED, dict(n=33)), (UNSUPPORTED, dict(dtype=2)), (UNSUPPORTED, dict(T=1 << 31)),
    (UNSUPPORTED, dict(V=1 << 31, ld=1 << 31)), (UNSUPPORTED, dict(ld=1 << 40)),
    (UNSUPPORTED, dict(T=1 << 24)), (UNSUPPORTED, dict(T=1 << 23, V=10000, ld=10000)),  # launches of 2^32 threads
    (OK, dict(T=0)), (OK, dict(T=0, logits=None)),
    (OK, dict(tokens=None, logprob=None, entropy=None, n=0, idx=None, top=None)),
])
def test_logprobs_validation(status, kw):
    assert _scores(**kw) == status


def test_logprobs_workspace():
    assert m.logprobs_workspace_size(0, 100, 5) == 0
    need = m.logprobs_workspace_size(2, 151939, 20)
    if need:
        big = dict(T=2, V=151939, ld=151939, n=20)
        assert _scores(**big, ws=None) == WORKSPACE
        assert _scores(**big, nb=need - 1) == WORKSPACE
        assert _scores(**big, ws=FAKE + 8, nb=need) == INVALID


@pytest.mark.parametrize("T", [1, 2])
def test_linear_outputs_are_at_most_a_row_of_y(T):
    """2^22 outputs, the longest distance of rows, whatever the number of tokens."""
    assert _linear(N=(1 << 22) + 1, T=T) == UNSUPPORTED
    assert _linear(N=1 << 22, T=0) == OK
