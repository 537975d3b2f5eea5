"""Capped scores of moe_q4_attention at caps of any size (needs an MI355X).

Caps up to 64: a score is off by at most 10 half steps of the cap.  1 - 2 / (1 +
e^2x): an exponential and a reciprocal of a step each, a sum, a difference, the
argument's rounding (which moves the result by x / cosh^2 x < 1/2 of it).  Beyond:
at most 12 half steps of the score itself, a polynomial of x = s / cap up to |x| =
1/2 (the roundings of x, of the polynomial and of two products), beyond it 1 - 2 / (1
+ e^2|x|), whose error is 10 half steps of the result from 1/2 on; 16 are allowed.
"""
from __future__ import annotations

import pytest
import torch

from attention_cases import HALF, U, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def check(c, cap, **kw):
    o = c.run(cap=cap, **kw)
    torch.cuda.synchronize()
    few = c.T * (c.hq // c.hkv) <= 16 * len(c.lens)
    if cap < 1e7:
        ref, mag, off = c.expect(cap=cap, **kw)
        off = off - 16 * U * cap  # what is left has 8 half steps of the score
    else:
        ref, mag, off = c.expect(**kw)  # (s - s^3 / (3 cap^2): the same to 2^-40)
    off = 2 * off + (10 * U * cap if cap <= 64 else 0)
    keys = max(c.kv)
    weights = HALF ** 2 if few else HALF  # two bf16, or one
    tol = HALF * ref.abs() + mag * (weights + 2.2 * off + 2 * (keys + 64) * U) + 1e-30
    worst = float(((o.double() - ref).abs() / tol).max())
    print(f"cap {cap}: largest error / tolerance {worst:.3f}", flush=True)
    assert torch.isfinite(o).all() and worst <= 1, f"cap {cap}: {worst}"


@pytest.mark.parametrize("cap", [0.5, 30.0, 64.0, 65.0, 300.0, 1e4, 1e5, 1e6, 1e8, 1e20, 3e38])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens,hist", [([1, 1, 1], [3, 12, 700]), ([30], [0]), ([150, 9], [40, 3])])
@pytest.mark.parametrize("q_scale", [1.5, 30.0])
def test_caps(lens, hist, d, cap, q_scale):
    c = Case(lens, hist, 4, 2, d, 16, seed=5, q_scale=q_scale)
    check(c, cap)
    check(c, cap, slopes=torch.tensor([0.3, 0.01, 0.0, 0.1], device="cuda"))


@pytest.mark.parametrize("scale", [-0.2, 1e-20, 3.0])
@pytest.mark.parametrize("cap", [65.0, 1e6, 3e38])
@pytest.mark.parametrize("lens,hist", [([1, 1], [3, 500]), ([40], [0])])
def test_caps_and_scales(lens, hist, cap, scale):
    c = Case(lens, hist, 4, 2, 128, 16, seed=5)
    c.scale = scale
    check(c, cap)


@pytest.mark.parametrize("cap", [1e-45, 1e-38, 1e-20])
def test_caps_that_leave_no_score(cap):
    """Scores between cap and -cap: the mean of the values."""
    for lens, hist in (([1], [40]), ([30], [0])):
        check(Case(lens, hist, 4, 2, 64, 16, seed=5, v_mean=2.0), cap)
