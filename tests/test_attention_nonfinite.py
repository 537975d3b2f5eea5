"""moe_q4_attention where queries, keys or values are NaN or infinite (needs an
MI355X): whole and split keys, both kernels, both ways to join.

The formula decides: weights exp(s - max s) over what a query sees, a weight of 0
times NaN is NaN, and scores that are all -inf leave no weight to divide by.
Where the formula is finite the tolerance is that of attention_cases.Case.check,
where it is not the row has to hold a NaN or an infinity; rows that see nothing
of it keep their bits.
"""
from __future__ import annotations

import pytest
import torch

from attention_cases import HALF, U, Case

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


# (new rows, rows before, query heads, heads of the cache): single tokens whose last part holds one key
# (385, 4097), short ones and many; blocks of rows that are split, few joined rows and many; one block that is not
SHAPES = [([1], [384], 2, 2), ([1], [4096], 8, 1), ([1, 1, 1, 1], [20, 700, 0, 2100], 4, 2), ([2, 1], [3, 1300], 4, 1),
          ([129], [0], 1, 1), ([40], [6000], 4, 1), ([700], [500], 8, 2), ([150, 30], [0, 900], 2, 1), ([50], [0], 4, 2)]
OPTIONS = ["plain", "capped", "biased"]


def options(name, hq):
    return {"plain": {}, "capped": {"cap": 30.0},
            "biased": {"slopes": torch.linspace(0.001, 0.05, hq, device="cuda")}}[name]


def place(c, b, key):
    """(page, place in it) of a key"""
    return int(c.table[b, key // c.page]), key % c.page


def row_formula(c, b, t, h, seen, cap=0.0, slopes=None):
    """(float64 o of row t of the call, tolerance) over the keys in seen, as they lie in the cache"""
    at = torch.tensor([place(c, b, j) for j in seen], device="cuda")
    g = h // (c.hq // c.hkv)
    k, v = (x[at[:, 0], g, at[:, 1]].double() for x in (c.k, c.v))
    q = c.q[t, h].double()
    s = (k * q).sum(1) * c.scale
    off = (c.d + 8) * U * (torch.nan_to_num(k, 0, 0, 0).abs() * torch.nan_to_num(q, 0, 0, 0).abs()).sum(1) * abs(c.scale)
    if cap:
        s = torch.tanh(s / cap) * cap
        off = off + 16 * U * cap
    if slopes is not None:
        own = c.kv[b] - c.lens[b] + t - sum(c.lens[:b])
        gap = (own - torch.tensor(seen, device="cuda")).abs().double()
        s = s - float(slopes[h]) * gap
        off = off + 4 * U * float(slopes[h]) * gap
    off = float((off + 8 * U * torch.nan_to_num(s, 0, 0, 0).abs()).amax())
    p = torch.exp(s - s.amax())
    o = (p[:, None] * v).sum(0) / p.sum()
    mag = (p[:, None] * v.abs()).sum(0) / p.sum()
    return o, HALF * o.abs() + mag * (HALF + 2.2 * off + 2 * (len(seen) + 64) * U) + 1e-30


def check_rows(c, o, rows, **kw):
    """rows: (sequence, row of it)"""
    for b, i in rows:
        t = sum(c.lens[:b]) + i
        seen = list(range(c.kv[b] - c.lens[b] + i + 1))
        for h in range(c.hq):
            ref, tol = row_formula(c, b, t, h, seen, **kw)
            if not torch.isfinite(ref).all():
                assert not torch.isfinite(o[t, h]).all(), (b, i, h, "finite")
            else:
                assert bool(((o[t, h].double() - ref).abs() <= tol).all()), (b, i, h)


@pytest.mark.parametrize("every", [False, True])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens,hist,hq,hkv", SHAPES)
def test_capped_scores_of_minus_infinity(lens, hist, hq, hkv, d, every):
    """Products of -inf are scores of -cap: all of them, or the newest 70 and some before."""
    c = Case(lens, hist, hq, hkv, d, 16, seed=2)
    c.q[:, :, 2] = c.q[:, :, 2].abs() + 0.5
    for b, e in enumerate(c.kv):
        for j in range(e):
            if every or j >= e - 70 or j % 50 == 3:
                p, at = place(c, b, j)
                c.k[p, :, at, 2] = -INF
    o = c.run(cap=30.0)
    torch.cuda.synchronize()
    check_rows(c, o, sorted({(b, i) for b, n in enumerate(lens) for i in (0, n // 2, n - 1)}), cap=30.0)
    assert torch.isfinite(o).all()
