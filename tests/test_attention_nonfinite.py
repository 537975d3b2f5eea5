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

from attention_cases import HALF, U, Case, random_tree

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
    """(page, place in it) of a key, or of a list of them"""
    key = torch.as_tensor(key, device="cuda")
    return c.table[b].long()[key // c.page], key % c.page


def row_formula(c, b, t, h, seen, cap=0.0, slopes=None):
    """(float64 o of row t of the call, tolerance) over the keys in seen, as they lie in the cache"""
    page, at = place(c, b, seen)
    g = h // (c.hq // c.hkv)
    k, v = (x[page, g, at].double() for x in (c.k, c.v))
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
        p, at = place(c, b, [j for j in range(e) if every or j >= e - 70 or j % 50 == 3])
        c.k[p, :, at, 2] = -INF
    o = c.run(cap=30.0)
    torch.cuda.synchronize()
    check_rows(c, o, sorted({(b, i) for b, n in enumerate(lens) for i in (0, n // 2, n - 1)}), cap=30.0)
    assert torch.isfinite(o).all()


@pytest.mark.parametrize("opt", OPTIONS)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens,hist,hq,hkv", SHAPES)
def test_nan_in_a_query(lens, hist, hq, hkv, d, opt):
    c = Case(lens, hist, hq, hkv, d, 16, seed=2)
    kw = options(opt, hq)
    clean = c.run(**kw)
    for t, h in {(0, 0), (c.T - 1, hq - 1), (c.T // 2, hq // 2)}:
        q = c.q.clone()
        q[t, h, 3] = NAN
        o = c.run(q=q, **kw)
        torch.cuda.synchronize()
        assert torch.isnan(o[t, h]).all(), (t, h)
        same = (o == clean).all(-1)
        same[t, h] = True
        assert same.all(), (t, h)


@pytest.mark.parametrize("what", ["k", "v"])
@pytest.mark.parametrize("opt", OPTIONS)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens,hist,hq,hkv", SHAPES)
def test_nan_in_one_key_or_value(lens, hist, hq, hkv, d, opt, what):
    """The last token's (alone in its part in some of the shapes), and others."""
    kw = options(opt, hq)
    clean = Case(lens, hist, hq, hkv, d, 16, seed=2).run(**kw)
    for back in (0, 1, 64, 100):
        c = Case(lens, hist, hq, hkv, d, 16, seed=2)
        spoiled = []
        for b, e in enumerate(c.kv):
            spoiled.append(e - 1 - back)
            if e - 1 - back >= 0:
                p, at = place(c, b, e - 1 - back)
                getattr(c, what)[p, hkv - 1, at, d - 5] = NAN
        o = c.run(**kw)
        torch.cuda.synchronize()
        t = 0
        for b, n in enumerate(lens):
            for i in range(n):
                mine, was = o[t].unflatten(0, (hkv, -1)), clean[t].unflatten(0, (hkv, -1))
                sees = 0 <= spoiled[b] <= hist[b] + i
                assert torch.equal(mine[:-1], was[:-1])
                if sees:
                    assert torch.isnan(mine[-1]).any(-1).all(), (b, i, spoiled[b])
                else:
                    assert torch.equal(mine[-1], was[-1]), (b, i, spoiled[b])
                t += 1


@pytest.mark.parametrize("lens", [[1], [20]])
def test_nan_in_a_drafted_key(lens):
    c = Case([n * 3 for n in lens], [380], 4, 2, 128, 16, seed=4)
    tree = random_tree(c.lens, 3)
    clean = c.run(tree=tree)
    j = c.lens[0] - 1
    p, at = place(c, 0, 380 + j)
    c.k[p, :, at, 7] = NAN
    o = c.run(tree=tree)
    torch.cuda.synchronize()
    for t, x in enumerate(tree.tolist()):
        if x >> j & 1:
            assert torch.isnan(o[t]).all()
        else:
            assert torch.equal(o[t], clean[t])


@pytest.mark.parametrize("every", [False, True])
@pytest.mark.parametrize("opt", OPTIONS)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens,hist,hq,hkv", SHAPES)
def test_scores_of_minus_infinity(lens, hist, hq, hkv, d, opt, every):
    """Keys whose scores are -inf: all of them (no weight is left to divide by;
    under a cap they are scores like any other), or the newest 70 and some before."""
    c = Case(lens, hist, hq, hkv, d, 16, seed=2)
    kw = options(opt, hq)
    c.q[:, :, 2] = c.q[:, :, 2].abs() + 0.5
    for b, e in enumerate(c.kv):
        p, at = place(c, b, [j for j in range(e) if every or j >= e - 70 or j % 50 == 3])
        c.k[p, :, at, 2] = -INF
    o = c.run(**kw)
    torch.cuda.synchronize()
    rows = sorted({(b, i) for b, n in enumerate(lens) for i in (0, n // 2, n - 1)})
    check_rows(c, o, rows, **kw)
    if every and opt != "capped":
        assert torch.isnan(o).all()


@pytest.mark.parametrize("opt", OPTIONS)
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens,hist,hq,hkv", SHAPES)
def test_scores_of_infinity(lens, hist, hq, hkv, d, opt):
    c = Case(lens, hist, hq, hkv, d, 16, seed=2)
    kw = options(opt, hq)
    c.q[:, :, 2] = c.q[:, :, 2].abs() + 0.5
    for b, e in enumerate(c.kv):
        p, at = place(c, b, e - 1)
        c.k[p, :, at, 2] = INF
    o = c.run(**kw)
    torch.cuda.synchronize()
    check_rows(c, o, sorted({(b, i) for b, n in enumerate(lens) for i in (0, n // 2, n - 1)}), **kw)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens,hist,hq,hkv", SHAPES)
def test_nan_value_under_a_score_of_minus_infinity(lens, hist, hq, hkv, d):
    """A weight of 0 times NaN: the last key's score is -inf, its value NaN."""
    c = Case(lens, hist, hq, hkv, d, 16, seed=2)
    c.q[:, :, 2] = c.q[:, :, 2].abs() + 0.5
    for b, e in enumerate(c.kv):
        p, at = place(c, b, e - 1)
        c.k[p, :, at, 2] = -INF
        c.v[p, :, at, 1] = NAN
    o = c.run()
    torch.cuda.synchronize()
    for b, n in enumerate(lens):
        last = sum(lens[:b + 1]) - 1
        assert torch.isnan(o[last]).any(-1).all(), b
        if n > 1:
            assert torch.isfinite(o[last - 1]).all(), b
