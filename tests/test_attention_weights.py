"""What the bound of attention_cases.Case.check does not tell (needs an MI355X):
every key of every part and tile counts once, and single tokens' weights keep
16 bits.

Keys: with q = 0 all weights are 1 (exp(0)), and where entry d of the values is
1 for one key alone, o[d] is 1 / (keys seen), rounded twice (the quotient's and its
product's half steps of fp32, then half a step of bf16), or 0 for a query that does not
see that key.  A key that is lost gives 0, one that counts twice 2 / (keys seen).

Weights: bf16 value and bf16 remainder; a half step of a half step is 2^-16.
"""
from __future__ import annotations

import pytest
import torch

from attention_cases import HALF, U, Case, random_tree

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("opt", ["plain", "window", "prefix", "tree"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens,hist,hq,hkv", [([1], [1300], 2, 1), ([1, 1, 1], [0, 700, 31], 8, 2), ([3, 1], [1000, 64], 4, 1),
                                              ([1] * 70, [(i * 37) % 400 for i in range(70)], 2, 2), ([40], [900], 4, 2),
                                              ([64, 17], [130, 600], 8, 1), ([300, 5], [0, 500], 2, 1), ([700], [100], 1, 1)])
def test_every_key_counts_once(lens, hist, hq, hkv, d, opt):
    c = Case(lens, hist, hq, hkv, d, 16, seed=3, q_scale=0.0)
    kw = {"plain": {}, "window": {"window": 150},
          "prefix": {"window": 40, "prefix": torch.tensor([(i * 29) % 200 for i in range(len(lens))], dtype=torch.int32, device="cuda")},
          "tree": {"tree": random_tree(lens, 4)}}[opt]
    seen = [c.seen(b, kw.get("window", 0), kw.get("prefix"), kw.get("tree"))[0] for b in range(len(lens))]
    places = []
    for b, e in enumerate(c.kv):
        j = torch.arange(e, device="cuda")
        places.append((c.table[b].long()[j // 16], j % 16))
    entry = torch.arange(d, device="cuda")
    for first in range(0, max(c.kv), d):  # d keys of each sequence at a time
        for e, (page, at) in zip(c.kv, places):
            v = torch.zeros(e, hkv, d, dtype=torch.bfloat16, device="cuda")
            n = min(d, e - first)
            if n > 0:
                v[first + entry[:n], :, entry[:n]] = 1.0
            c.v[page, :, at] = v
        o = c.run(**kw)
        torch.cuda.synchronize()
        t = 0
        for b, n in enumerate(lens):
            want = torch.zeros(n, d, dtype=torch.float64, device="cuda")
            mine = seen[b][:, first:first + d].double()
            want[:, :mine.shape[1]] = mine / seen[b].sum(1, keepdim=True).clamp(min=1)
            err = (o[t:t + n].double() - want[:, None]).abs()
            assert bool((err <= (HALF + 3 * U) * want[:, None]).all()), (b, first)
            t += n


def rounded_once(c):
    """float64 o if each weight were one bf16"""
    o, t, r = torch.zeros(c.q.shape, dtype=torch.float64, device="cuda"), 0, c.hq // c.hkv
    for b, n in enumerate(c.lens):
        ok, _ = c.seen(b)
        for h in range(c.hq):
            k, v = (x[:, h // r].double() for x in c.dense[b])
            s = torch.where(ok, c.q[t:t + n, h].double() @ k.t().contiguous() * c.scale, -torch.inf)
            w = torch.exp(s - s.amax(1, keepdim=True))
            o[t:t + n, h] = w.bfloat16().double() @ v / w.sum(1, keepdim=True)
        t += n
    return o


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens,hist,hq,hkv", [([1], [5], 2, 1), ([1, 1, 1], [3, 40, 700], 4, 2), ([2, 1], [9000, 100], 4, 1),
                                              ([1, 1], [20000, 1], 8, 2)])
@pytest.mark.parametrize("opt", [{}, {"cap": 30.0}, {"cap": 200.0}, {"window": 100}, {"slopes": True}])
def test_single_tokens_keep_the_remainder(lens, hist, hq, hkv, d, opt):
    """Small scores, so that their own error does not cover the weights'."""
    c = Case(lens, hist, hq, hkv, d, 16, seed=7, q_scale=0.15)
    assert c.T * (hq // hkv) <= 16 * len(lens)  # the kernel for few rows
    kw = dict(opt)
    if kw.get("slopes"):
        kw["slopes"] = torch.linspace(0.001, 0.05, hq, device="cuda")
    o = c.run(**kw)
    torch.cuda.synchronize()
    ref, mag, off = c.expect(**kw)
    if kw.get("cap"):  # (10 half steps of the cap up to 64, 16 of the score beyond)
        off = off - 16 * U * kw["cap"]
        off = off + 10 * U * kw["cap"] if kw["cap"] <= 64 else 2 * off
    tol = HALF * ref.abs() + mag * (HALF ** 2 + 2.2 * off + 2 * (max(c.kv) + 64) * U) + 1e-30
    worst = float(((o.double() - ref).abs() / tol).max())
    print(f"{lens} {hist} d={d} {opt}: largest error / tolerance {worst:.3f}", flush=True)
    assert worst <= 1, worst
    if not opt and max(c.kv) < 1000:
        assert bool(((rounded_once(c) - ref).abs() > tol).any()), "the bound tells a remainder that is lost"
