"""moe_q4_kv_append against a float64 form (needs an MI355X).

Tolerance per output: a norm's sum of d squares and its root are off by at
most (d / 8 + 12) 2^-24 relative (8 squares a lane, then a tree), each turned
value by eight roundings of |a| + |b| beside it and by the angle (the cosine and
sine of the float64 angle, rounded to float32, which the eight hold; the
angle itself is off by 2^-50 of its value); then the last rounding.
"""
from __future__ import annotations

import pytest
import torch

import quantized_moe_expert_amd as m

pytestmark = pytest.mark.gpu
U, HALF = 2.0 ** -24, 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


class Append:
    def __init__(self, lens, hist, hq, hkv, d, page, rot=0, norm=False, interleaved=False, far=None, tail=0, seed=0,
                 pool=None, size=1.0, cols=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.lens, self.kv = lens, [n + h for n, h in zip(lens, hist)]
        self.hq, self.hkv, self.d, self.page, self.rot, self.interleaved = hq, hkv, d, page, rot, interleaved
        need = [-(-max(n, 1) // page) for n in self.kv]
        n_pages = sum(need) + 2 if pool is None else pool
        ids = torch.randperm(sum(need) + 2, generator=gen, device="cuda").int()
        if pool is not None:
            ids = n_pages - 1 - ids
        self.table = torch.full((len(lens), max(need + [cols])), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = ids[at:at + n]
            at += n
        self.k = torch.empty(n_pages, hkv, page, d, dtype=torch.bfloat16, device="cuda")
        self.v = torch.empty_like(self.k)
        if pool is None:
            self.k.copy_(torch.randn(self.k.shape, generator=gen, device="cuda"))
            self.v.copy_(torch.randn(self.k.shape, generator=gen, device="cuda"))
        self.live = sum(lens)
        self.T = T = self.live + tail
        self.rows = (torch.randn(T, (hq + 2 * hkv) * d + 8, generator=gen, device="cuda") * size).bfloat16()
        w = self.rows[:, 8:]
        self.q = w[:, :hq * d].unflatten(1, (hq, d))
        self.kn = w[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
        self.vn = w[:, (hq + hkv) * d:].unflatten(1, (hkv, d))
        self.inv_freq = (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)).float() if rot else None
        self.positions = None
        if far is not None:
            self.positions = torch.randint(-far, far, (T,), generator=gen, device="cuda").int()
        self.q_norm, self.k_norm = (torch.randn(d, generator=gen, device="cuda") if norm else None for _ in range(2))
        self.eps = 1e-6
        self.start = torch.tensor([sum(lens[:b]) for b in range(len(lens) + 1)], dtype=torch.int32, device="cuda")
        self.kv_len = torch.tensor(self.kv, dtype=torch.int32, device="cuda")
        self.cache = m.kv_cache_struct(self.k, self.v, self.table, self.kv_len)

    def run(self, q_out, with_q=True):
        m.moe_q4_kv_append(self.q if with_q else None, self.kn, self.vn, self.start, self.cache,
                           q_out if with_q else None, self.inv_freq, self.positions, self.q_norm if with_q else None,
                           self.k_norm, self.eps, self.interleaved)

    def places(self):
        """(row, page, place in it) of every token that is stored"""
        out, t, table = [], 0, self.table.tolist()
        for b, n in enumerate(self.lens):
            for i in range(n):
                at = self.kv[b] - n + i
                if 0 <= at < len(table[b]) * self.page and 0 <= table[b][at // self.page] < self.k.shape[0]:
                    out.append((t, table[b][at // self.page], at % self.page))
                t += 1
        return torch.tensor(out, dtype=torch.long, device="cuda").reshape(-1, 3)

    def turned(self, x, w):
        """(x normed and turned, tolerance), float64"""
        x = x[:self.live].double()
        off = torch.zeros_like(x)
        if w is not None:
            x = x / (x.square().mean(-1, keepdim=True) + self.eps).sqrt() * w.double()
            off = (self.d / 8 + 12) * U * x.abs()
        if not self.rot:
            return x, HALF * x.abs() + off if w is not None else off
        if self.positions is None:
            pos = torch.cat([torch.arange(n, device="cuda") + e - n for n, e in zip(self.lens, self.kv)])
        else:
            pos = self.positions[:self.live]
        ang = pos.double()[:, None] * self.inv_freq.double()
        c, s = ang.cos()[:, None], ang.sin()[:, None]
        wrong = (2.0 ** -50 * ang.abs() + 8 * U)[:, None]
        i = torch.arange(self.rot // 2, device="cuda")
        i, j = (2 * i, 2 * i + 1) if self.interleaved else (i, i + self.rot // 2)
        y, tol = x.clone(), off.clone()
        y[..., i], y[..., j] = x[..., i] * c - x[..., j] * s, x[..., j] * c + x[..., i] * s
        more = wrong * (x[..., i].abs() + x[..., j].abs()) + off[..., i] + off[..., j]
        tol[..., i], tol[..., j] = more, more
        plain = torch.ones(self.d, dtype=torch.bool, device="cuda")
        plain[:self.rot] = False
        tol = tol + HALF * y.abs()
        if w is None:
            tol[..., plain] = 0  # copied
        return y, tol

    def check(self, what, with_q=True, in_place=False):
        k0, v0 = self.k.clone(), self.v.clone()
        want_q, tol_q = self.turned(self.q, self.q_norm)
        want_k, tol_k = self.turned(self.kn, self.k_norm)
        want_v = self.vn.clone()
        q_out = self.q if in_place else torch.full((self.T, self.hq, self.d), 7.0, dtype=torch.bfloat16, device="cuda")
        tail = self.q[self.live:].clone() if in_place else torch.full_like(self.q[self.live:], 7.0)
        self.run(q_out, with_q)
        torch.cuda.synchronize()
        worst = 0.0
        if with_q:
            err = (q_out[:self.live].double() - want_q).abs()
            worst = float((err / (tol_q + 1e-30)).max())
            assert torch.equal(q_out[self.live:], tail), "rows behind the last sequence"
        t, p, at = self.places().unbind(1)
        if len(t):
            err = (self.k[p, :, at].double() - want_k[t]).abs()
            worst = max(worst, float((err / (tol_k[t] + 1e-30)).max()))
            assert torch.equal(self.v[p, :, at], want_v[t]), "values are copied"
        self.k[p, :, at], self.v[p, :, at] = k0[p, :, at], v0[p, :, at]
        assert torch.equal(self.k, k0) and torch.equal(self.v, v0), "the rest of the cache"
        print(f"{what}: largest error / tolerance {worst:.3f}", flush=True)
        assert worst <= 1, f"{what}: {worst}"


@pytest.mark.parametrize("d,rot", [(64, 0), (64, 16), (64, 48), (64, 64), (128, 32), (128, 112), (128, 128), (256, 64), (256, 256)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (16, 2), (15, 3)])
def test_heads(d, rot, interleaved, norm, hq, hkv):
    Append([1, 3, 0, 20], [0, 15, 7, 30], hq, hkv, d, 16, rot, norm, interleaved, seed=d + rot).check(f"d={d} rot={rot}")


@pytest.mark.parametrize("lens,hist,page", [([1], [0], 16), ([1] * 70, list(range(70)), 48), ([300, 0, 0, 1, 17], [0, 5, 0, 63, 64], 64),
                                            ([1000], [24], 1024), ([0, 0, 5], [1, 0, 0], 16)])
def test_lengths(lens, hist, page):
    Append(lens, hist, 6, 2, 128, page, 64, True, seed=1, tail=2).check(f"{lens}")


@pytest.mark.parametrize("B", [63, 64, 65, 127, 4097, 9000])
def test_many_sequences(B):
    """Starts found in one, two and three steps, empty sequences among them."""
    Append([i % 3 for i in range(B)], [i % 5 for i in range(B)], 1, 1, 64, 16, 16, seed=2, tail=5).check(f"{B} sequences")


@pytest.mark.parametrize("far", [1000, 1 << 20, (1 << 31) - 1])
@pytest.mark.parametrize("interleaved", [False, True])
def test_far_positions(far, interleaved):
    Append([40, 3], [0, 9], 2, 1, 128, 16, 128, False, interleaved, far=far, seed=3).check(f"positions to {far}")


def test_far_from_one():
    """Values whose squares are small beside eps, and large ones."""
    for size in (1e-6, 1e-3, 1e4):
        Append([9], [3], 4, 2, 64, 16, 32, True, seed=4, size=size).check(f"size {size}")


def test_without_q_and_in_place():
    Append([5, 9], [2, 40], 4, 2, 128, 16, 64, True, seed=5, tail=3).check("without q", with_q=False)
    for interleaved in (False, True):
        Append([5, 9], [2, 40], 4, 2, 128, 16, 64, True, interleaved, seed=5, tail=3).check("in place", in_place=True)


def test_nothing_before_the_sequence_or_behind_the_table():
    """Indices below 0, behind the table and in pages that are not there are not stored."""
    a = Append([20, 20, 40], [-8, 0, 0], 2, 1, 64, 16, 16, seed=6)
    a.table[1, 0] = -1
    a.table[2, 1] = a.k.shape[0]
    a.kv_len[2] = a.kv[2] = 55
    a.check("not there")


def test_far_pages():
    pool = (1 << 32) // (2 * 64 * 128) + 50
    a = Append([70], [10], 4, 2, 128, 64, 64, True, seed=7, pool=pool)
    far = a.table[0, :2].long()
    a.k[far], a.v[far] = 1.0, 2.0
    want_k, tol = a.turned(a.kn, a.k_norm)
    a.run(torch.empty(a.T, 4, 128, dtype=torch.bfloat16, device="cuda"))
    torch.cuda.synchronize()
    t, p, at = a.places().unbind(1)
    assert bool(((a.k[p, :, at].double() - want_k[t]).abs() <= tol[t]).all()) and torch.equal(a.v[p, :, at], a.vn[t])
    assert (a.k[far[0], :, :10] == 1).all() and (a.v[far[1], :, 16:] == 2).all()


def test_captured():
    """A decode step in a graph: the cache grows between replays."""
    a = Append([1, 1, 1], [0, 20, 5], 4, 2, 64, 16, 32, True, seed=8, cols=4)
    a.table.copy_(torch.randperm(12, device="cuda").reshape(3, 4))
    pages = torch.randn(12, 2, 16, 64, device="cuda").bfloat16()
    a.k, a.v = pages.clone(), pages.clone()
    a.cache = m.kv_cache_struct(a.k, a.v, a.table, a.kv_len)
    q_out = torch.zeros(3, 4, 64, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a.run(q_out)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.run(q_out)
    for i in range(4):
        a.kv_len += 1
        a.rows.copy_(torch.randn(a.rows.shape, device="cuda"))
        k0, v0 = a.k.clone(), a.v.clone()
        g.replay()
        torch.cuda.synchronize()
        got = a.k.clone(), a.v.clone(), q_out.clone()
        a.k.copy_(k0)
        a.v.copy_(v0)
        a.run(q_out)
        torch.cuda.synchronize()
        assert torch.equal(got[0], a.k) and torch.equal(got[1], a.v) and torch.equal(got[2], q_out), i
        assert not torch.equal(a.k, k0)


def test_binding_refusals():
    a = Append([3], [4], 4, 2, 64, 16, 32)
    q_out = torch.empty(3, 4, 64, dtype=torch.bfloat16, device="cuda")
    for bad in (lambda: m.moe_q4_kv_append(None, a.kn, a.vn, a.start, a.cache, q_out),
                lambda: m.moe_q4_kv_append(a.q, a.kn[:, :1], a.vn, a.start, a.cache, q_out),
                lambda: m.moe_q4_kv_append(a.q, a.kn, a.vn.float(), a.start, a.cache, q_out),
                lambda: m.moe_q4_kv_append(a.q, a.kn, a.vn, a.start[:1], a.cache, q_out),
                lambda: m.moe_q4_kv_append(a.q, a.kn, a.vn, a.start, a.cache, q_out, a.inv_freq.double()),
                lambda: m.moe_q4_kv_append(a.q, a.kn, a.vn, a.start, a.cache, q_out, k_norm=torch.ones(32, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
