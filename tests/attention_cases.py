"""Caches, inputs and the float64 form of moe_q4_attention for its tests."""
from __future__ import annotations

import torch

import quantized_moe_expert_amd as m

U = 2.0 ** -24      # half a step of float32, relative
HALF = 2.0 ** -8    # half a step of bf16, relative


class Case:
    """Sequences of ``lens`` new tokens after ``hist`` cached ones; the pool's
    pages in a random order, whatever no sequence uses is NaN."""

    def __init__(self, lens, hist, hq, hkv, d, page, seed=0, spare=2, cols=None, q_scale=1.5, v_mean=0.0, tail=0,
                 pool=None):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.lens, self.hist, self.hq, self.hkv, self.d, self.page = list(lens), list(hist), hq, hkv, d, page
        self.kv = [n + h for n, h in zip(lens, hist)]
        need = [-(-max(n, 0) // page) for n in self.kv]
        total = sum(need)
        n_pages = total + spare if pool is None else pool
        cols = max(need + [1]) if cols is None else cols
        ids = torch.randperm(total + spare, generator=gen, device="cuda").int()
        if pool is not None:
            ids = n_pages - 1 - ids  # the far end of a large pool
        table = torch.full((len(lens), cols), 2 ** 30, dtype=torch.int32, device="cuda")
        self.k = torch.empty(n_pages, hkv, page, d, dtype=torch.bfloat16, device="cuda")
        self.v = torch.empty_like(self.k)
        used = ids.long()
        self.k[used] = float("nan")
        self.v[used] = float("nan")
        self.dense, at = [], 0
        for b, n in enumerate(self.kv):
            n = max(n, 0)
            mine = ids[at:at + need[b]]
            table[b, :need[b]] = mine
            at += need[b]
            kd = torch.randn(n, hkv, d, generator=gen, device="cuda").bfloat16()
            vd = (torch.randn(n, hkv, d, generator=gen, device="cuda") + v_mean).bfloat16()
            i = torch.arange(n, device="cuda")
            p = mine.long()[i // page]
            self.k[p, :, i % page] = kd
            self.v[p, :, i % page] = vd
            self.dense.append((kd, vd))
        self.table = table
        self.kv_len = torch.tensor(self.kv, dtype=torch.int32, device="cuda")
        start = [0]
        for n in lens:
            start.append(start[-1] + n)
        self.start = torch.tensor(start, dtype=torch.int32, device="cuda")
        self.T = start[-1] + tail
        self.q = (torch.randn(self.T, hq, d, generator=gen, device="cuda") * q_scale).bfloat16()
        self.scale = d ** -0.5
        self.cache = m.kv_cache_struct(self.k, self.v, self.table, self.kv_len)

    def run(self, q=None, o=None, ws=None, stream=None, **kw):
        q = self.q if q is None else q
        o = torch.full_like(self.q, float("nan")) if o is None else o
        if ws is None:
            size = m.attention_workspace_size(self.T, len(self.lens), self.hq, self.cache)
            ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
        m.moe_q4_attention(q, self.start, self.cache, o, self.scale, ws, stream=stream, **kw)
        return o

    def seen(self, b, window=0, prefix=None, tree=None):
        """(which keys each new row of sequence b sees, their distances)"""
        n, e = self.lens[b], max(self.kv[b], 0)
        before, t0 = self.kv[b] - n, sum(self.lens[:b])
        key = torch.arange(e, device="cuda")
        row = before + torch.arange(n, device="cuda")
        kpos, qpos = key.clone(), row.clone()
        if tree is None:
            ok = key[None] <= row[:, None]
        else:
            masks = [x % (1 << 64) for x in tree[t0:t0 + n].tolist()]
            ok = key[None].expand(n, e) < before
            ok = ok.clone()
            for i, x in enumerate(masks):
                depth = bin(x & ~(1 << i) if i < 64 else x).count("1")
                qpos[i] = before + depth
                if 0 <= before + i < e:
                    kpos[before + i] = before + depth
                for j in range(min(n, 64)):
                    if x >> j & 1 and 0 <= before + j < e:
                        ok[i, before + j] = True
        gap = qpos[:, None] - kpos[None]
        if window:
            ok = ok & (gap < window)
        if prefix is not None:
            ok = ok | (key[None] < int(prefix[b]))
        there = self.table[b, key // self.page] if e else key
        ok = ok & ((there >= 0) & (there < self.k.shape[0]))[None]
        return ok, gap.abs().double()

    def expect(self, cap=0.0, window=0, slopes=None, prefix=None, tree=None):
        """float64: (o, sum of the weights times |v|, bound of a score's error, keys) per row and head"""
        r, d = self.hq // self.hkv, self.d
        o = torch.zeros(self.T, self.hq, d, dtype=torch.float64, device="cuda")
        mag, off = torch.zeros_like(o), torch.zeros(self.T, self.hq, 1, dtype=torch.float64, device="cuda")
        t0 = 0
        for b, n in enumerate(self.lens):
            e = max(self.kv[b], 0)
            if n and e:
                ok, gap = self.seen(b, window, prefix, tree)
                for h in range(self.hq):
                    kd, vd = (x[:, h // r].double() for x in self.dense[b])
                    q = self.q[t0:t0 + n, h].double()
                    kd = torch.where(ok.any(0)[:, None], kd, 0)  # what nobody sees may be anything
                    vd = torch.where(ok.any(0)[:, None], vd, 0)
                    s = q @ kd.t().contiguous() * self.scale
                    err = (d + 8) * U * (q.abs() @ kd.abs().t().contiguous()) * abs(self.scale)
                    if cap:
                        s = torch.tanh(s / cap) * cap
                        err = err + 16 * U * cap
                    if slopes is not None:
                        s = s - float(slopes[h]) * gap
                        err = err + 4 * U * abs(float(slopes[h])) * gap
                    err = err + 8 * U * s.abs()
                    s = torch.where(ok, s, -torch.inf)
                    p = torch.where(ok.any(1)[:, None], torch.softmax(s, 1), 0)
                    o[t0:t0 + n, h] = p @ vd
                    mag[t0:t0 + n, h] = p @ vd.abs()
                    off[t0:t0 + n, h, 0] = torch.where(ok, err, 0).amax(1)
            t0 += n
        return o, mag, off

    def check(self, o, what="", **kw):
        """Each weight's error: twice its score's (its own and the sum's), its
        own rounding to bf16 (half a step; 2^-17 where the remainder is kept
        as well), the exponential's and the products' and sums' roundings
        over the keys; then the last rounding."""
        ref, mag, off = self.expect(**kw)
        keys = max(max(self.kv), 1)
        tol = HALF * ref.abs() + mag * (HALF + 2.2 * off + 2 * (keys + 64) * U) + 1e-30
        live = sum(self.lens)
        err = (o[:live].double() - ref[:live]).abs()
        worst = float((err / tol[:live]).max()) if live else 0.0
        print(f"{what}: largest error / tolerance {worst:.3f}", flush=True)
        assert torch.isfinite(o[:live]).all() and worst <= 1, f"{what}: {worst}"


def random_tree(lens, seed, reach=6):
    """int64 [sum lens] masks of random drafts: each row follows an earlier one, or none."""
    import random
    rng, out = random.Random(seed), []
    for n in lens:
        mine = []
        for i in range(n):
            parent = rng.randint(max(-1, i - reach), i - 1)
            mine.append((mine[parent] if parent >= 0 else 0) | (1 << i if i < 64 else 0))
        out += mine
    return torch.tensor([x - (1 << 64) if x >> 63 else x for x in out], dtype=torch.int64, device="cuda")
