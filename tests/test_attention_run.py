"""The attention layers' operators together with those that were there, as a
backbone uses them (needs an MI355X): norm -> attention mixer -> norm ->
experts -> norm -> output head -> scores, for a prompt, the tokens after it and
a tree of drafts."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
import quantized_moe_expert_amd as m
import synth
from attention_cases import random_tree
from gpu_cases import assert_close, np_u16

pytestmark = pytest.mark.gpu

H, HQ, HKV, D, V, PAGE, ROT = 512, 8, 2, 64, 1001, 16, 32
HALF = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


class Layer:
    """One layer (attention mixer, routed experts), its norms and the output head."""

    def __init__(self, max_tokens, max_seqs, pages_each, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def int8(n, k):
            q = torch.randint(-127, 128, (n, k), generator=gen, device="cuda", dtype=torch.int8)
            return q, (torch.rand(n, k // 128, generator=gen, device="cuda") + 0.5).mul(1.0 / 64 / k ** 0.5).half()

        def vec(n):
            return 1 + 0.2 * torch.randn(n, generator=gen, device="cuda")

        self.win, self.wout = int8((HQ + 2 * HKV) * D, H), int8(H, HQ * D)
        self.norms, self.q_norm, self.k_norm = [vec(H) for _ in range(3)], vec(D), vec(D)
        self.inv_freq = (10000.0 ** (-torch.arange(0, ROT, 2, device="cuda") / ROT)).float()
        n = max_seqs * pages_each
        self.k, self.v = (torch.full((n, HKV, PAGE, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        self.table = torch.randperm(n, generator=gen, device="cuda").int().reshape(max_seqs, pages_each)
        self.kv_len = torch.zeros(max_seqs, dtype=torch.int32, device="cuda")
        self.cache = m.kv_cache_struct(self.k, self.v, self.table, self.kv_len)
        self.mixer = m.AttentionMixer(m.linear_struct(*self.win), m.linear_struct(*self.wout), HQ, self.cache, max_tokens,
                                      max_seqs, self.inv_freq, self.q_norm, self.k_norm)
        self.experts_w = synth.random_layer(32, H, 128, synth.FMT_ASYM_G64, seed=seed, device="cuda")
        self.router = synth.bf16_bits(synth.normal((32, H), 0.05, seed, "ar/router", "cuda"))
        self.experts = m.MoeQ4Layer(self.experts_w, 4, max_tokens)
        self.head_w = (torch.randn(V, H, generator=gen, device="cuda") * 0.1).bfloat16()
        self.head = m.linear_struct(self.head_w)
        new = dict(dtype=torch.bfloat16, device="cuda")
        self.a, self.b, self.stream, self.h = (torch.empty(max_tokens, H, **new) for _ in range(4))
        self.logits = torch.empty(max_tokens, V, **new)

    def step(self, x, start, positions, tree, tokens, out):
        """(x normed, mixed, its norm, experts' y, the next stream, its norm, logits)"""
        T = x.shape[0]
        a, b, stream, h, logits = (t[:T] for t in (self.a, self.b, self.stream, self.h, self.logits))
        m.moe_q4_add_norm(x, None, None, a, self.norms[0])
        mixed = self.mixer.forward(a, start, b, positions, None, tree, residual=x)
        h1 = torch.empty_like(mixed)
        m.moe_q4_add_norm(mixed, None, None, h1, self.norms[1])
        y = self.experts.forward(h1.view(torch.int16), self.router)
        m.moe_q4_add_norm(mixed, y, stream, h, self.norms[2])
        m.moe_q4_linear(h, self.head, logits)
        m.moe_q4_logprobs(logits, tokens, *out, None)
        return a, mixed, h1, y, stream, h, logits


def scores(T, n=5):
    return (torch.zeros(T, device="cuda"), torch.zeros(T, device="cuda"),
            torch.zeros(T, n, dtype=torch.int32, device="cuda"), torch.zeros(T, n, device="cuda"))


def rms(x, w):
    return x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt() * w.double().cpu()


def mixer_expect(lay, residual, x, lens, pos, hist, tree):
    """float64 with the bf16 roundings between the steps; hist: keys and values of each sequence so far, extended."""
    def weights(q, s):
        return q.double().cpu() * s.double().cpu().repeat_interleave(128, 1)
    x = x.double().cpu()
    rows = (x @ weights(*lay.win).t()).bfloat16().double()
    q, k, v = (t.unflatten(1, (-1, D)) for t in rows.split((HQ * D, HKV * D, HKV * D), 1))
    ang = pos.double().cpu()[:, None] * lay.inv_freq.double().cpu()
    c, s = ang.cos()[:, None], ang.sin()[:, None]

    def turn(t, w):
        t = rms(t, w)
        a, b = t[..., :ROT // 2], t[..., ROT // 2:ROT]
        return torch.cat((a * c - b * s, b * c + a * s, t[..., ROT:]), -1).bfloat16().double()

    q, k = turn(q, lay.q_norm), turn(k, lay.k_norm)
    o, t0 = torch.zeros_like(q), 0
    for b, n in enumerate(lens):
        before = hist[b][0].shape[0]
        kk, vv = torch.cat((hist[b][0], k[t0:t0 + n])), torch.cat((hist[b][1], v[t0:t0 + n]))
        ok = torch.ones(n, before + n, dtype=torch.bool).tril(before)
        if tree is not None:
            bits = [int(u) for u in tree[t0:t0 + n].tolist()]
            ok[:, before:] = torch.tensor([[u >> j & 1 == 1 for j in range(n)] for u in bits])
        for h in range(HQ):
            w = (q[t0:t0 + n, h] @ kk[:, h * HKV // HQ].t() * D ** -0.5).masked_fill(~ok, -torch.inf).softmax(1)
            o[t0:t0 + n, h] = w @ vv[:, h * HKV // HQ]
        if tree is None:
            hist[b] = (kk, vv)
        t0 += n
    return residual.double().cpu() + o.bfloat16().double().flatten(1) @ weights(*lay.wout).t()


@pytest.mark.parametrize("lens", [[70], [5, 130, 64]])
def test_prompt_tokens_and_drafts(lens):
    B = len(lens)
    lay = Layer(max(sum(lens), 12 * B), B, 10)
    gen = torch.Generator(device="cuda").manual_seed(3)
    hist, length = [(torch.zeros(0, HKV, D, dtype=torch.float64),) * 2] * B, [0] * B
    for ls, drafted in ((lens, False), ([1] * B, False), ([2] * B, False), ([6] * B, True), ([1] * B, False)):
        n = sum(ls)
        x = torch.randn(n, H, generator=gen, device="cuda").bfloat16()
        start = torch.tensor([sum(ls[:i]) for i in range(B + 1)], dtype=torch.int32, device="cuda")
        tokens = torch.randint(0, V, (n,), generator=gen, device="cuda", dtype=torch.int32)
        lay.kv_len.copy_(torch.tensor([a + b for a, b in zip(length, ls)], dtype=torch.int32))
        tree = random_tree(ls, 7) if drafted else None
        depth = [bin(u).count("1") - 1 for u in tree.tolist()] if drafted else [i for l in ls for i in range(l)]
        pos = torch.tensor([length[b] for b in range(B) for _ in range(ls[b])]) + torch.tensor(depth)
        out = scores(n)
        a, mixed, h1, y, stream, h, logits = lay.step(x, start, pos.int().cuda() if drafted else None, tree, tokens, out)
        torch.cuda.synchronize()
        want = rms(x.double().cpu(), lay.norms[0])
        assert bool(((a.double().cpu() - want).abs() <= 1.01 * HALF * want.abs()).all())
        # the roundings between the mixer's steps (projection, heads, weights, o) can
        # each be met from the other side (half a bf16 step of a row's entries), and the last one
        want = mixer_expect(lay, x, a, ls, pos, hist, tree)
        assert float((mixed.double().cpu() - want).abs().max()) <= 5 * HALF * float(want.abs().amax())
        # experts: against the oracle on the norm's own output
        want = rms(mixed.double().cpu(), lay.norms[1])
        assert bool(((h1.double().cpu() - want).abs() <= 1.01 * HALF * want.abs()).all())
        xb = np_u16(h1.view(torch.int16))
        lr = oracle.router(xb, np_u16(lay.router), n, H, 32)
        ir, gr = oracle.topk(lr, n, 32, 4)
        w = lay.experts_w
        assert_close(y.cpu().numpy(), oracle.experts(w.fmt, 32, H, 128, *oracle.layer_np(w), xb, ir, gr, n, 4), "experts")
        want = mixed.double().cpu() + y.double().cpu()
        assert bool(((stream.double().cpu() - want).abs() <= 1.01 * HALF * want.abs() + 1e-6).all())
        want = rms(stream.double().cpu(), lay.norms[2])
        assert bool(((h.double().cpu() - want).abs() <= 1.01 * HALF * want.abs()).all())
        z = h.double().cpu() @ lay.head_w.double().cpu().t()
        assert float(((logits.double().cpu() - z).abs() / (z.abs() + z.abs().amax())).max()) <= HALF
        order = torch.argsort(-logits.double().cpu(), dim=1, stable=True)[:, :5]
        assert np.array_equal(out[2].cpu().numpy(), order.numpy())
        if not drafted:  # drafts are not kept: the next call's tokens take their places
            length = [i + j for i, j in zip(length, ls)]


@pytest.mark.parametrize("lens", [[1, 1, 1], [3, 40]])
def test_captured_run(lens):
    """The whole step in one graph while the cache grows, against eager calls."""
    T, B = sum(lens), len(lens)
    lay, ref = Layer(T, B, 16, 1), Layer(T, B, 16, 1)
    gen = torch.Generator(device="cuda").manual_seed(4)
    start = torch.tensor([sum(lens[:i]) for i in range(B + 1)], dtype=torch.int32, device="cuda")
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    tokens, out = torch.zeros(T, dtype=torch.int32, device="cuda"), scores(T)
    lay.kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
    h1 = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")

    def run(l, out):
        a, b = l.a[:T], l.b[:T]
        m.moe_q4_add_norm(x, None, None, a, l.norms[0])
        l.mixer.forward(a, start, b, residual=x)
        m.moe_q4_add_norm(b, a, l.stream[:T], l.h[:T], l.norms[2], l.norms[1], x, m.ACT_SIGMOID, 0.5)
        m.moe_q4_linear(l.h[:T], l.head, l.logits[:T])
        m.moe_q4_logprobs(l.logits[:T], tokens, *out, None)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(lay, out)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(lay, out)
    lay.kv_len.zero_()
    for i in range(4):
        for l in (lay, ref):
            l.kv_len += torch.tensor(lens, dtype=torch.int32, device="cuda")
        x.copy_(torch.randn(T, H, generator=gen, device="cuda"))
        tokens.copy_(torch.randint(0, V, (T,), generator=gen, device="cuda", dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        want = scores(T)
        run(ref, want)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), i
        assert torch.equal(lay.stream[:T], ref.stream[:T]) and torch.equal(lay.h[:T], ref.h[:T])
        for a, b in ((lay.k, ref.k), (lay.v, ref.v)):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_mixers_on_two_streams():
    jobs = []
    for seed, lens in ((1, [1, 1]), (2, [70, 3])):
        lay = Layer(80, 2, 12, seed)
        gen = torch.Generator(device="cuda").manual_seed(seed)
        x = torch.randn(sum(lens), H, generator=gen, device="cuda").bfloat16()
        start = torch.tensor([0, lens[0], sum(lens)], dtype=torch.int32, device="cuda")
        lay.kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
        y = torch.empty_like(x)
        lay.mixer.forward(x, start, y)
        jobs.append((lay, x, start, y, y.clone(), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for lay, x, start, y, _, s in jobs:
            with torch.cuda.stream(s):
                lay.mixer.forward(x, start, y)
    torch.cuda.synchronize()
    for _, _, _, y, want, _ in jobs:
        assert torch.equal(y, want)


def test_rows_that_fill_up_the_batch():
    """A batch of a fixed size of which a part is in use: the other rows are
    sequences of no tokens.  Outputs of those in use are the bits of the call
    without them, the others' the residual's, and no other place of the cache changes."""
    T, used = 6, 4
    lay = Layer(T, T, 4, 5)
    gen = torch.Generator(device="cuda").manual_seed(5)
    start = torch.arange(T + 1, dtype=torch.int32, device="cuda")
    for i in range(3):
        lay.kv_len.copy_(torch.tensor([i + 1] * used + [0] * (T - used), dtype=torch.int32))
        x = torch.randn(T, H, generator=gen, device="cuda").bfloat16()
        x[used:] = 0
        k0, v0 = lay.k.clone(), lay.v.clone()
        y = torch.empty_like(x)
        lay.mixer.forward(x, start, y)
        torch.cuda.synchronize()
        k1, v1 = lay.k.clone(), lay.v.clone()
        changed = (k1.view(torch.int16) != k0.view(torch.int16)).any(-1).any(1)
        places = [(int(lay.table[b, i // PAGE]), i % PAGE) for b in range(used)]
        assert sorted(places) == sorted(map(tuple, changed.nonzero().tolist()))
        few = m.kv_cache_struct(lay.k, lay.v, lay.table[:used], lay.kv_len[:used])
        mixer = m.AttentionMixer(lay.mixer.w_in, lay.mixer.w_out, HQ, few, used, used, lay.inv_freq, lay.q_norm, lay.k_norm)
        want = mixer.forward(x[:used], start[:used + 1], torch.empty_like(x[:used]))
        torch.cuda.synchronize()
        assert torch.equal(y[:used], want) and torch.equal(y[used:], x[used:])


def test_mixer_refusals():
    lay = Layer(8, 2, 2)
    win, wout = m.linear_struct(*lay.win), m.linear_struct(*lay.wout)
    for bad in (lambda: m.AttentionMixer(win, wout, HQ + 2, lay.cache, 8), lambda: m.AttentionMixer(wout, win, HQ, lay.cache, 8),
                lambda: lay.mixer.forward(torch.zeros(9, H, dtype=torch.bfloat16, device="cuda"), lay.kv_len, None)):
        with pytest.raises(ValueError):
            bad()


@pytest.mark.parametrize("max_tokens,max_seqs", [(1, 1), (7, 3), (64, 64), (300, 20), (5000, 4)])
def test_mixer_workspace_fits_every_batch(max_tokens, max_seqs):
    lay = Layer(max_tokens, max_seqs, 80)
    for n in range(1, max_seqs + 1):
        for t in sorted({1, n, 2 * n, 4 * n, 4 * n + 1, max_tokens // 2, max_tokens} - {0}):
            if t <= max_tokens:
                assert m.attention_workspace_size(t, n, HQ, lay.cache) <= lay.mixer.ws.numel()
