"""The operators beside the experts together with them, as a backbone uses
them (needs an MI355X): mixer -> experts -> output head -> scores, a prompt
and the tokens after it."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
import quantized_moe_expert_amd as m
import synth
from gpu_cases import assert_close, np_u16

pytestmark = pytest.mark.gpu

H, HK, HV, DK, DV, V = 512, 2, 4, 64, 128, 1001


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


class Backbone:
    """One layer (delta mixer, routed experts) and the output head."""

    def __init__(self, max_tokens, max_seqs, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        width = 2 * HK * DK + HV * DV

        def int8(n, k):
            q = torch.randint(-127, 128, (n, k), generator=gen, device="cuda", dtype=torch.int8)
            s = (torch.rand(n, k // 128, generator=gen, device="cuda") + 0.5).mul(1.0 / 64 / k ** 0.5).half()
            return q, s

        self.win, self.wout = int8(width, H), int8(H, HV * DV)
        self.head_w = (torch.randn(V, H, generator=gen, device="cuda") * 0.1).bfloat16()
        self.head = m.linear_struct(self.head_w)
        self.experts_w = synth.random_layer(32, H, 128, synth.FMT_ASYM_G64, seed=seed, device="cuda")
        self.router = synth.bf16_bits(synth.normal((32, H), 0.05, seed, "bb/router", "cuda"))
        self.mixers = {mode: m.DeltaMixer(m.linear_struct(*self.win), m.linear_struct(*self.wout), HK, HV, DK, DV,
                                          max_tokens, max_seqs, mode) for mode in ("decode", "prefill")}
        self.experts = m.MoeQ4Layer(self.experts_w, 4, max_tokens)
        self.mixed = torch.empty(max_tokens, H, dtype=torch.bfloat16, device="cuda")
        self.logits = torch.empty(max_tokens, V, dtype=torch.bfloat16, device="cuda")

    def step(self, mode, x, g, beta, start, states, tokens, out):
        T = x.shape[0]
        mixed = self.mixers[mode].forward(x, g, beta, start, states, states, self.mixed[:T])
        y = self.experts.forward(mixed.view(torch.int16), self.router)
        stream = torch.empty_like(mixed)
        m.moe_q4_residual_bf16(mixed, y, T * H, stream)
        logits = self.logits[:T]
        m.moe_q4_linear(stream, self.head, logits)
        lp, ent, idx, top = out
        m.moe_q4_logprobs(logits, tokens, lp, ent, idx, top, None)
        return mixed, y, stream, logits


def scores(T, n=5):
    return (torch.zeros(T, device="cuda"), torch.zeros(T, device="cuda"),
            torch.zeros(T, n, dtype=torch.int32, device="cuda"), torch.zeros(T, n, device="cuda"))


def gates(T, gen):
    return (-torch.rand(T, HV, generator=gen, device="cuda") ** 3, torch.rand(T, HV, generator=gen, device="cuda"))


def mixer_expect(bb, x, g, beta, lens, s0):
    """float64: every step of the mixer, with the two bf16 roundings between."""
    def weights(q, s):
        return q.double().cpu() * s.double().cpu().repeat_interleave(128, 1)
    rows = (x.double().cpu() @ weights(*bb.win).t()).bfloat16().double()
    q = rows[:, :HK * DK].unflatten(1, (HK, DK))
    k = rows[:, HK * DK:2 * HK * DK].unflatten(1, (HK, DK))
    v = rows[:, 2 * HK * DK:].unflatten(1, (HV, DV))
    q, k = (t / (t.square().sum(-1, keepdim=True) + 1e-6).sqrt() for t in (q, k))
    q, k = q.repeat_interleave(HV // HK, 1), k.repeat_interleave(HV // HK, 1)
    g, beta = g.double().cpu(), beta.double().cpu()
    o, S, t = torch.zeros_like(v), s0.double().cpu(), 0
    for b, n in enumerate(lens):
        for _ in range(n):
            S[b] *= g[t].exp()[:, None, None]
            u = beta[t][:, None] * (v[t] - (S[b] * k[t][..., None]).sum(1))
            S[b] += k[t][..., None] * u[:, None, :]
            o[t] = (S[b] * q[t][..., None]).sum(1) * DK ** -0.5
            t += 1
    return x.double().cpu() + o.bfloat16().double().flatten(1) @ weights(*bb.wout).t(), S


@pytest.mark.parametrize("lens", [[70], [5, 130, 64]])
def test_prompt_then_tokens(lens):
    T, B = sum(lens), len(lens)
    bb = Backbone(T, B)
    gen = torch.Generator(device="cuda").manual_seed(3)
    states = torch.randn(B, HV, DK, DV, generator=gen, device="cuda") * 0.1
    for mode, ls in (("prefill", lens), ("decode", [1] * B), ("decode", [2] * B)):
        n = sum(ls)
        x = torch.randn(n, H, generator=gen, device="cuda").bfloat16()
        g, beta = gates(n, gen)
        start = torch.tensor([sum(ls[:i]) for i in range(B + 1)], dtype=torch.int32, device="cuda")
        tokens = torch.randint(0, V, (n,), generator=gen, device="cuda", dtype=torch.int32)
        want, want_s = mixer_expect(bb, x, g, beta, ls, states)
        out = scores(n)
        mixed, y, stream, logits = bb.step(mode, x, g, beta, start, states, tokens, out)
        torch.cuda.synchronize()
        # mixer: the roundings between its steps can each be met from the other
        # side (half a bf16 step, 2^-8, of a row's entries), and the last one
        scale = want.abs().amax()
        assert float((mixed.double().cpu() - want).abs().max()) <= 3 * 2.0 ** -8 * float(scale)
        assert float((states.double().cpu() - want_s).norm() / want_s.norm()) <= 2.0 ** -8
        # experts: against the oracle on the mixer's own output
        xb = np_u16(mixed.view(torch.int16))
        lr = oracle.router(xb, np_u16(bb.router), n, H, 32)
        ir, gr = oracle.topk(lr, n, 32, 4)
        w = bb.experts_w
        yr = oracle.experts(w.fmt, 32, H, 128, *oracle.layer_np(w), xb, ir, gr, n, 4)
        assert_close(y.cpu().numpy(), yr, f"experts after the mixer, {mode}")
        # head and scores: float64 on the stream
        z = stream.double().cpu() @ bb.head_w.double().cpu().t()
        assert float(((logits.double().cpu() - z).abs() / (z.abs() + z.abs().amax())).max()) <= 2.0 ** -8
        lp = torch.log_softmax(logits.double().cpu(), 1)
        at = lp.gather(1, tokens.cpu().long()[:, None])[:, 0]
        assert float((out[0].double().cpu() - at).abs().max()) <= 1e-5
        order = torch.argsort(-logits.double().cpu(), dim=1, stable=True)[:, :5]
        assert np.array_equal(out[2].cpu().numpy(), order.numpy())


@pytest.mark.parametrize("mode,lens", [("prefill", [70, 66]), ("decode", [1, 2])])
def test_captured_run(mode, lens):
    """The mixer, head and scores in one graph, replayed with other inputs
    against eager calls."""
    T, B = sum(lens), len(lens)
    bb = Backbone(T, B, 1)
    gen = torch.Generator(device="cuda").manual_seed(4)
    start = torch.tensor([sum(lens[:i]) for i in range(B + 1)], dtype=torch.int32, device="cuda")
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    g, beta = torch.zeros(T, HV, device="cuda"), torch.zeros(T, HV, device="cuda")
    tokens = torch.zeros(T, dtype=torch.int32, device="cuda")
    states, out = torch.zeros(B, HV, DK, DV, device="cuda"), scores(T)

    def step(states, out):
        mixed = bb.mixers[mode].forward(x, g, beta, start, states, states, bb.mixed[:T])
        m.moe_q4_linear(mixed, bb.head, bb.logits[:T])
        m.moe_q4_logprobs(bb.logits[:T], tokens, *out, None)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(states, out)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(states, out)
    s0 = torch.randn(states.shape, generator=gen, device="cuda") * 0.1
    states.copy_(s0)
    eager = s0.clone()
    for i in range(3):
        x.copy_(torch.randn(T, H, generator=gen, device="cuda"))
        gi, bi = gates(T, gen)
        g.copy_(gi)
        beta.copy_(bi)
        tokens.copy_(torch.randint(0, V, (T,), generator=gen, device="cuda", dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        want = scores(T)
        step(eager, want)
        torch.cuda.synchronize()
        assert torch.equal(states, eager) and all(torch.equal(a, b) for a, b in zip(out, want)), i


def test_mixer_refusals():
    bb = Backbone(8, 2)
    win, wout = m.linear_struct(*bb.win), m.linear_struct(*bb.wout)
    for bad in (lambda: m.DeltaMixer(win, wout, HK, HV, DK, DV, 8, mode="both"),
                lambda: m.DeltaMixer(win, wout, HK + 1, HV, DK, DV, 8), lambda: m.DeltaMixer(wout, win, HK, HV, DK, DV, 8)):
        with pytest.raises(ValueError):
            bad()
    mx = bb.mixers["decode"]
    x = torch.zeros(9, H, dtype=torch.bfloat16, device="cuda")
    start = torch.tensor([0, 9], dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        mx.forward(x, torch.zeros(9, HV, device="cuda"), torch.zeros(9, HV, device="cuda"), start, None, None, x)


@pytest.mark.parametrize("mode", ["prefill", "decode"])
def test_mixer_rows_that_fill_up_the_batch(mode):
    """A batch of a fixed size, captured, of which a part is in use: the other
    rows are sequences without a state.  Outputs and states of those in use are
    the bits of a call with them alone, and no other state changes."""
    T, used = 6, 4
    bb = Backbone(T, T, 2)
    mixer = bb.mixers[mode]
    gen = torch.Generator(device="cuda").manual_seed(5)
    start = torch.arange(T + 1, dtype=torch.int32, device="cuda")
    idx = torch.tensor([7, 2, 5, 0, -1, -1], dtype=torch.int32, device="cuda")
    x, y = (torch.zeros(T, H, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    g, beta = torch.zeros(T, HV, device="cuda"), torch.zeros(T, HV, device="cuda")
    states = torch.randn(8, HV, DK, DV, generator=gen, device="cuda") * 0.1
    s0 = states.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        mixer.forward(x, g, beta, start, states, states, y, idx)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mixer.forward(x, g, beta, start, states, states, y, idx)
    states.copy_(s0)
    eager = s0.clone()
    for i in range(3):
        x.copy_(torch.randn(T, H, generator=gen, device="cuda"))
        x[used:] = float("nan")  # whatever the unused rows hold
        gi, bi = gates(T, gen)
        g.copy_(gi)
        beta.copy_(bi)
        graph.replay()
        torch.cuda.synchronize()
        want = torch.empty(used, H, dtype=torch.bfloat16, device="cuda")
        mixer.forward(x[:used], g[:used], beta[:used], start[:used + 1], eager, eager, want, idx[:used])
        torch.cuda.synchronize()
        assert torch.equal(y[:used], want) and torch.equal(states, eager), i
    for unnamed in (1, 3, 4, 6):
        assert torch.equal(states[unnamed], s0[unnamed])
    assert not torch.equal(states[7], s0[7])


@pytest.mark.parametrize("mode", ["prefill", "decode"])
def test_mixers_on_two_streams(mode):
    """A mixer for each stream, with the same weights."""
    lens = [70, 66] if mode == "prefill" else [1, 2]
    T, B = sum(lens), len(lens)
    bb = Backbone(T, B, 3)
    win, wout = m.linear_struct(*bb.win), m.linear_struct(*bb.wout)
    start = torch.tensor([sum(lens[:i]) for i in range(B + 1)], dtype=torch.int32, device="cuda")
    jobs = []
    for seed in (1, 2):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        mixer = m.DeltaMixer(win, wout, HK, HV, DK, DV, T, B, mode)
        x = torch.randn(T, H, generator=gen, device="cuda").bfloat16()
        s0 = torch.randn(B, HV, DK, DV, generator=gen, device="cuda") * 0.1
        args = (x, *gates(T, gen), start, s0)
        s1, y = torch.empty_like(s0), torch.empty_like(x)
        mixer.forward(*args, s1, y)
        jobs.append((mixer, args, s1.clone(), y.clone(), s1, y, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for mixer, args, _, _, s1, y, stream in jobs:
            with torch.cuda.stream(stream):
                mixer.forward(*args, s1, y)
    torch.cuda.synchronize()
    for _, _, want_s, want_y, s1, y, _ in jobs:
        assert torch.equal(s1, want_s) and torch.equal(y, want_y)
