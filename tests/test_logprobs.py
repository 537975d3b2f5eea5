"""moe_q4_logprobs against a plain float64 form (needs an MI355X).

Tolerance: a log probability l - m - log z takes the difference (one
rounding), the sum z of V exponentials, whose relative error is at most (the
longest run of additions into one partial sum, below V / 64 + 40, plus 4 for
the exponential and its argument) 2^-24, and two roundings of the result; an
argument d <= 104 in magnitude of an exponential that counts is itself off by
|d| 2^-24.  The entropy's second sum has the same relative error per term.
"""
from __future__ import annotations

import pytest
import torch

import quantized_moe_expert_amd as m

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def expect(l, tokens, n):
    """float64 on the CPU; NaN as -inf, an empty row has logprob -inf and entropy 0."""
    l = l.detach().cpu().double()
    l = torch.where(torch.isnan(l), -INF, l)
    top = l.amax(1, keepdim=True)
    d = torch.where(l == top, 0.0, l - top)
    e = d.exp()
    z = e.sum(1, keepdim=True)
    lp = torch.where(top == -INF, -INF, d - z.log())
    ent = (z.log() - torch.where(e > 0, e * d, 0.0).sum(1, keepdim=True) / z)[:, 0]
    ent = torch.where(top[:, 0] == -INF, 0.0, ent)
    order = torch.argsort(-l, dim=1, stable=True)[:, :n]
    t = tokens.cpu().long()
    ok = (t >= 0) & (t < l.shape[1])
    own = torch.where(ok, lp.gather(1, t.clamp(0, l.shape[1] - 1)[:, None])[:, 0], 0.0)
    return own, ent, order, lp.gather(1, order)


def score(l, tokens, n, poison=True):
    T, V = l.shape
    lp, ent = torch.full((T,), 9.0, device="cuda"), torch.full((T,), 9.0, device="cuda")
    idx = torch.full((T, n), -7, dtype=torch.int32, device="cuda")
    top = torch.full((T, n), 9.0, device="cuda")
    ws = torch.full((max(m.logprobs_workspace_size(T, V, n), 1),), 255, dtype=torch.uint8, device="cuda")
    m.moe_q4_logprobs(l, tokens, lp, ent, idx if n else None, top if n else None, ws)
    torch.cuda.synchronize()
    return lp, ent, idx, top


def near(got, want, V, what, wide=1.0):
    got = got.cpu().double()
    fin = torch.isfinite(want)
    assert torch.equal(fin, torch.isfinite(got)) and torch.equal(got[~fin], want[~fin]), what
    tol = 2.0 ** -24 * (V / 64 + 44 + 104 + 4 * want[fin].abs()) * wide
    err = (got[fin] - want[fin]).abs()
    assert (err <= tol).all(), f"{what}: {float((err / tol).max())} of the tolerance"


def check(l, tokens, n, what):
    own, ent, order, top = expect(l, tokens, n)
    glp, gent, gidx, gtop = score(l, tokens, n)
    V = l.shape[1]
    near(glp, own, V, what + " logprob")
    near(gent, ent, V, what + " entropy", wide=2 + float(ent.max()))
    assert torch.equal(gidx.cpu().long(), order), what + " top_idx"
    near(gtop, top, V, what + " top_logprob")


def rows(T, V, dtype, seed, spread=2.5):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    l = torch.randn(T, V, generator=gen, device="cuda") * spread
    tok = torch.randint(0, V, (T,), generator=gen, device="cuda", dtype=torch.int32)
    return (l.bfloat16() if dtype == "bf16" else l), tok


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [1, 2, 3, 31, 63, 64, 65, 255, 256, 1000, 2047, 2049, 4097, 8191, 8193, 16385, 50001])
@pytest.mark.parametrize("T,n", [(1, 1), (3, 20), (9, 32)])
def test_sizes(dtype, V, T, n):
    l, tok = rows(T, V, dtype, V)
    check(l, tok, min(n, V), f"{dtype} {T}x{V} top {n}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V", [(700, 4097), (65, 151939), (2, 400000)])
def test_large(dtype, T, V):
    l, tok = rows(T, V, dtype, 5)
    check(l, tok, 20, f"{dtype} {T}x{V}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [5, 300, 5000, 70001])
def test_ties_and_orders(dtype, V):
    """Equal logits everywhere, few distinct values, rising, falling, the
    largest at the end, both zeros."""
    ramp = torch.arange(V, device="cuda", dtype=torch.float32) / V
    l = torch.stack([torch.zeros(V, device="cuda"), torch.full((V,), -3e38, device="cuda"),
                     (torch.arange(V, device="cuda") % 3).float(), ramp, -ramp, (ramp == ramp[-1]).float() * 20,
                     torch.where(torch.arange(V, device="cuda") % 2 == 0, -0.0, 0.0), ramp.round()])
    l = l.bfloat16() if dtype == "bf16" else l
    tok = torch.arange(8, device="cuda", dtype=torch.int32) % V
    for n in (1, 5, min(32, V)):
        check(l, tok, n, f"ties {dtype} V={V} n={n}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [7, 1000, 40000])
def test_masked_rows(dtype, V):
    """-inf, NaN, the type's lowest value, +inf, an empty row, one logit left,
    fewer logits left than are asked for."""
    l, tok = rows(9, V, "f32", 3)
    lowest = torch.finfo(torch.bfloat16).min
    l[0] = -INF
    l[1] = float("nan")
    l[2] = -INF
    l[2, V // 2] = 1.5
    l[3, ::2] = -INF
    l[4, 1::3] = float("nan")
    l[5] = lowest
    l[6, :V // 2] = lowest
    l[7, 3], l[7, V - 1] = INF, INF
    l[8] = -INF
    l[8, V - 2:] = 0.25
    tok[2], tok[7] = V // 2, 3
    l = l.bfloat16() if dtype == "bf16" else l
    check(l, tok, min(20, V), f"masked {dtype} V={V}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("magnitude", [1e-30, 1e4, 1e30])
def test_magnitudes(dtype, magnitude):
    l, tok = rows(4, 3000, "f32", 8, magnitude)
    check(l.bfloat16() if dtype == "bf16" else l, tok, 10, f"{dtype} {magnitude}")


def test_tokens_outside_are_not_scored():
    l, _ = rows(6, 500, "bf16", 2)
    tok = torch.tensor([-1, -100, 500, 2 ** 31 - 1, -2 ** 31, 499], dtype=torch.int32, device="cuda")
    check(l, tok, 3, "outside")
    assert (score(l, tok, 3)[0][:5] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,off,gap", [(4097, 1, 2), (30001, 3, 10), (100, 7, 1)])
def test_rows_in_wider_rows(dtype, V, off, gap):
    """Odd element offsets and distances; NaN and infinities lie around the rows."""
    l, tok = rows(5, V, dtype, 4)
    whole = torch.full((5, V + off + gap), INF, dtype=l.dtype, device="cuda")
    whole[:, ::2] = float("nan")
    whole[:, off:off + V] = l
    check(whole[:, off:off + V], tok, min(32, V), f"strided {dtype} V={V}")


def test_parts():
    """Each output alone gives what all of them together give."""
    l, tok = rows(7, 20001, "bf16", 6)
    lp, ent, idx, top = score(l, tok, 9)
    ws = torch.empty(max(m.logprobs_workspace_size(7, 20001, 9), 1), dtype=torch.uint8, device="cuda")
    a, b, c, d = (torch.zeros_like(t) for t in (lp, ent, idx, top))
    m.moe_q4_logprobs(l, tok, a, None, None, None, ws)
    m.moe_q4_logprobs(l, None, None, b, None, None, ws)
    m.moe_q4_logprobs(l, None, None, None, c, d, ws)
    torch.cuda.synchronize()
    assert torch.equal(a, lp) and torch.equal(b, ent) and torch.equal(c, idx) and torch.equal(d, top)


def test_graph_replays_and_streams():
    for T, V in ((5, 4097), (2, 60001)):
        l, tok = rows(T, V, "bf16", 1)
        want = score(l, tok, 8)
        out = [torch.zeros_like(t) for t in want]
        ws = torch.empty(max(m.logprobs_workspace_size(T, V, 8), 1), dtype=torch.uint8, device="cuda")
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            m.moe_q4_logprobs(l, tok, *out, ws)
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            m.moe_q4_logprobs(l, tok, *out, ws)
        for i in range(3):
            l.copy_(rows(T, V, "bf16", 20 + i)[0])
            want = score(l, tok, 8)
            for t in out:
                t.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want)), (V, i)


def test_far_rows():
    """Rows 2^23 elements apart (offsets beyond 2^32), of one and of several
    segments."""
    for V in (5000, 20000):
        l, tok = rows(600, V, "bf16", 6)
        far = torch.empty(600, 1 << 23, dtype=torch.bfloat16, device="cuda")[:, 3:3 + V]
        far.copy_(l)
        check(far, tok, 7, f"far rows V={V}")


def test_two_streams():
    """Calls on two streams at once, each with buffers of its own."""
    jobs = []
    for i, (T, V) in enumerate(((3, 4097), (5, 60001), (40, 9000), (7, 300))):
        l, tok = rows(T, V, "bf16", i)
        ws = torch.empty(max(m.logprobs_workspace_size(T, V, 9), 1), dtype=torch.uint8, device="cuda")
        jobs.append((l, tok, ws, score(l, tok, 9), [torch.zeros_like(t) for t in score(l, tok, 9)]))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for i, (l, tok, ws, _, out) in enumerate(jobs):
            m.moe_q4_logprobs(l, tok, *out, ws, stream=streams[i % 2])
    torch.cuda.synchronize()
    for _, _, _, want, out in jobs:
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_refusals():
    l, tok = rows(4, 100, "bf16", 0)
    f, i = torch.zeros(4, device="cuda"), torch.zeros(4, 5, dtype=torch.int32, device="cuda")
    top = torch.zeros(4, 5, device="cuda")
    ws = torch.empty(max(m.logprobs_workspace_size(4, 100, 5), 1), dtype=torch.uint8, device="cuda")
    for bad in (lambda: m.moe_q4_logprobs(l.half(), tok, f, f, i, top, ws),
                lambda: m.moe_q4_logprobs(l.cpu(), tok, f, f, i, top, ws),
                lambda: m.moe_q4_logprobs(l.t(), tok, f, f, i, top, ws),
                lambda: m.moe_q4_logprobs(l, tok.long(), f, f, i, top, ws),
                lambda: m.moe_q4_logprobs(l, tok[:3], f, f, i, top, ws),
                lambda: m.moe_q4_logprobs(l, tok, f.double(), f, i, top, ws),
                lambda: m.moe_q4_logprobs(l, tok, f, f, i, top[:, :4], ws),
                lambda: m.moe_q4_logprobs(l, tok, f, f, i.long(), top, ws)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(m.MoeQ4Error):
        m.moe_q4_logprobs(l, tok, None, f, i, top, ws)
    with pytest.raises(m.MoeQ4Error):
        m.moe_q4_logprobs(l, tok, f, f, i, None, ws)
    m.moe_q4_logprobs(l[:0], tok[:0], f[:0], f[:0], i[:0], top[:0], ws)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [262144 + 5, 2200000])
def test_many_segments(dtype, V):
    """Top lists of more keys than the joining workgroup holds at once (33 and
    269 segments of 32 keys), and more segments than it has threads: ordinary
    rows, few distinct values (ties across the segments), the largest all in the
    last segments, all in the first, one left."""
    l, tok = rows(5, V, "f32", 11)
    l[1] = l[1].round()
    l[2, -20000:] += 40
    l[3, :9000] += 40
    l[4] = -INF
    l[4, V - 1] = 2.0
    tok[2], tok[4] = V - 3, V - 1
    check(l.bfloat16() if dtype == "bf16" else l, tok, 32, f"many segments {dtype} V={V}")


@pytest.mark.parametrize("V", [300, 20001])
def test_signalling_nan_counts_as_minus_infinity(V):
    l, tok = rows(4, V, "bf16", 12)
    want = l.clone()
    want[:, 5::3] = -INF
    bits = l.view(torch.int16)
    bits[:, 5::3] = 0x7f81  # a NaN whose quiet bit is clear
    bits[1, 5::3] = -0x7f  # 0xff81
    for a, b in ((l, want), (bits, want)):
        assert all(torch.equal(p, q) for p, q in zip(score(a, tok, 20), score(b, tok, 20)))
    f = want.float()
    f.view(torch.int32)[:, 5::3] = 0x7f800001
    assert all(torch.equal(p, q) for p, q in zip(score(f, tok, 20), score(want.float(), tok, 20)))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_rows(dtype):
    l, tok = rows((1 << 20) + 3, 5, dtype, 13)
    check(l, tok, 2, f"many rows {dtype}")


def test_graphs_that_share_a_workspace():
    """Two captured calls with one workspace, replayed in turn."""
    shapes = ((3, 60001), (5, 20001))
    ws = torch.empty(max(m.logprobs_workspace_size(T, V, 8) for T, V in shapes), dtype=torch.uint8, device="cuda")
    jobs = []
    for i, (T, V) in enumerate(shapes):
        l, tok = rows(T, V, "bf16", 30 + i)
        want = score(l, tok, 8)
        out = [torch.zeros_like(t) for t in want]
        m.moe_q4_logprobs(l, tok, *out, ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            m.moe_q4_logprobs(l, tok, *out, ws)
        jobs.append((graph, out, want, l, tok))
    for _ in range(3):
        for graph, out, *_ in jobs:
            for t in out:
                t.zero_()
            graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for _, out, want, *_ in jobs for a, b in zip(out, want))
