"""moe_q4_delta_decode and moe_q4_delta_prefill against the rule token by
token in float64 (needs an MI355X).

Tolerance: with unit keys (or keys normalised in the call), beta in [0, 1] and
g <= 0 a step does not lengthen a state's error, so the errors of the steps
add up.  One step takes inner products over k_dim and a handful of roundings
of numbers of the size of the state and of v; a chunk of 64 tokens takes sums
over k_dim and 64 and the operands of its products carry at least 22 bits
(4 units of 2^-24 each).  So after L tokens, with M the largest norm of a
column of the state or of |v| on the way, a column's error is at most
(L + 64) (k_dim + 64 + 16) 2^-24 M.  An output o = scale S^T q adds that error
times scale |q|; its products (rounded to 12 bits on the matrix cores, 2^-12
each, relative to scale |q| times a column of the state or to the sum of the
chunk's scale |q.k| |u| <= 64 scale |q| 2 M, taken as independent: 8 instead
of 64) and half a step of bf16.
"""
from __future__ import annotations

import pytest
import torch

import quantized_moe_expert_amd as m

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def rule(q, k, v, g, beta, lens, s0, scale, norm):
    """Outputs, final states and, per sequence and head, the largest column
    norm (of states and values) on the way; float64, on the CPU."""
    q, k, v, g, beta, s0 = (t.detach().cpu().double() for t in (q, k, v, g, beta, s0))
    hv, r = v.shape[1], v.shape[1] // k.shape[1]
    if norm:
        q, k = (t / (t.square().sum(-1, keepdim=True) + 1e-6).sqrt() for t in (q, k))
    q, k = q.repeat_interleave(r, 1), k.repeat_interleave(r, 1)
    o = torch.zeros(v.shape, dtype=torch.float64)
    S, big, t = s0.clone(), torch.zeros(len(lens), hv, dtype=torch.float64), 0
    for b, n in enumerate(lens):
        H = S[b]
        big[b] = H.norm(dim=1).amax(-1)
        for _ in range(n):
            H = H * g[t].exp()[:, None, None]
            u = beta[t][:, None] * (v[t] - (H * k[t][..., None]).sum(1))
            H = H + k[t][..., None] * u[:, None, :]
            o[t] = (H * q[t][..., None]).sum(1) * scale
            big[b] = torch.maximum(big[b], torch.maximum(H.norm(dim=1).amax(-1), v[t].abs().amax(-1)))
            t += 1
        S[b] = H
    return o, S, big, q


def inputs(lens, hk, hv, dk, dv, norm, seed=0, g_scale=1.0, tail=0, wide=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    T = sum(lens) + tail

    def rows(h, d, unit):
        x = torch.randn(T, h * d + wide, generator=gen, device="cuda")
        if unit:
            part = x[:, :h * d].unflatten(1, (h, d))
            part /= part.norm(dim=-1, keepdim=True) * (1 + 2.0 ** -7)  # stays below 1 after rounding
        return x.bfloat16()[:, :h * d].unflatten(1, (h, d))

    q, k, v = rows(hk, dk, not norm), rows(hk, dk, not norm), rows(hv, dv, False)
    g = -torch.rand(T, hv, generator=gen, device="cuda") ** 3 * g_scale
    beta = torch.rand(T, hv, generator=gen, device="cuda")
    s0 = torch.randn(len(lens), hv, dk, dv, generator=gen, device="cuda") * 0.3
    start = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")
    return q, k, v, g, beta, s0, start


def call(kind, q, k, v, g, beta, start, idx, s_in, s_out, o, scale, norm):
    args = (q, k, v, g, beta, start, idx, s_in, s_out, o, scale, norm)
    if kind == "decode":
        m.moe_q4_delta_decode(*args)
    else:
        need = m.delta_workspace_size(q.shape[0], start.numel() - 1, k.shape[1], v.shape[1], k.shape[2], v.shape[2])
        m.moe_q4_delta_prefill(*args, torch.full((max(need, 1),), 255, dtype=torch.uint8, device="cuda"))


def check(o, s, ref, lens, scale, dk, what):
    want_o, want_s, big, qn = ref
    o, s = o.detach().cpu().double(), s.detach().cpu().double()
    assert torch.isfinite(o).all() and torch.isfinite(s).all(), what
    t = 0
    worst_o = worst_s = 0.0
    for b, n in enumerate(lens):
        M = big[b] + 1e-30
        col = (n + 64) * (dk + 80) * 2.0 ** -24 * M  # [hv]
        worst_s = max(worst_s, float(((s[b] - want_s[b]).norm(dim=1).amax(-1) / col).max()))
        if n:
            oo, ww = o[t:t + n], want_o[t:t + n]
            ql = abs(scale) * qn[t:t + n].norm(dim=-1)  # [n, hv]
            tol = 2.0 ** -8 * ww.abs() + (ql * (col + 17 * 2.0 ** -12 * M))[..., None]
            worst_o = max(worst_o, float(((oo - ww).abs() / tol).max()))
        t += n
    print(f"{what}: largest error / tolerance: o {worst_o:.3f}, state {worst_s:.3f}", flush=True)
    assert worst_o <= 1 and worst_s <= 1, what


def run(kind, lens, hk=2, hv=4, dk=128, dv=128, norm=True, seed=0, g_scale=1.0, scale=None, wide=0, **change):
    q, k, v, g, beta, s0, start = inputs(lens, hk, hv, dk, dv, norm, seed, g_scale, wide=wide)
    if change:
        g, beta = change.get("g", lambda x: x)(g), change.get("beta", lambda x: x)(beta)
        k = change.get("k", lambda x: x)(k)
    scale = dk ** -0.5 if scale is None else scale
    o = torch.full((sum(lens), hv, dv), float("nan"), dtype=torch.bfloat16, device="cuda")
    s1 = torch.full_like(s0, float("nan"))
    call(kind, q, k, v, g, beta, start, None, s0, s1, o, scale, norm)
    torch.cuda.synchronize()
    ref = rule(q, k, v, g, beta, lens, s0, scale, norm)
    check(o, s1, ref, lens, scale, dk, f"{kind} {lens} heads {hk}/{hv} dims {dk}x{dv} norm={norm} {list(change)}")


KINDS = ["decode", "prefill"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("L", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128)])
def test_lengths(kind, L, dk, dv):
    run(kind, [L], dk=dk, dv=dv, seed=L)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dk", [64, 128])
@pytest.mark.parametrize("dv", [64, 128])
@pytest.mark.parametrize("hk,hv", [(1, 1), (1, 3), (2, 8), (3, 3)])
@pytest.mark.parametrize("norm", [True, False])
def test_heads(kind, dk, dv, hk, hv, norm):
    run(kind, [70, 3], hk, hv, dk, dv, norm, seed=hv)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("lens", [[0], [0, 5, 0, 64, 0], [1] * 9, [64, 64, 64], [63, 1, 65, 130, 2], [200, 0, 1]])
def test_packed(kind, lens):
    run(kind, lens, seed=len(lens), wide=40)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("lens,hk,hv,dk,dv", [([70] * 10, 4, 8, 128, 128), ([65, 3] * 16, 2, 8, 64, 64),
                                              ([130, 1, 64, 63, 200, 0], 8, 16, 64, 128), ([100] * 9, 8, 16, 128, 64)])
def test_many_columns(kind, lens, hk, hv, dk, dv):
    """More state columns than workgroups of 16 of them are used for."""
    assert len(lens) * hv * dv // 16 > 512
    run(kind, lens, hk, hv, dk, dv, True, seed=hv)


@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 64)])
def test_many_chunks(dk, dv):
    """Chunks and heads enough for the preparation to take two heads of a key
    head at a time (2048 pairs)."""
    lens = [64, 5] * 44 + [63, 65, 130]
    assert (sum(lens) // 64 + len(lens)) * 16 >= 2048
    run("prefill", lens, 4, 16, dk, dv, True, seed=dk)


@pytest.mark.parametrize("dk,dv", [(64, 128), (128, 128)])
@pytest.mark.parametrize("extra", [0, 1])
def test_chunks_about_the_paired_heads(dk, dv, extra):
    """Just below and at the 1024 or 4096 chunks and heads from which two heads
    of a key head share their preparation; the scan at and above 256 tiles of 16
    columns."""
    limit = 1024 if dk == 128 else 4096
    hv = 32
    lens = [limit // hv // 2 * 64 - 64, 63, 1 + 64 * extra]
    lens[0] -= 64 * (sum(lens) // 64 + len(lens) - limit // hv - extra + 1)
    assert (sum(lens) // 64 + len(lens)) * hv == limit + (extra - 1) * hv
    run("prefill", lens, 16, hv, dk, dv, False, seed=dk + extra)


@pytest.mark.parametrize("n", [16, 17])
def test_columns_about_the_shared_rows(n):
    run("prefill", [130] * n, 2, 4, 64, 64, True, seed=n)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("name,change", [
    ("no decay", dict(g=lambda g: g * 0)), ("full decay", dict(g=lambda g: g * 0 - 200)),
    ("infinite decay", dict(g=lambda g: torch.where(g < -0.3, float("-inf"), g))),
    ("mixed decay", dict(g=lambda g: torch.where(g < -0.5, g * 120, g))),
    ("beta 0", dict(beta=lambda b: b * 0)), ("beta 1", dict(beta=lambda b: b * 0 + 1)),
    ("beta 0 or 1", dict(beta=lambda b: b.round())),
    ("one key", dict(k=lambda k: k[:1].expand(k.shape).contiguous())),
    ("zero keys", dict(k=lambda k: k * 0)),
])
def test_values(kind, name, change):
    run(kind, [150, 20], seed=4, **change)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("size", [1e-6, 1e-3, 1e4])
def test_key_and_query_magnitudes(kind, size):
    """Keys far from unit length, normalised in the call (1e-6 enters the root)."""
    run(kind, [100], norm=True, seed=5, k=lambda k: (k.float() * size).bfloat16())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("scale", [1.0, -0.25, 0.0])
def test_scale(kind, scale):
    run(kind, [66], scale=scale, norm=False, seed=6)


@pytest.mark.parametrize("kind", KINDS)
def test_states_pool(kind):
    """Entries in another order, one that nobody names, sequences without an
    entry, the states in place, and rows behind the last sequence."""
    lens = [70, 3, 0, 65, 5]
    q, k, v, g, beta, _, start = inputs(lens, 2, 4, 64, 128, True, 7, tail=9)
    pool = torch.randn(6, 4, 64, 128, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)) * 0.3
    idx = torch.tensor([4, -1, 0, 2, 6], dtype=torch.int32, device="cuda")
    s0 = torch.stack([pool[4], pool[0] * 0, pool[0], pool[2], pool[0] * 0])
    ref = rule(q, k, v, g, beta, lens, s0, 0.2, True)
    for place in ("in place", "apart"):
        s_in = pool.clone()
        s_out = s_in if place == "in place" else torch.full_like(pool, 7.0)
        o = torch.full((sum(lens) + 9, 4, 128), 3.0, dtype=torch.bfloat16, device="cuda")
        call(kind, q, k, v, g, beta, start, idx, s_in, s_out, o, 0.2, True)
        torch.cuda.synchronize()
        final = torch.stack([s_out[4], ref[1][1].float().cuda(), s_out[0], s_out[2], ref[1][4].float().cuda()])
        check(o[:sum(lens)], final, ref, lens, 0.2, 64, f"{kind} {place}")
        assert torch.equal(s_out[0], pool[0])  # no tokens: handed on
        assert (o[sum(lens):] == 3).all()
        for unnamed in (1, 3, 5):
            assert torch.equal(s_out[unnamed], pool[unnamed] if place == "in place" else torch.full_like(pool[0], 7.0))
        if place == "apart":
            assert torch.equal(s_in, pool)


@pytest.mark.parametrize("kind", KINDS)
def test_no_states(kind):
    """From zero states, and with the final ones dropped."""
    lens = [80, 4]
    q, k, v, g, beta, s0, start = inputs(lens, 2, 4, 128, 64, True, 8)
    ref = rule(q, k, v, g, beta, lens, s0 * 0, 0.1, True)
    o, o2 = (torch.zeros(84, 4, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    s1 = torch.full_like(s0, float("nan"))
    call(kind, q, k, v, g, beta, start, None, None, s1, o, 0.1, True)
    call(kind, q, k, v, g, beta, start, None, None, None, o2, 0.1, True)
    torch.cuda.synchronize()
    check(o, s1, ref, lens, 0.1, 128, f"{kind} zero states")
    assert torch.equal(o, o2)


@pytest.mark.parametrize("kind", KINDS)
def test_malformed_starts_stay_in_bounds(kind):
    """Starts beyond T or falling are clamped; nothing outside o is written."""
    q, k, v, g, beta, s0, _ = inputs([50, 50], 2, 4, 64, 64, True, 9)
    whole = torch.full((100 + 40, 4, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    for starts in ([0, 1000, 2000], [-5, 40, 2 ** 31 - 1], [90, 10, 60], [2 ** 31 - 1, -2 ** 31, 5]):
        start = torch.tensor(starts, dtype=torch.int32, device="cuda")
        call(kind, q, k, v, g, beta, start, None, s0, torch.empty_like(s0), whole[20:120], 0.1, True)
        torch.cuda.synchronize()
        assert (whole[:20] == 3).all() and (whole[120:] == 3).all(), starts


@pytest.mark.parametrize("kind", KINDS)
def test_nan_stays_in_its_sequence(kind):
    """Other sequences and the chunks (tokens, in decode) before it keep
    their bits."""
    lens = [140, 70]
    q, k, v, g, beta, s0, start = inputs(lens, 2, 4, 128, 128, True, 10)
    outs = []
    for bad in (False, True):
        if bad:
            v[80], k[100, 0, 3] = float("nan"), float("inf")
        o, s1 = torch.zeros(210, 4, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros_like(s0)
        call(kind, q, k, v, g, beta, start, None, s0, s1, o, 0.1, True)
        outs.append((o, s1))
    torch.cuda.synchronize()
    assert torch.equal(outs[0][0][140:], outs[1][0][140:]) and torch.equal(outs[0][1][1], outs[1][1][1])
    before = 80 if kind == "decode" else 64
    assert torch.equal(outs[0][0][:before], outs[1][0][:before])
    assert torch.isnan(outs[1][0][80]).all()


def test_decode_continues_a_prompt():
    """A prompt by prefill, then tokens by decode from its states, against
    the whole by decode."""
    L, n = 150, 4
    q, k, v, g, beta, s0, start = inputs([L + n], 2, 4, 128, 128, True, 11)
    ref = rule(q, k, v, g, beta, [L + n], s0, 0.1, True)
    o, s = torch.empty(L + n, 4, 128, dtype=torch.bfloat16, device="cuda"), s0.clone()
    one = lambda a: torch.tensor([0, a], dtype=torch.int32, device="cuda")
    call("prefill", q[:L], k[:L], v[:L], g[:L], beta[:L], one(L), None, s, s, o[:L], 0.1, True)
    for t in range(L, L + n):
        w = slice(t, t + 1)
        call("decode", q[w], k[w], v[w], g[w], beta[w], one(1), None, s, s, o[w], 0.1, True)
    torch.cuda.synchronize()
    check(o, s, ref, [L + n], 0.1, 128, "prefill then decode")


@pytest.mark.parametrize("kind", KINDS)
def test_same_input_same_bits(kind):
    lens = [130, 70]
    q, k, v, g, beta, s0, start = inputs(lens, 2, 4, 128, 128, True, 12)
    got = []
    for _ in range(3):
        o, s1 = torch.zeros(200, 4, 128, dtype=torch.bfloat16, device="cuda"), torch.zeros_like(s0)
        call(kind, q, k, v, g, beta, start, None, s0, s1, o, 0.1, True)
        got.append((o, s1))
    torch.cuda.synchronize()
    assert all(torch.equal(got[0][0], o) and torch.equal(got[0][1], s) for o, s in got[1:])


@pytest.mark.parametrize("kind", KINDS)
def test_graph_replays_and_streams(kind):
    """Captured with states in place and replayed: each replay takes the
    next step of the states, as eager calls do."""
    lens = [70, 3]
    q, k, v, g, beta, s0, start = inputs(lens, 2, 4, 128, 128, True, 13)
    need = m.delta_workspace_size(73, 2, 2, 4, 128, 128)
    ws = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
    s, o = s0.clone(), torch.zeros(73, 4, 128, dtype=torch.bfloat16, device="cuda")

    def step(s, o):
        if kind == "decode":
            m.moe_q4_delta_decode(q, k, v, g, beta, start, None, s, s, o, 0.1, True)
        else:
            m.moe_q4_delta_prefill(q, k, v, g, beta, start, None, s, s, o, 0.1, True, ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(s, o)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(s, o)
    s.copy_(s0)
    es, eo = s0.clone(), torch.zeros_like(o)
    for i in range(3):
        graph.replay()
        torch.cuda.synchronize()
        step(es, eo)
        torch.cuda.synchronize()
        assert torch.equal(s, es) and torch.equal(o, eo), i


@pytest.mark.parametrize("kind", KINDS)
def test_far_rows_and_states(kind):
    """Rows 2^22 elements apart and a state beyond 2^31 elements."""
    lens, ld, n = [1040, 3], 1 << 22, 2 ** 31 // (4 * 64 * 64) + 2
    T = sum(lens)
    q, k, v, g, beta, s0, start = inputs(lens, 2, 4, 64, 64, True, 14)
    far = torch.empty(T, ld, dtype=torch.bfloat16, device="cuda")
    parts = [far[:, 0:128].unflatten(1, (2, 64)), far[:, 2 ** 21:2 ** 21 + 128].unflatten(1, (2, 64)),
             far[:, ld - 256:].unflatten(1, (4, 64)), far[:, 1024:1024 + 256].unflatten(1, (4, 64))]
    for a, b in zip(parts, (q, k, v)):
        a.copy_(b)
    pool = torch.empty(n, 4, 64, 64, device="cuda")
    idx = torch.tensor([n - 1, n - 2], dtype=torch.int32, device="cuda")
    pool[n - 1], pool[n - 2] = s0[0], s0[1]
    call(kind, parts[0], parts[1], parts[2], g, beta, start, idx, pool, pool, parts[3], 0.1, True)
    torch.cuda.synchronize()
    check(parts[3].contiguous(), torch.stack([pool[n - 1], pool[n - 2]]), rule(q, k, v, g, beta, lens, s0, 0.1, True),
          lens, 0.1, 64, f"{kind} far")


@pytest.mark.parametrize("kind", KINDS)
def test_two_streams(kind):
    """Calls on two streams at once, each with buffers of its own."""
    jobs = []
    for seed, lens in enumerate(([70, 3], [200], [64] * 30, [1] * 9)):
        q, k, v, g, beta, s0, start = inputs(lens, 2, 4, 128, 128, True, seed)
        T = sum(lens)
        need = m.delta_workspace_size(T, len(lens), 2, 4, 128, 128)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        o, s1 = torch.empty(T, 4, 128, dtype=torch.bfloat16, device="cuda"), torch.empty_like(s0)
        args = [q, k, v, g, beta, start, None, s0, s1, o, 0.1, True] + ([ws] if kind == "prefill" else [])
        fn = m.moe_q4_delta_prefill if kind == "prefill" else m.moe_q4_delta_decode
        fn(*args)
        jobs.append((fn, args, o, s1, o.clone(), s1.clone()))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(4):
        for i, (fn, args, o, s1, _, _) in enumerate(jobs):
            fn(*args, stream=streams[i % 2])
    torch.cuda.synchronize()
    for _, _, o, s1, want_o, want_s in jobs:
        assert torch.equal(o, want_o) and torch.equal(s1, want_s)


def test_refusals():
    q, k, v, g, beta, s0, start = inputs([5], 2, 4, 64, 64, True)
    o = torch.empty_like(v)
    args = dict(q=q, k=k, v=v, g=g, beta=beta, seq_start=start, state_idx=None, state_in=s0, state_out=s0, o=o, scale=1.0)
    for bad in (dict(q=q.float()), dict(k=k[:4]), dict(g=g[:, :2]), dict(beta=beta.double()), dict(state_in=s0.half()),
                dict(state_out=s0[:, :2]), dict(o=o[:, :2]), dict(seq_start=start.long()), dict(seq_start=start.cpu()),
                dict(state_idx=start), dict(q=q.transpose(1, 2)), dict(state_in=torch.cat([s0, s0])),
                dict(seq_start=start[:0])):
        with pytest.raises(ValueError):
            m.moe_q4_delta_decode(**{**args, **bad})
    with pytest.raises(m.MoeQ4Error):  # dims
        half = torch.zeros(5, 2, 32, dtype=torch.bfloat16, device="cuda")
        m.moe_q4_delta_decode(**{**args, "q": half, "k": half, "state_in": None, "state_out": None})
    if m.delta_workspace_size(5, 1, 2, 4, 64, 64):
        with pytest.raises(m.MoeQ4Error):
            m.moe_q4_delta_prefill(**args)


@pytest.mark.parametrize("n_seq", [1, 9])
@pytest.mark.parametrize("L", [1, 2, 17, 63, 64, 65, 129])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128)])
def test_prefill_operands_have_22_bits(dk, dv, L, n_seq):
    """States and outputs as near as operands of two f16 make them, on both
    layouts of the scan (few columns and many).

    A chunk takes the state through three products after one another (K S,
    T' X, K^T W).  Each has operands of 22 bits (2^-22 for either, of what is
    multiplied) and fp32 sums of 64 or k_dim + 64 terms, whose roundings are
    taken as independent (14 x 2^-24 < 2^-20): 3 (2^-21 + 2^-20) < 5 x 2^-20 of
    M, and the chunks' errors add.  An output's two products (with q.k_j of
    random directions, whose norm over a chunk is below 2) add at most
    2 x 3 x 2^-20 of scale |q| M before it is rounded, by at most half a bf16
    step.  (The file's own bound allows the output's operands 12 bits.)  The
    same algorithm in fp32 on the CPU is within 0.05 of either bound; without
    the remainder of one operand it is, at the worst of these lengths, 13 (S),
    52 (T'), 62 (X) and 75 (W) times the state's and, where only the output
    sees it, 5 times the output's (S in Q S, P, U).
    """
    lens = [L] * n_seq
    q, k, v, g, beta, s0, start = inputs(lens, 4, 8, dk, dv, True, seed=L)
    scale = dk ** -0.5
    o = torch.full((sum(lens), 8, dv), float("nan"), dtype=torch.bfloat16, device="cuda")
    s1 = torch.full_like(s0, float("nan"))
    call("prefill", q, k, v, g, beta, start, None, s0, s1, o, scale, True)
    torch.cuda.synchronize()
    want_o, want_s, big, qn = rule(q, k, v, g, beta, lens, s0, scale, True)
    chunks = (L + 63) // 64
    off_s = (s1.cpu().double() - want_s).norm(dim=2).amax(-1) / (5 * chunks * 2.0 ** -20 * big)
    half = torch.ldexp(torch.ones_like(want_o), torch.frexp(want_o).exponent - 9)
    tol = (5 * chunks + 6) * 2.0 ** -20 * scale * qn.norm(dim=-1) * big.repeat_interleave(L, 0)
    off_o = ((o.cpu().double() - want_o).abs() - half) / tol[..., None]
    print(f"{n_seq} x {L}, {dk}x{dv}: largest error / bound: o {float(off_o.max()):.4f}, state {float(off_s.max()):.4f}",
          flush=True)
    assert float(off_o.max()) <= 1 and float(off_s.max()) <= 1


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n_seq", [1, 9])
@pytest.mark.parametrize("power", [-40, 60])
def test_powers_of_two_pass_through(kind, n_seq, power):
    """The rule is linear in v and the state: a power of two on both comes out
    of every output, bit for bit."""
    lens = [130] * n_seq
    q, k, v, g, beta, s0, start = inputs(lens, 2, 8, 64, 128, True, 15)
    got = []
    for f in (1.0, 2.0 ** power):
        o, s1 = torch.zeros(v.shape, dtype=torch.bfloat16, device="cuda"), torch.zeros_like(s0)
        call(kind, q, k, (v.float() * f).bfloat16(), g, beta, start, None, s0 * f, s1, o, 0.1, True)
        got.append((o.float(), s1))
    torch.cuda.synchronize()
    assert torch.equal(got[0][0] * 2.0 ** power, got[1][0]) and torch.equal(got[0][1] * 2.0 ** power, got[1][1])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n_seq", [1, 9])
def test_large_values_behind_a_token(kind, n_seq):
    """Tokens whose values are 2^16 times larger, in the same chunk, leave the
    outputs before them as near as the 22 bits (test above) make them; the bound
    is doubled for the operands' absolute step there (2^-39 of the largest, 2^-23
    of the smaller ones)."""
    L, cut = 64, 40
    lens = [L] * n_seq
    q, k, v, g, beta, s0, start = inputs(lens, 2, 8, 64, 128, True, 16)
    v = v.unflatten(0, (n_seq, L)).clone()
    v[:, cut:] *= 2.0 ** 16
    v = v.flatten(0, 1)
    o, s1 = torch.zeros(v.shape, dtype=torch.bfloat16, device="cuda"), torch.zeros_like(s0)
    call(kind, q, k, v, g, beta, start, None, s0, s1, o, 0.1, True)
    torch.cuda.synchronize()
    before = lambda t: t.unflatten(0, (n_seq, L))[:, :cut].flatten(0, 1)
    want, _, big, qn = rule(*(before(t) for t in (q, k, v, g, beta)), [cut] * n_seq, s0, 0.1, True)
    half = torch.ldexp(torch.ones_like(want), torch.frexp(want).exponent - 9)
    tol = 2 * 11 * 2.0 ** -20 * 0.1 * qn.norm(dim=-1) * big.repeat_interleave(cut, 0)
    worst = float((((before(o).cpu().double() - want).abs() - half) / tol[..., None]).max())
    print(f"{kind} {n_seq}: largest error / bound {worst:.4f}", flush=True)
    assert worst <= 1


@pytest.mark.parametrize("kind", KINDS)
def test_long_sequence(kind):
    """2^17 tokens.  With 0.1 of decay a token, what lies 1000 tokens back is
    gone (e^-100): the last ones are those of the last 1064 tokens alone."""
    T, tail = 2 ** 17 + 5, 1064
    q, k, v, g, beta, s0, start = inputs([T], 1, 2, 64, 64, True, 17)
    g = g * 0 - 0.1
    o, s1 = torch.zeros(v.shape, dtype=torch.bfloat16, device="cuda"), torch.zeros_like(s0)
    call(kind, q, k, v, g, beta, start, None, s0, s1, o, 0.1, True)
    torch.cuda.synchronize()
    ref = rule(*(t[-tail:] for t in (q, k, v, g, beta)), [tail], s0 * 0, 0.1, True)
    want_o, want_s, big, qn = ref
    check(o[-64:], s1, (want_o[-64:], want_s, big, qn[-64:]), [64], 0.1, 64, f"{kind} {T} tokens")


@pytest.mark.parametrize("kind", KINDS)
def test_many_sequences(kind):
    gen = torch.Generator().manual_seed(1)
    run(kind, torch.randint(0, 4, (3000,), generator=gen).tolist(), 1, 1, 64, 64, True, seed=18)


@pytest.mark.parametrize("kind", KINDS)
def test_most_heads(kind):
    run(kind, [3, 65], 2, 1024, 64, 64, True, seed=19)


def test_graphs_that_share_a_workspace():
    """Two captured prompts with one workspace, replayed in turn."""
    ws, jobs = None, []
    for seed, lens in ((20, [70, 3]), (21, [200])):
        q, k, v, g, beta, s0, start = inputs(lens, 2, 4, 128, 128, True, seed)
        need = m.delta_workspace_size(sum(lens), len(lens), 2, 4, 128, 128)
        ws = torch.empty(1 << 20 if need < 1 << 20 else need, dtype=torch.uint8, device="cuda") if ws is None else ws
        assert need <= ws.numel()
        o, s1 = torch.zeros(v.shape, dtype=torch.bfloat16, device="cuda"), torch.zeros_like(s0)
        args = (q, k, v, g, beta, start, None, s0, s1, o, 0.1, True, ws)
        m.moe_q4_delta_prefill(*args)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            m.moe_q4_delta_prefill(*args)
        jobs.append((graph, o, s1, o.clone(), s1.clone(), args))
    for _ in range(3):
        for graph, o, s1, *_ in jobs:
            o.zero_()
            s1.zero_()
            graph.replay()
    torch.cuda.synchronize()
    for _, o, s1, want_o, want_s, _ in jobs:
        assert torch.equal(o, want_o) and torch.equal(s1, want_s)
