"""moe_q4_linear against a plain float64 form (needs an MI355X).

Tolerance per output: with S = sum |x w| over the inputs (scales included),
the fp32 sum of K exact products is off by at most (K + K/32 + 8) 2^-24 S (a
group's partial sum takes up to four more roundings, its scale factors among them);
bias and activation add a few roundings of the result (their slopes are below
1.13) and the last rounding is half a step of the output type.
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


def weights(fmt, N, K, gen, zero_scales=False):
    if fmt == "int8":
        q = torch.randint(-128, 128, (N, K), generator=gen, device="cuda", dtype=torch.int8)
        s = (torch.rand(N, K // 128, generator=gen, device="cuda") + 0.5).mul(0.02).half()
        if zero_scales:
            s[torch.rand(s.shape, generator=gen, device="cuda") < 0.4] = 0
            s[0] = 0
            s[-1, -1] = 6e-8  # the smallest f16
        w = q.double() * s.double().repeat_interleave(128, 1)
        return q, s, w
    q = (torch.randn(N, K, generator=gen, device="cuda") * 0.1).bfloat16()
    return q, None, q.double()


def expect(x, w, bias, act, residual):
    z = x.double() @ w.t().contiguous()
    if bias is not None:
        z = z + bias.double()
    if act == m.ACT_SILU:
        z = z * torch.sigmoid(z)
    elif act == m.ACT_GELU:
        z = z * torch.special.ndtr(z)
    return z if residual is None else z + residual.double()


def check(y, x, w, bias, act, residual, what):
    K = x.shape[1]
    ref = expect(x, w, bias, act, residual)
    mag = x.double().abs() @ w.abs().t().contiguous()
    half_step = torch.finfo(y.dtype).eps / 2
    parts = mag + (0 if bias is None else bias.double().abs()) + (0 if residual is None else residual.double().abs())
    tol = half_step * ref.abs() + 1.13 * (K + K / 32 + 8) * 2.0 ** -24 * parts + 1e-30
    err = (y.double() - ref).abs()
    worst = float((err / tol).max())
    print(f"{what}: largest error / tolerance {worst:.3f}", flush=True)
    assert torch.isfinite(y).all() and worst <= 1, f"{what}: {worst}"


def run(fmt, T, K, N, act=0, bias=False, residual=False, out=torch.bfloat16, seed=0, zero_scales=False):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    q, s, w = weights(fmt, N, K, gen, zero_scales)
    x = torch.randn(T, K, generator=gen, device="cuda").bfloat16()
    b = torch.randn(N, generator=gen, device="cuda") if bias else None
    r = torch.randn(T, N, generator=gen, device="cuda").bfloat16() if residual else None
    y = torch.full((T, N), float("nan"), dtype=out, device="cuda")
    m.moe_q4_linear(x, m.linear_struct(q, s, b), y, act, r)
    torch.cuda.synchronize()
    check(y, x, w, b, act, r, f"{fmt} T={T} K={K} N={N} act={act} bias={bias} residual={residual} {out}")


@pytest.mark.parametrize("fmt", ["int8", "bf16"])
@pytest.mark.parametrize("T", [1, 2, 3, 7, 15, 16, 17, 31, 33, 48, 63, 64, 65, 100, 127, 129, 200, 257, 300])
@pytest.mark.parametrize("K,N", [(256, 100), (1152, 257)])
def test_lengths(fmt, T, K, N):
    run(fmt, T, K, N, seed=T)


@pytest.mark.parametrize("fmt,K", [("int8", 128), ("int8", 384), ("int8", 4096), ("bf16", 8), ("bf16", 24),
                                   ("bf16", 136), ("bf16", 1000), ("bf16", 4096)])
@pytest.mark.parametrize("N", [1, 2, 15, 17, 64, 255, 1025])
@pytest.mark.parametrize("T", [1, 5, 40, 150])
def test_sizes(fmt, K, N, T):
    run(fmt, T, K, N, seed=K + N + T)


@pytest.mark.parametrize("fmt", ["int8", "bf16"])
@pytest.mark.parametrize("act", [0, 1, 2])
@pytest.mark.parametrize("bias,residual,out", [(True, True, torch.bfloat16), (True, False, torch.float32),
                                               (False, True, torch.float32), (False, False, torch.bfloat16)])
@pytest.mark.parametrize("T", [4, 130])
def test_epilogue(fmt, act, bias, residual, out, T):
    run(fmt, T, 512, 333, act, bias, residual, out, seed=act)


@pytest.mark.parametrize("T", [1, 20, 90, 300])
def test_zero_and_tiny_scales(T):
    """Groups whose scale is 0, next to ordinary ones and to the smallest f16."""
    run("int8", T, 1024, 200, out=torch.float32, seed=T, zero_scales=True)


@pytest.mark.parametrize("fmt,K", [("int8", 128), ("int8", 640), ("int8", 8192), ("int8", 8320), ("int8", 16512),
                                   ("bf16", 392), ("bf16", 8200)])
@pytest.mark.parametrize("T,N", [(70, 100), (300, 2050), (449, 1441)])
def test_small_tiles(fmt, K, T, N):
    """Rows of one group to more than two fills of the scales; one workgroup per tile row to more than the card has."""
    run(fmt, T, K, N, out=torch.float32, seed=K)


def test_small_tiles_zero_scales():
    run("int8", 300, 1024, 2050, residual=True, seed=3, zero_scales=True)


@pytest.mark.parametrize("fmt,T,N,K", [("int8", 2050, 2100, 640), ("bf16", 2050, 2100, 648), ("int8", 600, 4097, 2048),
                                       ("bf16", 1000, 1025, 512), ("int8", 1000, 513, 1024)])
def test_large(fmt, T, N, K):
    run(fmt, T, K, N, 1, True, True, seed=9)


@pytest.mark.parametrize("fmt", ["int8", "bf16"])
@pytest.mark.parametrize("T", [3, 70, 300])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_rows_in_wider_rows(fmt, T, out):
    """Strided x, residual and y at odd element offsets; what lies between the rows stays."""
    K, N = 384, 130
    gen = torch.Generator(device="cuda").manual_seed(T)
    q, s, w = weights(fmt, N, K, gen)
    x = torch.randn(T, K + 72, generator=gen, device="cuda").bfloat16()[:, 8:8 + K]
    r = torch.randn(T, N + 5, generator=gen, device="cuda").bfloat16()[:, 3:3 + N]
    whole = torch.full((T, N + 7), 5.0, dtype=out, device="cuda")
    m.moe_q4_linear(x, m.linear_struct(q, s), whole[:, 1:1 + N], m.ACT_NONE, r)
    torch.cuda.synchronize()
    check(whole[:, 1:1 + N], x, w, None, 0, r, f"strided {fmt} T={T}")
    assert (whole[:, :1] == 5).all() and (whole[:, 1 + N:] == 5).all()


@pytest.mark.parametrize("fmt", ["int8", "bf16"])
@pytest.mark.parametrize("T", [2, 100])
def test_residual_in_place(fmt, T):
    gen = torch.Generator(device="cuda").manual_seed(T)
    q, s, w = weights(fmt, 300, 256, gen)
    x = torch.randn(T, 256, generator=gen, device="cuda").bfloat16()
    y = torch.randn(T, 300, generator=gen, device="cuda").bfloat16()
    r = y.clone()
    m.moe_q4_linear(x, m.linear_struct(q, s), y, m.ACT_SILU, y)
    torch.cuda.synchronize()
    check(y, x, w, None, m.ACT_SILU, r, f"in place {fmt} T={T}")


@pytest.mark.parametrize("fmt", ["int8", "bf16"])
@pytest.mark.parametrize("T", [1, 40, 130])
def test_infinities_and_nan_stay_in_their_row(fmt, T):
    """A token with an infinity or a NaN changes no other token's outputs."""
    gen = torch.Generator(device="cuda").manual_seed(T)
    q, s, _ = weights(fmt, 200, 512, gen)
    x = torch.randn(T + 1, 512, generator=gen, device="cuda").bfloat16()
    w = m.linear_struct(q, s)
    ref, y = torch.empty(T + 1, 200, device="cuda"), torch.empty(T + 1, 200, device="cuda")
    m.moe_q4_linear(x, w, ref)
    x[0, 3], x[0, 100] = float("inf"), float("nan")
    m.moe_q4_linear(x, w, y)
    torch.cuda.synchronize()
    assert torch.isnan(y[0]).all() and torch.equal(y[1:], ref[1:])


@pytest.mark.parametrize("T", [4, 40, 300])
def test_same_input_same_bits(T):
    gen = torch.Generator(device="cuda").manual_seed(T)
    q, s, _ = weights("int8", 500, 2048, gen)
    x = torch.randn(T, 2048, generator=gen, device="cuda").bfloat16()
    w, y = m.linear_struct(q, s), [torch.empty(T, 500, device="cuda") for _ in range(3)]
    for z in y:
        m.moe_q4_linear(x, w, z)
    torch.cuda.synchronize()
    assert torch.equal(y[0], y[1]) and torch.equal(y[0], y[2])


def test_graph_replays_and_streams():
    """Captured and replayed with other inputs, and on another stream."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    q, s, _ = weights("int8", 500, 1024, gen)
    w = m.linear_struct(q, s)
    for T in (3, 200):
        x, y = torch.zeros(T, 1024, dtype=torch.bfloat16, device="cuda"), torch.zeros(T, 500, device="cuda")
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            m.moe_q4_linear(x, w, y)
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            m.moe_q4_linear(x, w, y)
        for i in range(3):
            x.copy_(torch.randn(T, 1024, generator=gen, device="cuda"))
            want = torch.empty_like(y)
            m.moe_q4_linear(x, w, want)
            y.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(y, want), (T, i)


@pytest.mark.parametrize("fmt", ["int8", "bf16"])
def test_far_rows(fmt):
    """Rows 2^22 elements apart: element offsets pass 2^32."""
    T, K, N, ld = 1100, 256, 130, 1 << 22
    gen = torch.Generator(device="cuda").manual_seed(1)
    q, s, w = weights(fmt, N, K, gen)
    x = torch.empty(T, ld, dtype=torch.bfloat16, device="cuda")[:, :K]
    y = torch.empty(T, ld, dtype=torch.bfloat16, device="cuda")[:, 5:5 + N]
    x.copy_(torch.randn(T, K, generator=gen, device="cuda"))
    for rows in (slice(0, T), slice(T - 20, T)):
        m.moe_q4_linear(x[rows], m.linear_struct(q, s), y[rows])
        torch.cuda.synchronize()
        check(y[rows], x[rows], w, None, 0, None, f"far rows {fmt}")
        y[rows] = float("nan")


def test_two_streams():
    """Calls on two streams at once, each with buffers of its own."""
    gen = torch.Generator(device="cuda").manual_seed(2)
    jobs = []
    for T in (5, 40, 300, 700):
        q, s, _ = weights("int8", 700, 1024, gen)
        x = torch.randn(T, 1024, generator=gen, device="cuda").bfloat16()
        w, want = m.linear_struct(q, s), torch.empty(T, 700, device="cuda")
        m.moe_q4_linear(x, w, want)
        jobs.append((x, w, want, torch.empty_like(want), (q, s)))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for i, (x, w, _, y, _) in enumerate(jobs):
            m.moe_q4_linear(x, w, y, stream=streams[i % 2])
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for _, _, want, y, _ in jobs)


def test_refusals():
    x = torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda")
    q, s = torch.zeros(32, 256, dtype=torch.int8, device="cuda"), torch.zeros(32, 2, dtype=torch.float16, device="cuda")
    y, w = torch.zeros(4, 32, device="cuda"), m.linear_struct(q, s)
    for bad in (lambda: m.linear_struct(q), lambda: m.linear_struct(q, s[:, :1]), lambda: m.linear_struct(q.float()),
                lambda: m.linear_struct(q.cpu(), s.cpu()), lambda: m.linear_struct(q[:, ::2], s),
                lambda: m.linear_struct(q, s, torch.zeros(31, device="cuda")),
                lambda: m.moe_q4_linear(x.float(), w, y), lambda: m.moe_q4_linear(x[:, :128], w, y),
                lambda: m.moe_q4_linear(x, w, y[:3]), lambda: m.moe_q4_linear(x.cpu(), w, y),
                lambda: m.moe_q4_linear(x.t().contiguous().t(), w, y), lambda: m.moe_q4_linear(x, w, y.half()),
                lambda: m.moe_q4_linear(x, w, y, 0, torch.zeros(4, 32, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(m.MoeQ4Error):
        m.moe_q4_linear(x, w, y, 7)
    m.moe_q4_linear(x[:0], w, y[:0])


@pytest.mark.parametrize("T,N", [(1, 300), (40, 70), (100, 70), (1100, 2400)])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_gelu_keeps_its_relative_accuracy(T, N, out):
    """z (1 + erf(z / sqrt 2)) / 2 for z in [-12, 9], far into the tail where
    the parenthesis cancels.  One input per output, so that z is exact; the
    argument of the error function takes two roundings (2^-24 each), which its
    slope makes at most 2 z^2 2^-24 of the value, the function itself up to 16
    steps (32 x 2^-24), the products 8 x 2^-24."""
    gen = torch.Generator(device="cuda").manual_seed(T)
    x, w = torch.zeros(T, 8, device="cuda"), torch.zeros(N, 8, device="cuda")
    x[:, 5] = torch.rand(T, generator=gen, device="cuda") * 6 - 4
    w[:, 5] = torch.rand(N, generator=gen, device="cuda") * 2 + 1
    x[0, 5] = -4.0
    x, w = x.bfloat16(), w.bfloat16()
    y = torch.empty(T, N, dtype=out, device="cuda")
    m.moe_q4_linear(x, m.linear_struct(w), y, m.ACT_GELU)
    torch.cuda.synchronize()
    z = (x[:, 5:6].double() * w[None, :, 5].double()).cpu()
    want = z * torch.special.erfc(-z * 0.5 ** 0.5) / 2
    rel = (2 * z * z + 40) * 2.0 ** -24 + (2.0 ** -8 if out == torch.bfloat16 else 2.0 ** -24)
    worst = float(((y.cpu().double() - want).abs() / (rel * want.abs() + 1e-44)).max())
    print(f"gelu T={T} N={N} {out}: largest error / tolerance {worst:.3f}, z from {float(z.min()):.2f}", flush=True)
    assert worst <= 1


# (T, N) of the three large tiles: 128 x 128 (165 of them), 128 x 256 (153), 256 x 256 (400)
LARGE = [(600, 4097), (2050, 2100), (5000, 5100)]


def mixed_scales(N, K, gen):
    """Scales of either sign over 2^-24 .. 2^5, a third of them 0 (or -0), whole
    rows of 0 and of the smallest f16 among them."""
    s = torch.exp2(torch.randint(-24, 6, (N, K // 128), generator=gen, device="cuda").float())
    s = s * (1 + torch.rand(s.shape, generator=gen, device="cuda")) * torch.randn(s.shape, generator=gen, device="cuda").sign()
    s[torch.rand(s.shape, generator=gen, device="cuda") < 0.33] = 0
    s[3], s[5], s[-1, -1] = 0, 2.0 ** -24, -(2.0 ** -24)
    s[7, 0] = -0.0
    return s.half()


@pytest.mark.parametrize("T,N", LARGE)
@pytest.mark.parametrize("fmt,K", [("int8", 128), ("int8", 256), ("int8", 1280), ("bf16", 8), ("bf16", 264), ("bf16", 1000)])
def test_large_tiles(fmt, K, T, N):
    """Every large tile with float outputs at odd offsets of wider rows, x and
    residual rows in wider ones, and scales of any size and sign.  (A change of
    a group's unit takes up to six roundings of the sums: K / 16 in all.)"""
    gen = torch.Generator(device="cuda").manual_seed(K)
    q, s, w = weights(fmt, N, K, gen)
    if fmt == "int8":
        s = mixed_scales(N, K, gen)
        w = q.double() * s.double().repeat_interleave(128, 1)
    x = torch.randn(T, K + 24, generator=gen, device="cuda").bfloat16()[:, 8:8 + K]
    b = torch.randn(N, generator=gen, device="cuda")
    r = torch.randn(T, N + 3, generator=gen, device="cuda").bfloat16()[:, 1:1 + N]
    whole = torch.full((T, N + 6), 5.0, device="cuda")
    y = whole[:, 3:3 + N]
    m.moe_q4_linear(x, m.linear_struct(q, s, b), y, m.ACT_NONE, r)
    torch.cuda.synchronize()
    ref = expect(x, w, b, 0, r)
    parts = x.double().abs() @ w.abs().t().contiguous() + b.double().abs() + r.double().abs()
    tol = 2.0 ** -24 * (ref.abs() + (K + K / 16 + 8) * parts)
    worst = float(((y.double() - ref).abs() / tol).max())
    print(f"{fmt} T={T} K={K} N={N}: largest error / tolerance {worst:.3f}", flush=True)
    assert torch.isfinite(y).all() and worst <= 1
    assert (whole[:, :3] == 5).all() and (whole[:, 3 + N:] == 5).all()


@pytest.mark.parametrize("T,N", LARGE)
@pytest.mark.parametrize("fmt,K", [("int8", 384), ("bf16", 392)])
@pytest.mark.parametrize("act", [0, 1, 2])
def test_large_tiles_in_place(fmt, K, T, N, act):
    gen = torch.Generator(device="cuda").manual_seed(act)
    q, s, w = weights(fmt, N, K, gen, zero_scales=True)
    x = torch.randn(T, K, generator=gen, device="cuda").bfloat16()
    b = torch.randn(N, generator=gen, device="cuda")
    y = torch.randn(T, N, generator=gen, device="cuda").bfloat16()
    r = y.clone()
    m.moe_q4_linear(x, m.linear_struct(q, s, b), y, act, y)
    torch.cuda.synchronize()
    check(y, x, w, b, act, r, f"in place {fmt} T={T} N={N} act={act}")


@pytest.mark.parametrize("T,N", LARGE)
@pytest.mark.parametrize("fmt,K", [("int8", 384), ("bf16", 392)])
def test_large_tiles_keep_infinities_and_nan_apart(fmt, K, T, N):
    """Tokens with an infinity or a NaN, and bf16 weight rows with one, change
    no other outputs; the same input gives the same bits."""
    gen = torch.Generator(device="cuda").manual_seed(K)
    q, s, _ = weights(fmt, N, K, gen)
    x = torch.randn(T, K, generator=gen, device="cuda").bfloat16()
    w = m.linear_struct(q, s)
    ref, again, y = (torch.empty(T, N, device="cuda") for _ in range(3))
    m.moe_q4_linear(x, w, ref)
    m.moe_q4_linear(x, w, again)
    bad = torch.zeros(T, N, dtype=torch.bool, device="cuda")
    for t in (0, T // 2, T - 1):
        x[t, K - 1], x[t, 100] = float("inf"), float("nan")
        bad[t] = True
    if fmt == "bf16":
        for n in (1, N - 1):
            q[n, K - 1] = float("nan")
            bad[:, n] = True
    m.moe_q4_linear(x, w, y)
    torch.cuda.synchronize()
    assert torch.equal(ref, again)
    assert torch.isnan(y[bad]).all() and torch.equal(y[~bad], ref[~bad])


@pytest.mark.parametrize("fmt", ["int8", "bf16"])
@pytest.mark.parametrize("T,N", [(2, 130), (40, 70), (100, 130), (600, 4097)])
def test_most_inputs(fmt, T, N):
    """65536 inputs."""
    run(fmt, T, 65536, N, out=torch.float32, seed=N)


@pytest.mark.parametrize("T,N", [(1, 1 << 22), (20, (1 << 22) - 3), (70, 1 << 22), ((1 << 22) + 3, 17), ((1 << 22) + 3, 100)])
def test_most_outputs_and_tokens(T, N):
    """2^22 outputs (the longest rows) and more than 2^22 tokens, compared part by part."""
    gen = torch.Generator(device="cuda").manual_seed(N)
    q, s, w = weights("int8", N, 128, gen)
    x = torch.randn(T, 128, generator=gen, device="cuda").bfloat16()
    y = torch.full((T, N), float("nan"), device="cuda")
    m.moe_q4_linear(x, m.linear_struct(q, s), y)
    torch.cuda.synchronize()
    step = 1 << 20
    for t in range(0, T, step):
        for n in range(0, N, step):
            check(y[t:t + step, n:n + step], x[t:t + step], w[n:n + step], None, 0, None, f"T={T} N={N} at {t}, {n}")
