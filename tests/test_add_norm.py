"""moe_q4_add_norm against a float64 form (needs an MI355X).

Tolerance: a row's sum of squares is a lane's (at most 64 of them), a wave's
tree and up to 16 waves': off by at most 90 * 2^-24 relative, half of that in
the root; with the roundings of root, quotient and products 60 * 2^-24.  The
gate adds 8 * 2^-24 of its product.  x_out: the error of scale r, the sum's and the
last rounding.  y is held against the norm of the x_out that was stored.
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


def run(T, H, u="bf16", x=True, post=False, gate=None, act=0, pre=True, scale=0.7, eps=1e-6, x_out=True, in_place=False,
        seed=0, size=1.0, pad=8):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def rows(dtype=torch.bfloat16):
        return (torch.randn(T, H + pad, generator=gen, device="cuda") * size).to(dtype)[:, :H]

    def vec(on):
        return torch.randn(H, generator=gen, device="cuda") if on else None

    xs = rows() if x else None
    us = rows(torch.float32 if u == "f32" else torch.bfloat16) if u else None
    w_post, w_pre = vec(post), vec(pre)
    g = None
    if gate == "rows":
        g = rows() * 3
    elif gate == "one":
        g = rows()[:1]
    out = torch.full((T, H + 2 * pad), 5.0, dtype=torch.bfloat16, device="cuda")
    x_keep = None if xs is None else xs.clone()
    xo = xs if in_place else out[:, :H] if x_out else None
    yb = torch.full((T, H + pad), 5.0, dtype=torch.bfloat16, device="cuda")
    m.moe_q4_add_norm(xs, us, xo, yb[:, :H] if pre else None, w_pre, w_post, g, act, scale, eps)
    torch.cuda.synchronize()
    s = torch.zeros(T, H, dtype=torch.float64, device="cuda") if x_keep is None else x_keep.double()
    tol = torch.zeros_like(s)
    if us is not None:
        r = us.double()
        rel = 4 * U
        if post:
            r = r / (r.square().mean(1, keepdim=True) + eps).sqrt() * w_post.double()
            rel += 60 * U
        if g is not None:
            gd = g.double()
            r = r * (gd if act == m.ACT_NONE else torch.sigmoid(gd) if act == m.ACT_SIGMOID else gd * torch.sigmoid(gd))
            rel += 8 * U
        s = s + scale * r
        tol = rel * (scale * r).abs() + (2 * U + HALF) * s.abs()
    what = f"T={T} H={H} u={u} x={x} post={post} gate={gate} act={act} pre={pre}"
    worst = 0.0
    if xo is not None:
        worst = float(((xo.double() - s).abs() / (tol + 1e-30)).max())
        if us is None:
            assert torch.equal(xo, x_keep)
        if not in_place:
            assert (out[:, H:] == 5).all()
    if pre:
        # of the stored x_out; where it is not stored it may be the neighbour of the rounded value
        z = xo.double() if xo is not None else s.bfloat16().double()
        norm = (z.square().mean(1, keepdim=True) + eps).sqrt()
        want = z / norm * w_pre.double()
        bound = (HALF + 61 * U) * want.abs()
        if xo is None:
            bound = bound + (2 * HALF * s.abs() + tol) / norm * w_pre.double().abs() + 2 * HALF * want.abs()
        worst = max(worst, float(((yb[:, :H].double() - want).abs() / (bound + 1e-30)).max()))
        assert (yb[:, H:] == 5).all() and torch.isfinite(yb).all()
    print(f"{what}: largest error / tolerance {worst:.3f}", flush=True)
    assert worst <= 1, f"{what}: {worst}"


@pytest.mark.parametrize("H", [8, 16, 56, 64, 72, 128, 136, 256, 264, 512, 520, 1000, 2048, 2056, 4096, 4104, 8192, 8200, 16384,
                               16392, 32768, 32776, 65536])
@pytest.mark.parametrize("T", [1, 2, 33])
def test_widths(H, T):
    run(T, H, "f32", post=True, seed=H + T)
    run(T, H, "bf16", seed=H + T)


@pytest.mark.parametrize("u", ["bf16", "f32"])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate,act", [(None, 0), ("rows", 0), ("rows", 1), ("rows", 3), ("one", 0), ("one", 3)])
@pytest.mark.parametrize("pre,x,x_out", [(True, True, True), (False, True, True), (True, False, True), (True, True, False),
                                         (False, False, True), (True, False, False)])
@pytest.mark.parametrize("T,H", [(5, 128), (3, 1032)])
def test_forms(u, post, gate, act, pre, x, x_out, T, H):
    run(T, H, u, x, post, gate, act, pre, x_out=x_out, seed=3)


@pytest.mark.parametrize("T,H", [(1, 64), (7, 2048), (100, 4096)])
def test_plain_norm(T, H):
    """Without a block's output: the norm of x."""
    run(T, H, None, pad=0)
    run(T, H, None, x_out=False)


@pytest.mark.parametrize("T,H", [(9, 64), (9, 2048), (5, 20000)])
def test_in_place(T, H):
    run(T, H, "f32", post=True, in_place=True)
    run(T, H, "bf16", gate="rows", act=3, pre=False, in_place=True)


@pytest.mark.parametrize("size", [1e-12, 1e-4, 1e6, 1e15])
def test_sizes_of_values(size):
    run(6, 512, "f32", post=True, size=size)
    run(6, 512, "bf16", size=size, eps=0.0)


def test_zero_rows():
    """Rows of zeros, with eps and the norm's weight: zeros."""
    x = torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(256, device="cuda")
    xo, y = torch.ones_like(x), torch.ones_like(x)
    m.moe_q4_add_norm(x, x.float(), xo, y, w, w)
    torch.cuda.synchronize()
    assert (xo == 0).all() and (y == 0).all()


def test_a_row_does_not_touch_another():
    """NaN and infinities stay in their rows (several rows share a wave)."""
    for H in (8, 64, 200, 1024):
        gen = torch.Generator(device="cuda").manual_seed(H)
        x = torch.randn(40, H, generator=gen, device="cuda").bfloat16()
        u = torch.randn(40, H, generator=gen, device="cuda")
        w = torch.ones(H, device="cuda")
        outs = []
        for bad in (False, True):
            if bad:
                u[3, 0], u[17, H - 1], x[30, 2] = float("nan"), float("inf"), float("-inf")
            xo, y = torch.empty_like(x), torch.empty_like(x)
            m.moe_q4_add_norm(x, u, xo, y, w, w)
            outs.append((xo, y))
        torch.cuda.synchronize()
        keep = [i for i in range(40) if i not in (3, 17, 30)]
        for a, b in zip(*outs):
            assert torch.equal(a[keep], b[keep])
        assert torch.isnan(outs[1][1][3]).all()


def test_many_rows():
    run(70001, 64, "bf16", post=True)
    run(5000, 4096, "f32", gate="rows", act=1)


def test_the_same_input_twice():
    """u, gate and x may be the same memory."""
    x = torch.randn(9, 384, device="cuda").bfloat16()
    xo, y, w = torch.empty_like(x), torch.empty_like(x), torch.ones(384, device="cuda")
    m.moe_q4_add_norm(x, x, xo, y, w, None, x, m.ACT_SIGMOID)
    torch.cuda.synchronize()
    s = x.double() + x.double() * torch.sigmoid(x.double())
    assert bool(((xo.double() - s).abs() <= (HALF + 16 * U) * s.abs() + 16 * U * x.double().abs()).all())


def test_captured():
    x, u = torch.zeros(20, 512, dtype=torch.bfloat16, device="cuda"), torch.zeros(20, 512, device="cuda")
    w, y = torch.randn(512, device="cuda"), torch.zeros(20, 512, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        m.moe_q4_add_norm(x, u, x, y, w, w)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.moe_q4_add_norm(x, u, x, y, w, w)
    for _ in range(3):
        x.copy_(torch.randn(20, 512, device="cuda"))
        u.copy_(torch.randn(20, 512, device="cuda"))
        xe, ye = x.clone(), torch.empty_like(y)
        g.replay()
        torch.cuda.synchronize()
        m.moe_q4_add_norm(xe, u, xe, ye, w, w)
        torch.cuda.synchronize()
        assert torch.equal(x, xe) and torch.equal(y, ye)


def test_binding_refusals():
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    for bad in (lambda: m.moe_q4_add_norm(x, x[:3], x, None), lambda: m.moe_q4_add_norm(x, x.double(), x, None),
                lambda: m.moe_q4_add_norm(x, x, x.float(), None), lambda: m.moe_q4_add_norm(x, x, x.t(), None),
                lambda: m.moe_q4_add_norm(x, x, None, x, torch.ones(32, device="cuda")),
                lambda: m.moe_q4_add_norm(x, x, x, None, gate=x[:2])):
        with pytest.raises(ValueError):
            bad()
    w = torch.ones(64, device="cuda")
    for bad in (lambda: m.moe_q4_add_norm(x, None, None, None), lambda: m.moe_q4_add_norm(x, x.clone(), x, x, w),
                lambda: m.moe_q4_add_norm(x, None, torch.empty_like(x), None, gate=x),
                lambda: m.moe_q4_add_norm(x, x.clone(), torch.empty_like(x), None, gate=x, gate_act=m.ACT_GELU)):
        with pytest.raises(m.MoeQ4Error):
            bad()
