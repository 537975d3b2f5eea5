"""moe_q4_attention at the edges of its arguments (needs an MI355X)."""
from __future__ import annotations

import pytest
import torch

import quantized_moe_expert_amd as m
from attention_cases import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens,hist", [([1, 1], [7, 300]), ([40], [20]), ([200, 3], [0, 0])])
@pytest.mark.parametrize("cap", [0.0, 30.0, 1e6])
def test_slopes_near_the_largest_float(lens, hist, d, cap):
    """A distance of 1 costs everything: a row's own value is left."""
    c = Case(lens, hist, 4, 2, d, 16, seed=1)
    o = c.run(cap=cap, slopes=torch.full((4,), 3.3e38, device="cuda"))
    torch.cuda.synchronize()
    t = 0
    for b, n in enumerate(lens):
        own = c.dense[b][1][c.kv[b] - n:].repeat_interleave(2, 1)
        tol = 2.0 ** -7 * own.abs().float()  # the weight's rounding and the last one
        assert bool(((o[t:t + n].float() - own.float()).abs() <= tol).all()), b
        t += n


@pytest.mark.parametrize("used", [1, 2, 3])
def test_fewer_sequences_than_the_table_has(used):
    """seq_start of the first ones: the same as a table of that many rows."""
    lens, hist, T = [2, 1, 3, 1], [40, 0, 700, 5], sum([2, 1, 3, 1][:used])
    c = Case(lens, hist, 4, 2, 64, 16, seed=3)
    few = m.kv_cache_struct(c.k, c.v, c.table[:used], c.kv_len[:used])
    prefix = torch.full((used,), 3, dtype=torch.int32, device="cuda")
    ws = torch.empty(m.attention_workspace_size(T, used, 4, c.cache), dtype=torch.uint8, device="cuda")
    outs = []
    for cache in (c.cache, few):
        o = torch.empty_like(c.q[:T])
        m.moe_q4_attention(c.q[:T], c.start[:used + 1], cache, o, c.scale, ws, window=9, prefix=prefix)
        outs.append(o)
    assert torch.equal(*outs)
    new = torch.randn(T, 2, 64, device="cuda").bfloat16()
    for cache in (c.cache, few):
        k0 = c.k.clone()
        m.moe_q4_kv_append(None, new, new, c.start[:used + 1], cache, None)
        outs.append(c.k.clone())
        c.k.copy_(k0)
    assert torch.equal(outs[2].view(torch.int16), outs[3].view(torch.int16)) and not torch.equal(
        outs[2].view(torch.int16), c.k.view(torch.int16))
    torch.cuda.synchronize()
    for start in (c.start[:1], torch.zeros(6, dtype=torch.int32, device="cuda")):
        with pytest.raises(ValueError):
            m.moe_q4_attention(c.q[:T], start, c.cache, o, c.scale, ws)


@pytest.mark.parametrize("lens", [[1], [2, 5], [1, 1, 1], [30, 1, 2]])
def test_mixer_with_fewer_sequences(lens):
    """One mixer, batches of one to max_seqs sequences: as a mixer of that size."""
    hq, hkv, d, H, B = 4, 2, 64, 256, len(lens)
    gen = torch.Generator(device="cuda").manual_seed(1)
    w_in, w_out = ((torch.randn(n, k, generator=gen, device="cuda") / k ** 0.5).bfloat16()
                   for n, k in (((hq + 2 * hkv) * d, H), (H, hq * d)))
    k, v = (torch.zeros(12, hkv, 16, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = torch.arange(12, dtype=torch.int32, device="cuda").reshape(3, 4)
    kv_len = torch.tensor(lens + [0] * (3 - B), dtype=torch.int32, device="cuda")
    start = torch.tensor([sum(lens[:i]) for i in range(B + 1)], dtype=torch.int32, device="cuda")
    x = torch.randn(sum(lens), H, generator=gen, device="cuda").bfloat16()
    got = []
    for cache, n in ((m.kv_cache_struct(k, v, table, kv_len), 3), (m.kv_cache_struct(k, v, table[:B], kv_len[:B]), B)):
        mixer = m.AttentionMixer(m.linear_struct(w_in), m.linear_struct(w_out), hq, cache, 33, n)
        got.append(mixer.forward(x, start, torch.empty_like(x)))
        torch.cuda.synchronize()
    assert torch.equal(*got)


@pytest.mark.parametrize("window", [-1, 1 << 31, (1 << 32) + 5])
def test_windows_that_do_not_fit_are_refused(window):
    """Not cut to 32 bits: 2^32 + 5 would be a window of 5."""
    c = Case([1], [40], 4, 2, 64, 16)
    with pytest.raises((ValueError, m.MoeQ4Error)):
        c.run(window=window)
