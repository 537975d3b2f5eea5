"""moe_q4_attention against a float64 form (needs an MI355X).  The tolerance is
derived in attention_cases.Case.check."""
from __future__ import annotations

import pytest
import torch

import quantized_moe_expert_amd as m
from attention_cases import Case, random_tree

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def both(case, what, **kw):
    o = case.run(**kw)
    torch.cuda.synchronize()
    case.check(o, what, **kw)
    return o


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (2, 2), (8, 2), (5, 1), (7, 1), (16, 1), (18, 1), (40, 1)])
def test_single_tokens(d, hq, hkv):
    hist = [0, 1, 14, 15, 16, 17, 30, 31, 32, 33, 47, 62, 63, 64, 100, 127, 128, 500, 1023, 2000]
    both(Case([1] * len(hist), hist, hq, hkv, d, 16, seed=hq), f"single d={d} {hq}/{hkv}")


@pytest.mark.parametrize("d,page", [(64, 16), (128, 48), (256, 64), (128, 4096)])
@pytest.mark.parametrize("hq,hkv", [(8, 2), (3, 3)])
@pytest.mark.parametrize("lens", [[1, 2, 3, 4, 5], [2] * 7, [8, 1, 16, 3], [15, 17, 31, 33], [63, 64, 65, 66, 1], [127, 0, 129],
                                  [200, 300], [1, 257, 2, 0, 511]])
def test_lengths(d, page, hq, hkv, lens):
    hist = [(i * 37 + 11 * n) % 150 for i, n in enumerate(lens)]
    both(Case(lens, hist, hq, hkv, d, page, seed=sum(lens)), f"{lens} d={d}")
    both(Case(lens, [0] * len(lens), hq, hkv, d, page, seed=sum(lens)), f"{lens} d={d}, nothing before")


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens,hist", [([1], [9000]), ([1, 1, 1], [20000, 3, 700]), ([3, 1], [5000, 5001]),
                                       ([40], [6000]), ([700], [3100]), ([1500, 20], [0, 8000])])
def test_long(d, lens, hist):
    both(Case(lens, hist, 4, 1, d, 64, seed=7), f"long {lens} {hist} d={d}")


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lens,hist", [([1] * 6, [0, 5, 40, 200, 1000, 3000]), ([3, 2, 1], [100, 0, 700]),
                                       ([30, 40], [33, 900]), ([150, 260], [0, 700])])
@pytest.mark.parametrize("opt", ["cap", "window", "window1", "slopes", "prefix", "all"])
def test_scores_and_masks(d, lens, hist, opt):
    c = Case(lens, hist, 6, 2, d, 32, seed=5)
    gen = torch.Generator(device="cuda").manual_seed(1)
    kw = {}
    if opt in ("cap", "all"):
        kw["cap"] = 3.0 if opt == "cap" else 30.0
    if opt == "window":
        kw["window"] = 70
    if opt == "window1":
        kw["window"] = 1
    if opt == "all":
        kw["window"] = 129
    if opt in ("slopes", "all"):
        kw["slopes"] = 2.0 ** -(8 * torch.rand(6, generator=gen, device="cuda"))
    if opt in ("prefix", "all"):
        kw["prefix"] = torch.tensor([[0, 3, 20, 400, 1, 64, 9][i % 7] for i in range(len(lens))], dtype=torch.int32,
                                    device="cuda")
    both(c, f"{opt} {lens} d={d}", **kw)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv", [(8, 2), (2, 2), (16, 1)])
@pytest.mark.parametrize("lens,hist", [([1], [0]), ([2], [50]), ([16], [100]), ([64], [333]), ([5, 33, 64, 1, 12], [0, 31, 700, 9, 64]),
                                       ([64, 63], [3000, 5])])
@pytest.mark.parametrize("opts", [{}, {"window": 40, "cap": 20.0}, {"slopes": True, "window": 3}])
def test_trees(d, hq, hkv, lens, hist, opts):
    c = Case(lens, hist, hq, hkv, d, 16, seed=3)
    kw = dict(opts)
    if kw.get("slopes"):
        kw["slopes"] = torch.linspace(0.01, 0.4, hq, device="cuda")
    both(c, f"tree {lens} d={d} {hq}/{hkv} {opts}", tree=random_tree(lens, 5), **kw)


@pytest.mark.parametrize("lens,hist", [([7], [0]), ([40, 9], [0, 20])])
def test_tree_masks_that_are_no_tree(lens, hist):
    """Any bits: rows that see nothing new, all, later ones, not themselves, rows behind the draft's end."""
    c = Case(lens, hist, 4, 2, 64, 16, seed=8)
    pattern = [0, -1, 1, 2, 1 << 62, -(1 << 63), 0x5555555555555555, 1 << 8, 3]
    tree = torch.tensor([pattern[i % 9] for i in range(sum(lens))], dtype=torch.int64, device="cuda")
    for kw in ({}, {"window": 5}, {"slopes": torch.tensor([0.1, 0.2, 0.3, 0.0], device="cuda")}):
        o = both(c, f"masks {lens} {kw}", tree=tree, **kw)
        if hist[0] == 0:
            assert (o[0] == 0).all()  # nothing cached, nothing seen


@pytest.mark.parametrize("lens", [[65], [100, 3], [129]])
def test_more_rows_than_a_mask_has_bits(lens):
    c = Case(lens, [10] * len(lens), 4, 2, 64, 16, seed=9)
    both(c, f"{lens} rows", tree=random_tree(lens, 2, reach=80))


def test_causal_tree_is_a_prompt():
    """A chain as a tree: the same formula as without one."""
    c = Case([64, 20], [100, 0], 8, 2, 128, 16, seed=2)
    tree = torch.tensor([(1 << (i + 1)) - 1 - (1 << 64 if i == 63 else 0) for n in (64, 20) for i in range(n)],
                        dtype=torch.int64, device="cuda")
    o = both(c, "chain", tree=tree)
    c.check(o, "chain against causal")


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("n", [1, 6, 40])
def test_nothing_to_see(n, tree):
    """No key at all, rows before the first token, sequences without rows, pages that are not there."""
    c = Case([n, 0, n, n, n], [0, 30, -n, 40, 40], 4, 2, 128, 16, seed=4)
    c.kv_len[0] = 0
    c.kv[0] = 0
    c.kv_len[2] = -5  # nothing, however it is put
    c.kv[2] = 0
    c.table[3] = -1                       # none of its pages
    c.table[4, 1] = c.k.shape[0]          # one of them
    kw = {"tree": random_tree(c.lens, 1)} if tree else {}
    o = c.run(**kw)
    torch.cuda.synchronize()
    assert (o[:2 * n] == 0).all() and (o[2 * n:3 * n] == 0).all()
    c.check(o, f"nothing {n}", **kw)


def test_rows_before_the_first_token():
    """More rows than tokens: the first ones have no index and see nothing."""
    for n, kv in ((3, 1), (20, 7), (150, 100)):
        c = Case([n], [kv - n], 2, 1, 64, 16, seed=n)
        o = both(c, f"{n} rows of {kv}")
        assert (o[:n - kv] == 0).all()


@pytest.mark.parametrize("n,kv", [(20, 7), (64, 40), (3, 1)])
def test_drafts_before_the_first_token(n, kv):
    c = Case([n], [kv - n], 4, 2, 64, 16, seed=n)
    for kw in ({}, {"window": 4}, {"slopes": torch.tensor([0.1, 0.0, 0.3, 1.0], device="cuda")}):
        both(c, f"{n} drafted of {kv} tokens {kw}", tree=random_tree([n], 3), **kw)


def test_table_that_is_too_short():
    """Keys behind the table are seen by nobody."""
    for n in (1, 30, 140):
        c = Case([n], [200], 4, 2, 64, 16, seed=1)
        c.table = c.table[:, :8].contiguous()
        c.cache = m.kv_cache_struct(c.k, c.v, c.table, c.kv_len)
        o = c.run()
        torch.cuda.synchronize()
        ref = Case([n], [200], 4, 2, 64, 16, seed=1)
        ref.table[:, 8:] = -1
        ref.check(o, f"short table {n}")


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n,hist", [(1, 100), (9, 70), (64, 0), (200, 37), (300, 0)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_what_is_not_seen_does_not_count(d, n, hist, bad):
    """NaN and infinities in later tokens, outside the window and in the rest of the last page."""
    window = 50
    c = Case([n], [hist], 4, 2, d, 32, seed=6)
    clean = c.run(window=window)
    torch.cuda.synchronize()
    e = n + hist
    spoiled = [i for i in range(e) if i % 7 == 3 or i == e - 1]
    for i in spoiled:
        p, at = int(c.table[0, i // 32]), i % 32
        c.k[p, :, at, ::5] = bad
        c.v[p, :, at, 1::3] = bad
    o = c.run(window=window)
    torch.cuda.synchronize()
    for t in range(n):
        sees = [i for i in spoiled if hist + t - window < i <= hist + t]
        if not sees:
            assert torch.equal(o[t], clean[t]), t
        elif bad != bad:
            assert torch.isnan(o[t]).any(), t
    c2 = Case([n], [hist], 4, 2, d, 32, seed=6)
    prefix = torch.tensor([2], dtype=torch.int32, device="cuda")
    clean = c2.run(window=3, prefix=prefix)
    for i in range(2, e - n - 3):
        p, at = int(c2.table[0, i // 32]), i % 32
        c2.k[p, :, at], c2.v[p, :, at] = bad, bad
    assert torch.equal(c2.run(window=3, prefix=prefix), clean)


@pytest.mark.parametrize("n", [12, 40])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_siblings_in_a_tree_do_not_count(n, bad):
    c = Case([n], [37], 8, 2, 128, 16, seed=6)
    tree = random_tree([n], 11)
    clean = c.run(tree=tree)
    j = n // 2
    p, at = int(c.table[0, (37 + j) // 16]), (37 + j) % 16
    c.k[p, :, at], c.v[p, :, at] = bad, bad
    o = c.run(tree=tree)
    torch.cuda.synchronize()
    for t, x in enumerate(tree.tolist()):
        if x >> j & 1:
            assert not torch.isfinite(o[t]).all()
        else:
            assert torch.equal(o[t], clean[t]), t


@pytest.mark.parametrize("n,hist", [(1, 90), (5, 3), (70, 40), (200, 0)])
def test_strides_and_rows_behind_the_last(n, hist):
    """q and o as parts of wider rows; rows behind the last sequence stay."""
    c = Case([n, n], [hist, hist + 1], 4, 2, 64, 16, seed=n, tail=3)
    wide = torch.randn(c.T, 4 * 64 + 72, device="cuda").bfloat16()
    wide[:, 40:40 + 256] = c.q.flatten(1)
    out = torch.full((c.T, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    o = out[:, 128:384].unflatten(1, (4, 64))
    c.run(q=wide[:, 40:296].unflatten(1, (4, 64)), o=o)
    torch.cuda.synchronize()
    c.check(o, f"strides {n}")
    assert (out[:, :128] == 7).all() and (out[:, 384:] == 7).all() and (out[2 * n:] == 7).all()


@pytest.mark.parametrize("n", [1, 20, 150])
def test_far_pages(n):
    """Pages behind 2^32 elements of the pool."""
    pool = (1 << 32) // (2 * 64 * 128) + 50
    c = Case([n], [300], 4, 2, 128, 64, seed=1, pool=pool)
    both(c, f"far {n}")


def test_shared_pages():
    """Two sequences that read the same first pages."""
    c = Case([1, 1], [64, 64], 4, 2, 64, 32, seed=1)
    c.table[1, :2] = c.table[0, :2]
    c.dense[1] = tuple(torch.cat((a[:64], b[64:])) for a, b in zip(c.dense[0], c.dense[1]))
    both(c, "shared pages")


@pytest.mark.parametrize("B", [300, 5000])
def test_many_sequences(B):
    lens = [1 if i % 3 else (i // 3) % 3 for i in range(B)]
    both(Case(lens, [(i * 13) % 40 for i in range(B)], 2, 1, 64, 16, seed=1), f"{B} sequences")


@pytest.mark.parametrize("lens,hist", [([1, 1], [300, 2000]), ([50], [100]), ([300], [0])])
def test_large_scores(lens, hist):
    """Scores of hundreds: the maximum moves far, most weights vanish."""
    both(Case(lens, hist, 4, 2, 128, 16, seed=3, q_scale=60.0, v_mean=5.0), f"large {lens}")


def test_equal_scores():
    """q = 0: the mean of the values."""
    for n, h in ((1, 700), (30, 40), (200, 0)):
        both(Case([n], [h], 4, 2, 128, 16, seed=3, q_scale=0.0, v_mean=3.0), f"equal {n}")


@pytest.mark.parametrize("lens,hist", [([1] * 4, [100, 4000, 20, 900]), ([20], [700]), ([400, 3], [100, 2000])])
def test_same_bits(lens, hist):
    c = Case(lens, hist, 8, 2, 128, 16, seed=3)
    o = c.run()
    size = m.attention_workspace_size(c.T, len(lens), 8, c.cache)
    for fill in (0, 255, 127):
        assert torch.equal(c.run(ws=torch.full((size + 256,), fill, dtype=torch.uint8, device="cuda")), o)


@pytest.mark.parametrize("lens", [[1, 1, 1], [1, 2, 0], [30, 5, 2], [140, 7, 60]])
def test_captured(lens):
    """Two graphs that share a workspace, replayed in turn while the cache
    grows, each replay against an eager call."""
    hists = [[50, 700, 3], [60, 900, 40], [0, 0, 0], [2000, 10, 17]]
    cases = [Case(lens, [2001] * 3, 4, 2, 64, 16, seed=s, cols=140) for s in (1, 2)]
    size = max(m.attention_workspace_size(c.T, 3, 4, c.cache) for c in cases)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    outs, graphs = [torch.zeros_like(c.q) for c in cases], []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for c, o in zip(cases, outs):
            c.run(o=o, ws=ws)
    torch.cuda.current_stream().wait_stream(side)
    for c, o in zip(cases, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run(o=o, ws=ws)
        graphs.append(g)
    for hist in hists:
        for c in cases:
            c.kv_len.copy_(torch.tensor([n + h for n, h in zip(lens, hist)], dtype=torch.int32))
            c.q.copy_(torch.randn(c.q.shape, device="cuda"))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for c, o in zip(cases, outs):
            assert torch.equal(o, c.run())


def test_two_streams():
    jobs = [(Case(lens, hist, 8, 2, 128, 16, seed=3), torch.cuda.Stream()) for lens, hist in (([1, 1], [3000, 70]), ([90], [500]))]
    want = [c.run() for c, _ in jobs]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for c, s in jobs:
            with torch.cuda.stream(s):
                got.append(c.run())
    torch.cuda.synchronize()
    for i, o in enumerate(got):
        assert torch.equal(o, want[i % 2])


def test_binding_refusals():
    c = Case([2], [3], 4, 2, 64, 16)
    for bad in (lambda: c.run(q=c.q.float()), lambda: c.run(q=c.q[:, :, :32]), lambda: c.run(q=c.q.transpose(0, 1)),
                lambda: c.run(slopes=torch.zeros(3, device="cuda")), lambda: c.run(tree=torch.zeros(2, device="cuda")),
                lambda: c.run(prefix=torch.zeros(1, dtype=torch.int32)),
                lambda: m.kv_cache_struct(c.k[:, :, :, :32], c.v, c.table, c.kv_len),
                lambda: m.kv_cache_struct(c.k, c.v, c.table, c.kv_len.long()),
                lambda: m.kv_cache_struct(c.k.cpu(), c.v, c.table, c.kv_len)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(m.MoeQ4Error):
        c.run(prefix=torch.zeros(1, dtype=torch.int32, device="cuda"), tree=torch.zeros(2, dtype=torch.int64, device="cuda"))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("scale", [-0.1, 0.0, 1e-30, 2.0])
@pytest.mark.parametrize("lens,hist", [([1, 2], [100, 600]), ([70], [40])])
def test_scales(d, scale, lens, hist):
    for kw in ({}, {"cap": 5.0}, {"slopes": torch.tensor([0.5, 0.01, 0.0, 1.0], device="cuda")}):
        c = Case(lens, hist, 4, 2, d, 16, seed=3, q_scale=0.5)
        c.scale = scale
        both(c, f"scale {scale} {kw}", **kw)


@pytest.mark.parametrize("cap", [1e-30, 1e-3, 1e6])
def test_caps_of_any_size(cap):
    for lens, hist in (([1], [300]), ([60], [20])):
        both(Case(lens, hist, 4, 2, 128, 16, seed=3), f"cap {cap}", cap=cap)


@pytest.mark.parametrize("window", [2, 1000, (1 << 31) - 1])
@pytest.mark.parametrize("lens,hist", [([1, 1], [2500, 10]), ([100], [1500])])
def test_windows(window, lens, hist):
    both(Case(lens, hist, 4, 2, 64, 16, seed=3), f"window {window}", window=window)
    both(Case(lens, hist, 4, 2, 64, 16, seed=3), f"window {window} and prefix", window=window,
         prefix=torch.full((len(lens),), 70, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("hq", [100, 300, 1024])
def test_many_query_heads_on_one(hq):
    for lens, hist in (([1, 2], [50, 700]), ([5], [0])):
        both(Case(lens, hist, hq, 1, 64, 16, seed=1), f"{hq} heads on one")


@pytest.mark.parametrize("lens,hist", [([200] + [1] * 300, [50] + [7] * 300), ([300, 1, 1, 1], [10, 2000, 5, 0]),
                                       ([0] * 70 + [40], [3] * 71), ([0] * 200 + [1], [5] * 200 + [3000])])
def test_sequences_of_another_kind(lens, hist):
    """A prompt among single tokens, single tokens beside a prompt, sequences without rows."""
    both(Case(lens, hist, 4, 2, 64, 16, seed=1), f"{len(lens)} sequences")


@pytest.mark.parametrize("d,n", [(64, 1), (128, 1), (64, 33), (256, 20)])
def test_more_than_a_wave_of_sequences(d, n):
    """The plan over several waves, with blocks that are split."""
    B = 90
    hist = [(i * 17) % 60 for i in range(B)]
    hist[5], hist[70], hist[89] = 3000, 1500, 2200
    both(Case([n + i % 2 for i in range(B)], hist, 4, 1, d, 32, seed=1), f"{B} sequences of {n} rows")


def test_starts_that_do_not_ascend_stay_in_bounds():
    """Numbers are undefined; nothing outside o and the workspace is written (guard bytes on both sides)."""
    for B, n in ((40, 1), (300, 1), (40, 30), (300, 9)):
        c = Case([n] * B, [200] * B, 4, 2, 64, 16, seed=1)
        gen = torch.Generator().manual_seed(2)
        c.start.copy_(torch.randint(-5, c.T + 9, (B + 1,), generator=gen))
        size = m.attention_workspace_size(c.T, B, 4, c.cache)
        ws = torch.full((size + 512,), 77, dtype=torch.uint8, device="cuda")
        out = torch.full((c.T + 16, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        c.run(o=out[8:8 + c.T], ws=ws[256:256 + size])
        torch.cuda.synchronize()
        assert (ws[:256] == 77).all() and (ws[256 + size:] == 77).all()
        assert (out[:8] == 7).all() and (out[8 + c.T:] == 7).all()
