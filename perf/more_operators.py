"""Measured cases of a backbone's attention layers: the paged cache, the
attention that reads it and the norms around the blocks.

Three entry points: `moe_q4_kv_append` (norm of the heads, position rotation,
keys and values into the pages), `moe_q4_attention` (prompts, single tokens
and trees of drafted tokens over the pages) and `moe_q4_add_norm` (norm of a
block's output, gate, residual, norm before the next block).  With `own`
false, run() computes them in plain torch.
"""
import math
import random

import torch

own = False


# ------------------------------------------------------------------ cases

def _heads(q, kv, d, page):
    return {"hq": q, "hkv": kv, "d": d, "page": page}


def _append(lens, hist, heads, rot, norm, interleaved, far):
    """far: added to the cache index of a token to give its position"""
    return {"op": "append", "lens": lens, "hist": hist, **heads, "rot": rot, "norm": norm, "interleaved": interleaved,
            "far": far}


def _attention(lens, hist, heads, cap=0.0, window=0, slopes=False, prefix="", tree=False):
    """lens: new tokens of each sequence; hist: tokens before them"""
    return {"op": "attention", "lens": lens, "hist": hist, **heads, "cap": cap, "window": window, "slopes": slopes,
            "prefix": prefix, "tree": tree}


def _norm(T, H, u, post, gate, pre=True):
    return {"op": "norm", "T": T, "H": H, "u": u, "post": post, "gate": gate, "pre": pre}


def _text(v):
    return ",".join(str(x) for x in v)


def listed():
    spread = [100 + (7919 * i * i) % 24000 for i in range(63)]
    cases = {
        # one step of a batch of 16 streams: latency
        "append t16": _append(_text([1] * 16), _text(500 + 217 * i for i in range(16)), _heads(16, 2, 256, 64), 64, True,
                              False, 0),
        # packed prompts of very different lengths, far into their positions, small pages
        "append t8000": _append("1,300,2611,5088", "700,0,64,15", _heads(32, 8, 128, 16), 128, False, True, 1000000),
        # one token of one stream: latency
        "decode b1": _attention("1", "4096", _heads(16, 2, 256, 64)),
        # a decode batch whose streams are of very different ages
        "decode b64": _attention(_text([1] * 64), _text(spread + [32000]), _heads(32, 8, 128, 16)),
        # every score option at once, a head of keys for each head of queries, odd pages
        "decode capped b24": _attention(_text([1] * 23 + [3]), _text(13 + 389 * i for i in range(24)),
                                        _heads(12, 12, 64, 48), 30.0, 1024, True, _text([4] * 24)),
        # a small tree of drafted tokens of one stream: latency
        "tree b1": _attention("16", "2000", _heads(16, 2, 256, 64), tree=True),
        # drafts of a batch
        "tree b32": _attention(_text(33 + (i * 5) % 31 for i in range(32)), _text(500 + (i * 1327) % 7500 for i in range(32)),
                               _heads(32, 8, 128, 32), tree=True),
        # packed ragged prompts whose first part sees itself whole, scores biased by distance
        "prefill ragged": _attention("1,63,64,65,500,1307", "0,0,0,0,0,0", _heads(8, 2, 64, 16), slopes=True,
                                     prefix="1,10,64,33,100,257"),
        # one long prompt
        "prefill 1x8192": _attention("8192", "0", _heads(32, 8, 128, 64)),
        # the next pieces of long prompts over what the cache has of them, capped scores
        "prefill chunk": _attention("2048,1999,512", "6144,12001,29990", _heads(16, 2, 256, 64), cap=50.0),
        # between the experts' float output and the next mixer, one step of 16 streams
        "norm t16": _norm(16, 2048, "f32", False, "none"),
        # a prompt: norm, gate, residual, norm
        "norm t8192": _norm(8192, 4096, "bf16", True, "sigmoid"),
    }
    return [dict(c, name=n) for n, c in cases.items()]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_heads(rng):
    hkv = rng.choice([1, 2, 3, 4, 8])
    return _heads(hkv * rng.choice([1, 2, 4, 5, 7, 8]), hkv, rng.choice([64, 128, 256]), 16 * rng.choice([1, 2, 3, 4, 8, 16]))


def draw(rng):
    op = rng.choice(["append", "attention", "attention", "tree", "norm"])
    if op == "norm":
        H = 8 * _logint(rng, 8, 2048)
        T = _logint(rng, 1, 65536)
        while T * H > 8192 * 4096:
            T = max(1, T // 2)
        return _norm(T, H, rng.choice(["bf16", "f32"]), rng.random() < 0.5, rng.choice(["none", "none", "silu", "sigmoid"]),
                     rng.random() < 0.8)
    heads = _draw_heads(rng)
    d, hq, hkv = heads["d"], heads["hq"], heads["hkv"]
    if op == "append":
        B = _logint(rng, 1, 64)
        total = _logint(rng, B, 8000)
        cuts = sorted(rng.randint(0, total) for _ in range(B - 1))
        lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
        while sum(lens) * hq * d > 8000 * 32 * 128:
            lens = [n // 2 for n in lens]
        if not sum(lens):
            lens[0] = 1
        return _append(_text(lens), _text(rng.randint(0, 3000) for _ in lens), heads,
                       rng.choice([r for r in (16, 32, 64, 128, 256) if r <= d]), rng.random() < 0.5, rng.random() < 0.5,
                       rng.choice([0, 0, 1000000, 100000000]))
    if op == "tree":
        B = _logint(rng, 1, 32)
        lens = [rng.randint(1, 64) for _ in range(B)]
        hist = [_logint(rng, 1, 8000) for _ in range(B)]
    elif rng.random() < 0.5:  # single tokens, or a few
        B = _logint(rng, 1, 64)
        few = rng.choice([1, 1, 4])
        lens = [rng.randint(1, few) for _ in range(B)]
        hist = [_logint(rng, 1, 32000) - 1 for _ in range(B)]
    else:  # prompts, or pieces of prompts
        B = rng.randint(1, 8)
        total = _logint(rng, 64, 8192)
        cuts = sorted(rng.randint(0, total) for _ in range(B - 1))
        lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
        hist = [rng.choice([0, _logint(rng, 1, 30000)]) for _ in lens]

    def large():  # more than the largest listed cases: their batches filled up to the longest sequence, their products
        most = len(lens) * max(n + h for n, h in zip(lens, hist))
        pairs = sum(n * (n // 2 + h + 1) for n, h in zip(lens, hist))
        return (most * hkv * d > 64 * 32000 * 8 * 128 or most * max(lens) * hq > 3 * 32000 * 2048 * 16
                or 4 * d * hq * pairs > 4 * 128 * 32 * 8192 * 8192)

    while large():
        lens, hist = [(n + 1) // 2 for n in lens], [h // 2 for h in hist]
    prefix = ""
    if op == "attention" and rng.random() < 0.25:
        prefix = _text(rng.randint(0, n + h) for n, h in zip(lens, hist))
    return _attention(_text(lens), _text(hist), heads, rng.choice([0.0, 0.0, 20.0, 50.0]),
                      rng.choice([0, 0, 0, _logint(rng, 16, 8192)]), rng.random() < 0.25, prefix, op == "tree")


def _ints(text):
    return [int(n) for n in text.split(",")] if text else []


# ----------------------------------------------------------------- inputs

def _start(lens):
    start = [0]
    for n in lens:
        start.append(start[-1] + n)
    return start


def _draft_masks(lens, seed):
    """Random trees: each drafted token follows an earlier one of its draft, or
    the stream itself.  Bit j: the token follows token j, or is token j."""
    rng, masks = random.Random(seed), []
    for n in lens:
        own_masks = []
        for i in range(n):
            parent = rng.randint(max(-1, i - 6), i - 1)
            own_masks.append((own_masks[parent] if parent >= 0 else 0) | 1 << i)
        masks += own_masks
    return [v - (1 << 64) if v >> 63 else v for v in masks]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=dtype)

    st = {"case": dict(case)}
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        st["x"] = normal(T, H).mul_(3).bfloat16()
        st["u"] = normal(T, H) if case["u"] == "f32" else normal(T, H, dtype=torch.bfloat16)
        st["post"] = 1 + 0.2 * normal(H) if case["post"] else None
        st["pre"] = 1 + 0.2 * normal(H) if case["pre"] else None
        st["gate"] = normal(T, H, dtype=torch.bfloat16) if case["gate"] != "none" else None
        st["scale"], st["eps"] = 0.7, 1e-6
        st["x_out"] = torch.empty_like(st["x"])
        st["y"] = torch.empty_like(st["x"]) if case["pre"] else None
        if own:
            import quantized_moe_expert_amd as m
            st["m"] = m
            st["act"] = {"none": m.ACT_NONE, "silu": m.ACT_SILU, "sigmoid": m.ACT_SIGMOID}[case["gate"]]
        return st

    lens, hist = _ints(case["lens"]), _ints(case["hist"])
    hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]
    T, B = sum(lens), len(lens)
    kv = [n + h for n, h in zip(lens, hist)]
    need = [-(-n // page) for n in kv]
    # the pages of a sequence lie anywhere in the pool; entries behind its last page are not in use
    n_pages, cols = sum(need) + 3, max(need) + 1
    order = torch.randperm(n_pages, generator=gen, device="cuda").int()
    table = torch.full((B, cols), -1, dtype=torch.int32, device="cuda")
    filled = torch.arange(cols, device="cuda")[None] < torch.tensor(need, device="cuda")[:, None]
    table[filled] = order[:sum(need)]
    st["k_pages"], st["v_pages"] = (normal(n_pages, hkv, page, d, dtype=torch.bfloat16) for _ in range(2))
    st["table"], st["lens"], st["kv"] = table, lens, kv
    st["kv_len"] = torch.tensor(kv, dtype=torch.int32, device="cuda")
    st["seq_start"] = torch.tensor(_start(lens), dtype=torch.int32, device="cuda")
    if case["op"] == "append":
        # q, k and v are parts of the rows of one projection
        st["rows"] = rows = normal(T, (hq + 2 * hkv) * d, dtype=torch.bfloat16)
        st["q"] = rows[:, :hq * d].unflatten(1, (hq, d))
        st["k"] = rows[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
        st["v"] = rows[:, (hq + hkv) * d:].unflatten(1, (hkv, d))
        rot = case["rot"]
        st["inv_freq"] = (10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)).float()
        st["positions"] = None
        if case["far"]:
            at = [h + i + case["far"] for n, h in zip(lens, hist) for i in range(n)]
            st["positions"] = torch.tensor(at, dtype=torch.int32, device="cuda")
        st["q_norm"], st["k_norm"] = (1 + 0.2 * normal(d) if case["norm"] else None for _ in range(2))
        st["q_out"] = torch.empty(T, hq, d, dtype=torch.bfloat16, device="cuda")
        st["eps"] = 1e-6
    else:
        st["q"] = normal(T, hq, d).mul_(1.5).bfloat16()
        st["o"] = torch.empty_like(st["q"])
        st["scale"] = d ** -0.5
        # a token's distance costs from a ten-thousandth to a half
        st["slopes"] = 2.0 ** -(1 + 12 * torch.rand(hq, generator=gen, device="cuda")) if case["slopes"] else None
        st["prefix"] = torch.tensor(_ints(case["prefix"]), dtype=torch.int32, device="cuda") if case["prefix"] else None
        st["tree"] = None
        if case["tree"]:
            st["tree"] = torch.tensor(_draft_masks(lens, seed), dtype=torch.int64, device="cuda")
    if own:
        import quantized_moe_expert_amd as m
        st["m"] = m
        st["cache"] = m.kv_cache_struct(st["k_pages"], st["v_pages"], st["table"], st["kv_len"])
        if case["op"] == "attention":
            size = m.attention_workspace_size(T, B, hq, st["cache"])
            st["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    return st


# ------------------------------------------------------------- plain forms

def _rms(x, weight, eps):
    return x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * weight


def _plain_append(st):
    case = st["case"]
    T, page, rot = st["q"].shape[0], case["page"], case["rot"]
    t = torch.arange(T, device="cuda")
    seq = (t[:, None] >= st["seq_start"][None, 1:]).sum(1)
    index = st["kv_len"][seq] - st["seq_start"][seq + 1] + t
    pos = index if st["positions"] is None else st["positions"]
    angle = pos.double()[:, None] * st["inv_freq"].double()
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    q, k = st["q"].float(), st["k"].float()
    if case["norm"]:
        q, k = _rms(q, st["q_norm"], st["eps"]), _rms(k, st["k_norm"], st["eps"])

    def rotate(x):
        a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if case["interleaved"] else (x[..., :rot // 2], x[..., rot // 2:rot])
        a, b = a * cos - b * sin, b * cos + a * sin
        turned = torch.stack((a, b), -1).flatten(-2) if case["interleaved"] else torch.cat((a, b), -1)
        return torch.cat((turned, x[..., rot:]), -1)

    st["q_out"].copy_(rotate(q))
    at = st["table"][seq, index // page].long()
    st["k_pages"][at, :, index % page] = rotate(k).bfloat16()
    st["v_pages"][at, :, index % page] = st["v"]
    return [st["q_out"], st["k_pages"], st["v_pages"]]


def _plain_attention(st):
    """Every sequence filled up to the longest: scores, softmax, values."""
    case, lens = st["case"], st["lens"]
    hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]
    r, B, N, L = hq // hkv, len(lens), max(lens), max(st["kv"])
    key = torch.arange(L, device="cuda")
    at = st["table"][:, key // page].clamp(min=0).long()
    k = st["k_pages"][at, :, (key % page)[None]].permute(0, 2, 3, 1).float().contiguous()  # [B, hkv, d, L]
    v = st["v_pages"][at, :, (key % page)[None]].transpose(1, 2).float().contiguous()      # [B, hkv, L, d]
    there = key[None] < st["kv_len"][:, None]
    v = v * there[:, None, :, None]
    new = torch.arange(N, device="cuda")
    n = st["seq_start"].diff()[:, None]
    live = new[None] < n
    row = (st["seq_start"][:-1, None] + torch.minimum(new[None], (n - 1).clamp(min=0))).clamp(max=st["q"].shape[0] - 1).long()
    q = st["q"].float()[row].unflatten(2, (hkv, r)).permute(0, 2, 3, 1, 4).flatten(2, 3).contiguous()
    s = (q @ k).unflatten(2, (r, N)).mul_(st["scale"])  # [B, hkv, r, N, L]
    if case["cap"]:
        s = torch.tanh_(s.div_(case["cap"])).mul_(case["cap"])
    before = (st["kv_len"][:, None] - n)[..., None]  # tokens before the new ones
    if case["tree"]:
        bit = torch.arange(64, device="cuda")
        bits = (st["tree"][row][..., None] >> bit) & 1  # [B, N, 64]
        depth = bits.sum(-1) - bits.gather(-1, new.clamp(max=63)[None, :, None].expand(B, N, 1))[..., 0]
        drafted = key[None, None] - before  # key's place among the new tokens
        spot = drafted.clamp(0, 63)
        seen = (drafted < 0) | ((bits.gather(2, spot.expand(B, N, L)) == 1) & (drafted < n[..., None]))
        qpos = before + depth[..., None]
        kpos = torch.where(drafted < 0, key, before + depth.gather(1, spot[:, 0].clamp(max=N - 1))[:, None])
    else:
        qpos, kpos = before + new[:, None], key
        seen = kpos <= qpos
    if case["window"]:
        seen = seen & (qpos - kpos < case["window"])
    if case["prefix"]:
        seen = seen | (key < st["prefix"][:, None, None])
    seen = seen & there[:, None]
    if case["slopes"]:
        s = s - st["slopes"].view(hkv, r, 1, 1) * (qpos - kpos).abs()[:, None, None]
    s = s.masked_fill_(~seen[:, None, None], float("-inf"))
    top = s.amax(-1, keepdim=True)
    p = s.sub_(torch.where(top > float("-inf"), top, 0)).exp_()
    z = p.sum(-1, keepdim=True)
    o = (p.flatten(2, 3) @ v).unflatten(2, (r, N)) / torch.where(z > 0, z, 1)
    st["o"].copy_(o.permute(0, 3, 1, 2, 4).flatten(2, 3)[live])
    return st["o"]


def _plain_norm(st):
    case = st["case"]
    r = st["u"].float()
    if case["post"]:
        r = _rms(r, st["post"], st["eps"])
    if case["gate"] != "none":
        g = st["gate"].float()
        r = r * (1 / (1 + torch.exp(-g)) if case["gate"] == "sigmoid" else g / (1 + torch.exp(-g)))
    st["x_out"].copy_(st["x"].float() + st["scale"] * r)
    if not case["pre"]:
        return [st["x_out"]]
    st["y"].copy_(_rms(st["x_out"].float(), st["pre"], st["eps"]))
    return [st["x_out"], st["y"]]


# -------------------------------------------------------------------- run

def run(st):
    case = st["case"]
    op = case["op"]
    if not own:
        return {"append": _plain_append, "attention": _plain_attention, "norm": _plain_norm}[op](st)
    m = st["m"]
    if op == "append":
        m.moe_q4_kv_append(st["q"], st["k"], st["v"], st["seq_start"], st["cache"], st["q_out"], st["inv_freq"],
                           st["positions"], st["q_norm"], st["k_norm"], st["eps"], case["interleaved"])
        return [st["q_out"], st["k_pages"], st["v_pages"]]
    if op == "attention":
        m.moe_q4_attention(st["q"], st["seq_start"], st["cache"], st["o"], st["scale"], st["ws"], case["cap"],
                           case["window"], st["slopes"], st["prefix"], st["tree"])
        return st["o"]
    m.moe_q4_add_norm(st["x"], st["u"], st["x_out"], st["y"], st["pre"], st["post"], st["gate"], st["act"], st["scale"],
                      st["eps"])
    return [st["x_out"], st["y"]] if case["pre"] else [st["x_out"]]


def _seen(case):
    """(pairs of a query row and a key that it sees, keys that any row of their sequence sees)"""
    pairs = keys = 0
    w = case["window"] or 1 << 40
    prefixes = _ints(case["prefix"]) or [0] * len(_ints(case["lens"]))
    for n, h, pre in zip(_ints(case["lens"]), _ints(case["hist"]), prefixes):
        low = n + h
        for i in range(n):
            first = max(0, h + i + 1 - w)
            # a drafted token follows about three of its draft
            own_keys = min(i + 1, 3) if case["tree"] else i + 1
            pairs += max(0, h - first) + min(own_keys, w) if case["tree"] else h + i + 1 - first
            pairs += max(0, min(pre, first)) + max(0, pre - (h + i + 1))
            low = min(low, first)
        if n:
            keys += n + h - max(0, low - pre)
    return pairs, keys


def work(case):
    if case["op"] == "norm":
        T, H = case["T"], case["H"]
        b = T * H * (2 + (4 if case["u"] == "f32" else 2) + (2 if case["gate"] != "none" else 0) + (4 if case["pre"] else 2))
        return {"bytes": b + 4 * H * (case["post"] + case["pre"]), "flops": T * H * 12}
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    lens = _ints(case["lens"])
    T = sum(lens)
    if case["op"] == "append":
        return {"bytes": T * d * (hq + 2 * hkv) * 4 + 4 * T, "flops": T * d * (hq + hkv) * 6}
    pairs, keys = _seen(case)
    return {"bytes": 4 * T * hq * d + 4 * keys * hkv * d + (8 * T if case["tree"] else 0), "flops": 4 * d * hq * pairs}


# ------------------------------------------------------------ 64-bit forms

def _exact_append(st):
    case, lens = st["case"], st["lens"]
    page, rot = case["page"], case["rot"]
    q, k = st["q"].double(), st["k"].double()
    if case["norm"]:
        q, k = (x * torch.rsqrt(x.pow(2).mean(2, keepdim=True) + st["eps"]) * w.double()
                for x, w in ((q, st["q_norm"]), (k, st["k_norm"])))
    index = torch.cat([torch.arange(e - n, e, device="cuda") for n, e in zip(lens, st["kv"])])
    pos = index if st["positions"] is None else st["positions"].long()
    turn = torch.polar(torch.ones(1, dtype=torch.float64, device="cuda"), torch.outer(pos.double(), st["inv_freq"].double()))
    half = rot // 2
    a = torch.arange(half, device="cuda")
    a, b = (2 * a, 2 * a + 1) if case["interleaved"] else (a, a + half)

    def rotated(x):
        z = torch.complex(x[:, :, a], x[:, :, b]) * turn[:, None]
        x = x.clone()
        x[:, :, a], x[:, :, b] = z.real, z.imag
        return x

    pages = torch.cat([st["table"][i, torch.arange(e - n, e, device="cuda") // page] for i, (n, e) in enumerate(zip(lens, st["kv"]))])
    kp, vp = st["k_pages"].double(), st["v_pages"].double()
    kp[pages.long(), :, index % page] = rotated(k)
    vp[pages.long(), :, index % page] = st["v"].double()
    return [rotated(q), kp, vp]


def _exact_attention(st):
    case = st["case"]
    hq, hkv, d, page = case["hq"], case["hkv"], case["d"], case["page"]
    o = torch.zeros(st["o"].shape, dtype=torch.float64, device="cuda")
    masks = st["tree"].tolist() if case["tree"] else None
    t0 = 0
    for b, (n, e) in enumerate(zip(st["lens"], st["kv"])):
        if not n:
            continue
        pages = st["table"][b, :-(-e // page)].long()
        k, v = (x[pages].transpose(1, 2).reshape(-1, hkv, d)[:e].double().transpose(0, 1).contiguous()
                for x in (st["k_pages"], st["v_pages"]))
        place = torch.arange(e, device="cuda")
        where = torch.arange(e, dtype=torch.float64, device="cuda")
        ok = place[None] <= torch.arange(e - n, e, device="cuda")[:, None]
        if masks:
            own_masks = [x % (1 << 64) for x in masks[t0:t0 + n]]
            for i, x in enumerate(own_masks):
                where[e - n + i] = e - n + bin(x & ~(1 << i)).count("1")
            ok[:, e - n:] = torch.tensor([[x >> j & 1 == 1 for j in range(n)] for x in own_masks], device="cuda")
        step = max(1, (1 << 28) // (e * hq))
        for i in range(0, n, step):
            j = min(n, i + step)
            gap = where[e - n + i:e - n + j, None] - where[None]
            see = ok[i:j]
            if case["window"]:
                see = see & (gap < case["window"])
            if case["prefix"]:
                see = see | (place < int(st["prefix"][b]))[None]
            x = st["q"][t0 + i:t0 + j].double().reshape(j - i, hkv, hq // hkv, d).permute(1, 2, 0, 3)
            s = torch.matmul(x.reshape(hkv, -1, d), k.transpose(1, 2).contiguous()).view(hkv, hq // hkv, j - i, e) * st["scale"]
            if case["cap"]:
                s = torch.tanh(s / case["cap"]) * case["cap"]
            if case["slopes"]:
                s = s - st["slopes"].double().view(hkv, -1, 1, 1) * gap.abs()
            p = torch.softmax(torch.where(see, s, -torch.inf), -1)
            p = torch.where(see.any(-1)[:, None], p, torch.zeros_like(p))
            y = torch.matmul(p.reshape(hkv, -1, e), v).view(hkv, hq // hkv, j - i, d)
            o[t0 + i:t0 + j] = y.permute(2, 0, 1, 3).reshape(j - i, hq, d)
        t0 += n
    return o


def _exact_norm(st):
    case = st["case"]
    r = st["u"].double()
    if case["post"]:
        r = r * torch.rsqrt(r.pow(2).mean(1, keepdim=True) + st["eps"]) * st["post"].double()
    if case["gate"] == "silu":
        r = r * torch.nn.functional.silu(st["gate"].double())
    elif case["gate"] == "sigmoid":
        r = r * torch.sigmoid(st["gate"].double())
    x = st["x"].double() + st["scale"] * r
    if not case["pre"]:
        return [x]
    z = x.bfloat16().double()  # the next block reads the stream as it is stored
    return [x, z * torch.rsqrt(z.pow(2).mean(1, keepdim=True) + st["eps"]) * st["pre"].double()]


def exact(case, seed):
    st = prepare(case, seed)
    return {"append": _exact_append, "attention": _exact_attention, "norm": _exact_norm}[case["op"]](st)
