"""Measured cases of the operators beside the experts in a backbone layer.

Three operators: the linear layer (`moe_q4_linear`: int8 group-128 or bf16
weights, with bias, activation and residual), the gated delta rule
(`moe_q4_delta_decode`, `moe_q4_delta_prefill`) and the scores of given tokens
(`moe_q4_logprobs`).  With `own` false, run() computes them in plain torch.
"""
import math

import torch

own = False

GROUP = 128  # inputs per int8 weight scale
CHUNK = 64   # tokens per step of the plain delta rule


# ------------------------------------------------------------------ cases

def _linear(fmt, T, K, N, act="none", bias=False, residual=False, out="bf16"):
    return {"op": "linear", "fmt": fmt, "T": T, "K": K, "N": N, "act": act, "bias": bias, "residual": residual,
            "out": out}


def _delta(kind, lens, hk, hv, dk, dv, norm):
    return {"op": "delta", "kind": kind, "lens": lens, "hk": hk, "hv": hv, "dk": dk, "dv": dv, "norm": norm}


def _logprobs(T, V, n, dtype):
    return {"op": "logprobs", "T": T, "V": V, "n": n, "dtype": dtype}


def listed():
    cases = {
        # one token of one stream through the output head (4097 sampleable rows, bf16): latency
        "linear head t1": _linear("bf16", 1, 2048, 4097),
        # a decode batch through a mixer's fused input projection, int8 weights
        "linear in t16": _linear("int8", 16, 2048, 12288),
        # a short ragged prompt through a mixer's output projection, added to the stream
        "linear out t300": _linear("int8", 300, 4096, 2048, residual=True),
        # a long prompt through a wide int8 layer with bias and activation
        "linear wide t4096": _linear("int8", 4096, 2048, 8192, act="silu", bias=True),
        # scoring a prompt: the output head over many rows, odd width, float logits
        "linear head t1000": _linear("bf16", 1000, 2048, 4097, out="f32"),
        # one decoded token of one sequence: latency
        "delta decode b1": _delta("decode", "1", 16, 32, 128, 128, True),
        # a decode batch of 64 sequences
        "delta decode b64": _delta("decode", ",".join(["1"] * 64), 16, 32, 128, 128, True),
        # a packed batch of short ragged prompts, small heads, keys normalised by the caller
        "delta prefill ragged": _delta("prefill", "1,63,64,65,500,1307", 4, 8, 64, 64, False),
        # one long prompt: the state's chain is the bound
        "delta prefill 1x8192": _delta("prefill", "8192", 16, 32, 128, 128, True),
        # a batch of prompts
        "delta prefill 8x2048": _delta("prefill", ",".join(["2048"] * 8), 16, 32, 128, 128, True),
        # scores of one sampled token: latency
        "logprobs t1": _logprobs(1, 4097, 8, "bf16"),
        # scores of a prompt over a large vocabulary
        "logprobs t512": _logprobs(512, 151939, 20, "bf16"),
    }
    return [dict(c, name=n) for n, c in cases.items()]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "delta", "logprobs"])
    if op == "linear":
        fmt = rng.choice(["int8", "bf16"])
        T, N = _logint(rng, 1, 4096), _logint(rng, 16, 16384)
        K = GROUP * _logint(rng, 2, 64) if fmt == "int8" else 8 * _logint(rng, 32, 1024)
        while T * K * N > 4096 * 2048 * 8192:
            T = max(1, T // 2)
        return _linear(fmt, T, K, N, rng.choice(["none", "silu", "gelu"]), rng.random() < 0.5, rng.random() < 0.5,
                       rng.choice(["bf16", "bf16", "f32"]))
    if op == "delta":
        hk, r = rng.choice([1, 2, 4, 8, 16]), rng.choice([1, 2, 4])
        hv, dk, dv = min(32, hk * r), rng.choice([64, 128]), rng.choice([64, 128])
        if rng.random() < 0.5:
            lens = [rng.randint(1, 3) for _ in range(_logint(rng, 1, 64))]
            return _delta("decode", ",".join(map(str, lens)), hk, hv, dk, dv, rng.random() < 0.5)
        n = rng.randint(1, 12)
        total = _logint(rng, 64, 16384)
        cuts = sorted(rng.randint(0, total) for _ in range(n - 1))
        lens = [b - a for a, b in zip([0] + cuts, cuts + [total])]
        return _delta("prefill", ",".join(map(str, lens)), hk, hv, dk, dv, rng.random() < 0.5)
    T, V = _logint(rng, 1, 4096), _logint(rng, 1000, 160000)
    while T * V > 512 * 151939:
        T = max(1, T // 2)
    return _logprobs(T, V, rng.randint(1, 32), rng.choice(["bf16", "f32"]))


# ----------------------------------------------------------------- inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    st = {"case": dict(case)}
    if case["op"] == "linear":
        T, K, N = case["T"], case["K"], case["N"]
        st["x"] = normal(T, K).bfloat16()
        if case["fmt"] == "int8":
            st["q"] = torch.randint(-127, 128, (N, K), generator=gen, device="cuda", dtype=torch.int8)
            st["scale"] = (torch.rand(N, K // GROUP, generator=gen, device="cuda") + 0.5).mul(2.0 / 127 / K ** 0.5).half()
        else:
            st["q"], st["scale"] = (normal(N, K) / K ** 0.5).bfloat16(), None
        st["bias"] = normal(N) if case["bias"] else None
        st["residual"] = normal(T, N).bfloat16() if case["residual"] else None
        st["y"] = torch.empty(T, N, device="cuda", dtype=torch.float32 if case["out"] == "f32" else torch.bfloat16)
    elif case["op"] == "delta":
        lens = [int(n) for n in case["lens"].split(",")]
        hk, hv, dk, dv = case["hk"], case["hv"], case["dk"], case["dv"]
        T, B = sum(lens), len(lens)
        # q, k and v are parts of the rows of one projection
        rows = normal(T, 2 * hk * dk + hv * dv)
        if not case["norm"]:
            qk = rows[:, :2 * hk * dk].unflatten(1, (2 * hk, dk))
            qk /= qk.square().sum(-1, keepdim=True).sqrt()
        st["rows"] = rows = rows.bfloat16()
        st["q"] = rows[:, :hk * dk].unflatten(1, (hk, dk))
        st["k"] = rows[:, hk * dk:2 * hk * dk].unflatten(1, (hk, dk))
        st["v"] = rows[:, 2 * hk * dk:].unflatten(1, (hv, dv))
        # log decay -A softplus(a): heads forget over a few to a few thousand tokens
        rate = torch.exp(torch.rand(hv, generator=gen, device="cuda") * 7 - 7)
        st["g"] = -rate * torch.log1p(torch.exp(normal(T, hv)))
        st["beta"] = 1 / (1 + torch.exp(-normal(T, hv)))
        start = [0]
        for n in lens:
            start.append(start[-1] + n)
        st["lens"], st["seq_start"] = lens, torch.tensor(start, dtype=torch.int32, device="cuda")
        # states live in a pool, in another order than the sequences
        st["state_idx"] = torch.randperm(B, generator=gen, device="cuda").int()
        st["state_in"] = normal(B, hv, dk, dv) * 0.1
        st["state_out"] = torch.empty_like(st["state_in"])
        st["o"] = torch.empty(T, hv, dv, dtype=torch.bfloat16, device="cuda")
        st["scale"] = dk ** -0.5
    else:
        T, V, n = case["T"], case["V"], case["n"]
        st["logits"] = normal(T, V).mul_(2.5)
        # some tokens may not be sampled
        st["logits"].masked_fill_(torch.rand(V, generator=gen, device="cuda") < 0.05, float("-inf"))
        if case["dtype"] == "bf16":
            st["logits"] = st["logits"].bfloat16()
        st["tokens"] = torch.randint(0, V, (T,), generator=gen, device="cuda", dtype=torch.int32)
        st["tokens"][3::7] = -1  # positions that are not scored
        new = {"dtype": torch.float32, "device": "cuda"}
        st["logprob"], st["entropy"] = torch.empty(T, **new), torch.empty(T, **new)
        st["top_idx"], st["top_logprob"] = torch.empty(T, n, dtype=torch.int32, device="cuda"), torch.empty(T, n, **new)
    if own:
        import quantized_moe_expert_amd as m
        st["m"] = m
        if case["op"] == "linear":
            st["act"] = {"none": m.ACT_NONE, "silu": m.ACT_SILU, "gelu": m.ACT_GELU}[case["act"]]
            st["w"] = m.linear_struct(st["q"], st["scale"], st["bias"])
        elif case["op"] == "delta" and case["kind"] == "prefill":
            need = m.delta_workspace_size(T, B, hk, hv, dk, dv)
            st["ws"] = torch.empty(need, dtype=torch.uint8, device="cuda")
        elif case["op"] == "logprobs":
            need = m.logprobs_workspace_size(T, V, n)
            st["ws"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    return st


# ------------------------------------------------------------- plain forms

def _plain_linear(st):
    case = st["case"]
    w = st["q"].float()
    if st["scale"] is not None:
        w = (w.unflatten(1, (-1, GROUP)) * st["scale"].float()[..., None]).flatten(1)
    y = st["x"].float() @ w.t()
    if st["bias"] is not None:
        y = y + st["bias"]
    if case["act"] == "silu":
        y = y / (1 + torch.exp(-y))
    elif case["act"] == "gelu":
        y = 0.5 * y * (1 + torch.erf(y * 0.5 ** 0.5))
    if st["residual"] is not None:
        y = y + st["residual"].float()
    st["y"].copy_(y)
    return st["y"]


def _plain_delta(st):
    """The rule in chunks: within a chunk the updates u solve a unit lower
    triangular system; the state goes from chunk to chunk."""
    case, lens = st["case"], st["lens"]
    hk, hv, dk, dv = case["hk"], case["hv"], case["dk"], case["dv"]
    B, C = len(lens), min(CHUNK, max(max(lens), 1))
    N = max(1, -(-max(lens) // C))
    # packed rows -> [B, N * C] slots and back
    pos = torch.arange(N * C, device="cuda")
    n = st["seq_start"].diff()[:, None]
    live = pos[None] < n
    at = (st["seq_start"][:-1, None] + torch.minimum(pos[None], (n - 1).clamp(min=0))).clamp(max=st["g"].shape[0] - 1).long()

    def slots(t):  # [T, h, ...] -> [N, B * hv, C, ...], heads repeated, empty slots 0
        t = t.float()[at] * live.reshape(B, N * C, *[1] * (t.dim() - 1))
        t = t.repeat_interleave(hv // t.shape[2], dim=2)
        t = t.unflatten(1, (N, C)).transpose(2, 3)  # [B, N, hv, C, ...]
        return t.transpose(0, 1).flatten(1, 2).contiguous()

    q, k, v, g, beta = (slots(st[x]) for x in ("q", "k", "v", "g", "beta"))
    if case["norm"]:
        q = q / (q.square().sum(-1, keepdim=True) + 1e-6).sqrt()
        k = k / (k.square().sum(-1, keepdim=True) + 1e-6).sqrt()
    q = q * st["scale"]
    G = g.cumsum(-1)
    low = torch.ones(C, C, dtype=torch.bool, device="cuda").tril()
    decay = torch.exp((G[..., :, None] - G[..., None, :]).masked_fill(~low, float("-inf")))
    kt = k.transpose(-1, -2).contiguous()
    A = beta[..., None] * decay * (k @ kt)
    P = decay * (q @ kt)
    rhs = torch.cat([beta[..., None] * v, (beta * torch.exp(G))[..., None] * k], -1)
    for i in range(1, C):  # forward substitution, all chunks at once
        rhs[..., i, :] -= (A[..., i, :i, None] * rhs[..., :i, :]).sum(-2)
    U, W = rhs[..., :dv].contiguous(), rhs[..., dv:].contiguous()
    qg = q * torch.exp(G)[..., None]
    last = torch.exp(G[..., -1])[..., None, None]
    kd = (kt * torch.exp(G[..., -1:] - G)[..., None, :]).contiguous()
    idx = st["state_idx"].long()
    S = st["state_in"][idx].flatten(0, 1)
    o = torch.empty(N, B * hv, C, dv, device="cuda")
    for c in range(N):
        u = U[c] - W[c] @ S
        o[c] = qg[c] @ S + P[c] @ u
        S = last[c] * S + kd[c] @ u
    st["state_out"][idx] = S.unflatten(0, (B, hv))
    o = o.unflatten(1, (B, hv)).permute(1, 0, 3, 2, 4).flatten(1, 2)  # [B, N * C, hv, dv]
    st["o"].copy_(o[live])
    return [st["o"], st["state_out"]]


def _plain_logprobs(st):
    n, V = st["case"]["n"], st["case"]["V"]
    l = st["logits"].float()
    top, idx = torch.sort(l, dim=1, descending=True, stable=True)
    idx = idx[:, :n].int()
    top, m = top[:, :n], top[:, :1]
    x = l - m
    e = torch.exp(x)
    z = e.sum(1, dtype=torch.float64)
    logz = torch.log(z)
    t = st["tokens"].long()
    lp = (x.gather(1, t.clamp(0, V - 1)[:, None])[:, 0] - logz).masked_fill((t < 0) | (t >= V), 0)
    ent = logz - torch.where(e > 0, e * x, 0).sum(1, dtype=torch.float64) / z
    return [lp.float(), ent.float(), idx, (top - m - logz[:, None]).float()]


# -------------------------------------------------------------------- run

def run(st):
    case = st["case"]
    op = case["op"]
    if not own:
        return {"linear": _plain_linear, "delta": _plain_delta, "logprobs": _plain_logprobs}[op](st)
    m = st["m"]
    if op == "linear":
        m.moe_q4_linear(st["x"], st["w"], st["y"], st["act"], st["residual"])
        return st["y"]
    if op == "delta":
        args = (st["q"], st["k"], st["v"], st["g"], st["beta"], st["seq_start"], st["state_idx"], st["state_in"],
                st["state_out"], st["o"], st["scale"], case["norm"])
        if case["kind"] == "decode":
            m.moe_q4_delta_decode(*args)
        else:
            m.moe_q4_delta_prefill(*args, st["ws"])
        return [st["o"], st["state_out"]]
    m.moe_q4_logprobs(st["logits"], st["tokens"], st["logprob"], st["entropy"], st["top_idx"], st["top_logprob"],
                      st["ws"])
    return [st["logprob"], st["entropy"], st["top_idx"], st["top_logprob"]]


def work(case):
    if case["op"] == "linear":
        T, K, N = case["T"], case["K"], case["N"]
        w = N * K + N * (K // GROUP) * 2 if case["fmt"] == "int8" else N * K * 2
        b = w + T * K * 2 + T * N * (4 if case["out"] == "f32" else 2)
        return {"bytes": b + (4 * N if case["bias"] else 0) + (2 * T * N if case["residual"] else 0),
                "flops": 2 * T * K * N}
    if case["op"] == "delta":
        lens = [int(n) for n in case["lens"].split(",")]
        hk, hv, dk, dv = case["hk"], case["hv"], case["dk"], case["dv"]
        T = sum(lens)
        # per token and head: decay, S^T k, the rank-one update, S^T q
        return {"bytes": T * (4 * hk * dk + 4 * hv * dv + 8 * hv) + len(lens) * (8 * hv * dk * dv + 8),
                "flops": T * hv * 7 * dk * dv}
    T, V, n = case["T"], case["V"], case["n"]
    return {"bytes": T * V * (2 if case["dtype"] == "bf16" else 4) + T * (12 + 8 * n), "flops": 4 * T * V}


# ------------------------------------------------------------ 64-bit forms

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "linear":
        x, w = st["x"].double(), st["q"].double()
        if st["scale"] is not None:
            w *= st["scale"].double().repeat_interleave(GROUP, 1)
        z = torch.mm(x, w.t().contiguous())
        if st["bias"] is not None:
            z += st["bias"].double()
        if case["act"] == "silu":
            z = z * torch.sigmoid(z)
        elif case["act"] == "gelu":
            z = z * torch.special.ndtr(z)
        return z if st["residual"] is None else z + st["residual"].double()
    if case["op"] == "delta":
        # token by token, every sequence that still has one
        r = case["hv"] // case["hk"]
        q, k, v = st["q"].double(), st["k"].double(), st["v"].double()
        if case["norm"]:
            q, k = (t * torch.rsqrt(t.pow(2).sum(2, keepdim=True) + 1e-6) for t in (q, k))
        a, beta = torch.exp(st["g"].double()), st["beta"].double()
        order = sorted(range(len(st["lens"])), key=lambda b: -st["lens"][b])
        sizes = [st["lens"][b] for b in order]
        first = st["seq_start"].long()[torch.tensor(order, device="cuda")]
        slot = st["state_idx"].long()[torch.tensor(order, device="cuda")]
        S = st["state_in"].double()[slot]
        o = torch.zeros(st["o"].shape, dtype=torch.float64, device="cuda")
        for t in range(max(sizes)):
            b = sum(n > t for n in sizes)
            row = first[:b] + t
            kt, qt = (x[row].repeat_interleave(r, 1) for x in (k, q))
            H = S[:b] * a[row][..., None, None]
            u = beta[row][..., None] * (v[row] - (H * kt[..., None]).sum(2))
            H = H + kt[..., None] * u[..., None, :]
            o[row] = (H * qt[..., None]).sum(2) * st["scale"]
            S[:b] = H
        out = torch.empty_like(S)
        out[slot] = S
        return [o, out]
    V, n = case["V"], case["n"]
    res = [[], [], [], []]
    for l in st["logits"].split(64):
        lp = torch.log_softmax(l.double(), 1)
        order = torch.argsort(-l.double(), dim=1, stable=True)[:, :n]
        res[1].append(-torch.special.xlogy(lp.exp(), lp.exp()).sum(1))
        res[2].append(order.int())
        res[3].append(lp.gather(1, order))
        t = st["tokens"].long()[sum(x.numel() for x in res[0]):][:len(l)]
        own_lp = lp.gather(1, t.clamp(0, V - 1)[:, None])[:, 0]
        res[0].append(torch.where((t >= 0) & (t < V), own_lp, torch.zeros_like(own_lp)))
    return [torch.cat(x) for x in res]
