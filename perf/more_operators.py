"""Workloads of the recurrent mixer's and the block edges' operators of the library.

Four operators: linear_attn_step (linear attention with a decay for each head, one new token per sequence),
linear_attn (the same over prompts of ragged lengths), gated_norm_q8_1 (per-head RMSNorm times a gate, to Q8_1 codes
or fp32) and residual_norm_q8_1 (the norm after a block, its gate and residual scale, the residual addition, and the
norm before the next block to Q8_1 codes).

`own` chooses what run() calls: the library's entry points, or the operators' plain form in elementary torch
operations.
"""
import math

import torch

own = False

_EPS = 1e-6


def listed():
    return [
        # one decoded token, small heads: launch latency
        dict(name="step_one", op="step", B=1, Hk=8, Hv=8, Dk=64, Dv=64),
        # a decode batch of the recurrent layer whose output projection is 6144 wide: 48 value heads of 128
        dict(name="step_decode_61", op="step", B=61, Hk=16, Hv=48, Dk=128, Dv=128),
        # many sequences of a state-space layer: one key for all the heads of a group, narrow values
        dict(name="step_batch_200", op="step", B=200, Hk=2, Hv=32, Dk=128, Dv=64),
        # a short question: one chunk that is not full, latency
        dict(name="prompt_37", op="prompt", B=1, Hk=8, Hv=8, Dk=64, Dv=64, lo=37, hi=37, pad=0, fresh=True),
        # a long prompt of the recurrent layer
        dict(name="prompt_4096", op="prompt", B=1, Hk=16, Hv=48, Dk=128, Dv=128, lo=4096, hi=4096, pad=0, fresh=True),
        # a batch of prompts of different lengths, some continued from their state, an empty one, rows behind the last
        dict(name="prompt_ragged_24", op="prompt", B=24, Hk=4, Hv=32, Dk=128, Dv=64, lo=0, hi=1500, pad=7, fresh=False),
        # one long document and few heads: the length has to be split over the whole GPU
        dict(name="prompt_16384", op="prompt", B=1, Hk=8, Hv=8, Dk=128, Dv=128, lo=16384, hi=16384, pad=0, fresh=False),
        # one decoded token's mixer output on its way to the 6144-wide output projection: latency
        dict(name="gated_one", op="gated", B=1, H=48, D=128, norm=True, act="silu", to="codes"),
        # a prompt's attention output under a sigmoid gate, wide heads, no norm, kept in fp32
        dict(name="gated_prompt_1777", op="gated", B=1777, H=24, D=256, norm=False, act="sigmoid", to="fp32"),
        # one decoded token of the small model: residual and norm, latency
        dict(name="edge_one", op="edge", B=1, K=1024, post=False, gate="none", scale=1.0),
        # a decode batch of the 27B-class layer, with a norm after the block and a residual scale
        dict(name="edge_decode_61", op="edge", B=61, K=5120, post=True, gate="none", scale=0.5),
        # a long prompt of the 27B-class layer, with a norm after the block and a gate for each token and channel
        dict(name="edge_prompt_4096", op="edge", B=4096, K=5120, post=True, gate="sigmoid", scale=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["step", "step", "prompt", "prompt", "prompt", "gated", "edge"])
    if kind in ("step", "prompt"):
        Hk = rng.randint(1, 16)
        c = dict(op=kind, Hk=Hk, Hv=Hk * rng.randint(1, 4), Dk=rng.choice([64, 128]), Dv=rng.choice([64, 128, 256]))
        if kind == "step":
            return dict(c, B=_log(rng, 1, min(512, 48_000_000 // (c["Hv"] * c["Dk"] * c["Dv"]))))
        B = _log(rng, 1, 32)
        # the plain form looks at every pair of a sequence's tokens
        most = math.isqrt(2_000_000_000 // (B * c["Hv"]))
        hi = _log(rng, 1, min(16384, most, max(1, 24_000_000 // (B * c["Hv"] * c["Dv"]))))
        return dict(c, B=B, lo=min(hi, rng.choice([0, 1, hi // 2, hi])), hi=hi, pad=rng.choice([0, 0, 5]),
                    fresh=rng.random() < 0.5)
    if kind == "gated":
        D = rng.choice([64, 128, 256])
        H = rng.randint(1, 6144 // D)
        return dict(op="gated", B=_log(rng, 1, min(4096, 20_000_000 // (H * D))), H=H, D=D, norm=rng.random() < 0.7,
                    act=rng.choice(["silu", "sigmoid", "linear"]), to=rng.choice(["codes", "fp32"]))
    K = 32 * _log(rng, 8, 640)
    return dict(op="edge", B=_log(rng, 1, min(4096, 20_000_000 // K)), K=K, post=rng.random() < 0.5,
                gate=rng.choice(["none", "none", "channel", "sigmoid"]), scale=rng.choice([1.0, 0.5, 0.22]))


def _lens(c):
    """Lengths between lo and hi, most of them short: a fixed spread of the case."""
    g = [(i * 0.6180339887498949) % 1.0 for i in range(c["B"])]
    return [c["lo"] + int(round((c["hi"] - c["lo"]) * u * u)) for u in g[::-1]]


def _continued(c):
    """The sequences that go on from their state."""
    return [not c["fresh"] and b % 3 != 1 for b in range(c["B"])]


def work(c):
    if c["op"] in ("step", "prompt"):
        state = 4 * c["Hv"] * c["Dk"] * c["Dv"]
        row = 4 * (2 * c["Hk"] * c["Dk"] + 2 * c["Hv"] * c["Dv"] + c["Hv"])
        T = c["B"] if c["op"] == "step" else sum(_lens(c))
        moved = 2 * c["B"] if c["op"] == "step" else c["B"] + sum(_continued(c))
        return {"bytes": moved * state + T * row, "flops": 4 * T * c["Hv"] * c["Dk"] * c["Dv"]}
    if c["op"] == "gated":
        n = c["B"] * c["H"] * c["D"]
        return {"bytes": n * (8 + (4 if c["to"] == "fp32" else 1.125)), "flops": n * 8}
    n = c["B"] * c["K"]
    return {"bytes": n * (12 + 1.125 + (4 if c["gate"] == "sigmoid" else 0)), "flops": n * 8}


def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    s = dict(c)
    B = c["B"]
    if c["op"] in ("step", "prompt"):
        Hk, Hv, Dk, Dv = c["Hk"], c["Hv"], c["Dk"], c["Dv"]
        T = B if c["op"] == "step" else sum(_lens(c)) + c["pad"]
        T = max(T, 1)
        n = B + 3
        # the stacked projection's output: queries, keys (of unit length or so) and values beside each other in a row
        s["qkv"] = torch.cat((randn(T, Hk * Dk), randn(T, Hk * Dk) / math.sqrt(Dk), randn(T, Hv * Dv)), 1)
        # decays: each head forgets at a rate of its own, some over a few tokens, some over thousands
        rate = torch.exp(uniform(Hv) * math.log(1000.0)) * 1e-3
        s["g"] = -rate * torch.nn.functional.softplus(randn(T, Hv))
        s["pool"] = randn(n, Hv, Dk, Dv) * 0.3
        s["slots"] = torch.randperm(n, generator=g, device="cuda")[:B].to(torch.int32)
        s["out"] = torch.zeros(T, Hv * Dv, device="cuda")
        if c["op"] == "prompt":
            lens = torch.tensor(_lens(c))
            s["starts"] = torch.cat((torch.zeros(1, dtype=torch.int64), lens.cumsum(0))).to(torch.int32).cuda()
            s["anew"] = torch.tensor([not x for x in _continued(c)], dtype=torch.int32).cuda()
        if own:
            import gemm_zq_rmsnorm_gb300 as zq
            s["state"] = zq.LinearState(s["pool"])
            if c["op"] == "prompt":
                need = zq.linear_attn_workspace_bytes(T, B, Hv, Dk, Dv)
                s["workspace"] = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
        return s
    if c["op"] == "gated":
        n = c["H"] * c["D"]
        s["x"] = randn(B, n) * 0.7
        # the gate is a part of a stacked projection's row
        s["stacked"] = randn(B, 2 * n) * 1.5
        s["gamma"] = 0.5 + uniform(c["D"]) if c["norm"] else None
        if c["to"] == "fp32":
            s["out"] = torch.empty(B, n, device="cuda")
        K = n
    else:
        K = c["K"]
        s["x"] = randn(B, K) * 2.0
        s["y"] = randn(B, K) * 0.8
        s["gamma_post"] = 0.5 + uniform(K) if c["post"] else None
        s["gamma"] = 0.5 + uniform(K)
        s["gate_rows"] = {"none": None, "channel": uniform(K), "sigmoid": randn(B, K)}[c["gate"]]
        s["x_out"] = torch.empty(B, K, device="cuda")
    if own:
        import gemm_zq_rmsnorm_gb300 as zq
        if c["op"] == "edge" or c["to"] == "codes":
            s["q8"] = zq.empty_q8_1(B, K)
            s["values"] = torch.empty(B, K, dtype=torch.float16, device="cuda")
    return s


def run(s):
    if own:
        return _OWN[s["op"]](s)
    return _PLAIN[s["op"]](s)


def _qkv(s):
    return s["qkv"].split((s["Hk"] * s["Dk"], s["Hk"] * s["Dk"], s["Hv"] * s["Dv"]), 1)


# ---------------------------------------------------------------- the library's calls
def _own_step(s):
    import gemm_zq_rmsnorm_gb300 as zq
    q, k, v = _qkv(s)
    out = zq.linear_attn_step(q, k, v, s["g"], s["state"], s["slots"], out=s["out"])
    return {"out": out, "state": s["pool"]}


def _own_prompt(s):
    import gemm_zq_rmsnorm_gb300 as zq
    q, k, v = _qkv(s)
    out = zq.linear_attn(q, k, v, s["g"], s["starts"], s["state"], s["slots"], fresh=s["anew"], out=s["out"],
                         workspace=s["workspace"])
    return {"out": out, "state": s["pool"]}


def _own_codes(s):
    import gemm_zq_rmsnorm_gb300 as zq
    q8 = s["q8"]
    return {"codes": zq.q8_1_dequant_f16(q8, out=s["values"]), "d": q8.d, "s": q8.s}


def _own_gated(s):
    import gemm_zq_rmsnorm_gb300 as zq
    gate = s["stacked"][:, s["H"] * s["D"]:]
    if s["to"] == "fp32":
        return {"out": zq.gated_norm_q8_1(s["x"], gate, s["gamma"], _EPS, s["D"], act=s["act"], out=s["out"])}
    zq.gated_norm_q8_1(s["x"], gate, s["gamma"], _EPS, s["D"], act=s["act"], q8_out=s["q8"])
    return _own_codes(s)


def _own_edge(s):
    import gemm_zq_rmsnorm_gb300 as zq
    act = "sigmoid" if s["gate"] == "sigmoid" else "linear"
    x = zq.residual_norm_q8_1(s["x"], s["y"], s["gamma"], _EPS, gamma_post=s["gamma_post"], gate=s["gate_rows"],
                              act=act, scale=s["scale"], x_out=s["x_out"], q8_out=s["q8"])
    return {"x": x, **_own_codes(s)}


_OWN = {"step": _own_step, "prompt": _own_prompt, "gated": _own_gated, "edge": _own_edge}


# ---------------------------------------------------------------- plain forms
def _plain_step(s):
    B, Hk, Hv, Dk, Dv = s["B"], s["Hk"], s["Hv"], s["Dk"], s["Dv"]
    q, k, v = _qkv(s)
    slots = s["slots"].long()
    q, k = (x.view(B, Hk, 1, Dk).expand(B, Hk, Hv // Hk, Dk).reshape(B, Hv, Dk, 1) for x in (q, k))
    state = s["pool"][slots] * torch.exp(s["g"])[..., None, None] + k * v.view(B, Hv, 1, Dv)
    s["pool"][slots] = state
    out = (q * state).sum(2) * (1.0 / math.sqrt(Dk))
    return {"out": out.view(B, Hv * Dv), "state": s["pool"]}


def _plain_prompt(s):
    B, Hk, Hv, Dk, Dv = s["B"], s["Hk"], s["Hv"], s["Dk"], s["Dv"]
    starts, slots = s["starts"].long(), s["slots"].long()
    lens = starts[1:] - starts[:-1]
    at = torch.arange(max(1, s["hi"]), device="cuda")
    L = at.numel()
    here = at < lens[:, None]                                            # [B][L]
    rows = (starts[:-1, None] + at).clamp(max=s["qkv"].shape[0] - 1)
    q, k, v = (x[rows] * here[..., None] for x in _qkv(s))
    q, k = (x.view(B, L, Hk, 1, Dk).expand(B, L, Hk, Hv // Hk, Dk).reshape(B, L, Hv, Dk).transpose(1, 2) for x in (q, k))
    v = v.view(B, L, Hv, Dv).transpose(1, 2)                             # [B][Hv][L][Dv]
    G = (s["g"][rows].double() * here[..., None]).cumsum(1).transpose(1, 2)   # [B][Hv][L]: sums of thousands of decays
    q = q * (1.0 / math.sqrt(Dk))
    first = s["pool"][slots] * (1 - s["anew"])[:, None, None, None]
    decay = (G[..., :, None] - G[..., None, :]).float()
    decay.masked_fill_(at[None, :] > at[:, None], -math.inf).exp_()      # [B][Hv][L][L], of each earlier token
    out = (q @ k.transpose(2, 3)).mul_(decay) @ v + torch.exp(G.float())[..., None] * (q @ first)
    last = G[..., -1:]
    s["pool"][slots] = (torch.exp(last.float())[..., None] * first
                        + (k * torch.exp((last - G).float())[..., None]).transpose(2, 3) @ v)
    full = s["out"].clone()
    full[rows[here]] = out.transpose(1, 2).reshape(B, L, Hv * Dv)[here]
    return {"out": full, "state": s["pool"]}


def _act(gate, act):
    if act == "linear":
        return gate
    sig = 1.0 / (1.0 + torch.exp(-gate))
    return gate * sig if act == "silu" else sig


def _norm(x, gamma):
    return x * (1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + _EPS)) * gamma


def _plain_codes(x):
    """Q8_1: blocks of 32 codes, halves away from zero, with their scale and scaled sum; the values they stand for."""
    b = x.reshape(x.shape[0], -1, 32)
    d = b.abs().amax(-1) / 127.0
    a = b.abs() * torch.where(d > 0, 1.0 / d, 0.0)[..., None]
    q = a.floor()
    q = (q + (a - q >= 0.5)).clamp(max=127.0) * b.sign()
    return {"codes": (q * d.half().float()[..., None]).view(x.shape).half(), "d": d.half(), "s": (d * q.sum(-1)).half()}


def _plain_gated(s):
    B, H, D = s["B"], s["H"], s["D"]
    x = s["x"].view(B, H, D)
    if s["norm"]:
        x = _norm(x, s["gamma"])
    x = (x * _act(s["stacked"][:, H * D:].reshape(B, H, D), s["act"])).view(B, H * D)
    return {"out": x} if s["to"] == "fp32" else _plain_codes(x)


def _plain_edge(s):
    y = _norm(s["y"], s["gamma_post"]) if s["post"] else s["y"]
    if s["gate"] != "none":
        y = y * _act(s["gate_rows"], "sigmoid" if s["gate"] == "sigmoid" else "linear")
    x = s["x"] + s["scale"] * y
    return {"x": x, **_plain_codes(_norm(x, s["gamma"]))}


_PLAIN = {"step": _plain_step, "prompt": _plain_prompt, "gated": _plain_gated, "edge": _plain_edge}


# ---------------------------------------------------------------- 64 bits, from the definitions
def exact(c, seed):
    global own
    was, own = own, False
    try:
        s = prepare(c, seed)
    finally:
        own = was
    return {"step": _exact_recurrence, "prompt": _exact_recurrence, "gated": _exact_gated, "edge": _exact_edge}[c["op"]](s)


def _exact_recurrence(s):
    """Token after token, all sequences at the same time."""
    B, Hk, Hv, Dk, Dv = s["B"], s["Hk"], s["Hv"], s["Dk"], s["Dv"]
    T = s["qkv"].shape[0]
    nk = Hk * Dk
    head = torch.arange(Hv, device="cuda") // (Hv // Hk)
    q = s["qkv"][:, :nk].double().view(T, Hk, Dk)
    k = s["qkv"][:, nk:2 * nk].double().view(T, Hk, Dk)
    v = s["qkv"][:, 2 * nk:].double().view(T, Hv, Dv)
    a = s["g"].double().exp()
    pool, out = s["pool"].double(), torch.zeros(T, Hv, Dv, dtype=torch.float64, device="cuda")
    slots = s["slots"].long()
    if s["op"] == "step":
        first, lens = list(range(B)), [1] * B
    else:
        lens = _lens(s)
        first = [sum(lens[:b]) for b in range(B)]
        pool[slots[[b for b, goes_on in enumerate(_continued(s)) if not goes_on]]] = 0
    order = sorted(range(B), key=lambda b: -lens[b])                     # the longest first
    start = torch.tensor([first[b] for b in order], device="cuda")
    where = slots[order]
    state = pool[where]                                                  # [B][Hv][Dk][Dv]
    for t in range(max(lens)):
        n = sum(m > t for m in lens)
        r = start[:n] + t
        st = state[:n]
        st *= a[r][..., None, None]
        st += k[r][:, head][..., None] * v[r][:, :, None]
        out[r] = torch.matmul(q[r][:, head][:, :, None], st)[:, :, 0] / math.sqrt(Dk)
    pool[where] = state
    return {"out": out.view(T, Hv * Dv), "state": pool}


def _exact_act(gate, act):
    g = gate.double()
    return {"linear": g, "silu": g * torch.sigmoid(g), "sigmoid": torch.sigmoid(g)}[act]


def _exact_norm(x, gamma):
    return x * gamma.double() / torch.sqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + _EPS)


def _exact_d(x):
    return x.abs().unflatten(-1, (-1, 32)).amax(-1) / 127


def _exact_gated(s):
    x = s["x"].double().unflatten(1, (s["H"], s["D"]))
    if s["norm"]:
        x = _exact_norm(x, s["gamma"])
    x = x.flatten(1) * _exact_act(s["stacked"][:, s["H"] * s["D"]:], s["act"])
    return {"out": x} if s["to"] == "fp32" else {"codes": None, "d": _exact_d(x), "s": None}


def _exact_edge(s):
    y = s["y"].double()
    if s["post"]:
        y = _exact_norm(y, s["gamma_post"])
    if s["gate"] != "none":
        y = y * _exact_act(s["gate_rows"], "sigmoid" if s["gate"] == "sigmoid" else "linear")
    x = s["x"].double() + s["scale"] * y
    return {"x": x, "codes": None, "d": _exact_d(_exact_norm(x, s["gamma"])), "s": None}
