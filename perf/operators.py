"""Workloads of the attention-side and adapter operators of the library.

Three operators: head_norm_rope (per-head RMSNorm of queries and keys, rotary
positions with one to three axes, and the write into the paged key-value
cache), paged_attn (attention of one new token per sequence over that cache)
and lora (low-rank adapters of many requests beside a shared projection).

`own` chooses what run() calls: the library's entry points, or the operators'
plain form in elementary torch operations.
"""
import math

import numpy as np
import torch

own = False

_TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
_BYTES = {"f16": 2, "bf16": 2, "e4m3": 1}
_EPS = 1e-6
_THETA = 1.0e6


def listed():
    return [
        # one decoded token of the small model: launch latency
        dict(name="norm_rope_one_token", op="norm_rope", T=1, Hq=16, Hk=8, D=128, rot=128, axes=1, interleaved=False,
             type="f16", page=16, far=2000),
        # a decode batch of the 27B-class layer's widths (48 x 128 queries, 8 x 128 keys), far positions
        dict(name="norm_rope_decode_61", op="norm_rope", T=61, Hq=48, Hk=8, D=128, rot=128, axes=1, interleaved=False,
             type="bf16", page=64, far=900000),
        # a prompt with an image: three position axes, a quarter of each 256-wide head rotated, 8-bit cache
        dict(name="norm_rope_image_prompt", op="norm_rope", T=777, Hq=24, Hk=4, D=256, rot=64, axes=3,
             interleaved=False, type="e4m3", page=32, far=5000),
        # a long prompt in one call, neighbouring values paired
        dict(name="norm_rope_prefill_4096", op="norm_rope", T=4096, Hq=48, Hk=8, D=128, rot=128, axes=1,
             interleaved=True, type="f16", page=128, far=4096),
        # one user, a short conversation, the small model's heads: launch latency
        dict(name="attn_one_1000", op="attn", B=1, Hq=16, Hk=8, D=128, type="f16", page=16, lo=1000, hi=1000,
             window=0),
        # a serving batch whose sequences differ widely in length
        dict(name="attn_ragged_48", op="attn", B=48, Hq=48, Hk=8, D=128, type="bf16", page=64, lo=1, hi=12000,
             window=0),
        # one long document: the length has to be split over the whole GPU
        dict(name="attn_one_131071", op="attn", B=1, Hq=24, Hk=4, D=256, type="bf16", page=64, lo=131071, hi=131071,
             window=0),
        # many short sequences, empty ones among them, a sliding window, small heads, 8-bit cache
        dict(name="attn_window_200", op="attn", B=200, Hq=32, Hk=8, D=64, type="e4m3", page=32, lo=0, hi=4000,
             window=1024),
        # a full batch of long sequences on an 8-bit cache
        dict(name="attn_long_e4m3_64", op="attn", B=64, Hq=48, Hk=8, D=128, type="e4m3", page=64, lo=8000, hi=24000,
             window=0),
        # one decoded token of the small model's q projection with an adapter
        dict(name="lora_one_token", op="lora", B=1, K=1024, N=2048, R=16, n=4, type="f16", runs=False, without=False),
        # a decode batch of many requests on the 27B-class gate projection, some without an adapter
        dict(name="lora_decode_56", op="lora", B=56, K=5120, N=17408, R=16, n=12, type="bf16", runs=False,
             without=True),
        # prompts of a few requests on the 27B-class down projection, large rank
        dict(name="lora_prefill_512", op="lora", B=512, K=17408, N=5120, R=64, n=4, type="f16", runs=True,
             without=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["norm_rope", "attn", "attn", "lora"])
    if kind == "norm_rope":
        D = rng.choice([64, 128, 256])
        Hk = rng.randint(1, 8)
        T = _log(rng, 1, 4096)
        return dict(op="norm_rope", T=T, Hq=Hk * rng.randint(1, max(1, (7168 // D - Hk) // Hk)), Hk=Hk, D=D,
                    rot=16 * rng.randint(1, D // 16), axes=rng.randint(1, 3), interleaved=rng.random() < 0.5,
                    type=rng.choice(list(_TYPES)), page=rng.choice([16, 32, 64, 128, 256]), far=_log(rng, T, 1 << 20))
    if kind == "attn":
        D = rng.choice([64, 128, 256])
        Hk = rng.randint(1, 8)
        B = _log(rng, 1, 256)
        kind = rng.choice(list(_TYPES))
        hi = min(_log(rng, 1, 131072), max(1, 800_000_000 // (B * Hk * D * _BYTES[kind])))
        lo = rng.choice([0, 1, hi // 2, hi])
        return dict(op="attn", B=B, Hq=Hk * rng.randint(1, 6), Hk=Hk, D=D, type=kind,
                    page=rng.choice([16, 32, 64, 128, 256]), lo=min(lo, hi), hi=hi,
                    window=rng.choice([0, 0, 0, _log(rng, 1, 8192)]))
    B = _log(rng, 1, 512)
    return dict(op="lora", B=B, K=256 * _log(rng, 1, 68), N=_log(rng, 33, 17408), R=rng.choice([8, 16, 32, 64]),
                n=_log(rng, 1, 16), type=rng.choice(["f16", "bf16"]), runs=rng.random() < 0.5,
                without=rng.random() < 0.5)


def _lens(c):
    """Lengths between lo and hi, most of them short: a fixed spread of the case."""
    g = [(i * 0.6180339887498949) % 1.0 for i in range(c["B"])]
    return [c["lo"] + int(round((c["hi"] - c["lo"]) * u * u)) for u in g[::-1]]


def _seen(c):
    w = c["window"]
    return [min(n, w) if w else n for n in _lens(c)]


def _ids(c):
    """The adapter of each token: requests one after another, or scattered as in a decode batch."""
    B, n = c["B"], c["n"]
    ids = [i * n // B for i in range(B)] if c["runs"] else [(i * 7919 + 1) % n for i in range(B)]
    return [-1 if c["without"] and i % 7 == 3 else a for i, a in enumerate(ids)]


def _axis(c):
    """Pairs of the rotation take their position axes in three runs, as time, height and width do."""
    half = c["rot"] // 2
    return [min(i * c["axes"] // half, c["axes"] - 1) for i in range(half)]


def work(c):
    if c["op"] == "norm_rope":
        T, Hq, Hk, D = c["T"], c["Hq"], c["Hk"], c["D"]
        by = 4 * T * D * (2 * Hq + 2 * Hk) + 2 * _BYTES[c["type"]] * T * Hk * D + 4 * T * (c["axes"] + 1)
        return {"bytes": by, "flops": T * (Hq + Hk) * (4 * D + 3 * c["rot"])}
    if c["op"] == "attn":
        n = sum(_seen(c))
        pages = sum(-(-m // c["page"]) for m in _seen(c))
        by = 2 * n * c["Hk"] * c["D"] * _BYTES[c["type"]] + 8 * c["B"] * c["Hq"] * c["D"] + 4 * pages + 4 * c["B"]
        return {"bytes": by, "flops": 4 * n * c["Hq"] * c["D"]}
    B, K, N, R = c["B"], c["K"], c["N"], c["R"]
    used, with_one = len({a for a in _ids(c) if a >= 0}), sum(a >= 0 for a in _ids(c))
    by = 2 * used * R * (K + N) + with_one * K * (1 + 2 / 32) + 8 * B * N + 4 * B
    return {"bytes": by, "flops": 2 * with_one * R * (K + N)}


def prepare(c, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    s = dict(c)
    if c["op"] == "lora":
        B, K, N, R, n = c["B"], c["K"], c["N"], c["R"], c["n"]
        x = randn(B, K // 32, 32)
        d = x.abs().amax(-1) / 127
        s["qs"] = torch.round(x / d[..., None]).to(torch.int8).reshape(B, K)
        s["d"] = d.half()
        s["s"] = (d * s["qs"].view(B, K // 32, 32).float().sum(-1)).half()
        s["A"] = (randn(n, R, K) / math.sqrt(K)).to(_TYPES[c["type"]])
        s["Bm"] = (randn(n, N, R) * 0.3).to(_TYPES[c["type"]])
        s["scales"] = 0.5 + torch.rand(n, generator=g, device="cuda")
        s["base"] = randn(B, N)
        s["y"] = torch.empty_like(s["base"])
        s["ids"] = torch.tensor(_ids(c), dtype=torch.int32, device="cuda")
        if own:
            import gemm_zq_rmsnorm_gb300 as zq
            s["x"] = zq.Q8_1(s["qs"], s["d"], s["s"])
            s["workspace"] = torch.empty(zq.lora_workspace_bytes(B, K, R), dtype=torch.uint8, device="cuda")
        return s

    Hq, Hk, D, page = c["Hq"], c["Hk"], c["D"], c["page"]
    s["k_scale"], s["v_scale"] = (0.05, 0.04) if c["type"] == "e4m3" else (1.0, 1.0)

    def pool(pages, scale):
        return (randn(pages, Hk, page, D) / scale).to(_TYPES[c["type"]])

    if c["op"] == "norm_rope":
        T = c["T"]
        pages = -(-T // page) + 3
        # the stacked projection's output, q, k and v beside each other in a row
        s["qkv"] = randn(T, (Hq + 2 * Hk) * D) * 1.7
        s["gamma_q"], s["gamma_k"] = 0.5 + torch.rand(2, D, generator=g, device="cuda")
        s["pos"] = torch.randint(0, c["far"], (c["axes"], T), generator=g, device="cuda", dtype=torch.int32)
        s["slots"] = torch.randperm(pages * page, generator=g, device="cuda")[:T].to(torch.int32)
        s["k"], s["v"] = pool(pages, s["k_scale"]), pool(pages, s["v_scale"])
        s["q_out"] = torch.empty(T, Hq * D, device="cuda")
        inv = _THETA ** (-2.0 * np.arange(c["rot"] // 2) / c["rot"])
        s["inv_freq"] = torch.from_numpy(inv).cuda()
        s["axis"] = torch.tensor(_axis(c), device="cuda")
    else:
        lens = _lens(c)
        need = [-(-m // page) for m in lens]
        width = max(max(need), 1)
        pages = sum(need) + 5
        order = torch.randperm(pages, generator=g, device="cuda")
        start = np.concatenate([[0], np.cumsum(need)])[:-1]
        at = torch.from_numpy(start[:, None] + np.arange(width)[None]).cuda()
        in_use = torch.from_numpy(np.arange(width)[None] < np.array(need)[:, None]).cuda()
        s["table"] = torch.where(in_use, order[at.clamp(max=pages - 1)], -1).to(torch.int32)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["k"], s["v"] = pool(pages, s["k_scale"]), pool(pages, s["v_scale"])
        s["q"] = randn(c["B"], Hq * D) * 1.5
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(c["B"], Hq, device="cuda")
    if own:
        import gemm_zq_rmsnorm_gb300 as zq
        s["cache"] = zq.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
        if c["op"] == "norm_rope":
            s["rope"] = zq.rope_table(inv, _axis(c))
        else:
            s["workspace"] = torch.empty(zq.paged_attn_workspace_bytes(Hq, Hk, D), dtype=torch.uint8, device="cuda")
    return s


def run(s):
    if own:
        return _OWN[s["op"]](s)
    return _PLAIN[s["op"]](s)


# ---------------------------------------------------------------- the library's calls
def _own_norm_rope(s):
    import gemm_zq_rmsnorm_gb300 as zq
    nq, nk = s["Hq"] * s["D"], s["Hk"] * s["D"]
    q, k, v = s["qkv"].split((nq, nk, nk), 1)
    q = zq.head_norm_rope(q, k, v, s["gamma_q"], s["gamma_k"], _EPS, s["rope"], s["pos"], s["cache"], s["slots"],
                          interleaved=s["interleaved"], q_out=s["q_out"])
    return {"q": q, "k": s["k"], "v": s["v"]}


def _own_attn(s):
    import gemm_zq_rmsnorm_gb300 as zq
    out = zq.paged_attn(s["q"], s["cache"], s["table"], s["lens"], window=s["window"], out=s["out"], lse=s["lse"],
                        workspace=s["workspace"])
    return {"out": out, "lse": s["lse"]}


def _own_lora(s):
    import gemm_zq_rmsnorm_gb300 as zq
    return {"y": zq.lora(s["x"], s["ids"], s["A"], s["Bm"], s["scales"], base=s["base"], y=s["y"],
                         workspace=s["workspace"])}


_OWN = {"norm_rope": _own_norm_rope, "attn": _own_attn, "lora": _own_lora}


# ---------------------------------------------------------------- plain forms
def _write(pool, x, scale, slots, page):
    """Rows x [T][Hk][D] into their slots of a pool [pages][Hk][page][D]."""
    x = x / scale
    at = (slots // page, slice(None), slots % page)
    if pool.dtype == torch.float8_e4m3fn:   # 8-bit pools saturate at the type's largest value
        pool.view(torch.uint8)[at] = x.clamp(-448, 448).to(pool.dtype).view(torch.uint8)
    else:
        pool[at] = x.to(pool.dtype)


def _plain_norm_rope(s):
    T, Hq, Hk, D, rot = s["T"], s["Hq"], s["Hk"], s["D"], s["rot"]
    q, k, v = s["qkv"].view(T, Hq + 2 * Hk, D).split((Hq, Hk, Hk), 1)
    angle = s["pos"].double()[s["axis"]].t() * s["inv_freq"]          # [T][rot/2], far positions need 64 bits
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]

    def norm_rotate(x, gamma):
        x = x * (1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + _EPS)) * gamma
        r, rest = x[..., :rot], x[..., rot:]
        if s["interleaved"]:
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
        else:
            a, b = r[..., :rot // 2], r[..., rot // 2:]
            r = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
        return torch.cat((r, rest), -1)

    slots = s["slots"].long()
    _write(s["k"], norm_rotate(k, s["gamma_k"]), s["k_scale"], slots, s["page"])
    _write(s["v"], v, s["v_scale"], slots, s["page"])
    return {"q": norm_rotate(q, s["gamma_q"]).reshape(T, Hq * D), "k": s["k"], "v": s["v"]}


def _rows(pool, table, scale):
    """The pages of each sequence one after another, fp32 [B][Hk][width * page][D]."""
    t = table.clamp(min=0).long()
    x = pool.view(torch.uint8)[t].view(pool.dtype) if pool.dtype == torch.float8_e4m3fn else pool[t]
    B, W, Hk, page, D = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(B, Hk, W * page, D).float() * scale


def _plain_attn(s):
    B, Hq, Hk, D = s["B"], s["Hq"], s["Hk"], s["D"]
    k, v = _rows(s["k"], s["table"], s["k_scale"]), _rows(s["v"], s["table"], s["v_scale"])
    j = torch.arange(k.shape[2], device="cuda")
    n = s["lens"][:, None]
    seen = j < n
    if s["window"]:
        seen = seen & (j >= n - s["window"])
    w = s["q"].view(B, Hk, Hq // Hk, D) @ k.transpose(2, 3) * (1.0 / math.sqrt(D))
    w = w.masked_fill(~seen[:, None, None], -math.inf)
    m = w.amax(-1, keepdim=True)
    p = torch.exp(w - m.clamp(min=-1e30))
    total = p.sum(-1, keepdim=True)
    out = (p @ v) / total.clamp(min=1e-30)
    return {"out": out.reshape(B, Hq * D), "lse": (m + torch.log(total)).reshape(B, Hq)}


def _plain_lora(s):
    B, N, R, n = s["B"], s["N"], s["R"], s["n"]
    x = (s["qs"].view(B, -1, 32).float() * s["d"].float()[..., None]).view(B, -1)
    # every adapter's rank values, then zeros but for the token's own adapter
    h = (x @ s["A"].float().view(n * R, -1).t()).view(B, n, R)
    mine = s["ids"][:, None] == torch.arange(n, device="cuda")
    h = (h * (mine * s["scales"])[..., None]).view(B, n * R)
    return {"y": s["base"] + h @ s["Bm"].float().transpose(1, 2).reshape(n * R, N)}


_PLAIN = {"norm_rope": _plain_norm_rope, "attn": _plain_attn, "lora": _plain_lora}


# ---------------------------------------------------------------- 64 bits, from the definitions
def exact(c, seed):
    global own
    was, own = own, False
    try:
        s = prepare(c, seed)
    finally:
        own = was
    return {"norm_rope": _exact_norm_rope, "attn": _exact_attn, "lora": _exact_lora}[c["op"]](s)


def _exact_norm_rope(s):
    T, Hq, Hk, D, page = s["T"], s["Hq"], s["Hk"], s["D"], s["page"]
    x = s["qkv"].double().view(T, Hq + 2 * Hk, D)
    half = s["rot"] // 2
    pairs = [(2 * i, 2 * i + 1) if s["interleaved"] else (i, i + half) for i in range(half)]
    first, second = (torch.tensor(p, device="cuda") for p in zip(*pairs))
    # rotation as a product of complex numbers
    turn = torch.polar(torch.ones(T, half, dtype=torch.float64, device="cuda"),
                       torch.stack([s["pos"][a].double() for a in _axis(s)], 1) * s["inv_freq"])

    def rotated(h, gamma):
        y = h * gamma.double() / torch.sqrt(h.square().sum(-1, keepdim=True) / D + _EPS)
        z = torch.complex(y[..., first], y[..., second]) * turn[:, None]
        y[..., first], y[..., second] = z.real, z.imag
        return y

    out = {"q": rotated(x[:, :Hq], s["gamma_q"]).reshape(T, Hq * D)}
    for name, rows in (("k", rotated(x[:, Hq:Hq + Hk], s["gamma_k"])), ("v", x[:, Hq + Hk:])):
        flat = s[name].double().transpose(1, 2).reshape(-1, Hk, D)      # [slot][Hk][D]
        most = 448.0 if s["type"] == "e4m3" else math.inf
        flat[s["slots"].long()] = (rows / s[name + "_scale"]).clamp(-most, most)
        out[name] = flat.view(-1, page, Hk, D).transpose(1, 2)
    return out


def _exact_attn(s):
    B, Hq, Hk, D, page = s["B"], s["Hq"], s["Hk"], s["D"], s["page"]
    out = torch.zeros(B, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq), -math.inf, dtype=torch.float64, device="cuda")
    at = torch.arange(int(s["table"].shape[1]) * page, device="cuda")
    for b, n in enumerate(_lens(s)):
        first = max(0, n - s["window"]) if s["window"] else 0
        if n == first:
            continue
        j = at[first:n]
        pages, row = s["table"][b].long()[j // page], j % page
        for h in range(Hk):
            if s["type"] == "e4m3":
                k, v = (s[x].view(torch.uint8)[pages, h, row].view(s[x].dtype) for x in ("k", "v"))
            else:
                k, v = s["k"][pages, h, row], s["v"][pages, h, row]
            G = Hq // Hk
            heads = slice(h * G, (h + 1) * G)
            w = (s["q"][b].view(Hq, D)[heads].double() @ k.double().t()) * (s["k_scale"] / math.sqrt(D))
            lse[b, heads] = torch.logsumexp(w, -1)
            out[b, heads] = torch.softmax(w, -1) @ v.double() * s["v_scale"]
    return {"out": out.view(B, Hq * D), "lse": lse}


def _exact_lora(s):
    x = s["qs"].double() * s["d"].double().repeat_interleave(32, 1)
    y = s["base"].double()
    ids = torch.tensor(_ids(s))
    for a in range(s["n"]):
        rows = torch.nonzero(ids == a)[:, 0].cuda()
        if len(rows):
            y[rows] += float(s["scales"][a]) * (x[rows] @ s["A"][a].double().t() @ s["Bm"][a].double().t())
    return {"y": y}
