"""Plain 64-bit forms of the attention-side operators, for the tests."""
import numpy as np
import torch


def norm_rope(x, gamma, eps, inv_freq, axis, pos, interleaved):
    """x fp32 [T][H][D] -> float64; gamma [D] or None; pos int [axes][T]."""
    x = x.astype(np.float64)
    if gamma is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + np.float64(np.float32(eps))) * gamma.astype(np.float64)
    out = x.copy()
    half = len(inv_freq)
    for p in range(half):
        ang = pos[min(axis[p], len(pos) - 1)].astype(np.float64) * inv_freq[p]
        c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
        i, j = (2 * p, 2 * p + 1) if interleaved else (p, p + half)
        out[..., i] = x[..., i] * c - x[..., j] * s
        out[..., j] = x[..., j] * c + x[..., i] * s
    return out


def to_type(x, dtype):
    """float64 -> the cache's type, by way of fp32; 8 bits saturate."""
    t = torch.from_numpy(np.ascontiguousarray(x)).float()
    if dtype == torch.float8_e4m3fn:
        t = t.clamp(-448, 448)
    return t.to(dtype)


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def attn(q, k, v, tokens, scale):
    """One sequence: q [Hq][D] float64, k and v [tokens][Hk][D] float64, over
    the rows `tokens`; (out, lse)."""
    Hq, D = q.shape
    out, lse = np.zeros((Hq, D)), np.full(Hq, -np.inf)
    if len(tokens) == 0:
        return out, lse
    G = Hq // k.shape[1]
    for h in range(Hq):
        w = k[tokens, h // G] @ q[h] * scale
        m = w.max()
        p = np.exp(w - m)
        out[h] = p @ v[tokens, h // G] / p.sum()
        lse[h] = m + np.log(p.sum())
    return out, lse


def q8_1(x):
    """Q8_1 planes (codes, d, s as float16) of fp32 rows [B][K], step by step as the library packs them."""
    b = x.reshape(x.shape[0], -1, 32)
    d = np.abs(b).max(-1) / np.float32(127)
    inv = np.where(d != 0, np.float32(1) / np.where(d != 0, d, np.float32(1)), np.float32(0))
    v = b * inv[..., None]
    a = np.abs(v)
    q = np.floor(a)
    q = np.minimum(q + (a - q >= 0.5), 127) * np.sign(v)
    s = d * q.sum(-1).astype(np.float32)
    return q.astype(np.int8).reshape(x.shape), d.astype(np.float16), s.astype(np.float16)
