"""Plain 64-bit forms of linear attention and of the block edges, for the tests."""
import torch


def recurrence(q, k, v, g, S0, scale):
    """One sequence, token after token: q, k [T][Hk][Dk], v [T][Hv][Dv], g
    [T][Hv] (or None), S0 [Hv][Dk][Dv].  Returns out [T][Hv][Dv], the last
    state, and what bounds them: |out[t][h]| <= bound[t][h], |S[h]| <= last[h],
    by the norms of the rows that went in."""
    T, Hv = v.shape[:2]
    rep = Hv // q.shape[1]
    q, k = (x.double().repeat_interleave(rep, 1) for x in (q, k))
    v, S = v.double(), S0.double().clone()
    a = torch.ones(T, Hv, dtype=torch.float64, device=v.device) if g is None else g.double().exp()
    out = torch.zeros(v.shape, dtype=torch.float64, device=v.device)
    size = S.norm(dim=1).amax(-1)
    sizes = []
    new = k.norm(dim=-1) * v.abs().amax(-1)
    for t in range(T):
        S = a[t][:, None, None] * S + k[t][:, :, None] * v[t][:, None, :]
        out[t] = scale * torch.einsum("hd,hde->he", q[t], S)
        size = a[t] * size + new[t]
        sizes.append(size)
    bound = torch.stack(sizes) * q.norm(dim=-1) * abs(scale) if T else out[..., 0]
    return out, S, bound, size


def act(g, kind):
    g = g.double()
    return {"linear": g, "sigmoid": torch.sigmoid(g), "silu": g * torch.sigmoid(g)}[kind]


def norm(x, gamma, eps):
    x = x.double()
    if gamma is None:
        return x
    return x * gamma.double() / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
