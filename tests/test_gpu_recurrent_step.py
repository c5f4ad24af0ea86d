"""Recurrent layers as a model runs them: projection, linear attention over a
ragged prompt and then token by token, the gated head norm to codes, the output
projection, and the edge to the next layer's codes.  Every stage against its
64-bit form on what it was given (the tolerances are those of the operators' own
tests), the steps eager, on a stream of their own, and as a graph replayed while
the states go on."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import gemm_zq_rmsnorm_gb300 as zq
from gemm_zq_rmsnorm_gb300 import inputs

import _attn_ref
import _mixer_ref as ref

pytestmark = pytest.mark.gpu

K, HK, HV, DK, DV, LAYERS, EPS = 512, 2, 4, 64, 64, 2, 1e-6
PARTS = (HK * DK, HK * DK, HV * DV, HV * DV)      # query, key, value, gate


def layer(i):
    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(i)
    return dict(win=torch.from_numpy(inputs.q4k_weights(40 + i, sum(PARTS), K)).cuda(),
                wout=torch.from_numpy(inputs.q4k_weights(50 + i, K, HV * DV)).cuda(),
                head=0.5 + randn(DV).abs(), post=0.5 + randn(K).abs(), before=0.5 + randn(K).abs(),
                rate=0.1 * torch.rand(HV, generator=g, device="cuda"))


def forward(layers, x, states, slots, starts=None, fresh=None, stream=None, seen=None):
    """The residual stream [T][K] after the layers; starts: a prompt, else one token per sequence."""
    a = zq.rmsnorm_q8_1(x, layers[0]["before"], EPS, stream=stream)
    for i, w in enumerate(layers):
        rows = zq.q4k_gemm(w["win"], sum(PARTS), K, a, len(x), stream=stream)
        q, k, v, z = rows.split(PARTS, 1)
        with torch.cuda.stream(stream or torch.cuda.current_stream()):
            decay = -w["rate"] * z[:, ::DV].abs()
        before = states[i].s.clone() if seen is not None else None
        if starts is None:
            o = zq.linear_attn_step(q, k, v, decay, states[i], slots, stream=stream)
        else:
            o = zq.linear_attn(q, k, v, decay, starts, states[i], slots, fresh=fresh, stream=stream)
        codes = zq.gated_norm_q8_1(o, z, w["head"], EPS, DV, q8_out=zq.empty_q8_1(len(x), HV * DV), stream=stream)
        y = zq.q4k_gemm(w["wout"], K, HV * DV, codes, len(x), stream=stream)
        a = zq.empty_q8_1(len(x), K)
        x_in, x = x, zq.residual_norm_q8_1(x, y, layers[(i + 1) % LAYERS]["before"], EPS, gamma_post=w["post"], scale=0.5,
                                           q8_out=a, stream=stream)
        if seen is not None:
            seen.append((q, k, v, z, decay, before, states[i].s.clone(), o, codes, x_in, y, x, a))
    return x


def check_stages(layers, seen, seqs, slots, fresh):
    for i, (q, k, v, z, decay, before, after, o, codes, x_in, y, x, a) in enumerate(seen):
        w = layers[i]
        for b, (t0, t1) in enumerate(seqs):
            n = t1 - t0
            S0 = torch.zeros_like(before[0]) if fresh[b] else before[slots[b]]
            want, S, bo, bs = ref.recurrence(q[t0:t1].view(n, HK, DK), k[t0:t1].view(n, HK, DK), v[t0:t1].view(n, HV, DV),
                                             decay[t0:t1], S0, DK ** -0.5)
            assert bool(((o[t0:t1].view(n, HV, DV) - want).abs() <= (2.0 ** -16 + n / 64 * 2.0 ** -17) * bo[..., None] + 1e-300).all())
            assert bool(((after[slots[b]] - S).abs() <= (1 + n / 64) * 2.0 ** -17 * bs[:, None, None] + 1e-300).all())
        full = zq.gated_norm_q8_1(o, z, w["head"], EPS, DV)
        normed = ref.norm(o.view(len(o), HV, DV), w["head"], EPS).view(o.shape)
        want = normed * ref.act(z, "silu")
        # a sigmoid below 2^-126 (z < -87.3) is flushed to zero: off by at most that, times z and the normalised value
        flushed = 2.0 ** -126 * z.abs().double() * normed.abs()
        assert bool(((full - want).abs() <= 2.0 ** -17 * want.abs() + flushed + 1e-37).all())
        for got, plane in zip((codes.qs, codes.d, codes.s), _attn_ref.q8_1(full.cpu().numpy())):
            assert np.array_equal(got.cpu().numpy(), plane)
        u = 0.5 * ref.norm(y, w["post"], EPS)
        want = x_in.double() + u
        assert bool(((x - want).abs() <= 2.0 ** -17 * u.abs() + 2.0 ** -24 * want.abs()).all())
        same = zq.rmsnorm_q8_1(x, layers[(i + 1) % LAYERS]["before"], EPS)
        assert torch.equal(a.qs, same.qs) and torch.equal(a.d, same.d) and torch.equal(a.s, same.s)


def test_prompt_then_steps():
    layers = [layer(i) for i in range(LAYERS)]
    lens, slots, B, steps = [130, 1, 67], [3, 0, 2], 3, 4
    T = sum(lens)
    g = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randn(T, K, generator=g, device="cuda")
    tokens = torch.randn(steps, B, K, generator=g, device="cuda")
    starts = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    slot = torch.tensor(slots, dtype=torch.int32, device="cuda")
    fresh = torch.tensor([1, 0, 1], dtype=torch.int32, device="cuda")
    states = [zq.LinearState(torch.randn(4, HV, DK, DV, generator=g, device="cuda")) for _ in layers]
    unused = [s.s[1].clone() for s in states]
    seen = []
    forward(layers, x, states, slot, starts, fresh, seen=seen)
    ends = starts.tolist()
    check_stages(layers, seen, list(zip(ends[:-1], ends[1:])), slots, [1, 0, 1])
    left = [s.s.clone() for s in states]

    eager = []
    for t in range(steps):
        seen = []
        eager.append(forward(layers, tokens[t], states, slot, seen=seen))
        check_stages(layers, seen, [(b, b + 1) for b in range(B)], slots, [0] * B)
    done = [s.s.clone() for s in states]

    # on a stream of their own
    stream = torch.cuda.Stream()
    for s, before in zip(states, left):
        s.s.copy_(before)
    torch.cuda.synchronize()
    for t in range(steps):
        again = forward(layers, tokens[t], states, slot, stream=stream)
        stream.synchronize()
        assert torch.equal(again, eager[t])
    assert all(torch.equal(s.s, d) for s, d in zip(states, done))

    # captured once, replayed while the states go on
    now = tokens[0].clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = forward(layers, now, states, slot)
    for s, before in zip(states, left):
        s.s.copy_(before)
    for t in range(steps):
        now.copy_(tokens[t])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager[t])
    assert all(torch.equal(s.s, d) and torch.equal(s.s[1], u) for s, d, u in zip(states, done, unused))
    assert zq.device_status() == 0
