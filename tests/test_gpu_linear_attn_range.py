"""Linear attention over prompts (zq_linear_attn) at the ends of the fp32 range:
states and tokens whose sizes are powers of two apart, value by value (not by the
norms of what went in) against the 64-bit recurrence.

Tolerance: a state's value passes through at most three chunks here.  A chunk
multiplies it by a power of two given as 2^(whole + broken), the broken part's power
to 2^-22 (ex2) and its sum of 64 decays to 64 * 2^-33 * ln 2, and rounds twice: under
2^-21 a chunk.  The queries' products with the state add what _mixer_ref's bound has:
2^-16 of the norms."""
import pytest

torch = pytest.importorskip("torch")

import gemm_zq_rmsnorm_gb300 as zq

import _mixer_ref as ref

pytestmark = pytest.mark.gpu

SHAPES = [(64, 64), (128, 128), (128, 256)]


def zeros(*shape):
    return torch.zeros(*shape, device="cuda")


def randn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def signs(seed, *shape):
    """Values of one size, 1 to 2, of both signs."""
    return randn(seed, *shape).sign() * (1.0 + torch.rand(*shape, generator=torch.Generator(device="cuda").manual_seed(seed + 1),
                                                          device="cuda"))


def call(q, k, v, g, S0, scale, heads):
    """One sequence of `heads` heads that are all alike, from S0; its outputs and state, and what they should be.  One
    head is cut into segments of a chunk, 80 are not cut."""
    Dk, Dv = S0.shape
    T = q.shape[0]
    pool = S0.repeat(1, heads, 1, 1)
    ints = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, T], [0])]
    assert (zq.linear_attn_workspace_bytes(T, 1, heads, Dk, Dv) > 0) == (heads == 1 and T > 128)
    out = zq.linear_attn(q, k, v.repeat(1, heads), g.repeat(1, heads), ints[0], zq.LinearState(pool), ints[1], scale=scale)
    o, S, _, _ = ref.recurrence(q[:, None], k[:, None], v[:, None], g, S0[None], scale)
    out = out.view(T, heads, Dv)
    assert all(torch.equal(out[:, 0], out[:, h]) and torch.equal(pool[0, 0], pool[0, h]) for h in range(heads))
    assert zq.device_status() == 0
    return out[:, 0].double(), pool[0, 0].double(), o[:, 0], S[0]


def near(got, want, tol):
    """Every value, relative to itself; what fp32 holds to fewer bits, by half a step of those."""
    assert torch.isfinite(got).all()
    off = (got - want).abs()
    worst = (off / (want.abs() + 1e-300)).max()
    assert (off <= tol * want.abs() + 2.0 ** -149).all(), float(worst)


@pytest.mark.parametrize("heads", [1, 80])
@pytest.mark.parametrize("Dk,Dv", SHAPES)
def test_a_state_that_shrinks_far(Dk, Dv, heads):
    """Chunks of zero keys, whose decays alone change a state of 4e4."""
    T = 192
    g = zeros(T, 1)
    g[:64], g[64:128] = -3.0 / 64, -86.6 / 64
    S0 = 4e4 * signs(1, Dk, Dv)
    out, S, o, want = call(randn(2, T, Dk), zeros(T, Dk), randn(3, T, Dv), g, S0, 1.0, heads)
    near(S, want, 3 * 2.0 ** -21)
    assert float((out - o).norm() / o.norm()) <= 2.0 ** -20


@pytest.mark.parametrize("heads", [1, 80])
@pytest.mark.parametrize("Dk,Dv", SHAPES)
def test_a_small_state_beside_large_tokens(Dk, Dv, heads):
    """A column of zero values keeps its state of 2^-100 while 2^60 is added to the others."""
    T = 70
    v = 2.0 ** 30 * randn(3, T, Dv)
    v[:, 5] = 0.0
    S0 = 2.0 ** -100 * signs(1, Dk, Dv)
    _, S, _, want = call(randn(2, T, Dk), 2.0 ** 30 * randn(4, T, Dk), v, -0.01 * randn(5, T, 1).abs(), S0, 1.0, heads)
    near(S[:, 5], want[:, 5], 2 * 2.0 ** -21)
    other = [c for c in range(Dv) if c != 5]
    assert float((S - want)[:, other].norm() / want[:, other].norm()) <= 2.0 ** -20
