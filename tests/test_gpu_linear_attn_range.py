"""Linear attention over prompts (zq_linear_attn) at the ends of the fp32 range:
states and tokens whose sizes are powers of two apart, value by value (not by the
norms of what went in) against the 64-bit recurrence.

Tolerances.  A state without new tokens: a chunk multiplies it by a power of two given
as 2^(whole + broken), the broken part's power to 2^-22 (ex2) and its sum of 64 decays to
64 * 2^-33 * ln 2, and rounds twice: under 2^-21 a chunk, and as much where a segment's
start is made.  Outputs, where nothing cancels or relative to a row's norm: both
factors' parts 2^-23 each, the low parts' product 2^-24, at most 24 additions that cut off
(2^-23 each), the rows' factors 2^-21: under 2^-18.  States of tokens of both signs are
judged by root mean squares of 2^-20, as in test_gpu_linear_attn.py."""
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
    assert (zq.linear_attn_workspace_bytes(T, 1, heads, Dk, Dv) > 0) == (heads < 80 and T > 128)
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


# heads for which a sequence of a few chunks is cut into many segments, into few that make their own starts, not at all
CUTS = {"join": lambda Dv: 1, "few": lambda Dv: 40 if Dv <= 128 else 20, "whole": lambda Dv: 80}
LN2 = 0.6931471805599453


def decays(T, powers):
    """[T][1] decays whose sum over chunk i is -ln 2 times powers[i]."""
    g = zeros(T, 1)
    for i, p in enumerate(powers):
        g[64 * i:64 * i + 64] = -LN2 * p / 64
    return g


@pytest.mark.parametrize("cut", CUTS)
@pytest.mark.parametrize("Dk,Dv", SHAPES)
@pytest.mark.parametrize("powers", [(200, 0, 0), (0, 190, 3), (110, 60, 20), (70, 80, 60)])
def test_a_large_state_after_large_decays(Dk, Dv, cut, powers):
    """2^110 after decays of 2^-190 to 2^-210: each token's decay, and what is left, is a number like any other."""
    T = 192
    S0 = 2.0 ** 110 * signs(11, Dk, Dv)
    q = randn(12, T, Dk)
    out, S, o, want = call(q, zeros(T, Dk), randn(13, T, Dv), decays(T, powers), S0, 0.5, CUTS[cut](Dv))
    near(S, want, 4 * 2.0 ** -21)
    for rows in (slice(0, 64), slice(64, 128), slice(128, 192)):
        assert float(((out - o)[rows].norm(dim=1) / o[rows].norm(dim=1)).max()) <= 2.0 ** -18


@pytest.mark.parametrize("cut", CUTS)
@pytest.mark.parametrize("Dk,Dv", SHAPES)
@pytest.mark.parametrize("eq,es,power,scale", [(-100, 120, 0, 0), (100, -100, 0, 0), (0, 100, 150, 0), (20, 90, 200, 0), (-60, 118, 30, 40),
                                               (-100, 90, 100, 100), (90, 60, 60, -100), (0, -90, 0, 60)])
def test_queries_and_states_far_apart(Dk, Dv, cut, eq, es, power, scale):
    """Queries of 2^eq for a state of 2^es under decays of 2^-power a chunk and a scale of 2^scale: the products are
    numbers like any other."""
    T = 70
    q = 2.0 ** eq * signs(21, T, Dk).abs()
    S0 = 2.0 ** es * signs(22, Dk, Dv).abs()          # (nothing cancels)
    out, S, o, want = call(q, zeros(T, Dk), zeros(T, Dv), decays(T, (power,)), S0, 2.0 ** scale, CUTS[cut](Dv))
    assert float(o.abs().max()) < 2.0 ** 120 and float(o.abs().min()) > 2.0 ** -120
    near(out, o, 2.0 ** -18)
    near(S, want, 2 * 2.0 ** -21)


@pytest.mark.parametrize("cut", CUTS)
@pytest.mark.parametrize("Dk,Dv", SHAPES)
@pytest.mark.parametrize("eq,ek,ev,scale", [(100, -55, -60, 0), (0, -55, -55, 0), (-50, 60, 50, 0), (-110, 50, 50, 90),
                                            (30, -110, 60, 0), (40, 30, -120, 30), (55, -20, 70, -90)])
def test_tokens_of_any_size(Dk, Dv, cut, eq, ek, ev, scale):
    """Queries of 2^eq, keys of 2^ek and values of 2^ev."""
    T = 192
    # (keys and queries of one sign: nothing cancels over them; values of both, so their sums are judged by their size)
    q, k, v = (2.0 ** e * signs(31 + i, T, D) for i, (e, D) in enumerate(((eq, Dk), (ek, Dk), (ev, Dv))))
    g = decays(T, (30, 10, 50))
    out, S, o, want = call(q.abs(), k.abs(), v, g, zeros(Dk, Dv), 2.0 ** scale, CUTS[cut](Dv))
    assert 2.0 ** -120 < float(o.norm(dim=1).min()) and float(o.abs().max()) < 2.0 ** 120
    assert float(((out - o).norm(dim=1) / o.norm(dim=1)).max()) <= 2.0 ** -18
    assert float((S - want).norm() / want.norm()) <= 2.0 ** -20


@pytest.mark.parametrize("cut", CUTS)
@pytest.mark.parametrize("Dk,Dv", SHAPES)
def test_tokens_that_become_small(Dk, Dv, cut):
    """A chunk of 2^100, decays that leave nothing of it, then a chunk of 2^-100: what comes last is what is left."""
    T = 192
    e = zeros(T, 1)
    e[:64], e[64:] = 50.0, -50.0
    k, v = torch.exp2(e) * signs(41, T, Dk).abs(), torch.exp2(e) * signs(42, T, Dv)
    out, S, o, want = call(signs(43, T, Dk).abs(), k, v, decays(T, (10, 400, 20)), zeros(Dk, Dv), 1.0, CUTS[cut](Dv))
    assert 2.0 ** -125 < float(want.norm()) < 2.0 ** -80
    assert float((S - want).norm() / want.norm()) <= 2.0 ** -20
    assert float(((out - o)[128:].norm(dim=1) / o[128:].norm(dim=1)).max()) <= 2.0 ** -18


@pytest.mark.parametrize("Dk,Dv", SHAPES)
def test_forgetting_leaves_nothing_of_the_largest_state(Dk, Dv):
    T = 70
    g = zeros(T, 1)
    g[3], g[66] = -float("inf"), -float("inf")
    S0 = 2.0 ** 126 * signs(51, Dk, Dv)
    q = 2.0 ** -20 * signs(52, T, Dk)
    q[3:] *= 2.0 ** 70
    q[3:] *= 2.0 ** 70
    out, S, o, want = call(q, zeros(T, Dk), zeros(T, Dv), g, S0, 1.0, 80)
    assert bool((out[3:] == 0).all()) and bool((S == 0).all()) and bool(torch.isfinite(out).all())


@pytest.mark.parametrize("Dk,Dv", SHAPES)
@pytest.mark.parametrize("e", [-40, -50, -60, -70, -85, -100])
def test_a_first_token_that_is_forgotten_in_its_chunk(Dk, Dv, e):
    """A state of zeros, one small token, and decays that leave nothing of it: sums of 2^-1000 are zeros."""
    T = 192
    k, v, g = zeros(T, Dk), randn(62, T, Dv), zeros(T, 1)
    k[0] = 2.0 ** e * signs(61, Dk)
    v[0] *= 2.0 ** e
    g[10] = -float("inf")
    for heads in (1, 80):
        out, S, o, want = call(randn(63, T, Dk), k, v, g, zeros(Dk, Dv), 1.0, heads)
        assert bool((want == 0).all()) and bool((S == 0).all())
        assert bool((out[10:] == 0).all()) and bool(torch.isfinite(out).all())
        # (below 2^-126 a value is held to half of 2^-149: the norm of the first ten rows to that much)
        assert float((out - o).norm()) <= 2.0 ** -18 * float(o.norm()) + (10 * Dv) ** 0.5 * 2.0 ** -149
