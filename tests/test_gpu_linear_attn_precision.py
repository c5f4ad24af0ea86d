"""What linear attention over prompts (zq_linear_attn) keeps of small values beside
large ones, as root mean squares against the 64-bit recurrence: a channel of one factor
that the other factor lacks is 1000 times the others, so that a bound by the rows' norms
would allow 1000 times the error.

Tolerance: both factors' binary16 parts to 2^-23 of each value, the low parts' product
2^-24, additions that cut off 2^-23 of the running sum: with random signs near 2^-22 of
the result's root mean square; 2^-20 is what the other tests of these products have."""
import pytest

torch = pytest.importorskip("torch")

import gemm_zq_rmsnorm_gb300 as zq

import _mixer_ref as ref

pytestmark = pytest.mark.gpu

LARGE = 1000.0


def run(q, k, v, g, S0):
    T, Hv, Dv = v.shape
    pool = S0.clone()[None]
    ints = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, T], [0])]
    out = zq.linear_attn(q, k, v, g, ints[0], zq.LinearState(pool), ints[1])
    o, S, _, _ = ref.recurrence(q, k, v, g, S0, q.shape[-1] ** -0.5)
    assert zq.device_status() == 0
    return out.double(), pool[0].double(), o, S


def rms(got, want, dims):
    """The largest share over what is left of the dimensions."""
    return float(((got - want).square().sum(dims).sqrt() / want.square().sum(dims).sqrt()).max())


@pytest.mark.parametrize("Dk,Dv", [(64, 64), (64, 128), (128, 64), (128, 128), (128, 256)])
@pytest.mark.parametrize("T,Hk,Hv", [(50, 1, 2), (333, 2, 2), (333, 40, 80)])
@pytest.mark.parametrize("where", ["q", "k", "v", "state"])
def test_a_channel_that_stands_out(Dk, Dv, T, Hk, Hv, where):
    g = torch.Generator(device="cuda").manual_seed(Dk + Dv + T)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    q, k, v = randn(T, Hk, Dk), randn(T, Hk, Dk) / Dk ** 0.5, randn(T, Hv, Dv)
    decay = -0.02 * randn(T, Hv).abs()
    S0 = randn(Hv, Dk, Dv) * 0.3
    if where == "q":          # keys and states lack it
        q[..., 5] *= LARGE
        k[..., 5] = 0.0
        S0[:, 5] = 0.0
    elif where == "k":        # queries lack it
        k[..., 5] *= LARGE
        q[..., 5] = 0.0
    elif where == "v":        # a column of its own
        v[..., 5] *= LARGE
    else:                     # the first state's largest values lie near 1, and queries lack them
        S0 = 4.0 * S0 / LARGE
        S0[:, 5] *= LARGE
        q[..., 5] = 0.0
        k *= 1e-3
    out, S, o, want = run(q, k, v, decay, S0)
    assert rms(out, o, (0,)) <= 2.0 ** -20            # every column of every head
    # columns of the state, or its rows where one of them would be all that a column's size is
    assert rms(S, want, (1,) if where in ("q", "v") else (2,)) <= 2.0 ** -20
