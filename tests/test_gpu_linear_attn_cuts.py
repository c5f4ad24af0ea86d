"""How zq_linear_attn cuts its sequences, each way against the 64-bit recurrence with
test_gpu_linear_attn's tolerances: two tiles of a 256-wide head that make their own
starts from the segments before (one tile's decays serve both), calls of as many
sequences as are still cut and of more, and the lengths where the cut sets in."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import gemm_zq_rmsnorm_gb300 as zq

import _mixer_ref as ref
from test_gpu_linear_attn import heads, make, prompts

pytestmark = pytest.mark.gpu


def cut(lens, Hv, Dv, first=2, pad=3):
    starts = np.concatenate([[0], np.cumsum(lens)]) + first
    return zq.debug_linear_segments(starts.tolist(), first + sum(lens) + pad, Hv, Dv)


@pytest.mark.parametrize("Hk,Hv,segments", [(19, 38, 2), (5, 25, 3), (19, 19, 4)])
@pytest.mark.parametrize("Dk", [64, 128])
def test_two_tiles_that_make_their_own_starts(Dk, Hk, Hv, segments):
    for lens, fresh in (([1900, 40, 0, 300], [False, True, False, False]), ([200], [True]), ([700, 900], [True, False])):
        s = cut(lens, Hv, 256)
        assert 0 < s["length"] and 2 <= max(n for _, n in s["of"]) <= segments
        prompts(lens, Hk, Hv, Dk, 256, seed=Hv, fresh=fresh)


@pytest.mark.parametrize("Hv,Dv", [(1, 64), (2, 128), (38, 256)])
@pytest.mark.parametrize("B", [512, 513, 700])
def test_calls_of_many_sequences(Hv, Dv, B):
    """The last that are cut, and the first that are not, two long ones among them.  Each sequence by the norms of its
    rows; root mean squares over the call (one token's (q . k) v has q . k's error, whatever is left of |q| |k|)."""
    Dk, rng = 64, np.random.default_rng(B)
    lens = [int(n) for n in rng.integers(0, 6, B)]
    lens[3], lens[B - 2] = 333, 650
    assert (cut(lens, Hv, Dv, 0, 0)["length"] > 0) == (B <= 512)
    T = sum(lens)
    q, k, v, g, pool = make(B + Hv, T, 1, Hv, Dk, Dv, B)
    starts = np.concatenate([[0], np.cumsum(lens)])
    slots = rng.permutation(B)
    fresh = [b % 3 == 1 for b in range(B)]
    before = pool.clone()
    ints = [torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda") for x in (starts, slots, fresh)]
    out = zq.linear_attn(q, k, v, g, ints[0], zq.LinearState(pool), ints[1], fresh=ints[2])
    off, size = torch.zeros(2, dtype=torch.float64, device="cuda"), torch.zeros(2, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        at = slice(int(starts[b]), int(starts[b]) + n)
        S0 = torch.zeros_like(before[0]) if fresh[b] else before[slots[b]]
        o, S, bo, bs = ref.recurrence(heads(q[at], Dk), heads(k[at], Dk), heads(v[at], Dv), g[at], S0, Dk ** -0.5)
        do, ds = heads(out[at], Dv).double() - o, pool[slots[b]].double() - S
        assert bool((do.abs() <= (2.0 ** -16 + n / 64 * 2.0 ** -17) * bo[..., None] + 1e-300).all()), (b, n, "out")
        assert bool((ds.abs() <= (1 + n / 64) * 2.0 ** -17 * bs[:, None, None] + 1e-300).all()), (b, n, "state")
        off += torch.stack([do.square().sum(), ds.square().sum()])
        size += torch.stack([o.square().sum(), S.square().sum()])
    assert bool(((off / size).sqrt() <= 2.0 ** -20).all()) and zq.device_status() == 0


@pytest.mark.parametrize("T", [127, 128, 129, 191, 192, 193, 256, 257])
@pytest.mark.parametrize("Hv", [1, 38])
def test_lengths_around_the_cut(T, Hv):
    assert (cut([T], Hv, 128, 0, 0)["length"] > 0) == (T > 128)
    prompts([T], 1, Hv, 128, 128, seed=T, first=0, pad=0, fresh=[False])
    prompts([T], 1, Hv, 64, 64, seed=T, first=0, pad=0, fresh=[True])
