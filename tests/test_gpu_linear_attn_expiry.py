"""Failure path of the prompt kernels' bounded waits (zq_linear_attn), on the GPU,
without a fault.

A call is made through its test hook with a short wait limit, and a barrier of the first
or second chunk, the queries and keys' or the values', expects one arrival more than there
are.  The waits for it must run out,
every kind of warp must return, the device status word must carry bit 0, what
belongs to nobody must be as it was, sequences that never come to that chunk must
be right, and an ordinary call afterwards must be right and raise nothing."""
import time

import pytest

torch = pytest.importorskip("torch")

import gemm_zq_rmsnorm_gb300 as zq

pytestmark = pytest.mark.gpu

LENS = (50, 330)


def make(Hv, Dk, Dv, lens):
    g = torch.Generator(device="cuda").manual_seed(Hv + Dk + Dv)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")
    T = sum(lens)
    starts = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")
    slots = torch.arange(len(lens), dtype=torch.int32, device="cuda")
    return (randn(T, Dk), randn(T, Dk) / Dk ** 0.5, randn(T, Hv * Dv), -0.1 * randn(T, Hv).abs(), starts), slots, \
        randn(len(lens) + 1, Hv, Dk, Dv)


# heads: sequences cut into many segments, into few, not at all
@pytest.mark.parametrize("Dk,Dv,Hv", [(64, 64, 1), (128, 128, 40), (128, 128, 80), (64, 256, 20), (128, 64, 80)])
@pytest.mark.parametrize("values", [False, True])
@pytest.mark.parametrize("chunk", [0, 1])
def test_wait_expires_and_reports(Dk, Dv, Hv, values, chunk):
    rows, slots, pool = make(Hv, Dk, Dv, LENS)
    T, B = sum(LENS), len(LENS)
    before = pool.clone()
    want = pool.clone()
    good = zq.linear_attn(*rows, zq.LinearState(want), slots)
    torch.cuda.synchronize()
    need = zq.linear_attn_workspace_bytes(T, B, Hv, Dk, Dv)
    room = torch.full((need + 4096,), 77, dtype=torch.uint8, device="cuda")
    out = torch.full((T + 1, Hv * Dv), 5.0, device="cuda")
    assert zq.device_status(clear=True) == 0
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    zq.debug_linear_attn_expiry(*rows, zq.LinearState(pool), slots, chunk, values=values, out=out[:T], workspace=room[:need])
    torch.cuda.synchronize()
    elapsed = time.perf_counter() - t0
    length = zq.debug_linear_segments(rows[4].tolist(), T, Hv, Dv)["length"]
    reached = chunk < (length or max(LENS)) / 64     # (a segment of one chunk has no chunk 1)
    assert zq.device_status(clear=True) == (zq.DEVICE_WAIT_EXPIRED if reached else 0)
    assert elapsed < 0.5, elapsed                      # the short limit, not the two-second default, ended the waits
    assert bool((room[need:] == 77).all()) and bool((out[T] == 5.0).all())
    assert torch.equal(pool[B], before[B])
    if not reached:
        assert torch.equal(out[:T], good) and torch.equal(pool, want)
    elif chunk == 1:                                   # the first sequence has one chunk
        assert torch.equal(out[:LENS[0]], good[:LENS[0]]) and torch.equal(pool[0], want[0])
    # the context is healthy: an ordinary call is right and raises nothing
    after = before.clone()
    again = zq.linear_attn(*rows, zq.LinearState(after), slots)
    torch.cuda.synchronize()
    assert zq.device_status() == 0
    assert torch.equal(again, good) and torch.equal(after, want)


def test_the_rest_of_a_long_sequence_does_not_wait():
    """128 chunks after the one that expires: none of their waits lasts."""
    rows, slots, pool = make(80, 64, 64, (64 * 130,))
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    zq.debug_linear_attn_expiry(*rows, zq.LinearState(pool), slots, 1)
    torch.cuda.synchronize()
    elapsed = time.perf_counter() - t0
    assert zq.device_status(clear=True) == zq.DEVICE_WAIT_EXPIRED
    assert elapsed < 0.25, elapsed


def test_argument_checks():
    rows, slots, pool = make(1, 64, 64, (10,))
    for chunk, wait_us in ((-1, 1000), (2, 1000), (0, 0), (0, 2_000_001)):
        with pytest.raises(zq.ZQError):
            zq.debug_linear_attn_expiry(*rows, zq.LinearState(pool), slots, chunk, wait_us=wait_us)
    assert zq.device_status() == 0
