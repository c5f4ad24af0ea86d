"""The cut of prompts into segments (zq_debug_linear_segments: the code that the
kernels run, here on the host): every segment that is read or written has its place
in the workspace, whatever the starts are."""
import ctypes
import random

import pytest

import gemm_zq_rmsnorm_gb300 as zq


def room(T, B, Hv, Dv, Dk=64):
    """Segments that the workspace has room for, by its size."""
    return zq.linear_attn_workspace_bytes(T, B, Hv, Dk, Dv) // (Hv * (Dk * Dv * 4 + 8))


def check(starts, T, Hv, Dv):
    B = len(starts) - 1
    s = zq.debug_linear_segments(starts, T, Hv, Dv)
    if s["length"] == 0:
        assert room(T, B, Hv, Dv) == 0 and s["segments"] == B
        return s
    assert s["length"] % 64 == 0 and s["segments"] == room(T, B, Hv, Dv)
    for first, count in s["of"]:
        assert first >= 0 and count >= 0
        assert count == 0 or first + count <= s["segments"], (starts, first, count)
    return s


def test_starts_that_decrease_stay_in_the_workspace():
    T = 1500
    s = check([0, T] * 5, T, 1, 64)
    assert s["length"] == 64 and s["segments"] == 32
    # 24 segments, one, 24 ...: the third sequence has room for seven, the fifth for none
    assert s["of"] == [(0, 24), (24, 1), (25, 7), (49, 0), (50, 0), (74, 0), (75, 0), (99, 0), (100, 0)]


@pytest.mark.parametrize("Hv,Dv", [(1, 64), (8, 128), (48, 128), (19, 256)])
def test_starts_of_any_kind(Hv, Dv):
    rng = random.Random(Hv)
    for _ in range(300):
        T, B = rng.randint(1, 6000), rng.randint(1, 20)
        starts = [rng.choice([0, T, rng.randint(-T, 2 * T), -2 ** 31, 2 ** 31 - 1]) for _ in range(B + 1)]
        check(starts, T, Hv, Dv)


@pytest.mark.parametrize("Hv,Dv", [(1, 64), (8, 128), (48, 128), (19, 256)])
def test_starts_that_do_not_decrease_have_all_their_segments(Hv, Dv):
    rng = random.Random(Hv)
    for _ in range(300):
        T, B = rng.randint(1, 6000), rng.randint(1, 20)
        starts = sorted(rng.randint(0, T) for _ in range(B + 1))
        s, first = check(starts, T, Hv, Dv), 0
        for b in range(B):
            n = starts[b + 1] - starts[b]
            count = max(1, -(-n // s["length"])) if s["length"] else 1
            assert s["of"][b] == (first, count)
            first += count


@pytest.mark.parametrize("bad,status", [(dict(T=0), -2), (dict(T=(1 << 24) + 1), -2), (dict(Hv=0), -2), (dict(Hv=1025), -2),
                                        (dict(Dv=96), -2)])
def test_refuses(bad, status):
    with pytest.raises(zq.ZQError) as e:
        zq.debug_linear_segments([0, 1], **{**dict(T=10, Hv=1, Dv=64), **bad})
    assert e.value.status == status
    out = zq.load()
    assert out.zq_debug_linear_segments(None, 10, 1, 1, 64, None) == -1


@pytest.mark.parametrize("chunk,wait_us,status", [(-1, 1000, -1), (2, 1000, -1), (0, 0, -1), (1, 2000001, -1)])
def test_expiry_hook_refuses(chunk, wait_us, status):
    """zq_debug_linear_attn_expiry: chunk and limit, then what zq_linear_attn refuses."""
    lib, at = zq.load(), 0x10000           # fake, never-dereferenced device addresses
    state = ctypes.byref(zq._LinearState(at, 4, 4, 128, 128))

    def call(c, us, T=30):
        return lib.zq_debug_linear_attn_expiry(at, 256, at, 256, at, 512, T, 3, 2, at, 4, at, state, at, None, 0.1, at, 512, at,
                                               1 << 40, 1, c, us, None)
    assert call(chunk, wait_us) == status and lib.zq_last_error()
    assert call(0, 1000, T=0) == -2
