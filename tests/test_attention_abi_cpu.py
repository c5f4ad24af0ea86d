"""CPU-only checks of the attention-side calls: refusals on the host with the
documented status, and the rotation table's values."""
import ctypes
import math

import numpy as np
import pytest

import gemm_zq_rmsnorm_gb300 as zq

A16, A8, A2 = 0x10000, 0x10008, 0x10002


@pytest.fixture(scope="module")
def lib():
    return zq.load()


def cache(k=A16, v=A16, type=1, pages=4, page=16, Hk=2, D=128, ks=1.0, vs=1.0):
    return ctypes.byref(zq._Cache(k, v, type, pages, page, Hk, D, ks, vs))


def norm_rope(lib, q=A16, qs=512, k=A16, ks=256, v=A16, vs=256, T=3, Hq=4, gq=A16, gk=A16, eps=1e-6, table=A16,
              rot=128, inter=0, pos=A16, axes=1, c=None, slots=A16, out=A16 + 4096, os=512):
    return lib.zq_head_norm_rope(q, qs, k, ks, v, vs, T, Hq, gq, gk, eps, table, rot, inter, pos, axes,
                                 cache() if c is None else c, slots, out, os, None)


BAD_CACHES = [
    (dict(k=None), -1), (dict(v=None), -1), (dict(k=A8), -3), (dict(v=A8), -3), (dict(type=0), -1), (dict(type=4), -1),
    (dict(D=96), -2), (dict(D=0), -2), (dict(page=8), -2), (dict(page=48), -2), (dict(page=512), -2),
    (dict(page=0), -2), (dict(Hk=0), -2), (dict(Hk=1025), -2), (dict(pages=0), -2), (dict(pages=2 ** 31 - 1), -2),
    (dict(ks=0.0), -1), (dict(vs=-1.0), -1), (dict(ks=1e-39), -1), (dict(ks=math.nan), -1), (dict(vs=math.inf), -1)]


@pytest.mark.parametrize("bad,status", BAD_CACHES)
def test_head_norm_rope_refuses_caches(lib, bad, status):
    assert norm_rope(lib, c=cache(**bad)) == status
    assert lib.zq_last_error()


@pytest.mark.parametrize("bad,status", [
    (dict(q=None), -1), (dict(q=A8), -3), (dict(qs=508), -2), (dict(qs=514), -2), (dict(k=None), -1),
    (dict(ks=252), -2), (dict(v=A8), -3), (dict(vs=0), -2), (dict(vs=-256), -2), (dict(T=0), -2), (dict(T=-1), -2),
    (dict(T=2 ** 30), -2), (dict(Hq=0), -2), (dict(T=1, Hq=65537, qs=1 << 24, os=1 << 24), -2), (dict(eps=-1.0), -1), (dict(eps=math.nan), -1), (dict(rot=8), -2),
    (dict(rot=144), -2), (dict(rot=-16), -2), (dict(axes=0), -2), (dict(axes=4), -2), (dict(table=None), -1),
    (dict(pos=None), -1), (dict(slots=None), -1), (dict(gq=A8), -3), (dict(slots=A2), -3), (dict(pos=A2), -3), (dict(table=A2), -3), (dict(out=None), -1),
    (dict(out=A8), -3), (dict(os=4), -2), (dict(out=A16, os=516), -1)])
def test_head_norm_rope_refuses(lib, bad, status):
    assert norm_rope(lib, **bad) == status
    assert lib.zq_last_error()


def test_valid_head_norm_rope_without_gpu(lib):
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert norm_rope(lib) == -5
    assert norm_rope(lib, gq=None, gk=None, table=None, rot=0, pos=None) == -5
    assert norm_rope(lib, out=A16) == -5          # in place


def test_null_cache_is_refused(lib):
    assert lib.zq_head_norm_rope(A16, 512, A16, 256, A16, 256, 3, 4, None, None, 0.0, None, 0, 0, None, 1, None, A16,
                                 A16, 512, None) == -1


def test_rope_table_values(lib):
    """Each entry is inv_freq / 2 pi as a fraction of 2^64 to the nearest multiple of four, plus the axis."""
    freq = np.array([0.0, 1.0, -1.0, 2 * math.pi * 0.25, 1e-9, 7.5, 2 * math.pi])
    axis = [0, 1, 2, 0, 1, 2, 0]
    out = np.zeros(len(freq), np.uint64)
    ax = (ctypes.c_int * len(axis))(*axis)
    assert lib.zq_rope_table(freq.ctypes.data, ctypes.addressof(ax), len(freq), out.ctypes.data) == 0
    for f, a, e in zip(freq, axis, out):
        e = int(e)
        assert e & 3 == a
        turns = f / (2 * math.pi) % 1.0
        off = ((e & ~3) - int(turns * 2 ** 64) + 2 ** 63) % 2 ** 64 - 2 ** 63
        assert abs(off) <= 2 ** 64 * 2.0 ** -52 * max(1.0, abs(f) / (2 * math.pi))


def inverse_two_pi(bits):
    """floor(2^bits / (2 pi)), by Machin's formula."""
    one = 1 << bits + 64

    def atan_inverse(n):
        total, power, k = one // n, one // n, 1
        while power:
            power //= -n * n
            k += 2
            total += power // k
        return total
    return (1 << 2 * bits + 64) // (8 * (4 * atan_inverse(5) - atan_inverse(239)))


def test_rope_table_is_exact(lib):
    """The nearest multiple of four of the exact quotient's 2^-64 turns, for frequencies of any size: at position 2^31
    the angle is right to 2^-32 turns.  A negative frequency has the negated entry."""
    g = np.random.default_rng(0)
    freq = np.concatenate([1e6 ** -(np.arange(64) / 64), [1.0, 100.0, 2 * math.pi, math.nextafter(2 * math.pi, 9), 6e9, 1e22,
                           2.0 ** 53, 2.0 ** -60, 1e-19, 5e-324, 1.7976931348623157e308, 0.0], 2.0 ** g.uniform(-70, 1024, 300)])
    freq = np.concatenate([freq, -freq])
    out = np.zeros(len(freq), np.uint64)
    assert lib.zq_rope_table(freq.ctypes.data, None, len(freq), out.ctypes.data) == 0
    bits = 2400
    inverse = inverse_two_pi(bits)
    for f, e in zip(freq, out):
        num, den = abs(float(f)).as_integer_ratio()
        turns = (num * inverse << 64) // den            # in 2^-64 turns, with `bits` more
        off = (int(e) * (1 if f >= 0 else -1) << bits) - turns
        off = (off + (1 << bits + 63)) % (1 << bits + 64) - (1 << bits + 63)
        assert int(e) % 4 == 0 and abs(off) <= 2 << bits, (f, off >> bits)


def test_rope_table_refuses(lib):
    out = np.zeros(2, np.uint64)
    f = np.array([1.0, 1.0])
    bad = np.array([1.0, math.inf])
    ax = (ctypes.c_int * 2)(0, 3)
    assert lib.zq_rope_table(None, None, 2, out.ctypes.data) == -1
    assert lib.zq_rope_table(f.ctypes.data, None, 0, out.ctypes.data) == -1
    assert lib.zq_rope_table(bad.ctypes.data, None, 2, out.ctypes.data) == -1
    assert lib.zq_rope_table(f.ctypes.data, ctypes.addressof(ax), 2, out.ctypes.data) == -1


def test_python_refusals_on_the_host():
    torch = pytest.importorskip("torch")
    k = torch.zeros(2, 1, 16, 64, dtype=torch.float16)
    with pytest.raises(ValueError):
        zq.KVCache(k, k)                                   # not on a GPU
    with pytest.raises(ValueError):
        zq.KVCache(k, k[:1])
    with pytest.raises(ValueError):
        zq.KVCache(k.float(), k.float())
    with pytest.raises(ValueError):
        zq.rope_table([1.0, 2.0], [0], device="cpu")


def test_tensors_of_a_call_come_from_its_streams_pool(monkeypatch):
    """Memory that the current stream has just given back may still be in use there: what a call on another stream
    allocates is of that stream's pool, and is kept until the current stream is done with it."""
    torch = pytest.importorskip("torch")
    log, active = [], ["current"]

    class Use:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            active.append(self.stream)

        def __exit__(self, *_):
            active.pop()

    class Made:
        def record_stream(self, stream):
            log.append(("record", stream))

    def empty(*args, **kw):
        log.append(("empty", active[-1]))
        return Made()

    monkeypatch.setattr(torch.cuda, "stream", Use)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: active[-1])
    monkeypatch.setattr(torch, "empty", empty)
    zq._new((4,), torch.float32, "cuda:0", "other")
    assert log == [("empty", "other"), ("record", "current")]
    del log[:]
    zq._new((4,), torch.float32, "cuda:0", "current")
    zq._new((4,), torch.float32, "cuda:0", None)
    assert log == [("empty", "current"), ("empty", "current")]


def test_workspaces_are_one_piece_of_memory():
    """A tensor whose elements share memory, or lie apart, has not the bytes that its size says."""
    torch = pytest.importorskip("torch")
    t = torch.zeros(64, dtype=torch.float32)
    assert zq._space(t, "x") == (t.data_ptr(), 256)
    for bad in (torch.zeros(1, dtype=torch.uint8).expand(1 << 20), t[::2], t.view(8, 8).t()):
        with pytest.raises(ValueError):
            zq._space(bad, "x")


def attn(lib, q=A16, qs=512, B=3, Hq=4, table=A16, width=2, lens=A16, scale=0.1, window=0, out=A16 + 4096, os=512,
         lse=A16, q8=None, ws=A16, wsb=1 << 30, c=None):
    return lib.zq_paged_attn(q, qs, B, Hq, cache() if c is None else c, table, width, lens, scale, window, out, os, lse,
                             q8, ws, wsb, None)


@pytest.mark.parametrize("bad,status", BAD_CACHES)
def test_paged_attn_refuses_caches(lib, bad, status):
    assert attn(lib, c=cache(**bad)) == status
    assert lib.zq_last_error()


@pytest.mark.parametrize("bad,status", [
    (dict(q=None), -1), (dict(q=A8), -3), (dict(qs=500), -2), (dict(qs=513), -2), (dict(B=0), -2), (dict(B=65536), -2),
    (dict(Hq=0), -2), (dict(Hq=1), -2), (dict(Hq=5, qs=1024, os=1024), -2), (dict(Hq=130, qs=1 << 20, os=1 << 20), -2),
    (dict(table=None), -1), (dict(table=A2), -3), (dict(width=0), -2), (dict(width=2 ** 31 - 1), -2),
    (dict(lens=None), -1), (dict(lens=A2), -3), (dict(scale=3e38, c=cache(ks=100.0)), -1), (dict(scale=0.0), -1), (dict(scale=-1.0), -1),
    (dict(scale=math.inf), -1), (dict(scale=math.nan), -1), (dict(window=-1), -1), (dict(out=None), -1),
    (dict(out=A8), -3), (dict(os=500), -2), (dict(out=A16), -1), (dict(lse=A2), -3),
    (dict(q8=ctypes.byref(zq._Q8(A16, A8, A16))), -3), (dict(q8=ctypes.byref(zq._Q8(A16, None, A16))), -1)])
def test_paged_attn_refuses(lib, bad, status):
    assert attn(lib, **bad) == status
    assert lib.zq_last_error()


def test_paged_attn_workspace(lib):
    assert lib.zq_paged_attn_workspace_bytes(4, 3, 128) == 0
    assert lib.zq_paged_attn_workspace_bytes(4, 2, 96) == 0
    small, large = (lib.zq_paged_attn_workspace_bytes(4, 2, D) for D in (64, 256))
    assert 0 < small < large < 64 << 20


def test_valid_paged_attn_without_gpu(lib):
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert attn(lib) == -5
    assert attn(lib, out=None, os=0, q8=ctypes.byref(zq._Q8(A16, A16, A16))) == -5


def lora(lib, q8=None, B=3, K=256, ids=A16, n=2, A=A16, Bm=A16, R=16, type=1, scales=A16, N=64, base=A16, bs=64,
         y=A16 + 4096, ys=64, ws=A16, wsb=1 << 30):
    return lib.zq_lora(zq._Q8(A16, A16, A16) if q8 is None else q8, B, K, ids, n, A, Bm, R, type, scales, N, base, bs, y,
                       ys, ws, wsb, None)


@pytest.mark.parametrize("bad,status", [
    (dict(q8=zq._Q8(None, A16, A16)), -1), (dict(q8=zq._Q8(A8, A16, A16)), -3), (dict(q8=zq._Q8(A16, A8, A16)), -3),
    (dict(B=0), -2), (dict(B=65537), -2), (dict(K=0), -2), (dict(K=48), -2), (dict(K=(1 << 20) + 32), -2),
    (dict(ids=None), -1), (dict(ids=A2), -3), (dict(n=0), -2), (dict(n=(1 << 20) + 1), -2), (dict(A=None), -1),
    (dict(A=A8), -3), (dict(Bm=None), -1), (dict(Bm=A8), -3), (dict(R=0), -2), (dict(R=24), -2), (dict(R=128), -2),
    (dict(type=3), -1), (dict(type=0), -1), (dict(scales=A2), -3), (dict(N=0), -2), (dict(N=(1 << 22) + 1), -2),
    (dict(base=A16 + 2), -3), (dict(bs=63), -2), (dict(y=None), -1), (dict(y=A16 + 2), -3), (dict(ys=63), -2),
    (dict(base=A16, y=A16, bs=64, ys=68), -1), (dict(ws=A8), -3)])
def test_lora_refuses(lib, bad, status):
    assert lora(lib, **bad) == status
    assert lib.zq_last_error()


def test_lora_workspace(lib):
    assert lib.zq_lora_workspace_bytes(0, 256, 16) == 0
    assert lib.zq_lora_workspace_bytes(4, 100, 16) == 0
    assert lib.zq_lora_workspace_bytes(4, 256, 12) == 0
    for B, K, R in ((1, 32, 8), (64, 5120, 16), (512, 17408, 64), (65536, 1024, 8)):
        need = lib.zq_lora_workspace_bytes(B, K, R)
        assert need % (B * R * 4) == 0 and 1 <= need // (B * R * 4) <= max(1, -(-K // 1024))


def test_valid_lora_without_gpu(lib):
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert lora(lib) == -5
    assert lora(lib, base=None, bs=0, scales=None) == -5
    assert lora(lib, base=A16 + 4096) == -5       # in place
