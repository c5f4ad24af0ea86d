"""Low-rank adapters beside a shared projection (zq_lora) against the 64-bit form.

Tolerance.  h = A x: the 32 products of a Q8_1 block are summed by two MMAs
(each off by at most 2^-21 of its terms' magnitudes), the blocks by a chain of
at most K/256 + 1 additions a warp, three levels of a tree and the splits (at
most 34): e_h = (K/256 + 42) 2^-23 sum |A x|.  h to its 16-bit parts: 2^-24 |h|
in three of bf16, 2^-22 of the token's largest |h| in two of f16.  The expansion sums R
products in MMAs (2^-21 of their magnitudes each 16, once more for each lower
part) and base in one rounding:
|y - ref| <= |scale| sum |B| (e_h + part + (R/16 + 2) 2^-21 |h|) + 2^-23 |ref|."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import gemm_zq_rmsnorm_gb300 as zq
from gemm_zq_rmsnorm_gb300 import inputs

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16


def make(seed, B, K, N, R, n, dtype, ids):
    g = np.random.default_rng(seed)
    x = g.standard_normal((B, K // 32, 32)).astype(np.float32)
    d = (np.abs(x).max(-1) / 127).astype(np.float16)
    qs = np.clip(np.round(x / d.astype(np.float32)[..., None]), -127, 127).astype(np.int8).reshape(B, K)
    a = zq.Q8_1(torch.from_numpy(qs).cuda(), torch.from_numpy(d).cuda(), torch.zeros(B, K // 32, dtype=F16).cuda())
    A = torch.from_numpy((g.standard_normal((n, R, K)) / K ** 0.5).astype(np.float32)).to(dtype).cuda()
    Bm = torch.from_numpy((g.standard_normal((n, N, R))).astype(np.float32)).to(dtype).cuda()
    scales = torch.from_numpy(g.uniform(-2, 2, n).astype(np.float32)).cuda()
    base = torch.from_numpy(g.standard_normal((B, N)).astype(np.float32)).cuda()
    return a, A, Bm, scales, base, torch.tensor(ids, dtype=torch.int32).cuda()


def check(y, a, A, Bm, scales, base, ids):
    y = y.cpu().numpy().astype(np.float64)
    B, K = a.qs.shape
    R, n = A.shape[1], A.shape[0]
    x = a.qs.cpu().numpy().astype(np.float64) * np.repeat(a.d.cpu().numpy().astype(np.float64), 32, 1)
    ids = ids.cpu().numpy()
    want = np.zeros_like(y) if base is None else base.cpu().numpy().astype(np.float64)
    tol = np.zeros_like(y)
    for i in np.unique(ids):
        if not 0 <= i < n:
            continue
        t = np.nonzero(ids == i)[0]
        Ai, Bi = A[i].float().cpu().numpy().astype(np.float64), Bm[i].float().cpu().numpy().astype(np.float64)
        s = 1.0 if scales is None else float(scales[i])
        h = x[t] @ Ai.T
        want[t] += s * (h @ Bi.T)
        e_h = (K / 256 + 42) * 2.0 ** -23 * (np.abs(x[t]) @ np.abs(Ai).T)
        part = 2.0 ** -24 * np.abs(h) if A.dtype == BF16 else 2.0 ** -22 * np.abs(h).max(-1, keepdims=True)
        tol[t] = abs(s) * ((e_h + part + (R / 16 + 2) * 2.0 ** -21 * np.abs(h)) @ np.abs(Bi).T)
    tol += 2.0 ** -23 * np.abs(want)
    off = np.abs(y - want)
    assert np.all(off <= tol), float((off - tol).max())


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("R", [8, 16, 32, 64])
@pytest.mark.parametrize("B,K,N,n", [(1, 32, 1, 1), (1, 1024, 2048, 3), (7, 288, 77, 5), (33, 1024, 260, 4),
                                     (64, 512, 1333, 64), (65, 5120, 512, 2), (200, 2048, 255, 9)])
def test_against_64_bits(dtype, R, B, K, N, n):
    g = np.random.default_rng(B)
    ids = g.integers(-1, n, B)
    a, A, Bm, scales, base, ids = make(B + R, B, K, N, R, n, dtype, ids)
    y = torch.full((B, N), 5.0, device="cuda")
    got = zq.lora(a, ids, A, Bm, scales, base=base, y=y)
    torch.cuda.synchronize()
    assert got is y and zq.device_status() == 0
    check(y, a, A, Bm, scales, base, ids)


@pytest.mark.parametrize("ids", [
    [0] * 70, list(range(64)) + [63] * 6, [-1] * 70, [i // 9 for i in range(70)], [3] + [-1] * 68 + [3],
    [2 ** 31 - 1, -2 ** 31, 64, 63] + [5, 6] * 33, [i % 2 for i in range(70)]],
    ids=["one", "all", "none", "runs", "ends", "outside", "alternating"])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_mixtures(ids, dtype):
    a, A, Bm, scales, base, ids = make(3, 70, 1024, 300, 16, 64, dtype, ids)
    check(zq.lora(a, ids, A, Bm, scales, base=base), a, A, Bm, scales, base, ids)
    check(zq.lora(a, ids, A, Bm), a, A, Bm, None, None, ids)


@pytest.mark.parametrize("N,dtype", [(512, F16), (301, BF16)])
def test_in_place_and_strided_rows(N, dtype):
    """base and y may be columns of a stacked output; what lies between stays."""
    B = 40
    a, A, Bm, scales, base, ids = make(5, B, 1024, N, 32, 3, dtype, [i % 4 - 1 for i in range(B)])
    want = zq.lora(a, ids, A, Bm, scales, base=base)
    for at in (64, 63):
        wide = torch.full((B, N + 200), 9.0, device="cuda")
        wide[:, at:at + N] = base
        part = wide[:, at:at + N]
        zq.lora(a, ids, A, Bm, scales, base=part, y=part)
        torch.cuda.synchronize()
        assert torch.equal(part, want)
        assert torch.all(wide[:, :at] == 9) and torch.all(wide[:, at + N:] == 9)


def test_tokens_without_an_adapter_are_base_bit_for_bit():
    a, A, Bm, scales, base, ids = make(7, 100, 256, 333, 8, 2, F16, [-1, 2, 1] * 33 + [-7])
    base[0, 0], base[3, 5] = float("nan"), float("-inf")
    y = zq.lora(a, ids, A, Bm, scales, base=base)
    none = (ids < 0) | (ids >= 2)
    assert torch.equal(y[none].view(torch.int32), base[none].view(torch.int32))
    y = zq.lora(a, ids, A, Bm, scales)
    assert torch.all(y[none] == 0)


def test_extreme_values():
    """Adapters of very large and very small values (binary16 parts follow the token's size) and the largest codes."""
    B, K, N, R = 6, 512, 64, 16
    a, A, Bm, scales, base, ids = make(9, B, K, N, R, 3, F16, [0, 1, 2, 0, 1, 2])
    a.qs[0], a.qs[1] = 127, -128
    A[1] *= 2.0 ** -10
    A[2] = 60000.0
    base.zero_()
    check(zq.lora(a, ids, A, Bm, scales, base=base), a, A, Bm, scales, base, ids)


@pytest.mark.parametrize("B,n,R", [(3, 2, 16), (56, 1, 16), (56, 12, 16), (17, 4, 64), (40, 3, 64)])
def test_long_rows_are_cut_by_the_units_of_a_tile(B, n, R):
    """17408-wide rows: four, two or one sums of parts of K, as the tile's tokens and adapters fill the GPU."""
    a, A, Bm, scales, base, ids = make(B, B, 17408, 160, R, n, F16, [i % (n + 1) - 1 for i in range(B)])
    check(zq.lora(a, ids, A, Bm, scales, base=base), a, A, Bm, scales, base, ids)


@pytest.mark.parametrize("R,dtype", [(8, F16), (16, BF16), (32, F16), (64, BF16)])
@pytest.mark.parametrize("B,N,runs", [(320, 20000, False), (512, 17409, True)])
def test_many_columns(R, dtype, B, N, runs):
    """Enough outputs for a warp to have many tasks one after the other, in place; the last columns a part of a block."""
    ids = np.random.default_rng(B + R).integers(-1, 6, B)
    a, A, Bm, scales, base, ids = make(B + R, B, 64, N, R, 6, dtype, np.sort(ids) if runs else ids)
    y = base.clone()
    check(zq.lora(a, ids, A, Bm, scales, base=y, y=y), a, A, Bm, scales, base, ids)


def test_large_batch_of_runs():
    B, K, N, R = 2500, 256, 128, 16
    ids = np.repeat(np.arange(7) - 1, 400)[:B]
    a, A, Bm, scales, base, ids = make(11, B, K, N, R, 6, BF16, ids)
    check(zq.lora(a, ids, A, Bm, scales, base=base), a, A, Bm, scales, base, ids)


def test_captured_replayed_and_same_every_time():
    B, K, N, R = 90, 2048, 640, 16
    a, A, Bm, scales, base, ids = make(13, B, K, N, R, 5, BF16, [i % 6 - 1 for i in range(B)])
    want = zq.lora(a, ids, A, Bm, scales, base=base)
    assert torch.equal(zq.lora(a, ids, A, Bm, scales, base=base), want)
    ws = torch.full((zq.lora_workspace_bytes(B, K, R),), 255, dtype=torch.uint8, device="cuda")
    y = torch.zeros(B, N, device="cuda")
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        zq.lora(a, ids, A, Bm, scales, base=base, y=y, workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)
    ids.copy_(torch.tensor([(i + 2) % 6 - 1 for i in range(B)], dtype=torch.int32))   # another batch, same graph
    graph.replay()
    torch.cuda.synchronize()
    check(y, a, A, Bm, scales, base, ids)


def test_beside_the_shared_projection():
    """As a decode step runs it: RMSNorm + Q8_1 once, the shared Q4_K projection and the adapters on its codes, in
    place; equal to the adapters on the projection's own output, computed in 64 bits from there."""
    for B in (1, 4, 8):
        K, N, R, n = 1024, 512, 16, 3
        x, g = inputs.activations(B, B, K), inputs.gamma(B, K)
        W = torch.from_numpy(inputs.q4k_weights(B, N, K)).cuda()
        q8 = zq.rmsnorm_q8_1(torch.from_numpy(x).cuda(), torch.from_numpy(g).cuda(), inputs.EPS)
        _, A, Bm, scales, _, ids = make(15, B, K, N, R, n, F16, [i % n for i in range(B)])
        y = zq.q4k_gemm(W, N, K, q8, B)
        base = y.clone()
        zq.lora(q8, ids, A, Bm, scales, base=y, y=y)
        torch.cuda.synchronize()
        check(y, q8, A, Bm, scales, base, ids)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,R", [(1, 16), (8, 64), (56, 16)])
def test_buffers_rewritten_by_the_kernels_before(B, R, in_place):
    """Back to back in one graph, over and over on the same buffers: the codes, the projection's output and the ids
    that a call reads are those of the kernels right before it, never of an earlier turn."""
    K, N, n, turns = 1024, 1536, 5, 12
    g = inputs.gamma(B, K)
    W = [torch.from_numpy(inputs.q4k_weights(B + i, N, K)).cuda() for i in range(2)]
    xs = [torch.from_numpy(inputs.activations(50 + i, B, K)).cuda() for i in range(turns)]
    gam = torch.from_numpy(g).cuda()
    _, A, Bm, scales, _, _ = make(19, B, K, N, R, n, BF16, [0] * B)
    all_ids = [torch.tensor([(i + 3 * t) % (n + 1) - 1 for t in range(B)], dtype=torch.int32).cuda() for i in range(turns)]
    q8, ids = zq.empty_q8_1(B, K), torch.zeros(B, dtype=torch.int32, device="cuda")
    base, y = torch.zeros(B, N, device="cuda"), torch.zeros(B, N, device="cuda")
    got = torch.zeros(turns, B, N, device="cuda")
    ws = torch.empty(max(zq.lora_workspace_bytes(B, K, R), 256), dtype=torch.uint8, device="cuda")
    gws = torch.empty(max(zq.gemm_workspace_bytes(N, K, B), 256), dtype=torch.uint8, device="cuda")

    def turn(i, sync):
        ids.copy_(all_ids[i])
        zq.rmsnorm_q8_1(xs[i], gam, inputs.EPS, out=q8)
        sync()
        zq.q4k_gemm(W[i % 2], N, K, q8, B, y=base, workspace=gws)
        sync()
        to = base if in_place else y
        zq.lora(q8, ids, A, Bm, scales, base=base, y=to, workspace=ws)
        sync()
        zq.lora(q8, ids, A, Bm, scales, base=to, y=got[i], workspace=ws)
        sync()

    for i in range(turns):
        turn(i, torch.cuda.synchronize)
    want = got.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for i in range(turns):
            turn(i, lambda: None)
    for _ in range(20):
        got.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)


def test_refusals():
    a, A, Bm, scales, base, ids = make(17, 4, 256, 64, 16, 2, F16, [0, 1, 0, 1])
    for bad in (dict(ids=ids.long()), dict(A=A.float()), dict(A=A.to(BF16)), dict(Bm=Bm[:, :, :8]), dict(ids=ids[:3]),
                dict(scales=scales.half()), dict(base=base.half()), dict(base=base[:3]), dict(y=base.t()),
                dict(A=A[:, :, :128]), dict(ids=ids.cpu())):
        kw = dict(a=a, ids=ids, A=A, Bm=Bm, scales=scales, base=base)
        kw.update(bad)
        with pytest.raises(ValueError):
            zq.lora(**kw)
    with pytest.raises(zq.ZQError) as e:
        zq.lora(a, ids, A, Bm, scales, base=base, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == -6
    with pytest.raises(zq.ZQError) as e:
        zq.lora(a, ids, A[:, :4].contiguous(), Bm[:, :, :4].contiguous(), scales, base=base)
    assert e.value.status == -2
    torch.cuda.synchronize()
