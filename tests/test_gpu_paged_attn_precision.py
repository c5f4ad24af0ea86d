"""The precision of paged attention as a root mean square over many outputs, so
tight that a part of q, a part of the weights, or sums over tiles in the tensor
core's truncating accumulator could not go missing unseen: each of these is
planted in the 64-bit form, and its error has to exceed the bound.

Bounds, for A = sum p |v| / sum p, in root mean squares (u = 2^-24, an error spread evenly over [-e, e] has e / sqrt 3):
* output: 2^x to 4u (2.3u), its argument to u a unit of |x| <= 3 (1.7u), three products in a row that are truncated
  by at most 2u of their sum each (3 x 1.2u), three roundings (1u): 4.8u, so 5u; and the heaviest row's score, which
  weighs against all others: it is the sum of D / 16 products in a row, and 1 to 2 nats lie in one or two binades of
  the unscaled sum (sqrt D to 2 sqrt D), whose last place is 2u nats at D = 64 and 256 and 1.4u or 2.8u at D = 128, so
  a truncated sum loses half of that a product on average, all of one sign: D / 16 x 1.1u more, in squares;
* the score of one row, which is its lse, against the root of the sum of its squared terms: D / 16 = 4 products a part, each
  truncated by at most 2u of the partial sum, all of one sign at worst (4.7u), additions of the parts, the scale, ln 2 and
  the result's rounding (2u), two binary16 parts of q 2^-22 of its largest value (four in a root of sums: 4 x 4u / sqrt 3 / 4
  of it): 6u, 8u with those;
* the mean (not its square) of the errors of sums of one sign over many tiles: the products' truncation, 3 x 1u, and
  the spread of the rest: 4u."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import gemm_zq_rmsnorm_gb300 as zq

from test_gpu_paged_attn import BF16, E4M3, F16, Case
from test_gpu_paged_attn_range import heads64

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def parts(x, dtype, n):
    """x as the sum of n 16-bit parts, each rounded to nearest, binary16 ones of 2^15 x."""
    up = 1.0 if dtype == BF16 else 2.0 ** 15
    left, got = torch.from_numpy(np.ascontiguousarray(x * up)), 0.0
    for _ in range(n):
        p = left.to(torch.float32).to(BF16 if dtype == BF16 else F16).double()
        left, got = left - p, got + p
    return (got / up).numpy()


def rms(x):
    return float(np.sqrt(np.mean(np.square(x))))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", [F16, BF16, E4M3])
def test_weights_keep_all_their_parts(dtype, D):
    """Three rows, the heaviest of them of value zero: the output's relative error is that of the others' weights."""
    B = 300
    c = Case(D, [3] * B, 2, 1, D, dtype, 16, gain=0.25)
    raw = torch.uint8 if dtype == E4M3 else torch.int16
    page = c.table[:, 0].long()
    one = int(torch.tensor(1.0).to(dtype).view(raw))
    c.k.view(raw)[page, :, :3, 0] = 0
    c.k.view(raw)[page, :, 1, 0] = one
    c.v.view(raw)[page, :, 1] = 0
    c.q[..., 0] = torch.from_numpy(np.random.default_rng(1).uniform(1.0, 2.0, (B, 2)).astype(np.float32)).cuda() * D ** 0.5
    out, _ = c.run()
    out = out.cpu().numpy().astype(np.float64)
    off, planted = [], []
    for b in range(B):
        s, v, _ = heads64(c, b)
        p = np.exp(s - s.max(0))
        total = p.sum(0)[:, None]
        A = np.einsum("th,thd->hd", p, np.abs(v)) / total
        want = np.einsum("th,thd->hd", p, v) / total
        cut = np.einsum("th,thd->hd", parts(p, dtype, 2 if dtype == BF16 else 1), v) / total
        keep = A > 1e-3
        off.append(((out[b] - want) / np.maximum(A, 1e-3))[keep])
        planted.append(((cut - want) / np.maximum(A, 1e-3))[keep])
    off, planted = np.concatenate(off), np.concatenate(planted)
    bound = np.hypot(5, D / 16 * 1.1) * U
    assert rms(planted) > 1.3 * bound, rms(planted) / U
    assert rms(off) <= bound, rms(off) / U


@pytest.mark.parametrize("dtype", [F16, BF16, E4M3])
def test_queries_keep_all_their_parts(dtype):
    B, D = 1000, 64
    c = Case(3, [1] * B, 4, 2, D, dtype, 16)
    _, lse = c.run()
    lse = lse.cpu().numpy().astype(np.float64)
    off, planted = [], []
    for b in range(B):
        k = np.repeat(c.rows(b)[0][0], 2, 0)
        q = c.q[b].cpu().numpy().astype(np.float64)
        size = c.scale * np.sqrt(np.square(q * k).sum(-1))
        q_cut = parts(q, BF16, 2) if dtype == BF16 else parts(q * 2.0 ** -15, F16, 1) * 2.0 ** 15
        want = c.scale * (q * k).sum(-1)
        off.append((lse[b] - want) / size)
        planted.append((c.scale * (q_cut * k).sum(-1) - want) / size)
    bound = (6 if dtype == BF16 else 8) * U
    assert rms(planted) > 1.5 * bound, rms(planted) / U
    assert rms(off) <= bound, rms(off) / U


@pytest.mark.parametrize("dtype", [F16, BF16, E4M3])
def test_sums_over_many_tiles_are_not_truncated(dtype):
    """Values of one sign: some forty tiles a warp, whose sums are rounded to nearest."""
    B, Hk, D, n, page = 64, 4, 64, 12000, 64
    g = torch.Generator(device="cuda").manual_seed(5)
    need = -(-n // page)
    shape = (B * need, Hk, page, D)
    k = torch.randn(*shape, generator=g, device="cuda").to(dtype)
    v = (1 + torch.rand(*shape, generator=g, device="cuda")).to(dtype)
    table = torch.arange(B * need, dtype=torch.int32, device="cuda").view(B, need)
    lens = torch.full((B,), n, dtype=torch.int32, device="cuda")
    q = 0.5 * torch.randn(B, Hk, D, generator=g, device="cuda")
    out = zq.paged_attn(q, zq.KVCache(k, v), table, lens)
    torch.cuda.synchronize()
    off = []
    for b in range(0, B, 4):
        kb, vb = (x[b * need:(b + 1) * need].double().transpose(1, 2).reshape(-1, Hk, D)[:n] if dtype != E4M3 else
                  x[b * need:(b + 1) * need].float().double().transpose(1, 2).reshape(-1, Hk, D)[:n] for x in (k, v))
        p = torch.softmax(torch.einsum("hd,thd->ht", q[b].double(), kb) * D ** -0.5, -1)
        want = torch.einsum("ht,thd->hd", p, vb)
        off.append(((out[b].double() - want) / want).cpu().numpy())
    # the same with two sums a tile of 32 rows truncated to 24 bits, forty tiles
    gen = np.random.default_rng(0)
    acc = exact = np.zeros(1000)
    for _ in range(80):
        y = gen.uniform(8, 40, 1000)
        exact = exact + y
        m, e = np.frexp(acc + y)
        acc = np.ldexp(np.floor(m * 2.0 ** 24) / 2.0 ** 24, e)
    assert abs(np.mean((acc - exact) / exact)) > 10 * U
    assert abs(np.mean(off)) <= 4 * U and rms(off) <= 5 * U, (np.mean(off) / U, rms(off) / U)
