"""What paged attention keeps over the range of its weights and of its cache's
values: rows far below a dominant one, infinities in the cache.

Weights.  A binary16 or e4m3 cache takes a weight, relative to the largest so
far, as two binary16 parts of its 2^15-fold: 2^-22 of itself, and 2^-40 (half a
step of 2^-24, over 2^15) where that is more.  With e_s the relative error of a
weight from its score (test_gpu_paged_attn.py), A = sum p |v| / sum p:
|out - ref| <= (2 e_s + 2^-21 + (tiles + pieces) 2^-22) A + 2^-40 max p sum |v| / sum p + 2^-23 |ref|;
the weights' floor is relative to a row of at most the largest weight, whose
share max p / sum p is at most 1."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import gemm_zq_rmsnorm_gb300 as zq

from test_gpu_paged_attn import BF16, E4M3, F16, Case

pytestmark = pytest.mark.gpu


def heads64(c, b):
    """Scores [rows][Hq], values [rows][Hq][D], |scale q k| summed [rows][Hq], of sequence b in 64 bits."""
    k, v = (np.repeat(x, c.Hq // c.Hk, 1) for x in c.rows(b))
    q = c.q[b].cpu().numpy().astype(np.float64)
    return (c.scale * np.einsum("hd,thd->th", q, k), v,
            c.scale * np.einsum("hd,thd->th", np.abs(q), np.abs(k)))


@pytest.mark.parametrize("gap", [6.0, 14.0, 16.0, 18.0])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", [F16, BF16, E4M3])
@pytest.mark.parametrize("lens", [[70] * 900, [1000], [3, 33, 2]], ids=["many", "long", "short"])
def test_rows_far_below_a_dominant_one_count(lens, dtype, D, gap):
    """One row `gap` nats above the others, whose value is zero (an attention sink): the output is the others' alone.
    With many sequences a warp holds whole ones; the dominant row is a sequence's first, or lies inside it."""
    c = Case(len(lens) + D, lens, 2, 1, D, dtype, 16, gain=0.25)
    c.k.view(torch.uint8 if dtype == E4M3 else dtype)[..., 0] = 0
    c.q[..., 0] = gap * D ** 0.5
    table = c.table.cpu().numpy()
    sink = np.array([0 if b % 2 else min(n - 1, 21) for b, n in enumerate(lens)])
    page = torch.from_numpy(table[np.arange(len(lens)), sink // 16].astype(np.int64)).cuda()
    row = torch.from_numpy((sink % 16).astype(np.int64)).cuda()
    one = int(torch.tensor(1.0).to(dtype).view(torch.uint8 if dtype == E4M3 else torch.int16))
    for pool, first in ((c.k, one), (c.v, 0)):
        x = pool.view(torch.uint8 if dtype == E4M3 else torch.int16)
        x[page, :, row] = 0
        x[page, :, row, 0] = first
    out, lse = (x.cpu().numpy().astype(np.float64) for x in c.run())
    for b in range(0, len(lens), 9):
        s, v, S = heads64(c, b)
        m = s.max(0)
        assert np.all(m - np.sort(s, 0)[-2] > gap - 2)
        p = np.exp(s - m)
        total = p.sum(0)
        want = np.einsum("th,thd->hd", p, v) / total[:, None]
        A = np.einsum("th,thd->hd", p, np.abs(v)) / total[:, None]
        K = S.max(0) + gap          # scale max |q| sum |k| is at most q's first value times a row's sum
        K = np.maximum(K, c.scale * np.abs(c.q[b].cpu().numpy()).max(-1) * np.abs(c.rows(b)[0]).sum(-1).max())
        e_s = (D / 32 + 8) * 2.0 ** -22 * S.max(0) + 2.0 ** -22 * K + 2.0 ** -21 * (1 + np.abs(s).max(0))
        tiles = -(-len(s) // 32) + 1
        tol = ((2 * e_s + 2.0 ** -21 + 2 * tiles * 2.0 ** -22)[:, None] * A
               + (0 if dtype == BF16 else 2.0 ** -40) * np.abs(v).sum(0) / total[:, None] + 2.0 ** -23 * np.abs(want))
        off = np.abs(out[b].reshape(want.shape) - want)
        assert np.all(off <= tol), (b, float((off / np.maximum(tol, 1e-300)).max()), float((off / A).max()))
        want_lse = m + np.log(total)
        assert np.all(np.abs(lse[b] - want_lse) <= e_s + 2 * tiles * 2.0 ** -24 + 2.0 ** -22 * (1 + np.abs(want_lse)))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("at", [0, 37, 599])
def test_scores_of_minus_infinity_weigh_nothing(D, dtype, at):
    """A key that overflowed to an infinity: where it makes a score -infinity the row weighs nothing, whatever the
    parts of q are (zeros, of either sign); where it makes one +infinity the head is NaN."""
    c = Case(D, [600, 40, 1], 8, 2, D, dtype, 16)
    page, row = int(c.table[0, at // 16]), at % 16
    c.q[0, 4:, 7] = torch.tensor([-1.0, -1.3, -0.7123, 0.01])
    c.k[page, 1, row, 7] = float("inf")
    c.k[page, 0, row, 9] = float("-inf")
    c.q[0, :4, 9] = torch.tensor([1.0, 1.3, 3.1e-5, 0.7123])
    one = int(c.table[2, 0])
    c.k[one, 1, 0, 5] = float("-inf")
    c.q[2, 4:, 5] = 1.0
    keys = c.k.clone()
    out, lse = c.run()
    assert out[0, 7].isnan().all() and lse[0, 7].isnan()
    # a sequence whose only score is -infinity has nothing to see
    assert torch.all(out[2, 4:] == 0) and torch.all(torch.isneginf(lse[2, 4:]))
    # the others: as if the row were not there
    keep = torch.ones(8, dtype=torch.bool)
    keep[7] = False
    c.k[page, :, row] = 0
    c.k[one, 1, 0, 5] = 0
    s, v, S = heads64(c, 0)
    rows = np.arange(600) != at
    s, v, S = s[rows], v[rows], S[rows]
    m = s.max(0)
    p = np.exp(s - m)
    want = np.einsum("th,thd->hd", p, v) / p.sum(0)[:, None]
    A = np.einsum("th,thd->hd", p, np.abs(v)) / p.sum(0)[:, None]
    K = c.scale * np.abs(c.q[0].cpu().numpy()).max(-1) * np.abs(c.rows(0)[0]).sum(-1).max()
    e_s = (D / 32 + 8) * 2.0 ** -22 * S.max(0) + 2.0 ** -22 * K + 2.0 ** -21 * (1 + np.abs(s).max(0))
    tol = (2 * e_s + 2.0 ** -21 + 2 * 20 * 2.0 ** -22)[:, None] * A + 2.0 ** -23 * np.abs(want)
    off = np.abs(out[0].cpu().numpy() - want)
    assert np.all(off[keep.numpy()] <= tol[keep.numpy()]), float((off / tol)[keep.numpy()].max())
    want_lse = (m + np.log(p.sum(0)))[keep.numpy()]
    assert np.all(np.abs(lse[0].cpu().numpy()[keep.numpy()] - want_lse) <= e_s.max() + 2.0 ** -20 * (1 + np.abs(want_lse)))
    # the sequence between them saw none of it
    c.k.copy_(keys)
    again, again_lse = c.run()
    assert torch.equal(again[1], out[1]) and not out[1].isnan().any()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_an_infinite_value_spoils_its_column_only(D, dtype):
    c = Case(D + 1, [600, 40], 8, 2, D, dtype, 16)
    want, want_lse = c.run()
    page = int(c.table[0, 3])
    c.v[page, 1, 5, 11] = float("inf")
    out, lse = c.run()
    assert not out[0, 4:, 11].isfinite().any()
    out[0, 4:, 11] = want[0, 4:, 11]
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
