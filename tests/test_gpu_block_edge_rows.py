"""Where the edge between two blocks (zq_residual_norm_q8_1) goes from a CTA for each
row to CTAs that take their rows in turn: both sides of every border, against the
64-bit form with test_gpu_block_edge's tolerances, codes byte for byte."""
import pytest

torch = pytest.importorskip("torch")

import gemm_zq_rmsnorm_gb300 as zq

import _mixer_ref as ref
from test_gpu_block_edge import EPS, edge_want, randn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K,values,gate", [(8192, 18000000, None), (5120, 18000000, None), (4128, 18000000, None),
                                           (4096, 10000000, None), (1024, 10000000, None), (32, 10000000, None),
                                           (8192, 9000000, "rows"), (1056, 9000000, "rows"), (1056, 9000000, "row"),
                                           (1024, 10000000, "rows"), (8224, 20000000, "rows")])
@pytest.mark.parametrize("post", [False, True])
def test_both_sides_of_the_border(K, values, gate, post):
    B = -(-values // K)
    for rows in (B - 1, B):
        x, y = randn(rows, rows, K), randn(K, rows, K)
        gamma, gamma_post = 0.5 + randn(1, K).abs(), 0.5 + randn(2, K).abs() if post else None
        gt = {None: None, "rows": randn(3, rows, K), "row": randn(4, K)}[gate]
        q8, out = zq.empty_q8_1(rows, K), torch.empty(rows, K, device="cuda")
        got = zq.residual_norm_q8_1(x, y, gamma, EPS, gamma_post=gamma_post, gate=gt, act="silu", scale=0.5, out=out, q8_out=q8)
        u, want = edge_want(x, y, gamma, gamma_post, gt, "silu", 0.5)
        tol = 2.0 ** -17 if post else 2.0 ** -20
        assert bool(((got.double() - want).abs() <= tol * u.abs() + 2.0 ** -24 * want.abs()).all())
        xh = ref.norm(got, gamma, EPS)
        assert bool(((out.double() - xh).abs() <= 2.0 ** -17 * xh.abs()).all())
        same = zq.rmsnorm_q8_1(got, gamma, EPS)
        assert torch.equal(q8.qs, same.qs) and torch.equal(q8.d, same.d) and torch.equal(q8.s, same.s)
    assert zq.device_status() == 0
