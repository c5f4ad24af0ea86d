"""The gated head norm (zq_gated_norm_q8_1) and the edge between two blocks
(zq_residual_norm_q8_1) against their 64-bit forms.

Tolerances.  A norm: squares added in at most 32 + 4 + 8 steps (the rows' sums
128 + 8), a mean, a sum, a root, a division and two products: under 160 * 2^-24
of the value, half of it from the sum's root; a gate: ex2 to 2^-22 and two
roundings, 1 + e, a reciprocal to 2^-23, two products: 11 * 2^-24 of itself; 2^-17
of the value together, 2^-20 without a norm.  A residual sum
takes that of its second part and half a step of the result.  Codes are those
that the library's packing gives for the fp32 values, byte for byte."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import gemm_zq_rmsnorm_gb300 as zq

import _attn_ref
import _mixer_ref as ref

pytestmark = pytest.mark.gpu

EPS = 1e-6


def randn(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def same_codes(q8, rows):
    qs, d, s = _attn_ref.q8_1(rows.cpu().numpy())
    assert np.array_equal(q8.qs.cpu().numpy(), qs)
    assert np.array_equal(q8.d.cpu().numpy(), d, equal_nan=True) and np.array_equal(q8.s.cpu().numpy(), s, equal_nan=True)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("B,H", [(1, 1), (1, 48), (7, 3), (61, 5), (1500, 2)])
@pytest.mark.parametrize("act", ["linear", "sigmoid", "silu"])
def test_gated_norm(D, B, H, act):
    stacked = randn(B + D, B, 4 + 2 * H * D) * 2.0
    x, gate = stacked[:, 4:4 + H * D], stacked[:, 4 + H * D:]
    gamma = 0.5 + randn(1, D).abs()
    q8 = zq.empty_q8_1(B, H * D)
    for norm, gated in ((True, True), (False, True), (True, False)):
        out = zq.gated_norm_q8_1(x, gate if gated else None, gamma if norm else None, EPS, D, act=act,
                                 out=torch.empty(B, H * D, device="cuda"), q8_out=q8)
        want = ref.norm(x.reshape(B, H, D), gamma if norm else None, EPS).reshape(B, H * D)
        if gated:
            want = want * ref.act(gate, act)
        tol = 2.0 ** -17 if norm else 2.0 ** -20
        assert bool(((out.double() - want).abs() <= tol * want.abs() + 1e-37).all())
        same_codes(q8, out)
        only = zq.gated_norm_q8_1(x, gate if gated else None, gamma if norm else None, EPS, D, act=act,
                                  q8_out=zq.empty_q8_1(B, H * D))
        assert torch.equal(only.qs, q8.qs) and torch.equal(only.d, q8.d) and torch.equal(only.s, q8.s)


def test_gates_of_any_size():
    g = torch.cat((torch.linspace(-120, 120, 4093, device="cuda"),
                   torch.tensor([0.0, -0.0, float("inf"), -float("inf"), float("nan"), 1e30, -1e30, 3e38, -3e38, 1e-30, 87.9],
                                device="cuda")))
    g = torch.cat((g, g.new_zeros(-len(g) % 64)))[None]
    one = torch.ones_like(g)
    got = zq.gated_norm_q8_1(one, g, None, 0.0, 64, act="sigmoid")
    want = torch.sigmoid(g.double())
    ok = ~want.isnan()
    assert bool(((got.double() - want)[ok].abs() <= 2.0 ** -20 * want[ok] + 2.0 ** -126).all())
    assert torch.equal(got.isnan(), g.isnan())
    got = zq.gated_norm_q8_1(one, g, None, 0.0, 64, act="silu")
    fine = torch.isfinite(g)
    want = g.double() * want
    assert bool(((got.double() - want)[fine].abs() <= 2.0 ** -20 * want[fine].abs() + 2.0 ** -118).all())


def test_gated_norm_of_what_is_not_finite_and_of_zeros():
    x = randn(3, 9, 3 * 128)
    x[2, 130] = float("nan")
    x[4, :128] = 0.0
    x[5, 300] = float("inf")
    gamma, gate = torch.ones(128, device="cuda"), torch.ones_like(x)
    out = zq.gated_norm_q8_1(x, gate, gamma, EPS, 128, act="linear")
    bad = torch.zeros(9, 3, dtype=torch.bool, device="cuda")
    bad[2, 1] = bad[5, 2] = True
    heads = out.view(9, 3, 128)
    assert torch.equal(heads.isnan().any(-1), bad) and bool((heads[4, 0] == 0).all())
    q8 = zq.gated_norm_q8_1(x[4:5], None, gamma, EPS, 128, q8_out=zq.empty_q8_1(1, 384))
    assert bool((q8.qs[0, :128] == 0).all()) and bool((q8.d[0, :4] == 0).all())
    zero = zq.gated_norm_q8_1(torch.zeros(2, 64, device="cuda"), None, torch.ones(64, device="cuda"), EPS, 64)
    assert bool((zero == 0).all())


def test_gated_norm_in_place_and_three_dimensions():
    x, gate, gamma = randn(4, 11, 3, 64), randn(5, 11, 3, 64), randn(6, 64)
    want = zq.gated_norm_q8_1(x, gate, gamma, EPS, 64)
    assert want.shape == x.shape
    got = zq.gated_norm_q8_1(x, gate, gamma, EPS, 64, out=x)
    assert got is x and torch.equal(x, want)


def edge_want(x, y, gamma, gamma_post, gate, act, scale):
    u = ref.norm(y, gamma_post, EPS)
    if gate is not None:
        u = u * ref.act(gate, act)
    return scale * u, x.double() + scale * u


@pytest.mark.parametrize("B,K", [(1, 32), (1, 1024), (3, 2048 + 32), (61, 5120), (2, 8192), (2, 8224), (3, 16384),
                                 (2, 17408), (2, 32768), (700, 256)])
@pytest.mark.parametrize("post,gate,act,scale", [(False, None, "linear", 1.0), (True, None, "linear", 0.22),
                                                 (True, "rows", "sigmoid", 1.0), (False, "row", "linear", -0.5),
                                                 (True, "rows", "silu", 2.0)])
def test_residual_norm(B, K, post, gate, act, scale):
    scale = float(np.float32(scale))
    stacked = randn(B + K, B, 2 * K + 8) * 1.5
    x, y = stacked[:, 4:4 + K], stacked[:, 4 + K:4 + 2 * K]
    gamma, gamma_post = 0.5 + randn(1, K).abs(), 0.5 + randn(2, K).abs() if post else None
    gt = {None: None, "rows": randn(3, B, K + 4)[:, :K], "row": randn(4, K)}[gate]
    q8, out = zq.empty_q8_1(B, K), torch.empty(B, K + 4, device="cuda")[:, :K]
    got = zq.residual_norm_q8_1(x, y, gamma, EPS, gamma_post=gamma_post, gate=gt, act=act, scale=scale, out=out, q8_out=q8)
    u, want = edge_want(x, y, gamma, gamma_post, gt, act, scale)
    tol = 2.0 ** -17 if post else 2.0 ** -20
    assert bool(((got.double() - want).abs() <= tol * u.abs() + 2.0 ** -24 * want.abs()).all())
    # the norm of what was stored, and its codes byte for byte
    xh = ref.norm(got, gamma, EPS)
    assert bool(((out.double() - xh).abs() <= 2.0 ** -17 * xh.abs()).all())
    same = zq.rmsnorm_q8_1(got, gamma, EPS)
    assert torch.equal(q8.qs, same.qs) and torch.equal(q8.d, same.d) and torch.equal(q8.s, same.s)
    same_codes(q8, out)


@pytest.mark.parametrize("B,K", [(2003, 5120), (1251, 8192), (9777, 1056), (312513, 32)])
@pytest.mark.parametrize("post,gate,act", [(False, None, "linear"), (True, "rows", "silu"), (True, "row", "sigmoid")])
def test_residual_norm_of_many_rows(B, K, post, gate, act):
    """From ten million values on, CTAs take their rows in turn while the next ones are on their way."""
    assert B * K >= 10 ** 7
    x, y = randn(B, B, K), randn(K, B, K + 4)[:, 4:]
    gamma, gamma_post = 0.5 + randn(1, K).abs(), 0.5 + randn(2, K).abs() if post else None
    gt = {None: None, "rows": randn(3, B, K + 4)[:, :K], "row": randn(4, K)}[gate]
    q8, out = zq.empty_q8_1(B, K), torch.empty(B, K, device="cuda")
    got = zq.residual_norm_q8_1(x, y, gamma, EPS, gamma_post=gamma_post, gate=gt, act=act, scale=0.5, out=out, q8_out=q8)
    u, want = edge_want(x, y, gamma, gamma_post, gt, act, 0.5)
    tol = 2.0 ** -17 if post else 2.0 ** -20
    assert bool(((got.double() - want).abs() <= tol * u.abs() + 2.0 ** -24 * want.abs()).all())
    xh = ref.norm(got, gamma, EPS)
    assert bool(((out.double() - xh).abs() <= 2.0 ** -17 * xh.abs()).all())
    same = zq.rmsnorm_q8_1(got, gamma, EPS)
    assert torch.equal(q8.qs, same.qs) and torch.equal(q8.d, same.d) and torch.equal(q8.s, same.s)
    for into in (x, y):                                   # in place of either
        before = into.clone()
        again = zq.residual_norm_q8_1(x, y, gamma, EPS, gamma_post=gamma_post, gate=gt, act=act, scale=0.5, x_out=into)
        assert again is into and torch.equal(into, got)
        into.copy_(before)
    assert zq.device_status() == 0


@pytest.mark.parametrize("B,H,D", [(701, 48, 128), (20837, 3, 64), (1303, 13, 256)])
def test_gated_norm_of_many_rows(B, H, D):
    """From four million values on a warp has two groups of rows on their way when it packs codes."""
    assert B * H * D >= 4 * 10 ** 6
    x, gate, gamma = randn(B, B, H * D), randn(H, B, H * D + 4)[:, 4:], 0.5 + randn(D, D).abs()
    q8 = zq.empty_q8_1(B, H * D)
    out = zq.gated_norm_q8_1(x, gate, gamma, EPS, D, out=torch.empty_like(x), q8_out=q8)
    want = ref.norm(x.reshape(B, H, D), gamma, EPS).reshape(B, H * D) * ref.act(gate, "silu")
    assert bool(((out.double() - want).abs() <= 2.0 ** -17 * want.abs() + 1e-37).all())
    same_codes(q8, out)
    alone = zq.gated_norm_q8_1(x, gate, gamma, EPS, D)    # fp32 rows: one group a warp
    assert torch.equal(alone, out)


def test_residual_in_place_alone_and_without_norm():
    x, y, gamma = randn(1, 9, 640), randn(2, 9, 640), randn(3, 640)
    want = zq.residual_norm_q8_1(x, y, None, 0.0, scale=0.5)
    assert torch.equal(want, torch.addcmul(x, y, torch.tensor(0.5, device="cuda"))) or bool(
        ((want.double() - (x.double() + 0.5 * y.double())).abs() <= 2.0 ** -24 * want.abs().double()).all())
    q8, q8b = zq.empty_q8_1(9, 640), zq.empty_q8_1(9, 640)
    zq.residual_norm_q8_1(x, y, None, 0.0, scale=0.5, q8_out=q8)             # codes of x_out itself
    same_codes(q8, want)
    zq.residual_norm_q8_1(x, y, gamma, EPS, scale=0.5, q8_out=q8)
    y2 = y.clone()
    assert torch.equal(zq.residual_norm_q8_1(x, y2, gamma, EPS, scale=0.5, x_out=y2, q8_out=q8b), want)
    assert torch.equal(q8.qs, q8b.qs)
    x2 = x.clone()
    assert zq.residual_norm_q8_1(x2, y, gamma, EPS, scale=0.5, x_out=x2, q8_out=q8b) is x2 and torch.equal(x2, want)
    assert torch.equal(q8.qs, q8b.qs) and torch.equal(q8.d, q8b.d)


def test_captured_edges_on_another_stream():
    x, y, gate, gamma = randn(1, 20, 1024), randn(2, 20, 1024), randn(3, 20, 1024), 0.5 + randn(4, 1024).abs()
    q8, q8g = zq.empty_q8_1(20, 1024), zq.empty_q8_1(20, 1024)

    def calls(stream=None):
        zq.residual_norm_q8_1(x, y, gamma, EPS, gamma_post=gamma, gate=gate, act="sigmoid", x_out=x, q8_out=q8, stream=stream)
        zq.gated_norm_q8_1(x, gate, gamma[:128], EPS, 128, q8_out=q8g, stream=stream)
    x0 = x.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    calls(s)
    torch.cuda.synchronize()
    want = [t.clone() for t in (x, q8.qs, q8g.qs, q8g.s)]
    x.copy_(x0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for t in (q8.qs, q8g.qs):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((x, q8.qs, q8g.qs, q8g.s), want))


def test_binding_refuses():
    x, g = randn(1, 4, 256), torch.ones(128, device="cuda")
    q8 = zq.empty_q8_1(4, 256)
    for bad in (dict(D=96), dict(gate=x[:, :128]), dict(gate=x.cpu()), dict(gamma=g[:64]), dict(act="relu"),
                dict(out=x[:3]), dict(q8_out=zq.empty_q8_1(4, 512))):
        a = dict(gate=x, gamma=g, D=128, act="silu", out=None, q8_out=q8)
        a.update(bad)
        with pytest.raises(ValueError):
            zq.gated_norm_q8_1(x, a["gate"], a["gamma"], EPS, a["D"], act=a["act"], out=a["out"], q8_out=a["q8_out"])
    gamma = torch.ones(256, device="cuda")
    for bad in (dict(y=x[:, :128]), dict(y=x.half()), dict(gamma=g), dict(gate=g), dict(gate=x.t()), dict(x_out=x.double()),
                dict(act="tanh"), dict(q8_out=zq.empty_q8_1(3, 256)), dict(gamma_post=gamma.cpu())):
        a = dict(y=x, gamma=gamma, gate=None, x_out=None, act="linear", q8_out=q8, gamma_post=None)
        a.update(bad)
        with pytest.raises(ValueError):
            zq.residual_norm_q8_1(x, a["y"], a["gamma"], EPS, gamma_post=a["gamma_post"], gate=a["gate"], act=a["act"],
                                  x_out=a["x_out"], q8_out=a["q8_out"])
