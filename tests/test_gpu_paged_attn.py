"""Attention of one new token over the paged cache (zq_paged_attn) against the
64-bit form, on caches whose unused places hold NaN.

Tolerances.  With S = scale sum |q k| of a row, A = sum p |v| / sum p and K =
scale max |q| sum |k|: a score passes through at most D/16 tensor-core sums of
16 products (each truncated to its accumulator's step, 2^-22 of S at most; half
of them in each of two chains at worst) and a few additions, q is off by 2^-22
of its largest value (two binary16 parts; three bf16 parts are exact), the
scaling and 2^x by 2^-21: e_s = (D/32 + 8) 2^-22 S + 2^-22 K + 2^-21 (1 + |s|).
A weight is off by e_s relatively and by 2^-22 for its parts, the sums by one
rounding of 2^-22 for each tile of a warp (all tiles at worst) and each joined
piece (< 320):
|out - ref| <= (2 e_s + 2^-21 + (tiles + 320) 2^-22) A + 2^-23 |ref|,
|lse - ref| <= e_s + (tiles + 320) 2^-24 + 2^-22 (1 + |ref|)."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import gemm_zq_rmsnorm_gb300 as zq

import _attn_ref as ref

pytestmark = pytest.mark.gpu

F16, BF16, E4M3 = torch.float16, torch.bfloat16, torch.float8_e4m3fn


class Case:
    """A cache of random pages, NaN wherever no row of a sequence is."""

    def __init__(self, seed, lens, Hq, Hk, D, dtype, page, window=0, scales=(1.0, 1.0), extra_width=0, gain=1.5):
        g = np.random.default_rng(seed)
        B = len(lens)
        self.lens, self.Hq, self.Hk, self.D, self.page, self.window = lens, Hq, Hk, D, page, window
        self.ks, self.vs = (float(np.float32(s)) for s in scales)
        need = [max(0, -(-n // page)) for n in lens]
        width = max(1, max(need)) + extra_width
        pages = sum(need) + 3
        order = g.permutation(pages)
        table = np.full((B, width), -1, np.int32)
        table[:] = g.choice(np.array([-1, pages, 2 ** 31 - 1, -2 ** 31], np.int64), (B, width)).astype(np.int32)
        used = np.zeros((pages, page), bool)
        at = 0
        for b, n in enumerate(lens):
            table[b, :need[b]] = order[at:at + need[b]]
            at += need[b]
            j = np.arange(max(0, n - window) if window else 0, max(n, 0))
            used[table[b, j // page], j % page] = True
        k = torch.from_numpy(g.standard_normal((pages, Hk, page, D)).astype(np.float32) / np.float32(self.ks)).to(dtype)
        v = torch.from_numpy(g.standard_normal((pages, Hk, page, D)).astype(np.float32) / np.float32(self.vs)).to(dtype)
        bad = torch.from_numpy(~used)[:, None, :, None].expand(pages, Hk, page, D)
        for x in (k, v):
            if dtype == E4M3:
                x.view(torch.uint8)[bad] = 0x7f
            else:
                x[bad] = float("nan")
        self.k, self.v, self.table, self.dtype = k.cuda(), v.cuda(), torch.from_numpy(table).cuda(), dtype
        self.q = torch.from_numpy((gain * g.standard_normal((B, Hq, D))).astype(np.float32)).cuda()
        self.t_lens = torch.tensor(lens, dtype=torch.int32).cuda()
        self.cache = zq.KVCache(self.k, self.v, self.ks, self.vs)
        self.scale = D ** -0.5

    def run(self, **kw):
        B = len(self.lens)
        lse = torch.full((B, self.Hq), 7.0, device="cuda")
        out = zq.paged_attn(self.q, self.cache, self.table, self.t_lens, window=self.window, lse=lse, **kw)
        torch.cuda.synchronize()
        assert zq.device_status() == 0
        return out, lse

    def rows(self, b):
        """K and V rows of sequence b, float64 [n][Hk][D], as the cache holds them."""
        n = max(0, self.lens[b])
        j = np.arange(n)
        pages = self.table[b].cpu().numpy().astype(np.int64)[j // self.page]
        if n:
            assert pages.min() >= 0
        got = []
        for pool, s in ((self.k, self.ks), (self.v, self.vs)):
            f = pool.float().transpose(1, 2).reshape(-1, self.Hk, self.D)
            got.append(f[torch.from_numpy(pages * self.page + j % self.page).cuda()].cpu().numpy().astype(np.float64) * s)
        return got

    def check(self, out, lse, left_out=()):
        q = self.q.cpu().numpy().astype(np.float64)
        out = out.cpu().numpy().astype(np.float64).reshape(q.shape)
        lse = lse.cpu().numpy().astype(np.float64)
        G = self.Hq // self.Hk
        for b, n in enumerate(self.lens):
            n = max(n, 0)
            first = max(0, n - self.window) if self.window else 0
            tok = np.array([j for j in range(first, n) if j // self.page not in left_out], int)
            k, v = self.rows(b)
            want, want_lse = ref.attn(q[b], k, v, tok, self.scale)
            if len(tok) == 0:
                assert np.all(out[b] == 0) and np.all(np.isneginf(lse[b])), b
                continue
            kr, vr = np.repeat(k[tok], G, 1), np.repeat(v[tok], G, 1)
            S = self.scale * np.einsum("hd,thd->th", np.abs(q[b]), np.abs(kr)).max(0)
            K = self.scale * (np.abs(kr).sum(-1) * np.abs(q[b]).max(-1)).max(0)
            s = self.scale * np.einsum("hd,thd->th", q[b], kr)
            p = np.exp(s - want_lse)
            A = np.einsum("th,thd->hd", p, np.abs(vr))
            e_s = (self.D / 32 + 8) * 2.0 ** -22 * S + 2.0 ** -22 * K + 2.0 ** -21 * (1 + np.abs(s).max(0))
            n_sum = -(-len(tok) // 16) + 1 + 320
            tol = (2 * e_s + 2.0 ** -21 + n_sum * 2.0 ** -22)[:, None] * A + 2.0 ** -23 * np.abs(want)
            off = np.abs(out[b] - want)
            assert np.all(off <= tol), (b, n, float((off / tol).max()))
            tol = e_s + n_sum * 2.0 ** -24 + 2.0 ** -22 * (1 + np.abs(want_lse))
            assert np.all(np.abs(lse[b] - want_lse) <= tol), (b, n, lse[b], want_lse)


LENS = [[1], [2, 0, 17], [15, 16, 31, 32, 33, 64, 65, 0, 1], [1000], [5000, 3], [0, 0], [129] * 40 + [0] * 5 + [2049]]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", [F16, BF16, E4M3])
@pytest.mark.parametrize("lens", LENS, ids=lambda x: f"{len(x)}x{max(x)}")
def test_against_64_bits(D, dtype, lens):
    scales = (0.05, 0.04) if dtype == E4M3 else (1.0, 1.0)
    c = Case(len(lens) + D, lens, 6, 2, D, dtype, 16 if len(lens) % 2 else 64, scales=scales)
    c.check(*c.run())


@pytest.mark.parametrize("Hq,Hk", [(1, 1), (2, 1), (8, 1), (9, 1), (16, 2), (17, 1), (64, 1), (33, 3), (5, 5), (48, 8)])
@pytest.mark.parametrize("D,dtype", [(64, E4M3), (128, BF16), (256, F16)])
def test_head_layouts(Hq, Hk, D, dtype):
    c = Case(Hq, [70, 0, 333, 1], Hq, Hk, D, dtype, 32)
    c.check(*c.run())


@pytest.mark.parametrize("window", [1, 15, 16, 17, 100, 4096])
@pytest.mark.parametrize("dtype", [BF16, E4M3])
def test_window(window, dtype):
    """Rows before the window hold NaN and are not met."""
    c = Case(window, [0, 1, 14, 16, 17, 99, 100, 101, 1500], 8, 2, 128, dtype, 32, window=window)
    c.check(*c.run())


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_pages(page):
    c = Case(page, [page - 1, page, page + 1, 3 * page + 7], 4, 1, 128, F16, page, extra_width=3)
    c.check(*c.run())


@pytest.mark.parametrize("dtype", [F16, BF16, E4M3])
def test_pages_outside_the_cache_are_left_out(dtype):
    lens = [200, 64, 31]
    c = Case(5, lens, 4, 2, 64, dtype, 32)
    good = c.table.clone()
    for bad in (-1, c.k.shape[0], 2 ** 31 - 1, -2 ** 31):
        c.table.copy_(good)
        c.table[:, 1] = bad
        out, lse = c.run()
        c.table.copy_(good)
        c.check(out, lse, left_out=(1,))
    c.table.fill_(-1)          # no page at all: empty rows
    out, lse = c.run()
    assert torch.all(out == 0) and torch.all(torch.isneginf(lse))


@pytest.mark.parametrize("dtype", [F16, BF16, E4M3])
@pytest.mark.parametrize("lens", [[3], [37, 0, 1024, 16], [4999], [1] * 300, list(range(1, 130))])
def test_every_row_counts_once(dtype, lens):
    """Zero queries weigh every row alike: sums of small whole values are exact, so a row lost, or met twice, shows."""
    D, Hk, Hq = 128, 2, 4
    c = Case(9, lens, Hq, Hk, D, dtype, 16)
    c.q.zero_()
    vals = torch.randint(-8, 9, c.v.shape, generator=torch.Generator().manual_seed(3)).float().cuda()
    c.v.copy_(vals.to(dtype)) if dtype != E4M3 else c.v.view(torch.uint8).copy_(vals.to(dtype).view(torch.uint8))
    c.k.view(torch.uint8).zero_()
    out, lse = c.run()
    out = out.cpu().numpy().astype(np.float64)
    for b, n in enumerate(lens):
        if n == 0:
            assert np.all(out[b] == 0)
            continue
        v = c.rows(b)[1]
        want = np.repeat(v.sum(0), Hq // Hk, 0) / n
        assert np.all(np.abs(out[b] - want) <= 2.0 ** -22 * np.abs(want))     # 1 / n and a product: two roundings
        # log2 n rounded, its product with ln 2: two steps of 2^-23
        assert np.all(np.abs(lse[b].cpu().numpy() - math.log(n)) <= 2.0 ** -21 * max(1.0, math.log(n)))


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_large_and_small_queries(dtype):
    """Rows of very different size: the parts of q follow each row's own size."""
    c = Case(21, [40, 700], 8, 2, 128, dtype, 16)
    for h, f in enumerate((1e-30, 1e-12, 1e-4, 1.0, 10.0, 0.0, 1e-42, 3.0)):
        c.q[:, h] *= f
    c.check(*c.run())


@pytest.mark.parametrize("D,dtype", [(64, E4M3), (128, BF16), (256, F16)])
@pytest.mark.parametrize("lens,Hq,Hk,window", [
    ([n], 8, 2, 0) for n in (255, 256, 257, 384, 385, 512, 513)] + [
    ([300, 0, 1, 256], 32, 2, 0), ([5000, 30, 700], 6, 3, 250), ([250] * 19, 8, 8, 0), ([250] * 20, 8, 8, 0),
    ([40] * 32, 4, 4, 0), ([256, 257], 20, 1, 0)])
def test_few_row_blocks_of_about_a_tile_for_each_warp(D, dtype, lens, Hq, Hk, window):
    """Around where row blocks stop having a CTA each: 8, 12 or 16 tiles of 32 rows, and as many blocks as SMs."""
    c = Case(sum(lens) + Hq, lens, Hq, Hk, D, dtype, 32, window=window)
    out, lse = c.run()
    c.check(out, lse)
    again, _ = c.run()
    assert torch.equal(out, again)


@pytest.mark.parametrize("k_scale", [2.0 ** -100, 2.0 ** 100])
@pytest.mark.parametrize("dtype", [F16, BF16, E4M3])
def test_cache_scales_far_from_one_and_queries_of_zeros(k_scale, dtype):
    """The scale of the scores may leave fp32's range where they are zeros: masked rows stay out, the others count alike."""
    c = Case(22, [40, 1, 700, 0], 8, 2, 64, dtype, 16)
    c.ks, c.cache = k_scale, zq.KVCache(c.k, c.v, k_scale, 1.0)
    c.q *= min(1.0, 1 / k_scale)
    c.q[:, 1::2] = 0.0
    c.check(*c.run())


@pytest.mark.parametrize("dtype", [F16, E4M3])
def test_keys_of_zeros_under_large_queries(dtype):
    c = Case(24, [33, 5], 4, 2, 128, dtype, 16)
    c.k.copy_(torch.zeros_like(c.k, dtype=torch.float32).to(dtype))
    c.cache = zq.KVCache(c.k, c.v, 2.0 ** 30, 1.0)
    c.q *= 1e30
    c.check(*c.run())


def test_large_scores_pick_one_row():
    """Scores in the thousands: all weight on one row, none overflows."""
    c = Case(23, [90], 4, 2, 128, BF16, 16)
    k, v = c.rows(0)
    for h in range(4):
        c.q[0, h] = torch.from_numpy((300 * k[50, h // 2]).astype(np.float32)).cuda()
    out, lse = c.run()
    want = np.repeat(v[50], 2, 0)
    # the weight is 1 to 2^-21, the other rows weigh nothing
    assert np.all(np.abs(out[0].cpu().numpy() - want) <= 2.0 ** -20 * np.abs(want))


def test_nan_and_infinity_of_a_row_stay_in_its_heads():
    c = Case(25, [60, 60], 4, 2, 128, F16, 16)
    page, row = int(c.table[0, 1]), 3
    want, _ = c.run()
    c.v[page, 0, row, 5] = float("nan")
    out, _ = c.run()
    assert out[0, :2, 5].isnan().all()
    out[0, :2, 5] = want[0, :2, 5]
    assert torch.equal(out, want)
    c.v[page, 0, row, 5] = 1.0
    c.k[page, 1, row, 7] = float("nan")
    out, lse = c.run()
    assert out[0, 2:].isnan().all() and lse[0, 2:].isnan().all() and not out[0, :2].isnan().any()
    assert torch.equal(out[1], want[1])


def test_strided_queries_and_outputs_and_rows_left_alone():
    c = Case(27, [50, 20, 3], 4, 2, 64, BF16, 16)
    want, _ = c.run()
    wide = torch.full((5, 3, 4 * 64 + 64), 9.0, device="cuda")
    wide[:3, 1, 64:] = c.q.view(3, -1)
    q = wide[:3, 1, 64:]
    hold = torch.full((5, 2, 4 * 64), 11.0, device="cuda")
    lse = torch.empty(3, 4, device="cuda")
    got = zq.paged_attn(q, c.cache, c.table, c.t_lens, out=hold[:3, 1], lse=lse)
    torch.cuda.synchronize()
    assert torch.equal(got.reshape(3, 4, 64), want)
    assert torch.all(hold[3:] == 11) and torch.all(hold[:, 0] == 11)


@pytest.mark.parametrize("D,dtype", [(64, F16), (64, E4M3), (128, BF16), (128, E4M3), (256, F16), (256, E4M3)])
@pytest.mark.parametrize("lens", [[7, 0, 16], [3000], [40] * 70], ids=["short", "long", "many"])
def test_codes_are_those_of_the_output(D, dtype, lens):
    Hq = 6
    c = Case(31, lens, Hq, 2, D, dtype, 16, scales=(0.05, 0.04) if dtype == E4M3 else (1.0, 1.0))
    q8 = zq.empty_q8_1(len(lens), Hq * D)
    out, lse = c.run(q8_out=q8, out=torch.empty_like(c.q))
    c.check(out, lse)
    q, d, s = ref.q8_1(out.cpu().numpy().reshape(len(lens), -1))
    assert np.array_equal(q8.qs.cpu().numpy(), q)
    assert np.array_equal(q8.d.cpu().numpy().view(np.uint16), d.view(np.uint16))
    assert np.array_equal(q8.s.cpu().numpy() + np.float16(0), s + np.float16(0))
    only = zq.empty_q8_1(len(lens), Hq * D)
    none, _ = c.run(q8_out=only)
    assert none is None and torch.equal(only.qs, q8.qs) and torch.equal(only.d, q8.d) and torch.equal(only.s, q8.s)


def test_same_result_every_time_and_on_another_stream():
    c = Case(33, [3000, 1, 700, 0, 90], 12, 2, 128, BF16, 16)
    want, want_lse = c.run()
    for _ in range(3):
        out, lse = c.run()
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        a = zq.paged_attn(c.q, c.cache, c.table, c.t_lens)
    b = zq.paged_attn(c.q, c.cache, c.table, c.t_lens)
    d = zq.paged_attn(c.q, c.cache, c.table, c.t_lens, stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert torch.equal(a, want) and torch.equal(b, want) and torch.equal(d, want)


def test_graph_follows_the_lengths():
    """One captured call, replayed as the sequences grow: the split is made on the device."""
    c = Case(35, [2000, 37, 600], 4, 2, 128, F16, 16)
    full = list(c.lens)
    ws = torch.empty(zq.paged_attn_workspace_bytes(4, 2, 128), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(c.q), torch.empty(3, 4, device="cuda")
    zq.paged_attn(c.q, c.cache, c.table, c.t_lens, out=out, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        zq.paged_attn(c.q, c.cache, c.table, c.t_lens, out=out, lse=lse, workspace=ws)
    for lens in ([1, 0, 5], [900, 37, 2], full):
        c.lens = lens
        c.t_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        ws.fill_(255)       # NaN: nothing is taken from an earlier call
        graph.replay()
        torch.cuda.synchronize()
        c.check(out, lse)


def test_two_graphs_with_their_own_workspaces_at_once():
    cs = [Case(37 + i, [1500 + 700 * i], 4, 2, 128, BF16, 16) for i in range(2)]
    want = [c.run()[0] for c in cs]
    streams, graphs, outs = [torch.cuda.Stream() for _ in cs], [], [torch.zeros_like(c.q) for c in cs]
    keep = []
    for c, s, o in zip(cs, streams, outs):
        ws = torch.empty(zq.paged_attn_workspace_bytes(4, 2, 128), dtype=torch.uint8, device="cuda")
        keep.append(ws)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            for _ in range(5):
                zq.paged_attn(c.q, c.cache, c.table, c.t_lens, out=o, workspace=ws)
        graphs.append(graph)
    torch.cuda.synchronize()
    for _ in range(4):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


@pytest.mark.parametrize("D,dtype", [(64, E4M3), (128, BF16)])
def test_thousands_of_short_sequences(D, dtype):
    """More sequences than threads plan them, empty ones among them."""
    g = np.random.default_rng(5)
    c = Case(5, [int(n) for n in g.choice([0, 1, 2, 17, 40], 2500)], 2, 1, D, dtype, 16)
    c.check(*c.run())


def test_parts_of_a_batchs_arrays():
    """Table rows, lengths and lse of a part of a batch: addresses of any multiple of four bytes."""
    c = Case(6, [5, 70, 33, 9], 4, 2, 128, F16, 16, extra_width=1)
    want, want_lse = c.run()
    lse = torch.full((5, 4), 3.0, device="cuda").view(-1)[1:9].view(2, 4)
    out = zq.paged_attn(c.q[1:3], c.cache, c.table[1:3], c.t_lens[1:3], lse=lse)
    torch.cuda.synchronize()
    # the work is shared out anew, so pieces join in other places: the tests' tolerance, not equality
    c.lens, c.q, c.table = c.lens[1:3], c.q[1:3], c.table[1:3]
    c.check(out, lse)


def test_lengths_beyond_the_table_and_below_zero():
    c = Case(41, [64, 64, 0], 4, 2, 64, F16, 16)
    c.t_lens.copy_(torch.tensor([2 ** 31 - 1, 64, -5], dtype=torch.int32))
    c.check(*c.run())


def test_offsets_past_32_bits():
    """Pages whose byte offsets pass 2^32 in the K and in the V pool."""
    Hk, page, D = 8, 256, 256
    per_page = Hk * page * D * 2
    pages = (5 << 30) // per_page
    k = torch.empty(pages, Hk, page, D, dtype=BF16, device="cuda")
    v = torch.empty_like(k)
    g = torch.Generator(device="cuda").manual_seed(1)
    picks = [pages - 1, 0, pages // 2, (2 ** 32) // per_page, (2 ** 31) // per_page]
    for p in picks:
        k[p] = torch.randn(Hk, page, D, generator=g, device="cuda").to(BF16)
        v[p] = torch.randn(Hk, page, D, generator=g, device="cuda").to(BF16)
    q = torch.randn(1, 24, D, generator=g, device="cuda")[:, :16].contiguous()
    lens = torch.tensor([5 * page - 3], dtype=torch.int32).cuda()
    table = torch.tensor([picks], dtype=torch.int32).cuda()
    out = zq.paged_attn(q, zq.KVCache(k, v), table, lens)
    small = zq.paged_attn(q, zq.KVCache(k[picks].clone(), v[picks].clone()),
                          torch.arange(5, dtype=torch.int32).cuda()[None], lens)
    torch.cuda.synchronize()
    assert torch.equal(out, small) and not out.isnan().any()


def test_step_with_norm_and_cache_write():
    """The pieces of a decode step together: ten tokens written one after another by head_norm_rope, each attended
    over the cache as it then is; against 64-bit attention over the values the cache holds."""
    Hq, Hk, D, page, B = 6, 2, 128, 16, 3
    g = torch.Generator(device="cuda").manual_seed(2)
    pages = 4
    k = torch.full((pages, Hk, page, D), float("nan"), dtype=F16, device="cuda")
    v = torch.full_like(k, float("nan"))
    cache, table = zq.KVCache(k, v), torch.tensor([[3], [0], [2]], dtype=torch.int32).cuda()
    freq = 1e4 ** (-2.0 * np.arange(D // 2) / D)
    rope = zq.rope_table(freq)
    gq, gk = (0.5 + torch.rand(D, generator=g, device="cuda") for _ in range(2))
    for t in range(10):
        qkv = torch.randn(B, (Hq + 2 * Hk) * D, generator=g, device="cuda")
        q, kk, vv = qkv.split((Hq * D, Hk * D, Hk * D), 1)
        pos = torch.full((B,), t, dtype=torch.int32, device="cuda")
        slots = (table[:, 0] * page + t).contiguous()
        q = zq.head_norm_rope(q, kk, vv, gq, gk, 1e-6, rope, pos, cache, slots)
        lse = torch.empty(B, Hq, device="cuda")
        out = zq.paged_attn(q, cache, table, pos + 1, lse=lse)
        torch.cuda.synchronize()
        c = Case.__new__(Case)
        c.lens, c.Hq, c.Hk, c.D, c.page, c.window, c.ks, c.vs = [t + 1] * B, Hq, Hk, D, page, 0, 1.0, 1.0
        c.q, c.k, c.v, c.table, c.scale = q.reshape(B, Hq, D), k, v, table, D ** -0.5
        c.check(out, lse)


def test_refusals():
    c = Case(43, [20], 4, 2, 128, F16, 16)
    with pytest.raises(ValueError):
        zq.paged_attn(c.q.half(), c.cache, c.table, c.t_lens)
    with pytest.raises(ValueError):
        zq.paged_attn(c.q, c.cache, c.table.long(), c.t_lens)
    with pytest.raises(ValueError):
        zq.paged_attn(c.q, c.cache, c.table, c.t_lens.cpu())
    with pytest.raises(ValueError):
        zq.paged_attn(c.q[..., :64], c.cache, c.table, c.t_lens)
    with pytest.raises(ValueError):
        zq.paged_attn(c.q, c.cache, c.table, c.t_lens, lse=torch.empty(1, 3, device="cuda"))
    with pytest.raises(ValueError):
        zq.paged_attn(c.q, c.cache, c.table, c.t_lens, q8_out=zq.empty_q8_1(1, 256))
    for kw, status in ((dict(workspace=torch.empty(16, dtype=torch.uint8, device="cuda")), -6), (dict(window=-1), -1),
                       (dict(scale=0.0), -1), (dict(scale=float("nan")), -1), (dict(out=c.q), -1)):
        with pytest.raises(zq.ZQError) as e:
            zq.paged_attn(c.q, c.cache, c.table, c.t_lens, **kw)
        assert e.value.status == status
    with pytest.raises(zq.ZQError):
        zq.paged_attn(c.q[:, :3].contiguous(), c.cache, c.table, c.t_lens)
    torch.cuda.synchronize()
