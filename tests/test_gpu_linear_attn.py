"""Linear attention with a decay for each head (zq_linear_attn_step,
zq_linear_attn) against the 64-bit recurrence.

Tolerances, as shares of what bounds a value by the norms of the rows that went
in (_mixer_ref.recurrence).  A step: expf (2 ulp), two roundings of a state's
value, a sum of at most 16 + 1 + 8 fp32 steps and the scale: under 36 * 2^-24 <
2^-18.  A prompt: a score is a sum of 3 * 128 products of binary16 parts in 24
additions (2^-23 each, the tensor core cuts off) with both factors taken to
2^-24 of their row's largest value (2 * sqrt(128) * 2^-24 of the norms) and the
product of the two low parts left out (2^-22): under 40 * 2^-23; the weights times
the values, and the queries times the state, alike; together under 120 * 2^-23 <
2^-16.  A chunk's update of the state adds at most 40 * 2^-23 and the decay's
rounding, for every 64 tokens at worst: T / 64 * 2^-17.
Root mean squares are near 2^-22 by the same steps with random signs; more than
2^-20 (2^-19 over thousands of tokens) would be a part that went missing."""
import math
import threading

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import gemm_zq_rmsnorm_gb300 as zq

import _mixer_ref as ref

pytestmark = pytest.mark.gpu

SHAPES = [(64, 64), (64, 128), (64, 256), (128, 64), (128, 128), (128, 256)]


def make(seed, T, Hk, Hv, Dk, Dv, n, rate=0.2):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    # the parts of a stacked row, behind 4 values that belong to something else
    rows = torch.cat((torch.full((T, 4), float("nan"), device="cuda"), randn(T, Hk * Dk), randn(T, Hk * Dk) / Dk ** 0.5,
                      randn(T, Hv * Dv)), 1)
    _, q, k, v = rows.split((4, Hk * Dk, Hk * Dk, Hv * Dv), 1)
    decay = -rate * torch.rand(Hv, generator=g, device="cuda") * randn(T, Hv).abs()
    return q, k, v, decay, randn(n, Hv, Dk, Dv) * 0.5


def heads(x, D):
    return x.reshape(x.shape[0], x.shape[1] // D, D)


def check(got, want, bound, tol, rms, what):
    got = got.double()
    off = (got - want).abs()
    assert torch.isfinite(got).all(), what
    assert (off <= tol * bound + 1e-300).all(), (what, float((off / (bound + 1e-300)).max()))
    if want.numel() and want.norm() > 0:
        assert float((got - want).norm() / want.norm()) <= rms, (what, float((got - want).norm() / want.norm()))


@pytest.mark.parametrize("Dk,Dv", SHAPES)
@pytest.mark.parametrize("B,Hk,Hv", [(1, 1, 1), (3, 2, 6), (17, 4, 4), (70, 1, 5)])
def test_step_against_64_bits(Dk, Dv, B, Hk, Hv):
    q, k, v, g, pool = make(B + Dk + Dv, B, Hk, Hv, Dk, Dv, B + 4)
    slots = torch.randperm(B + 4, generator=torch.Generator().manual_seed(B))[:B].to(torch.int32)
    if B > 2:
        slots[1], slots[2] = -1, B + 4          # padded rows: no state
    before = pool.clone()
    out = zq.linear_attn_step(q, k, v, g, zq.LinearState(pool), slots.cuda())
    torch.cuda.synchronize()
    untouched = torch.ones(B + 4, dtype=torch.bool)
    for b, slot in enumerate(slots.tolist()):
        kept = 0 <= slot < B + 4
        S0 = before[slot] if kept else torch.zeros_like(before[0])
        o, S, bo, bs = ref.recurrence(*(heads(x[b:b + 1], D) for x, D in ((q, Dk), (k, Dk), (v, Dv))), g[b:b + 1], S0,
                                      Dk ** -0.5)
        check(heads(out[b:b + 1], Dv), o, bo[..., None], 2.0 ** -18, 2.0 ** -21, "out")
        if kept:
            untouched[slot] = False
            check(pool[slot], S, bs[:, None, None], 2.0 ** -21, 2.0 ** -22, "state")
    assert torch.equal(pool[untouched.cuda()], before[untouched.cuda()])


def test_step_decays():
    """No decays, none at all, a decay of zero, of everything, and growth."""
    B, H, D = 6, 3, 64
    q, k, v, g, pool = make(1, B, H, H, D, D, B)
    slots = torch.arange(B, dtype=torch.int32).cuda()
    before = pool.clone()
    out = zq.linear_attn_step(q, k, v, None, zq.LinearState(pool), slots, scale=0.5)
    pool2 = before.clone()
    out2 = zq.linear_attn_step(q, k, v, torch.zeros_like(g), zq.LinearState(pool2), slots, scale=0.5)
    assert torch.equal(out, out2) and torch.equal(pool, pool2)
    g[0], g[1], g[2], g[3] = -math.inf, -1000.0, 2.0, -1e-9
    pool3 = before.clone()
    out3 = zq.linear_attn_step(q, k, v, g, zq.LinearState(pool3), slots, scale=-2.0)
    for b in range(B):
        o, S, bo, bs = ref.recurrence(heads(q[b:b + 1], D), heads(k[b:b + 1], D), heads(v[b:b + 1], D), g[b:b + 1],
                                      before[b], -2.0)
        check(heads(out3[b:b + 1], D), o, bo[..., None], 2.0 ** -18, 2.0 ** -20, b)
        check(pool3[b], S, bs[:, None, None], 2.0 ** -21, 2.0 ** -22, b)


def prompts(lens, Hk, Hv, Dk, Dv, seed=0, pad=3, rate=0.2, fresh=None, first=2, scale=None, alter=None):
    """A call over the lengths, checked against the recurrence of every sequence; returns its inputs and outputs."""
    B, T = len(lens), first + sum(lens) + pad
    q, k, v, g, pool = make(seed + T, T, Hk, Hv, Dk, Dv, B + 2, rate)
    if alter:
        alter(q, k, v, g, pool)
    starts = np.concatenate([[0], np.cumsum(lens)]) + first
    slots = np.random.default_rng(seed).permutation(B + 2)[:B]
    fresh = [(b + seed) % 3 == 1 for b in range(B)] if fresh is None else fresh
    before = pool.clone()
    for b in range(B):
        if fresh[b]:
            pool[slots[b]] = float("nan")       # not read
    for x in (q, k, v):                         # rows of no sequence: not read
        x[:first] = float("nan")
        x[T - pad:] = float("nan")
    out = torch.full((T, Hv * Dv), 7.0, device="cuda")
    ints = [torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda") for x in (starts, slots, fresh)]
    zq.linear_attn(q, k, v, g, ints[0], zq.LinearState(pool), ints[1], fresh=ints[2], scale=scale, out=out)
    torch.cuda.synchronize()
    assert zq.device_status() == 0
    assert bool((out[:first] == 7.0).all()) and bool((out[T - pad:] == 7.0).all())
    others = np.setdiff1d(np.arange(B + 2), slots)
    assert torch.equal(pool[others], before[others])
    s = Dk ** -0.5 if scale is None else scale
    rms = 2.0 ** -20 if max(lens) <= 1000 else 2.0 ** -19
    for b, n in enumerate(lens):
        at = slice(int(starts[b]), int(starts[b]) + n)
        S0 = torch.zeros_like(before[0]) if fresh[b] else before[slots[b]]
        o, S, bo, bs = ref.recurrence(heads(q[at], Dk), heads(k[at], Dk), heads(v[at], Dv), g[at], S0, s)
        check(heads(out[at], Dv), o, bo[..., None], 2.0 ** -16 + n / 64 * 2.0 ** -17, rms, (b, n, "out"))
        check(pool[slots[b]], S, bs[:, None, None], (1 + n / 64) * 2.0 ** -17, rms, (b, n, "state"))
        if n == 0 and not fresh[b]:
            assert torch.equal(pool[slots[b]], before[slots[b]])
    return q, k, v, g, before, pool, out, ints


@pytest.mark.parametrize("Dk,Dv", SHAPES)
@pytest.mark.parametrize("lens", [[1], [63], [64], [65], [3, 0, 64, 129, 1, 37]])
@pytest.mark.parametrize("Hk,Hv", [(1, 1), (2, 6)])
def test_prompts_against_64_bits(Dk, Dv, lens, Hk, Hv):
    prompts(lens, Hk, Hv, Dk, Dv, seed=len(lens) + Hv)


@pytest.mark.parametrize("Dk,Dv,Hk,Hv,lens", [
    (128, 128, 1, 1, [3001]), (64, 64, 2, 2, [2048]), (128, 64, 1, 2, [700, 1, 900]), (64, 256, 1, 3, [1500]),
    (128, 256, 1, 1, [640, 1111]), (128, 128, 4, 24, [777, 130])])
@pytest.mark.parametrize("rate", [0.003, 1.0])
def test_long_prompts(Dk, Dv, Hk, Hv, lens, rate):
    prompts(lens, Hk, Hv, Dk, Dv, rate=rate, seed=3)


def test_many_short_prompts():
    lens = [int(x) for x in np.random.default_rng(5).integers(0, 90, 300)]
    prompts(lens, 1, 2, 64, 64, seed=9)


def test_far_apart_sizes():
    """Tokens whose keys, values and queries differ by 2^60, zeros among them, and decays from none to everything:
    a small token's weight is right wherever no larger one drowns it."""
    def alter(q, k, v, g, pool):
        T = q.shape[0]
        e = torch.arange(T, device="cuda")
        k *= torch.exp2(((e * 7) % 41 - 20).float())[:, None]
        v *= torch.exp2(((e * 11) % 81 - 40).float())[:, None]
        q *= torch.exp2(((e * 5) % 61 - 30).float())[:, None]
        k[5], v[9], q[11] = 0.0, 0.0, 0.0
        g[::17] = -40.0
        g[::29] = -math.inf
        g[3::31] = -1e30
        g[1::5] = 0.0
    prompts([150, 64, 20], 1, 2, 128, 64, alter=alter, seed=2)
    prompts([333], 2, 2, 64, 128, alter=alter, seed=2)


def test_rows_after_a_huge_token_of_the_future():
    """A token 2^80 larger than the others changes nothing before it, bit for bit."""
    Dk, Dv, T = 128, 128, 100
    q, k, v, g, pool = make(4, T, 1, 1, Dk, Dv, 1)
    ints = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, T], [0], [1])]

    def go():
        return zq.linear_attn(q, k, v, g, ints[0], zq.LinearState(pool), ints[1], fresh=ints[2])
    want = go()
    for row, at in ((k, 77), (v, 77)):
        row[at] *= 2.0 ** 40
    got = go()
    assert torch.equal(got[:77], want[:77]) and bool(torch.isfinite(got).all())
    # a row whose query happens to be nearly orthogonal to that token's key is off by a share of |q| |k|, not of q . k
    o, _, bo, _ = ref.recurrence(heads(q, Dk), heads(k, Dk), heads(v, Dv), g, torch.zeros(1, Dk, Dv, device="cuda"),
                                 Dk ** -0.5)
    check(heads(got, Dv), o, bo[..., None], 2.0 ** -16 + T / 64 * 2.0 ** -17, math.inf, "out")


@pytest.mark.parametrize("where", ["q", "k", "v", "g"])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_what_is_not_finite_stays_behind_its_token(where, bad):
    Dk, Dv, lens, Hv = 64, 128, [70, 30, 20], 2
    T = sum(lens)
    q, k, v, g, pool = make(6, T, 2, Hv, Dk, Dv, 3)
    starts = torch.tensor([0, 70, 100, 120], dtype=torch.int32, device="cuda")
    slots = torch.tensor([2, 0, 1], dtype=torch.int32, device="cuda")
    clean_pool = pool.clone()
    want = zq.linear_attn(q, k, v, g, starts, zq.LinearState(clean_pool), slots)
    {"q": q, "k": k, "v": v, "g": g}[where][85, 1] = bad      # sequence 1, its token 15, head 0 (g: head 1)
    got = zq.linear_attn(q, k, v, g, starts, zq.LinearState(pool), slots)
    h = 1 if where == "g" else 0
    o, w = heads(got, Dv), heads(want, Dv)
    seen = torch.ones(T, Hv, dtype=torch.bool, device="cuda")
    seen[85 if where == "q" else slice(85, 100), h] = False
    assert torch.equal(o[seen], w[seen])
    assert not bool(torch.isfinite(o[85, h]).all())
    assert torch.equal(pool[2], clean_pool[2]) and torch.equal(pool[1], clean_pool[1])
    assert torch.equal(pool[0, 1 - h], clean_pool[0, 1 - h])
    if where != "q":
        assert not bool(torch.isfinite(o[99, h]).all()) and not bool(torch.isfinite(pool[0, h]).all())
    else:
        assert torch.equal(pool, clean_pool)


def test_a_prompt_in_parts_and_in_steps():
    """A prompt in one call, in three that go on from the state, and token by token."""
    Dk, Dv, Hk, Hv, T = 128, 64, 2, 4, 150
    q, k, v, g, pool = make(8, T, Hk, Hv, Dk, Dv, 1)
    slot = torch.zeros(1, dtype=torch.int32, device="cuda")

    def part(t0, t1, p):
        starts = torch.tensor([0, t1 - t0], dtype=torch.int32, device="cuda")
        return zq.linear_attn(q[t0:t1], k[t0:t1], v[t0:t1], g[t0:t1], starts, zq.LinearState(p), slot)
    p1, p2, p3 = pool.clone(), pool.clone(), pool.clone()
    whole = part(0, T, p1)
    parts = torch.cat([part(0, 41, p2), part(41, 105, p2), part(105, T, p2)])
    state = zq.LinearState(p3)
    steps = torch.cat([zq.linear_attn_step(q[t:t + 1], k[t:t + 1], v[t:t + 1], g[t:t + 1], state, slot)
                       for t in range(T)])
    o, S, bo, bs = ref.recurrence(heads(q, Dk), heads(k, Dk), heads(v, Dv), g, pool[0], Dk ** -0.5)
    for got, p, what in ((whole, p1, "whole"), (parts, p2, "parts"), (steps, p3, "steps")):
        check(heads(got, Dv), o, bo[..., None], 2.0 ** -15, 2.0 ** -20, what)
        check(p[0], S, bs[:, None, None], 2.0 ** -15, 2.0 ** -20, what)


def test_starts_outside_the_rows_are_cut_off():
    Dk = Dv = 64
    T = 40
    q, k, v, g, pool = make(12, T, 1, 1, Dk, Dv, 4)
    before = pool.clone()
    starts = torch.tensor([-5, 10, 35, 60, 20], dtype=torch.int32, device="cuda")   # rows 0..9, 10..34, 35..39, none
    slots = torch.tensor([0, 1, 2, 3], dtype=torch.int32, device="cuda")
    got = zq.linear_attn(q, k, v, g, starts, zq.LinearState(pool), slots)
    p2 = before.clone()
    want = zq.linear_attn(q, k, v, g, torch.tensor([0, 10, 35, 40, 40], dtype=torch.int32, device="cuda"),
                          zq.LinearState(p2), slots)
    assert torch.equal(got, want) and torch.equal(pool, p2) and torch.equal(pool[3], before[3])


@pytest.mark.parametrize("Hv", [1, 48])
def test_decreasing_starts_stay_inside(Hv):
    """Sequences that overlap are nobody's prompt; the call stays within its rows, states and workspace."""
    Dk, Dv, T, B = 64, 64, 1500, 9
    q, k, v, g, pool = make(14, T, 1, Hv, Dk, Dv, B + 1)
    kept = pool[B].clone()
    starts = torch.tensor([0, T, 0, T, 0, T, 0, T, 0, T], dtype=torch.int32, device="cuda")
    need = zq.linear_attn_workspace_bytes(T, B, Hv, Dk, Dv)
    room = torch.full((need + 4096,), 77, dtype=torch.uint8, device="cuda")
    out = torch.full((T + 1, Hv * Dv), 5.0, device="cuda")
    zq.linear_attn(q, k, v, g, starts, zq.LinearState(pool), torch.arange(B, dtype=torch.int32, device="cuda"), out=out[:T],
                   workspace=room[:need])
    torch.cuda.synchronize()
    assert need and bool((room[need:] == 77).all()) and bool((out[T] == 5.0).all()) and torch.equal(pool[B], kept)
    assert zq.device_status() == 0


@pytest.mark.parametrize("Dk,Dv", [(64, 64), (128, 256)])
def test_no_decay_and_one_row(Dk, Dv):
    """g left out is a decay of one; rows of one token may have any stride."""
    q, k, v, g, pool = make(15, 200, 2, 4, Dk, Dv, 2)
    slot = torch.tensor([1], dtype=torch.int32, device="cuda")
    for T in (1, 70, 200):
        starts = torch.tensor([0, T], dtype=torch.int32, device="cuda")
        before, p2 = pool.clone(), pool.clone()
        got = zq.linear_attn(q[:T], k[:T], v[:T], None, starts, zq.LinearState(pool), slot)
        same = zq.linear_attn(q[:T], k[:T], v[:T], torch.zeros_like(g[:T]), starts, zq.LinearState(p2), slot)
        assert torch.equal(got, same) and torch.equal(pool, p2) and torch.equal(pool[0], before[0])
        o, S, bo, bs = ref.recurrence(heads(q[:T], Dk), heads(k[:T], Dk), heads(v[:T], Dv), None, before[1], Dk ** -0.5)
        check(heads(got, Dv), o, bo[..., None], 2.0 ** -16 + T / 64 * 2.0 ** -17, 2.0 ** -20, T)
        check(pool[1], S, bs[:, None, None], (1 + T / 64) * 2.0 ** -17, 2.0 ** -20, T)
        step = zq.linear_attn_step(q[:1], k[:1], v[:1], None, zq.LinearState(before.clone()), slot)
        o, _, bo, _ = ref.recurrence(heads(q[:1], Dk), heads(k[:1], Dk), heads(v[:1], Dv), None, before[1], Dk ** -0.5)
        check(heads(step, Dv), o, bo[..., None], 2.0 ** -18, 2.0 ** -21, "step")


@pytest.mark.parametrize("Hk,Hv,Dv", [(16, 48, 128), (2, 38, 64), (20, 40, 256)])
def test_prompts_cut_into_few_segments(Hk, Hv, Dv):
    """Two to four segments of a sequence, going on from their state or fresh, beside sequences that are not cut."""
    prompts([2900, 40, 0, 700], Hk, Hv, 64, Dv, seed=Hv, fresh=[False, True, False, False])
    prompts([600, 1800], Hk, Hv, 128, Dv, seed=Hv + 1, fresh=[True, False])


def test_few_segments_captured_and_replayed():
    """One captured call whose sequences are cut into few segments serves other starts, slots and states."""
    Dk, Dv, Hk, Hv, T, B = 64, 64, 2, 40, 700, 3
    q, k, v, g, pool = make(40, T, Hk, Hv, Dk, Dv, B)
    ints = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 500, 600, 700], [0, 1, 2], [0, 1, 0])]
    ws = torch.empty(zq.linear_attn_workspace_bytes(T, B, Hv, Dk, Dv), dtype=torch.uint8, device="cuda")
    state, out = zq.LinearState(pool), torch.empty(T, Hv * Dv, device="cuda")

    def call():
        zq.linear_attn(q, k, v, g, ints[0], state, ints[1], fresh=ints[2], out=out, workspace=ws)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for starts, slots, fresh in (([0, 0, 700, 700], [1, 2, 0], [0, 0, 1]), ([0, 20, 300, 690], [2, 0, 1], [1, 0, 0])):
        for t, x in zip(ints, (starts, slots, fresh)):
            t.copy_(torch.tensor(x, dtype=torch.int32))
        v.neg_()
        before = pool.clone()
        ws.fill_(255)                      # NaN wherever something would be read that was not written
        graph.replay()
        graph.replay()                     # goes on from the first one's states
        torch.cuda.synchronize()
        got, left = out.clone(), pool.clone()
        pool.copy_(before)
        call()
        call()
        torch.cuda.synchronize()
        used = slice(starts[0], starts[-1])
        assert torch.equal(got[used], out[used]) and torch.equal(left, pool)
        assert torch.isfinite(got[used]).all() and torch.isfinite(left).all()


def test_two_threads_with_streams_of_their_own():
    """The first calls of new threads, at the same time, each on its stream and with its own workspace."""
    cases = [make(16 + i, 700, 1, 3, 128, 128, 2) for i in range(2)]
    ints = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 650, 700], [1, 0])]

    def run(i, pool, stream):
        q, k, v, g, _ = cases[i]
        outs = []
        for _ in range(4):
            outs.append(zq.linear_attn(q, k, v, g, ints[0], zq.LinearState(pool), ints[1], stream=stream))
            outs.append(zq.linear_attn_step(q[:2], k[:2], v[:2], g[:2], zq.LinearState(pool), ints[1], stream=stream))
        return outs
    wants = []
    for i in range(2):
        pool = cases[i][4].clone()
        wants.append((run(i, pool, None), pool))
    torch.cuda.synchronize()
    got = [None, None]

    def thread(i):
        stream, pool = torch.cuda.Stream(), cases[i][4].clone()
        torch.cuda.synchronize()
        got[i] = run(i, pool, stream), pool
        stream.synchronize()
    threads = [threading.Thread(target=thread, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for (a, pa), (b, pb) in zip(got, wants):
        assert torch.equal(pa, pb) and all(torch.equal(x, y) for x, y in zip(a, b))


def test_sequences_without_a_state():
    Dk, Dv = 64, 64
    q, k, v, g, pool = make(13, 50, 1, 2, Dk, Dv, 2)
    before = pool.clone()
    starts = torch.tensor([0, 20, 50], dtype=torch.int32, device="cuda")
    got = zq.linear_attn(q, k, v, g, starts, zq.LinearState(pool), torch.tensor([-1, 2], dtype=torch.int32, device="cuda"))
    assert torch.equal(pool, before)
    want = zq.linear_attn(q, k, v, g, starts, zq.LinearState(pool), torch.tensor([0, 1], dtype=torch.int32, device="cuda"),
                          fresh=torch.ones(2, dtype=torch.int32, device="cuda"))
    assert torch.equal(got, want) and not torch.equal(pool, before)


def test_captured_and_replayed_with_other_lengths():
    """One captured pair of calls (a prompt and a step) serves other starts, slots and inputs; two graphs with
    workspaces of their own run on two streams at once."""
    Dk, Dv, Hk, Hv, T, B = 128, 128, 1, 2, 600, 3

    def captured(i):
        q, k, v, g, pool = make(20 + i, T, Hk, Hv, Dk, Dv, B)
        ints = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 100, 150, 600], [0, 1, 2], [1, 1, 1])]
        ws = torch.empty(max(1, zq.linear_attn_workspace_bytes(T, B, Hv, Dk, Dv)), dtype=torch.uint8, device="cuda")
        state, out, out2 = zq.LinearState(pool), torch.empty(T, Hv * Dv, device="cuda"), torch.empty(B, Hv * Dv, device="cuda")

        def calls(stream=None):
            zq.linear_attn(q, k, v, g, ints[0], state, ints[1], fresh=ints[2], out=out, workspace=ws, stream=stream)
            zq.linear_attn_step(q[:B], k[:B], v[:B], g[:B], state, ints[1], out=out2, stream=stream)
        calls()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            calls()
        return graph, q, k, v, g, pool, ints, out, out2, calls
    graphs = [captured(0), captured(1)]
    for starts, slots, fresh in (([0, 600, 600, 600], [1, 0, 2], [0, 0, 1]), ([0, 1, 320, 590], [2, 1, 0], [1, 0, 1])):
        for _, q, _, _, _, pool, ints, out, _, _ in graphs:
            q.neg_()
            for t, x in zip(ints, (starts, slots, fresh)):
                t.copy_(torch.tensor(x, dtype=torch.int32))
            out.fill_(3.0)
        befores = [x[5].clone() for x in graphs]
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in graphs]
        for s, x in zip(streams, graphs):
            with torch.cuda.stream(s):
                x[0].replay()
        torch.cuda.synchronize()
        for before, (_, q, _, _, _, pool, _, out, out2, calls) in zip(befores, graphs):
            got, got2, left = out.clone(), out2.clone(), pool.clone()
            pool.copy_(before)
            out.fill_(3.0)
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            calls(stream=s)
            torch.cuda.synchronize()
            assert torch.equal(out, got) and torch.equal(out2, got2) and torch.equal(pool, left)
            assert bool((out[starts[-1]:] == 3.0).all())


def test_the_result_does_not_change():
    q, k, v, g, pool = make(30, 2000, 1, 3, 128, 128, 2)
    ints = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 1990, 2000], [1, 0])]
    runs = []
    for _ in range(3):
        p = pool.clone()
        runs.append((zq.linear_attn(q, k, v, g, ints[0], zq.LinearState(p), ints[1]), p))
    assert all(torch.equal(a, b) for r in runs[1:] for a, b in zip(r, runs[0]))


def test_binding_refuses():
    q, k, v, g, pool = make(31, 4, 2, 4, 64, 64, 4)
    state, ints = zq.LinearState(pool), torch.arange(4, dtype=torch.int32).cuda()
    for bad in (dict(q=q[:3]), dict(q=q.half()), dict(k=k[:, :64]), dict(v=v[:, :128]), dict(g=g[:, :3]), dict(g=g.double()),
                dict(slots=ints.long()), dict(slots=ints[:3]), dict(q=q.cpu()), dict(out=v[:, :64])):
        a = dict(q=q, k=k, v=v, g=g, slots=ints)
        a.update(bad)
        with pytest.raises(ValueError):
            zq.linear_attn_step(a["q"], a["k"], a["v"], a["g"], state, a["slots"], out=a.get("out"))
    starts = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    for bad in (dict(starts=starts.long()), dict(starts=ints), dict(fresh=ints), dict(workspace=torch.empty(4, 4).cuda().t())):
        a = dict(starts=starts, fresh=None, workspace=None)
        a.update(bad)
        with pytest.raises(ValueError):
            zq.linear_attn(q, k, v, g, a["starts"], state, ints[:1], fresh=a["fresh"], workspace=a["workspace"])
    with pytest.raises(ValueError):
        zq.LinearState(pool.half())
