"""Norm of query and key heads, rotation and cache write (zq_head_norm_rope)
against the 64-bit form.

Tolerances.  Queries: per value, the norm's rounding steps (sum of D squares by
lanes and a tree: at most D/32 + 5 additions, a mean, a sum, a root, a
division, two products: relative error under (D/64 + 12) 2^-24 of x) and the
rotation (two products, an addition, and the angle's and sincospi's errors,
under 2^-22 of the pair's norm): 2^-20 of the pair's larger value at D <= 256
(8 + 4 + ... < 16 half steps of 2^-24), plus one ulp of margin.  Cache values:
half a step of the type on top."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import gemm_zq_rmsnorm_gb300 as zq

import _attn_ref as ref

pytestmark = pytest.mark.gpu

F16, BF16, E4M3 = torch.float16, torch.bfloat16, torch.float8_e4m3fn
EPS = 1e-6
REL = 2.0 ** -20


def inv_freq(rot, theta=1e6):
    return theta ** (-2.0 * np.arange(rot // 2) / rot)


def as64(t):
    return t.float().cpu().numpy().astype(np.float64)


def make(seed, T, Hq, Hk, D, dtype, page, extra=2):
    g = np.random.default_rng(seed)
    qkv = torch.from_numpy(g.standard_normal((T, (Hq + 2 * Hk) * D)).astype(np.float32)).cuda()
    pages = -(-T // page) + extra
    k = torch.full((pages, Hk, page, D), 3.0).to(dtype).cuda()
    v = torch.full((pages, Hk, page, D), -5.0).to(dtype).cuda()
    slots = torch.from_numpy(g.permutation(pages * page)[:T].astype(np.int32)).cuda()
    gq, gk = (torch.from_numpy(g.uniform(0.5, 1.5, D).astype(np.float32)).cuda() for _ in range(2))
    return qkv, k, v, slots, gq, gk, g


def parts(qkv, Hq, Hk, D):
    return qkv.split((Hq * D, Hk * D, Hk * D), 1)


def check_cache(pool, rows, slots, dtype, scale, before, rel):
    """Every slot: the written ones hold `rows` (float64 [T][Hk][D]) / scale, the others what they held."""
    P, Hk, page, D = pool.shape
    got = as64(pool).transpose(0, 2, 1, 3).reshape(P * page, Hk, D)
    want = np.full_like(got, before)
    keep = (slots >= 0) & (slots < P * page)
    want[slots[keep]] = rows[keep] / scale
    if dtype == E4M3:
        want = np.clip(want, -448, 448)
    tiny = float(torch.finfo(dtype).smallest_normal) * ref.half_step(dtype) * 2
    pair = np.abs(want).max(-1, keepdims=True)          # the rotation mixes two values of a head
    tol = np.abs(want) * ref.half_step(dtype) * 1.0001 + pair * rel * 2 + tiny / 2
    tol[np.setdiff1d(np.arange(P * page), slots[keep])] = 0
    # a value a rounding error away from a tie may go to the tie's other side: covered by pair * rel * 2 and
    # the step at the upper binade's edge
    assert np.all(np.abs(got - want) <= tol), float(np.max(np.abs(got - want) - tol))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", [F16, BF16, E4M3])
@pytest.mark.parametrize("T,Hq,Hk,rot_part,axes,interleaved,page", [
    (1, 1, 1, 1.0, 1, False, 16),
    (5, 6, 3, 0.25, 3, False, 16),
    (37, 7, 1, 0.75, 2, True, 32),
    (300, 12, 2, 1.0, 1, True, 256),
    (129, 8, 8, 0.5, 3, False, 64),
])
def test_against_64_bits(D, dtype, T, Hq, Hk, rot_part, axes, interleaved, page):
    rot = int(D * rot_part) // 16 * 16
    qkv, k, v, slots, gq, gk, g = make(D + T, T, Hq, Hk, D, dtype, page)
    freq = inv_freq(rot)
    axis = [min(i * axes // (rot // 2), axes - 1) for i in range(rot // 2)]
    pos = g.integers(-3, 1 << 20, (axes, T)).astype(np.int32)
    ks, vs = (0.03, 0.02) if dtype == E4M3 else (1.0, 1.0)
    cache = zq.KVCache(k, v, ks, vs)
    qr, kr, vr = parts(qkv, Hq, Hk, D)
    out = zq.head_norm_rope(qr, kr, vr, gq, gk, EPS, zq.rope_table(freq, axis), torch.from_numpy(pos).cuda(), cache,
                            slots, interleaved=interleaved)
    torch.cuda.synchronize()
    assert zq.device_status() == 0
    x = qkv.cpu().numpy().reshape(T, Hq + 2 * Hk, D)
    want_q = ref.norm_rope(x[:, :Hq], gq.cpu().numpy(), EPS, freq, axis, pos, interleaved)
    want_k = ref.norm_rope(x[:, Hq:Hq + Hk], gk.cpu().numpy(), EPS, freq, axis, pos, interleaved)
    got = as64(out).reshape(T, Hq, D)
    assert np.all(np.abs(got - want_q) <= REL * 2 * np.abs(want_q).max(-1, keepdims=True))
    s = slots.cpu().numpy()
    check_cache(k, want_k, s, dtype, np.float64(np.float32(ks)), 3.0, REL)
    check_cache(v, x[:, Hq + Hk:].astype(np.float64), s, dtype, np.float64(np.float32(vs)), -5.0, 2.0 ** -23)


@pytest.mark.parametrize("D,dtype", [(64, E4M3), (128, BF16), (256, F16)])
@pytest.mark.parametrize("T,Hq,Hk", [(150, 48, 8), (700, 24, 4), (2000, 11, 3), (4500, 5, 1)])
def test_a_long_call_equals_short_ones(D, dtype, T, Hq, Hk):
    """How rows are dealt to warps depends on the number of tokens; what becomes of a row does not."""
    qkv, k, v, slots, gq, gk, g = make(T, T, Hq, Hk, D, dtype, 64)
    pos = torch.from_numpy(g.integers(0, 1 << 17, T).astype(np.int32)).cuda()
    table = zq.rope_table(inv_freq(D))
    q, kr, vr = parts(qkv, Hq, Hk, D)
    out = zq.head_norm_rope(q, kr, vr, gq, gk, EPS, table, pos, zq.KVCache(k, v), slots)
    k2, v2 = torch.full_like(k, 3.0), torch.full_like(v, -5.0)
    cache, out2 = zq.KVCache(k2, v2), torch.empty_like(out)
    for t in range(0, T, 61):
        at = slice(t, t + 61)
        zq.head_norm_rope(q[at], kr[at], vr[at], gq, gk, EPS, table, pos[at], cache, slots[at], q_out=out2[at])
    assert torch.equal(out, out2)
    assert torch.equal(k.view(torch.uint8), k2.view(torch.uint8))
    assert torch.equal(v.view(torch.uint8), v2.view(torch.uint8))


def test_no_norm_no_rotation_is_a_copy():
    """Without gammas and table queries are copied bit for bit, keys and values only rounded."""
    T, Hq, Hk, D = 19, 3, 2, 128
    qkv, k, v, slots, _, _, _ = make(3, T, Hq, Hk, D, F16, 16)
    qkv[4, 5] = float("inf")
    qkv[7, Hq * D + 9] = float("nan")
    qr, kr, vr = parts(qkv, Hq, Hk, D)
    out = zq.head_norm_rope(qr, kr, vr, None, None, EPS, None, None, zq.KVCache(k, v), slots)
    torch.cuda.synchronize()
    assert torch.equal(out, qr)
    rows = k.permute(0, 2, 1, 3).reshape(-1, Hk * D)[slots.long()]
    assert torch.equal(rows.isnan(), kr.isnan()) and torch.equal(rows.nan_to_num(), kr.half().nan_to_num())
    assert torch.equal(v.permute(0, 2, 1, 3).reshape(-1, Hk * D)[slots.long()], vr.half())


def test_in_place_equals_out_of_place_and_one_token_equals_its_row():
    T, Hq, Hk, D = 40, 5, 2, 128
    qkv, k, v, slots, gq, gk, g = make(5, T, Hq, Hk, D, BF16, 16)
    table, pos = zq.rope_table(inv_freq(D)), torch.arange(T, dtype=torch.int32).cuda()
    cache = zq.KVCache(k, v)
    qr, kr, vr = parts(qkv, Hq, Hk, D)
    out = zq.head_norm_rope(qr, kr, vr, gq, gk, EPS, table, pos, cache, slots)
    k1, v1 = torch.zeros_like(k), torch.zeros_like(v)
    one = zq.head_norm_rope(qr[9:10], kr[9:10], vr[9:10], gq, gk, EPS, table, pos[9:10].clone(), zq.KVCache(k1, v1),
                            slots[9:10].clone())
    copy = qkv.clone()
    q2, kk2, vv2 = parts(copy, Hq, Hk, D)
    same = zq.head_norm_rope(q2, kk2, vv2, gq, gk, EPS, table, pos, cache, slots, q_out=q2)
    torch.cuda.synchronize()
    assert same is q2 and torch.equal(q2, out) and torch.equal(one[0], out[9])
    assert torch.equal(copy[:, Hq * D:], qkv[:, Hq * D:])          # k and v rows untouched
    at = int(slots[9])
    assert torch.equal(k1[at // 16, :, at % 16], k[at // 16, :, at % 16])


def test_slots_outside_the_cache_are_not_written():
    T, Hq, Hk, D = 6, 2, 1, 64
    qkv, k, v, slots, gq, gk, _ = make(7, T, Hq, Hk, D, F16, 16, extra=1)
    n = k.shape[0] * 16
    slots = torch.tensor([-1, 0, n, n - 1, -2 ** 31, 2 ** 31 - 1], dtype=torch.int32).cuda()
    qr, kr, vr = parts(qkv, Hq, Hk, D)
    table, pos = zq.rope_table(inv_freq(D)), torch.arange(T, dtype=torch.int32).cuda()
    out = zq.head_norm_rope(qr, kr, vr, gq, gk, EPS, table, pos, zq.KVCache(k, v), slots)
    torch.cuda.synchronize()
    x = qkv.cpu().numpy().reshape(T, Hq + 2 * Hk, D)
    want = ref.norm_rope(x[:, :Hq], gq.cpu().numpy(), EPS, inv_freq(D), [0] * (D // 2), pos.cpu().numpy()[None], False)
    assert np.all(np.abs(as64(out).reshape(T, Hq, D) - want) <= REL * 2 * np.abs(want).max(-1, keepdims=True))
    check_cache(v, x[:, Hq + Hk:].astype(np.float64), slots.cpu().numpy().astype(np.int64), F16, 1.0, -5.0, 0.0)


def test_far_positions():
    """A rotation by a position and back by the same one is the identity wherever it is; the largest positions agree
    with 64 bits."""
    T, D = 8, 128
    pos = np.array([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 123456789, 2 ** 24 + 1, 10 ** 9], np.int32)
    qkv, k, v, slots, _, _, _ = make(11, T, 1, 1, D, F16, 16)
    qr, kr, vr = parts(qkv, 1, 1, D)
    freq = inv_freq(D)
    out = zq.head_norm_rope(qr, kr, vr, None, None, EPS, zq.rope_table(freq), torch.from_numpy(pos).cuda(),
                            zq.KVCache(k, v), slots)
    back = zq.head_norm_rope(out, kr, vr, None, None, EPS, zq.rope_table(-freq), torch.from_numpy(pos).cuda(),
                             zq.KVCache(k, v), slots)
    torch.cuda.synchronize()
    x = qkv.cpu().numpy().reshape(T, 3, D)
    want = ref.norm_rope(x[:, :1], None, EPS, freq, [0] * 64, pos[None], False)
    # 2^31 positions x a 2^-53 relative error of inv_freq / 2 pi and the table's 2^-63 turns: under 2^-20 radians
    assert np.max(np.abs(as64(out).reshape(T, 1, D) - want)) <= 2.0 ** -18 * np.abs(x).max()
    assert np.max(np.abs(as64(back) - as64(qr))) <= 2.0 ** -18 * np.abs(x).max()


def test_e4m3_saturates():
    T, D = 2, 64
    qkv, k, v, slots, _, _, _ = make(13, T, 1, 1, D, E4M3, 16)
    qkv[0, 2 * D] = 1e9
    qkv[0, 2 * D + 1] = -1e9
    qkv[1, 2 * D] = float("nan")
    qr, kr, vr = parts(qkv, 1, 1, D)
    zq.head_norm_rope(qr, kr, vr, None, None, EPS, None, None, zq.KVCache(k, v), slots)
    torch.cuda.synchronize()
    rows = v.view(torch.uint8).permute(0, 2, 1, 3).reshape(-1, D)[slots.long()].view(E4M3).float()
    assert rows[0, 0] == 448 and rows[0, 1] == -448 and rows[1, 0].isnan()


def test_captured_and_replayed_on_another_stream():
    T, Hq, Hk, D = 3, 4, 2, 128
    qkv, k, v, slots, gq, gk, _ = make(17, T, Hq, Hk, D, F16, 16)
    table, pos = zq.rope_table(inv_freq(D)), torch.arange(T, dtype=torch.int32).cuda()
    cache, out = zq.KVCache(k, v), torch.empty(T, Hq * D, device="cuda")
    qr, kr, vr = parts(qkv, Hq, Hk, D)
    want = zq.head_norm_rope(qr, kr, vr, gq, gk, EPS, table, pos, cache, slots).clone()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        zq.head_norm_rope(qr, kr, vr, gq, gk, EPS, table, pos, cache, slots, q_out=out)
    qkv.mul_(-1)          # the norm is odd: so is the output
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, -want)


@pytest.mark.parametrize("interleaved", [False, True])
def test_angles_at_the_farthest_positions(interleaved):
    """Frequencies up to a hundred radians a position at positions of any size, against the exact angle: 2^-25.9 turns of
    the table and its fp32 argument (2^-23.2 radians), 2^-22 of sine and cosine, three roundings, of a pair's norm."""
    from test_attention_abi_cpu import inverse_two_pi
    T, D = 12, 64
    pos = np.array([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 31 - 12345, 123456789, 2 ** 24 + 1, 10 ** 9, 777, -10 ** 6,
                    2 ** 30 + 1], np.int32)
    freq = np.concatenate([[1.0, 100.0, -1.0, -100.0, 6.3], 100.0 ** -(np.arange(27) / 27)])
    qkv, k, v, slots, _, _, _ = make(19, T, 1, 1, D, F16, 16)
    qr, kr, vr = parts(qkv, 1, 1, D)
    out = zq.head_norm_rope(qr, kr, vr, None, None, EPS, zq.rope_table(freq), torch.from_numpy(pos).cuda(),
                            zq.KVCache(k, v), slots, interleaved=interleaved)
    torch.cuda.synchronize()
    got, x = as64(out), qkv.cpu().numpy().astype(np.float64)[:, :D]
    inverse = inverse_two_pi(256)
    for p, f in enumerate(freq):
        i, j = (2 * p, 2 * p + 1) if interleaved else (p, p + D // 2)
        num, den = float(f).as_integer_ratio()
        turns = [((num * int(t) * inverse // den) % (1 << 256)) / 2.0 ** 256 for t in pos]
        c, s = np.cos(2 * np.pi * np.array(turns)), np.sin(2 * np.pi * np.array(turns))
        norm = np.hypot(x[:, i], x[:, j])
        tol = (2.0 ** -23.2 + 2.0 ** -22 + 3 * 2.0 ** -24) * norm
        assert np.all(np.abs(got[:, i] - (x[:, i] * c - x[:, j] * s)) <= tol), f
        assert np.all(np.abs(got[:, j] - (x[:, j] * c + x[:, i] * s)) <= tol), f
