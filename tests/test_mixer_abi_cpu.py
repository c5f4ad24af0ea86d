"""CPU-only checks of the recurrent mixer's and the block edges' calls: refusals
on the host with the documented status, before anything is launched."""
import ctypes
import math

import pytest

import gemm_zq_rmsnorm_gb300 as zq

A16, A8, A2 = 0x10000, 0x10008, 0x10002


@pytest.fixture(scope="module")
def lib():
    return zq.load()


def state(s=A16, n=4, Hv=4, Dk=128, Dv=128):
    return ctypes.byref(zq._LinearState(s, n, Hv, Dk, Dv))


def step(lib, q=A16, qs=256, k=A16, ks=256, v=A16, vs=512, B=3, Hk=2, g=A16, gs=4, st=None, slots=A16, scale=0.1,
         out=A16, os=512):
    return lib.zq_linear_attn_step(q, qs, k, ks, v, vs, B, Hk, g, gs, state() if st is None else st, slots, scale, out,
                                   os, None)


def prompt(lib, q=A16, qs=256, k=A16, ks=256, v=A16, vs=512, T=30, B=3, Hk=2, g=A16, gs=4, starts=A16, st=None,
           slots=A16, fresh=None, scale=0.1, out=A16, os=512, ws=A16, wb=1 << 40):
    return lib.zq_linear_attn(q, qs, k, ks, v, vs, T, B, Hk, g, gs, starts, state() if st is None else st, slots, fresh,
                              scale, out, os, ws, wb, None)


BOTH = [(dict(q=None), -1), (dict(q=A8), -3), (dict(qs=252), -2), (dict(qs=258), -2), (dict(k=None), -1),
        (dict(ks=0), -2), (dict(v=A8), -3), (dict(vs=508), -2), (dict(out=None), -1), (dict(out=A8), -3),
        (dict(os=-512), -2), (dict(g=A2), -3), (dict(gs=3), -2), (dict(gs=-4), -2), (dict(vs=1 << 29), -2), (dict(gs=1 << 29), -2), (dict(slots=None), -1),
        (dict(slots=A2), -3), (dict(scale=math.nan), -1), (dict(scale=math.inf), -1), (dict(Hk=0), -2),
        (dict(Hk=3), -2), (dict(Hk=8, qs=1024, ks=1024), -2), (dict(B=0), -2), (dict(B=65536), -2)]
STATES = [(dict(s=None), -1), (dict(s=A8), -3), (dict(n=0), -2), (dict(Hv=0), -2), (dict(Hv=1026), -2),
          (dict(Dk=96), -2), (dict(Dk=256), -2), (dict(Dv=32), -2), (dict(Dv=512), -2)]


@pytest.mark.parametrize("bad,status", BOTH)
def test_both_refuse(lib, bad, status):
    assert step(lib, **bad) == status
    assert lib.zq_last_error()
    assert prompt(lib, **bad) == status
    assert lib.zq_last_error()


@pytest.mark.parametrize("bad,status", STATES)
def test_both_refuse_states(lib, bad, status):
    assert step(lib, st=state(**bad), vs=1 << 20, os=1 << 20, gs=1 << 20) == status
    assert prompt(lib, st=state(**bad), vs=1 << 20, os=1 << 20, gs=1 << 20) == status


@pytest.mark.parametrize("bad,status", [(dict(T=0), -2), (dict(T=(1 << 24) + 1), -2), (dict(starts=None), -1),
                                        (dict(starts=A2), -3), (dict(fresh=A2), -3), (dict(ws=A8), -3)])
def test_prompt_refuses(lib, bad, status):
    assert prompt(lib, **bad) == status
    assert lib.zq_last_error()


def test_null_state_is_refused(lib):
    assert lib.zq_linear_attn_step(A16, 256, A16, 256, A16, 512, 3, 2, None, 0, None, A16, 0.1, A16, 512, None) == -1


def test_workspace_sizes(lib):
    assert lib.zq_linear_attn_workspace_bytes(0, 1, 4, 128, 128) == 0
    assert lib.zq_linear_attn_workspace_bytes(10, 1, 4, 96, 128) == 0
    assert lib.zq_linear_attn_workspace_bytes(1 << 24, 65535, 1024, 128, 256) < 1 << 34


def gated(lib, x=A16, xs=512, B=3, H=4, D=128, gamma=A16, eps=1e-6, gate=A16, gs=512, act=2, out=A16 + 65536, os=512,
          q8=None):
    return lib.zq_gated_norm_q8_1(x, xs, B, H, D, gamma, eps, gate, gs, act, out, os, q8, None)


def planes(qs=A16, d=A16, s=A16):
    return ctypes.byref(zq._Q8(qs, d, s))


@pytest.mark.parametrize("bad,status", [
    (dict(x=None), -1), (dict(x=A8), -3), (dict(xs=508), -2), (dict(xs=514), -2), (dict(B=0), -2), (dict(H=0), -2),
    (dict(H=65537), -2), (dict(B=1 << 30, H=4), -2), (dict(D=32), -2), (dict(D=512), -2), (dict(gamma=A8), -3),
    (dict(eps=-1.0), -1), (dict(eps=math.nan), -1), (dict(gate=A8), -3), (dict(gs=0), -2), (dict(act=3), -1),
    (dict(act=-1), -1), (dict(out=None), -1), (dict(out=A8), -3), (dict(os=4), -2), (dict(out=A16, os=516), -1),
    (dict(q8=planes(qs=None)), -1), (dict(q8=planes(d=A8)), -3)])
def test_gated_norm_refuses(lib, bad, status):
    assert gated(lib, **bad) == status
    assert lib.zq_last_error()


def edge(lib, x=A16, xs=512, y=A16 + 65536, ys=512, B=3, K=512, gp=A16, gate=A16, gs=512, act=1, scale=1.0,
         xo=A16 + 131072, xos=512, gamma=A16, eps=1e-6, out=None, os=0, q8=None):
    return lib.zq_residual_norm_q8_1(x, xs, y, ys, B, K, gp, gate, gs, act, scale, xo, xos, gamma, eps, out, os, q8, None)


@pytest.mark.parametrize("bad,status", [
    (dict(x=None), -1), (dict(x=A8), -3), (dict(xs=508), -2), (dict(y=None), -1), (dict(y=A8), -3), (dict(ys=0), -2),
    (dict(B=0), -2), (dict(B=(1 << 24) + 1), -2), (dict(K=0), -2), (dict(K=48), -2), (dict(K=32800, xs=32800), -2),
    (dict(gp=A8), -3), (dict(gate=A8), -3), (dict(gate=A8, gs=0), -3), (dict(gs=256), -2), (dict(act=9), -1),
    (dict(scale=math.nan), -1), (dict(scale=-math.inf), -1), (dict(xo=None), -1), (dict(xo=A8), -3),
    (dict(xos=510), -2), (dict(xo=A16, xos=516), -1), (dict(xo=A16 + 65536, xos=516), -1), (dict(gamma=A8), -3),
    (dict(eps=-1e-6), -1), (dict(out=A8, os=512), -3), (dict(out=A16, os=0), -2), (dict(q8=planes(s=None)), -1),
    (dict(q8=planes(qs=A8)), -3)])
def test_residual_norm_refuses(lib, bad, status):
    assert edge(lib, **bad) == status
    assert lib.zq_last_error()


def test_valid_calls_without_gpu(lib):
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert step(lib) == step(lib, g=None, gs=0) == -5
    assert prompt(lib) == prompt(lib, fresh=A16) == -5
    assert gated(lib) == gated(lib, gamma=None, gate=None) == gated(lib, out=None, q8=planes()) == gated(lib, out=A16) == -5
    assert edge(lib) == edge(lib, gs=0) == edge(lib, gate=None, gp=None, gamma=None) == edge(lib, xo=A16) == -5
    assert edge(lib, xo=A16 + 65536) == edge(lib, out=A16, os=512, q8=planes()) == -5


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros(2, 128)
    with pytest.raises(ValueError):
        zq.LinearState(torch.zeros(1, 2, 64, 64))
    with pytest.raises(ValueError):
        zq.gated_norm_q8_1(x, None, None, 1e-6, 64)
    with pytest.raises(ValueError):
        zq.residual_norm_q8_1(x, x, None, 1e-6)
