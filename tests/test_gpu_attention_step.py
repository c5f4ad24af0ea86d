"""The attention half of a decode step as it would be used, from the layer's
input to the o projection's output: RMSNorm + stacked q/k/v projection,
adapters on it in place, head norms + rotation + cache write, paged attention
straight to Q8_1 codes, o projection and its adapters; step by step against
64 bits, captured and replayed token after token."""
import threading

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import oracle
import gemm_zq_rmsnorm_gb300 as zq
from gemm_zq_rmsnorm_gb300 import inputs

import _attn_ref as ref
from test_gpu_lora import check as check_lora

pytestmark = pytest.mark.gpu

K, HQ, HK, D, PAGE, R, N_ADAPTERS = 1024, 8, 2, 128, 16, 16, 3
NQKV = (HQ + 2 * HK) * D


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Layer:
    def __init__(self, B, dtype):
        g = np.random.default_rng(B)
        self.B, self.dtype = B, dtype
        self.gamma = inputs.gamma(1, K)
        self.Wn = inputs.q4k_weights(2, NQKV, K), inputs.q4k_weights(3, K, HQ * D)
        self.W = [dev(w) for w in self.Wn]
        self.g = dev(self.gamma)
        self.gq, self.gk = (dev(g.uniform(0.5, 1.5, D).astype(np.float32)) for _ in range(2))
        self.freq = 1e4 ** (-2.0 * np.arange(D // 2) / D)
        self.rope = zq.rope_table(self.freq)
        half = [dev((g.standard_normal(s) / s[-1] ** 0.5).astype(np.float32)).half()
                for s in ((N_ADAPTERS, R, K), (N_ADAPTERS, NQKV, R), (N_ADAPTERS, R, HQ * D), (N_ADAPTERS, K, R))]
        self.lora_qkv, self.lora_o = half[:2], half[2:]
        self.scales = dev(g.uniform(0.5, 1.0, N_ADAPTERS).astype(np.float32))
        width = 3
        pages = B * width + 1
        self.k = torch.full((pages, HK, PAGE, D), float("nan"), device="cuda").to(dtype)
        self.v = self.k.clone()
        self.cache = zq.KVCache(self.k, self.v)
        self.table = dev(g.permutation(pages)[:B * width].astype(np.int32).reshape(B, width))
        # what a step is given, and what it leaves
        self.x = torch.empty(B, K, device="cuda")
        self.pos = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.slots, self.lens, self.ids = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(3))
        self.q8x, self.q8o = zq.empty_q8_1(B, K), zq.empty_q8_1(B, HQ * D)
        self.base = torch.empty(B, NQKV, device="cuda")
        self.qkv, self.q, self.o = (torch.empty(B, NQKV, device="cuda"), torch.empty(B, HQ * D, device="cuda"),
                                    torch.empty(B, HQ * D, device="cuda"))
        self.lse = torch.empty(B, HQ, device="cuda")
        self.y0, self.y = torch.empty(B, K, device="cuda"), torch.empty(B, K, device="cuda")

        def ws(n):
            return torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")
        self.ws = [ws(zq.gemm_workspace_bytes(NQKV, K, B)), ws(zq.lora_workspace_bytes(B, K, R)),
                   ws(zq.paged_attn_workspace_bytes(HQ, HK, D)), ws(zq.gemm_workspace_bytes(K, HQ * D, B)),
                   ws(zq.lora_workspace_bytes(B, HQ * D, R))]

    def step(self):
        B = self.B
        zq.rmsnorm_q8_1(self.x, self.g, inputs.EPS, out=self.q8x)
        zq.q4k_gemm(self.W[0], NQKV, K, self.q8x, B, y=self.base, workspace=self.ws[0])
        zq.lora(self.q8x, self.ids, *self.lora_qkv, self.scales, base=self.base, y=self.qkv, workspace=self.ws[1])
        q, k, v = self.qkv.split((HQ * D, HK * D, HK * D), 1)
        zq.head_norm_rope(q, k, v, self.gq, self.gk, 1e-6, self.rope, self.pos, self.cache, self.slots, q_out=self.q)
        zq.paged_attn(self.q, self.cache, self.table, self.lens, out=self.o, lse=self.lse, q8_out=self.q8o,
                      workspace=self.ws[2])
        zq.q4k_gemm(self.W[1], K, HQ * D, self.q8o, B, y=self.y0, workspace=self.ws[3])
        zq.lora(self.q8o, self.ids, *self.lora_o, self.scales, base=self.y0, y=self.y, workspace=self.ws[4])

    def give(self, t):
        """Token t of every sequence but those that have not begun (sequence b begins at step b % 3)."""
        at = np.maximum(t - np.arange(self.B) % 3, -1)
        table = self.table.cpu().numpy()
        slots = np.where(at >= 0, table[np.arange(self.B), np.maximum(at, 0) // PAGE] * PAGE + at % PAGE, -1)
        self.x.copy_(dev(inputs.activations(100 + t, self.B, K)))
        self.pos.copy_(dev(np.maximum(at, 0).astype(np.int32)))
        self.slots.copy_(dev(slots.astype(np.int32)))
        self.lens.copy_(dev((at + 1).astype(np.int32)))
        self.ids.copy_(dev(((np.arange(self.B) + t) % (N_ADAPTERS + 1) - 1).astype(np.int32)))
        return at

    def check(self, at):
        n = lambda x: x.detach().cpu().numpy()   # noqa: E731
        qs, d, s = oracle.rmsnorm_q8_1(n(self.x), self.gamma, inputs.EPS)
        assert np.array_equal(n(self.q8x.qs), qs)
        want, S = oracle.q4k_matmul(self.Wn[0], NQKV, K, qs, d, s)
        assert np.all(np.abs(n(self.base) - want) <= 1e-4 * S)
        check_lora(self.qkv, self.q8x, *self.lora_qkv, self.scales, self.base, self.ids)
        x = n(self.qkv).reshape(self.B, HQ + 2 * HK, D)
        pos = n(self.pos)[None]
        wq, wk = (ref.norm_rope(r, n(g), 1e-6, self.freq, [0] * (D // 2), pos, False)
                  for r, g in ((x[:, :HQ], self.gq), (x[:, HQ:HQ + HK], self.gk)))
        assert np.all(np.abs(n(self.q).reshape(wq.shape) - wq) <= 2.0 ** -19 * np.abs(wq).max(-1, keepdims=True))
        flat = [p.float().transpose(1, 2).reshape(-1, HK, D).cpu().numpy().astype(np.float64) for p in (self.k, self.v)]
        table = n(self.table)
        for b, t in enumerate(at):
            rows = table[b][np.arange(max(t + 1, 0)) // PAGE] * PAGE + np.arange(max(t + 1, 0)) % PAGE
            if t >= 0:      # the token's own row, to half a step of the cache's type
                for got, want in ((flat[0][rows[t]], wk[b]), (flat[1][rows[t]], x[b, HQ + HK:])):
                    assert np.all(np.abs(got - want) <= (ref.half_step(self.dtype) + 2.0 ** -18) *
                                  np.abs(want).max(-1, keepdims=True))
            o, lse = ref.attn(n(self.q)[b].reshape(HQ, D).astype(np.float64), flat[0][rows], flat[1][rows],
                              np.arange(len(rows)), D ** -0.5)
            # 2^-15: the bound of the attention's own tests for short rows of unit scores
            A = np.abs(flat[1][rows]).max() if len(rows) else 0
            assert np.all(np.abs(n(self.o)[b].reshape(HQ, D) - o) <= 2.0 ** -15 * A)
            assert np.array_equal(np.isneginf(n(self.lse)[b]), np.isneginf(lse))
        qs, d, s = ref.q8_1(n(self.o))
        assert np.array_equal(n(self.q8o.qs), qs)
        want, S = oracle.q4k_matmul(self.Wn[1], K, HQ * D, n(self.q8o.qs), n(self.q8o.d).view(np.uint16),
                                    n(self.q8o.s).view(np.uint16))
        assert np.all(np.abs(n(self.y0) - want) <= 1e-4 * np.maximum(S, 1e-30))
        check_lora(self.y, self.q8o, *self.lora_o, self.scales, self.y0, self.ids)


@pytest.mark.parametrize("B,dtype", [(1, torch.float16), (4, torch.bfloat16), (9, torch.float16)])
def test_steps_eager_and_captured(B, dtype):
    layer = Layer(B, dtype)
    for t in range(3):
        at = layer.give(t)
        layer.step()
        torch.cuda.synchronize()
        assert zq.device_status() == 0
        layer.check(at)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        layer.step()
    for t in range(3, 3 * PAGE, 7):
        for u in range(max(3, t - 6), t + 1):   # every token is written, every seventh step checked
            at = layer.give(u)
            graph.replay()
        torch.cuda.synchronize()
        layer.check(at)
    assert zq.device_status() == 0


def test_tensors_off_the_current_device_are_refused(monkeypatch):
    """A call launches on the current device: tensors of another one are refused before anything runs."""
    layer = Layer(1, torch.float16)
    layer.give(0)
    layer.step()
    torch.cuda.synchronize()
    was = layer.k.view(torch.int16).clone(), layer.q.clone(), layer.y.clone()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    q = layer.qkv[:, :HQ * D]
    for call in (lambda: zq.head_norm_rope(q, layer.qkv[:, HQ * D:-HK * D], layer.qkv[:, -HK * D:], layer.gq, layer.gk,
                                           1e-6, layer.rope, layer.pos, layer.cache, layer.slots, q_out=layer.q),
                 lambda: zq.paged_attn(layer.q, layer.cache, layer.table, layer.lens, out=layer.o),
                 lambda: zq.lora(layer.q8o, layer.ids, *layer.lora_o, layer.scales, base=layer.y0, y=layer.y)):
        with pytest.raises(ValueError, match="current device"):
            call()
    monkeypatch.undo()
    torch.cuda.synchronize()
    for now, then in zip((layer.k.view(torch.int16), layer.q, layer.y), was):
        assert torch.equal(now, then)


@pytest.mark.parametrize("op", ["norm", "attn", "lora"])
def test_outputs_and_workspaces_made_for_another_stream(op):
    """Work queued on the current stream goes on with tensors that Python has dropped already; a call on another
    stream, which allocates as much, leaves them alone, and its own result outlives the call."""
    layer = Layer(4, torch.bfloat16)
    layer.give(0)
    layer.step()
    q, k, v = layer.qkv.split((HQ * D, HK * D, HK * D), 1)
    call = {"norm": lambda s: zq.head_norm_rope(q, k, v, layer.gq, layer.gk, 1e-6, layer.rope, layer.pos, layer.cache,
                                                layer.slots, stream=s),
            "attn": lambda s: zq.paged_attn(layer.q, layer.cache, layer.table, layer.lens, stream=s),
            "lora": lambda s: zq.lora(layer.q8x, layer.ids, *layer.lora_qkv, layer.scales, base=layer.base, stream=s)}[op]
    want = call(None).clone()
    sizes = {want.numel() * 4, zq.paged_attn_workspace_bytes(HQ, HK, D), zq.lora_workspace_bytes(4, K, R)}
    other = torch.cuda.Stream()
    big = torch.randn(4096, 4096, device="cuda")
    for turn in range(3):
        # queued on the current stream: long products, then sums over temporaries of the call's sizes
        torch.cuda.synchronize()
        x = big
        for _ in range(20):
            x = torch.mm(x, big) * (1 / 64)
        sums = []
        for n in sizes:
            for _ in range(4):
                t = torch.full((n,), 1, dtype=torch.uint8, device="cuda")
                y = t + (x[0, 0] > 1e30).to(torch.uint8)     # waits for the products
                sums.append((n, (t.sum(dtype=torch.int64), y.sum(dtype=torch.int64))))
                del t, y
        got = call(other)
        back = torch.cuda.Event()
        back.record(other)
        torch.cuda.current_stream().wait_event(back)
        kept = got.clone()
        del got
        again = call(other)      # may not take what the current stream still copies
        torch.cuda.synchronize()
        assert torch.equal(kept, want) and torch.equal(again, want)
        for n, parts in sums:
            assert all(int(p) == n for p in parts)


def test_workspaces_that_are_not_one_piece_are_refused():
    layer = Layer(1, torch.float16)
    layer.give(0)
    layer.step()
    bad = torch.zeros(1, dtype=torch.uint8, device="cuda").expand(1 << 26)
    with pytest.raises(ValueError, match="contiguous"):
        zq.paged_attn(layer.q, layer.cache, layer.table, layer.lens, workspace=bad)
    with pytest.raises(ValueError, match="contiguous"):
        zq.lora(layer.q8x, layer.ids, *layer.lora_qkv, layer.scales, base=layer.base, workspace=bad)
    torch.cuda.synchronize()


def test_a_threads_first_call():
    """Each call as the first thing that a thread does on the GPU, after other threads have made the call."""
    layer = Layer(3, torch.float16)
    layer.give(0)
    layer.step()
    torch.cuda.synchronize()
    want = [t.clone() for t in (layer.q8x.qs, layer.base, layer.qkv, layer.q, layer.o, layer.y0)]
    q, k, v = layer.qkv.split((HQ * D, HK * D, HK * D), 1)
    calls = [lambda: zq.rmsnorm_q8_1(layer.x, layer.g, inputs.EPS, out=layer.q8x),
             lambda: zq.q4k_gemm(layer.W[0], NQKV, K, layer.q8x, 3, y=layer.base, workspace=layer.ws[0]),
             lambda: zq.lora(layer.q8x, layer.ids, *layer.lora_qkv, layer.scales, base=layer.base, y=layer.qkv,
                             workspace=layer.ws[1]),
             lambda: zq.head_norm_rope(q, k, v, layer.gq, layer.gk, 1e-6, layer.rope, layer.pos, layer.cache, layer.slots,
                                       q_out=layer.q),
             lambda: zq.paged_attn(layer.q, layer.cache, layer.table, layer.lens, out=layer.o, workspace=layer.ws[2]),
             lambda: zq.q4k_gemm(layer.W[1], K, HQ * D, layer.q8o, 3, y=layer.y0, workspace=layer.ws[3])]
    failed = []

    def work(call):
        try:
            call()
        except Exception as e:   # noqa: BLE001 -- handed to the test
            failed.append(e)

    for call in calls:
        t = threading.Thread(target=work, args=(call,))
        t.start()
        t.join()
    torch.cuda.synchronize()
    assert not failed
    for a, b in zip((layer.q8x.qs, layer.base, layer.qkv, layer.q, layer.o, layer.y0), want):
        assert torch.equal(a, b)


def test_threads_with_streams_of_their_own():
    """Calls from several threads at once, the first ones of their types and widths among them."""
    layers = [Layer(3, dtype) for dtype in (torch.float16, torch.bfloat16) * 2]
    for layer in layers:
        layer.give(0)
    torch.cuda.synchronize()
    failed, gate = [], threading.Barrier(len(layers))

    def work(layer):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                gate.wait(30)
                for _ in range(20):
                    layer.step()
                torch.cuda.current_stream().synchronize()
        except Exception as e:   # noqa: BLE001 -- handed to the test
            failed.append(e)

    threads = [threading.Thread(target=work, args=(layer,)) for layer in layers]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    for layer in layers:
        got = layer.y.clone(), layer.o.clone(), layer.k.view(torch.int16).clone()
        layer.step()
        torch.cuda.synchronize()
        assert zq.device_status() == 0
        assert all(torch.equal(a, b) for a, b in zip(got, (layer.y, layer.o, layer.k.view(torch.int16))))
