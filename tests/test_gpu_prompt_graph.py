"""A step of slots, pages, rotary positions, append, prompt attention and its
gradients captured into a HIP graph, replays against the same step launched
eagerly; calls on another stream than the tensors' own, and on two at once; the
checks of tensors' and the current GPU."""
import numpy as np
import pytest

from tests.gpu_helpers import assert_equal, dev, host, log

pytestmark = pytest.mark.gpu


class _Step:
    """Up to T new tokens for each of B sequences, all on the GPU: their number is data."""

    def __init__(self, q, B, T, heads, kv_heads, D, page, max_pages):
        import torch
        self.q, self.T, self.page = q, T, page
        self.cache = q.KVCache.empty(B * max_pages, kv_heads, D, page, 8)
        self.table = torch.full((B, max_pages), -1, dtype=torch.int32, device="cuda")
        self.held, self.lens, self.add = (torch.zeros(B, dtype=torch.int32, device="cuda") for _ in range(3))
        self.ring = torch.arange(B * max_pages, dtype=torch.int32, device="cuda")
        self.state = torch.tensor([0, B * max_pages], dtype=torch.int32, device="cuda")
        self.qkv = torch.zeros((T, heads + 2 * kv_heads, D), dtype=torch.float16, device="cuda")
        self.dout = torch.zeros((T, heads, D), dtype=torch.float16, device="cuda")
        self.split = [heads, kv_heads, kv_heads]
        self.freq, _ = q.qlin_rope_freqs(D)
        self.work = torch.empty(max(16, q.qlin_attn_prompt_work_bytes(heads, kv_heads, D, B, T, T)), dtype=torch.uint8,
                                device="cuda")
        self.grad_work = torch.empty(q.qlin_attn_prompt_backward_work_bytes(heads, kv_heads, D, B, T, T), dtype=torch.uint8,
                                     device="cuda")
        self.out = torch.zeros((T, heads, D), dtype=torch.float16, device="cuda")
        self.lse = torch.zeros((heads, T), device="cuda")
        self.grads = torch.zeros_like(self.qkv)
        self.missing = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.where = [torch.zeros(n, dtype=torch.int32, device="cuda") for n in (B + 1, T, T, T, B)]

    def feed(self, add, qkv, dout):
        for t, x in ((self.add, add), (self.qkv, qkv), (self.dout, dout)):
            t.copy_(x)

    def run(self):
        q = self.q
        cu, row, slot, position, lens = q.qlin_kv_slots(self.lens, self.add, self.T, None, *self.where)
        q.qlin_kv_pages(lens, self.page, self.table, self.held, self.ring, self.state, missing=self.missing)
        self.lens.copy_(lens)
        x = self.qkv.split(self.split, 1)
        q.qlin_rope(x[0], x[1], position, self.freq, q_out=x[0], k_out=x[1])
        q.qlin_kv_append(self.cache, x[1], x[2], self.table, slot, row)
        q.qlin_attn_prompt(*x, cu, out=self.out, lse=self.lse, work=self.work)
        g = self.grads.split(self.split, 1)
        q.qlin_attn_prompt_backward(self.dout, *x, self.out, self.lse, cu, dq=g[0], dk=g[1], dv=g[2],
                                    work=self.grad_work)
        q.qlin_rope(g[0], g[1], position, self.freq, inverse=True, q_out=g[0], k_out=g[1])

    def tensors(self):
        return dict(out=self.out, lse=self.lse, grads=self.grads, table=self.table, held=self.held, ring=self.ring,
                    state=self.state, lens=self.lens, missing=self.missing, k=self.cache.k, v=self.cache.v,
                    kmeta=self.cache.kmeta, **{f"where {i}": t for i, t in enumerate(self.where)})


def _inputs(g, B, T, shape, dshape):
    import torch
    add = torch.randint(0, T // B + 1, (B,), generator=g).int()
    return [x.cuda() for x in (add, torch.randn(shape, generator=g).half(), torch.randn(dshape, generator=g).half())]


@pytest.mark.parametrize("D,heads,kv_heads", [(64, 4, 2), (128, 4, 1), (256, 2, 2)])
def test_replays_match_eager(D, heads, kv_heads):
    import torch
    from outlier_aware_bit_amd import qlin as q
    log(f"graph replay of a prompt step, D={D}")
    B, T = 3, 400
    eager, graphed = (_Step(q, B, T, heads, kv_heads, D, 16, 40) for _ in range(2))
    g = torch.Generator().manual_seed(D)
    xs = _inputs(g, B, T, eager.qkv.shape, eager.dout.shape)
    for s in (eager, graphed):
        s.feed(*xs)
        s.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        graphed.run()
    for i in range(5):
        xs = _inputs(g, B, T, eager.qkv.shape, eager.dout.shape)
        for s in (eager, graphed):
            s.feed(*xs)
        eager.run()
        torch.randn(1 << 16, device="cuda").sum().item()  # unrelated work, synchronized
        graph.replay()
        torch.cuda.synchronize()
        for (name, a), b in zip(eager.tensors().items(), graphed.tensors().values()):
            assert_equal(host(b).view(np.uint8), host(a).view(np.uint8), f"{name}, replay {i}")
    assert int(eager.lens.sum()) > 0


def test_two_streams_at_once():
    import torch
    from outlier_aware_bit_amd import qlin as q
    log("prompt steps on two streams at once")
    g = torch.Generator().manual_seed(3)
    shape = (400, 8, 128)
    xs = _inputs(g, 3, 400, shape, (400, 4, 128))
    alone = _Step(q, 3, 400, 4, 2, 128, 16, 40)
    alone.feed(*xs)
    alone.run()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    steps = [_Step(q, 3, 400, 4, 2, 128, 16, 40) for _ in streams]
    for s in steps:
        s.feed(*xs)
    torch.cuda.synchronize()
    for s, st in zip(steps, streams):
        with torch.cuda.stream(st):
            s.run()
    torch.cuda.synchronize()
    for s in steps:
        for (name, a), b in zip(alone.tensors().items(), s.tensors().values()):
            assert_equal(host(b).view(np.uint8), host(a).view(np.uint8), name)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_divided_calls_on_two_streams_and_replayed(D):
    # Few heads of one long sequence: rows' keys and keys' queries are divided, workspaces hold the parts.
    import torch
    from outlier_aware_bit_amd import qlin as q
    log(f"divided prompt attention on two streams and in a graph, D={D}")
    T, heads = 900, 4
    sizes = (heads, 1, D, 1, T, T, True, 0)
    assert q.qlin_attn_prompt_work_bytes(*sizes) > 0
    assert q.qlin_attn_prompt_backward_work_bytes(*sizes) >= 2 * T * D * 8
    gen = torch.Generator().manual_seed(D)
    cu = dev(np.array([0, T], np.int32))

    def draw():
        return [torch.randn((T, n, D), generator=gen).half().cuda() for n in (heads, 1, 1, heads)]

    def step(qx, k, v, dout):
        out, lse = q.qlin_attn_prompt(qx, k, v, cu, want_lse=True)
        return (out, lse) + q.qlin_attn_prompt_backward(dout, qx, k, v, out, lse, cu)

    def same(got, want, what):
        for n, (a, b) in enumerate(zip(got, want)):
            assert_equal(host(a).view(np.uint8), host(b).view(np.uint8), f"{what}, output {n}")

    inputs = [draw() for _ in range(2)]
    alone = [step(*x) for x in inputs]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [None, None]
    for _ in range(3):
        for n, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[n] = step(*inputs[n])
    torch.cuda.synchronize()
    for n in range(2):
        same(got[n], alone[n], f"stream {n}")
    held = [x.clone() for x in inputs[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        replayed = step(*held)
    for i in range(4):
        x = draw()
        for a, b in zip(held, x):
            a.copy_(b)
        want = step(*x)
        torch.randn(1 << 16, device="cuda").sum().item()  # unrelated work, synchronized
        graph.replay()
        torch.cuda.synchronize()
        same(replayed, want, f"replay {i}")


@pytest.fixture
def calls():
    import torch
    from outlier_aware_bit_amd import qlin as q
    x = torch.ones((5, 2, 64), dtype=torch.float16, device="cuda")
    one, cu = torch.ones(1, dtype=torch.int32, device="cuda"), dev(np.array([0, 5], np.int32))
    pos, freq = dev(np.arange(5, dtype=np.int32)), q.qlin_rope_freqs(64)[0]
    out, lse = q.qlin_attn_prompt(x, x, x, cu, want_lse=True)
    table, ring, state = dev(np.array([[-1]], np.int32)), dev(np.array([0, 1], np.int32)), dev(np.array([0, 2], np.int32))
    return q, [lambda: q.qlin_rope(x, x, pos, freq), lambda: q.qlin_attn_prompt(x, x, x, cu),
               lambda: q.qlin_attn_prompt_backward(x, x, x, x, out, lse, cu), lambda: q.qlin_kv_slots(one, one, 3),
               lambda: q.qlin_kv_pages(one, 16, table, one * 0, ring, state)]


def test_another_current_gpu_is_refused(calls, monkeypatch):
    q, run = calls
    for f in run:
        f()
    monkeypatch.setattr(q, "_current_device", lambda: 1)
    for f in run:
        with pytest.raises(ValueError, match="current"):
            f()


def test_tensors_that_are_not_on_a_gpu_are_refused(calls):
    import torch
    q, _ = calls
    x, i = torch.ones((5, 2, 64), dtype=torch.float16), torch.zeros(2, dtype=torch.int32)
    y = x.cuda()
    for f in (lambda: q.qlin_rope(x, None, i, i.double()), lambda: q.qlin_rope(y, x, i, i.double()),
              lambda: q.qlin_attn_prompt(x, x, x, i), lambda: q.qlin_attn_prompt(y, y, y, i),
              lambda: q.qlin_attn_prompt(y, y, y, i.cuda(), out=x),
              lambda: q.qlin_kv_slots(i, i, 3), lambda: q.qlin_kv_slots(i.cuda(), i, 3),
              lambda: q.qlin_kv_pages(i, 16, i[None], i, i, i)):
        with pytest.raises(ValueError, match="GPU"):
            f()
