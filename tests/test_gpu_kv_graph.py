"""A decoding step over the paged cache (append, attention with the slots'
weights, eviction back to a budget) captured into a HIP graph and replayed, bit
for bit against the same step launched eagerly on a cache of its own.  Lengths
grow and shrink on the GPU alone; unrelated eager work and synchronisations lie
between the replays."""
import numpy as np
import pytest

from tests.gpu_helpers import assert_equal, dev, host, log
from tests.kv_helpers import HostCache

pytestmark = pytest.mark.gpu


class _Step:
    def __init__(self, q, c, budget, recent, group, seed):
        import torch
        rng = np.random.default_rng(seed)
        B, self.max_len = len(c.lens), c.max_pages * c.page
        self.q, self.budget, self.recent = q, budget, recent
        self.cache, self.table, self.lens = c.device(q), dev(c.table), dev(c.lens)
        self.position = dev(c.lens + 1000)
        shape = (B, c.heads, self.max_len)
        self.mass = dev(rng.random(shape).astype(np.float32))
        self.pos = dev(np.broadcast_to(np.arange(self.max_len, dtype=np.int32), shape).copy())
        self.qin = torch.zeros(B, c.heads * group, c.D, dtype=torch.float16, device="cuda")
        self.kin, self.vin = (torch.zeros(B, c.heads, c.D, dtype=torch.float16, device="cuda") for _ in range(2))
        self.out = torch.empty_like(self.qin)
        self.left = torch.empty_like(self.lens)
        self.kept = torch.empty((B, c.heads, budget), dtype=torch.int32, device="cuda")
        self.attn_work = torch.empty(q.qlin_attn_decode_work_bytes(self.cache, c.heads * group, B, self.max_len,
                                                                   mass=True), dtype=torch.uint8, device="cuda")
        self.evict_work = torch.empty(q.qlin_kv_evict_work_bytes(self.cache, B, self.max_len, budget),
                                      dtype=torch.uint8, device="cuda")

    def feed(self, xs):
        for t, x in zip((self.qin, self.kin, self.vin), xs):
            t.copy_(x)

    def run(self):
        q = self.q
        q.qlin_kv_append(self.cache, self.kin, self.vin, self.table, self.lens, None, self.position, self.mass, self.pos)
        self.lens += 1
        self.position += 1
        q.qlin_attn_decode(self.cache, self.qin, self.table, self.lens, self.max_len, mass=self.mass,
                           mass_out=self.mass, out=self.out, work=self.attn_work)
        q.qlin_kv_evict(self.cache, self.table, self.lens, self.max_len, self.budget, self.recent, self.mass, self.pos,
                        lens_out=self.left, kept=self.kept, work=self.evict_work)
        self.lens.copy_(self.left)

    def state(self):
        c = self.cache
        return [host(t) for t in (self.out, self.lens, self.mass, self.pos, self.kept, c.k, c.v) ] + \
               [host(t) for t in (c.kmeta, c.vmeta) if t is not None]


@pytest.mark.parametrize("bits,D,rotate,budget", [(4, 128, True, 700), (16, 64, False, 20), (8, 256, False, 300)])
def test_replays_match_eager(bits, D, rotate, budget):
    import torch
    from outlier_aware_bit_amd import qlin as q
    log(f"graph replay of a decoding step, {bits} bits, D={D}, budget={budget}")
    lens = [budget, budget // 2, 0, budget - 2]
    steps = []
    for _ in range(2):
        c = HostCache(np.random.default_rng(bits), lens, budget + 40, 2, D, 16, bits, rotate)
        for b in range(len(lens)):  # every page of a sequence's table is its own
            free = sorted(set(range(c.pages)) - set(c.table[c.table >= 0].tolist()))
            for p in range(c.max_pages):
                if c.table[b, p] < 0 and free:
                    c.table[b, p] = free.pop()
        steps.append(_Step(q, c, budget, 8, 4, 7))
    eager, graphed = steps
    g = torch.Generator().manual_seed(bits)
    def inputs(step):
        return [torch.randn(t.shape, generator=g).half().cuda() for t in (step.qin, step.kin, step.vin)]
    xs = inputs(eager)
    for s in steps:  # both states take the first step eagerly
        s.feed(xs)
        s.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        graphed.run()
    for i in range(6):
        xs = inputs(eager)
        for s in steps:
            s.feed(xs)
        eager.run()
        torch.randn(1 << 16, device="cuda").sum().item()  # unrelated work, synchronized
        graph.replay()
        torch.cuda.synchronize()
        for name, a, b in zip(("out", "lens", "mass", "pos", "kept", "k", "v", "kmeta", "vmeta"), eager.state(),
                              graphed.state()):
            assert_equal(b.view(np.uint8), a.view(np.uint8), f"{name}, replay {i}")
    assert host(graphed.lens).tolist() == [budget, min(budget // 2 + 7, budget), 7, budget]
