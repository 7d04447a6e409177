"""examples/serve_kv4.py: slots, pages, rotary positions, append, prompt
attention and decoding as one layer's steps, each checked against the float64
oracle over what the oracle's own cache holds by then."""
import importlib.util
import os

import numpy as np
import pytest

from oracle import prompt
from tests.gpu_helpers import assert_equal, host, log
from tests.prompt_helpers import HALF, TINY, Packed, within
from tests.test_gpu_decode_example import Mirror

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serve_kv4.py")


@pytest.fixture(scope="module")
def example():
    import torch
    assert torch.cuda.is_available()
    spec = importlib.util.spec_from_file_location("serve_kv4", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


class Watch:
    """A server whose projections' results and attention's outputs are kept on the host."""

    def __init__(self, server):
        self.server, self.mirror = server, Mirror(server)
        self.lens = np.zeros(server.table.shape[0], np.int64)
        qkv, turned, out = server.qkv, server._turned, server.out

        def watched_qkv(x):
            y = qkv(x)
            self.raw = host(y).reshape(x.shape[0], -1, 128)
            return y

        def watched_turned(x, position):
            got = turned(x, position)
            self.q, self.k, self.v = (host(t) for t in got)
            self._check_positions(host(position))
            return got

        def watched_out(o):
            self.o = host(o).reshape(self.q.shape)
            return out(o)

        server.qkv, server._turned, server.out = watched_qkv, watched_turned, watched_out

    def _check_positions(self, position):
        n, m = self.server.heads, self.server.kv_heads
        freq, amp = host(self.server.freq), self.server.amplitude
        for got, x in ((self.q, self.raw[:, :n]), (self.k, self.raw[:, n:n + m])):
            want = prompt.rope(x, position, freq, amplitude=amp)
            size = np.abs(x.astype(np.float64))
            size = amp * (size + np.roll(size, 64, -1))
            tol = np.where((position >= 0)[:, None, None], HALF * np.abs(want) + TINY + size * 2.0 ** -20, 0.0)
            assert np.all(np.abs(got - want) <= tol)
        assert_equal(self.v, self.raw[:, n + m:], "v is not turned")

    def pages(self):
        """Every page once, each row's by its length."""
        s = self.server
        page, table, held = s.page, host(s.table), host(s.held)
        assert_equal(host(s.lens), self.lens.astype(np.int32), "lens")
        assert_equal(held, (-(-self.lens // page)).astype(np.int32), "held")
        assert np.all((table >= 0) == (np.arange(table.shape[1]) < held[:, None]))
        head, count = host(s.state)
        free = host(s.ring)[(head + np.arange(count)) % s.ring.numel()]
        assert sorted(table[table >= 0].tolist() + free.tolist()) == list(range(s.ring.numel()))

    def prefill(self, x, add):
        import torch
        y, missing = self.server.prefill(x, torch.tensor(add, dtype=torch.int32).cuda())
        assert int(missing) == 0
        n = [a for a in add]
        c = Packed(0, n, n, self.server.heads, self.server.kv_heads, 128)
        c.q, c.k, c.v = self.q, self.k, self.v
        want, tol, _, _ = c.forward()
        within(self.o, want, tol, "prompt attention")
        at = 0
        for b, m in enumerate(add):
            for t in range(at, at + m):
                self.mirror.append(b, self.k[t], self.v[t])
            at += m
            self.lens[b] += m
        self.pages()
        return y

    def step(self, x, running):
        import torch
        y, missing = self.server.step(x, torch.tensor(running, dtype=torch.int32).cuda())
        assert int(missing) == 0
        for b, r in enumerate(running):
            if r:
                self.mirror.append(b, self.k[b], self.v[b])
                want, tol = self.mirror.attend(b, self.q[b])
                assert np.all(np.abs(self.o[b].astype(np.float64) - want) <= tol), b
            elif self.lens[b] == 0:  # no request; one that pauses attends to what it has
                assert np.all(self.o[b] == 0.0), b
        self.lens += running
        self.pages()
        return y

    def end(self, going):
        import torch
        self.server.end(torch.tensor(going, dtype=torch.int32).cuda())
        for b, g in enumerate(going):
            if g:
                self.mirror.rows[b] = [([], []) for _ in self.mirror.rows[b]]
                self.lens[b] = 0
        self.pages()


@pytest.mark.parametrize("bits", [4, 16])
def test_every_step_against_the_oracle(example, bits):
    import torch
    log(f"serving example, {bits} bits")
    hidden, rows = 256, 4
    server = example.Server4(hidden, 4, 2, rows, pages=13, max_pages=8, bits=bits, page=16, scaling="ramp", factor=4.0,
                             original_len=64, seed=bits)
    w = Watch(server)
    g = torch.Generator(device="cuda").manual_seed(bits)

    def states(n):
        return torch.randn(n, hidden, generator=g, device="cuda", dtype=torch.float16)

    w.prefill(states(57), [40, 0, 17, 0])
    for _ in range(3):
        w.step(states(rows), [1, 0, 1, 0])
    w.prefill(states(68), [0, 67, 0, 1])  # the rest of the pool, but for one page
    for _ in range(12):
        w.step(states(rows), [1, 1, 1, 1])
    w.end([1, 0, 0, 1])
    w.prefill(states(30), [30, 0, 0, 0])
    w.step(states(rows), [1, 1, 0, 0])


def test_a_pool_that_runs_short(example):
    import torch
    log("serving example, a pool that runs short")
    server = example.Server4(256, 2, 1, 2, pages=3, max_pages=4, bits=16, page=16)
    y, missing = server.prefill(torch.zeros(40, 256, dtype=torch.float16, device="cuda"),
                                torch.tensor([33, 7], dtype=torch.int32, device="cuda"))
    assert int(missing) == 1 and host(server.held).tolist() == [3, 0]
    assert torch.isfinite(y).all()


def test_command(example, capsys):
    log("serving example, its command")
    server, x = example.main(["--hidden", "512", "--heads", "4", "--kv-heads", "1", "--rows", "3", "--prompt", "200",
                              "--new-tokens", "9", "--steps", "25"])
    assert tuple(x.shape) == (3, 512)
    out = capsys.readouterr().out
    assert "requests ended" in out and "last states finite: True" in out
