"""One attention layer in W4A4KV4 that serves requests as they come and go: every
step takes new prompts and one token of every running request, and the GPU
works out from their lengths which pages they hold and where their rows go.

Per step: new lengths -> qlin_kv_pages (the block table) and qlin_kv_slots (rows,
slots, positions, borders) -> qkv projection -> qlin_rope -> qlin_kv_append ->
qlin_attn_prompt for the new prompts, qlin_attn_decode for the running requests
-> output projection.  A request that has its tokens ends: its pages go back to
the ring.

    python examples/serve_kv4.py [--bits 4] [--rows 16] [--steps 128] ...

Weights and hidden states are random; a summary is printed.  Needs the GPU and a
built library.
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from examples.decode_kv4 import HEAD_DIM, Linear4, random_signs  # noqa: E402
from outlier_aware_bit_amd import qlin  # noqa: E402


class Server4:
    """Projections, pool and block table of one layer for up to `rows` requests at a time."""

    def __init__(self, hidden, heads, kv_heads, rows, pages, max_pages, bits=4, page=64, scaling="plain", factor=1.0,
                 original_len=0, seed=0):
        g = torch.Generator().manual_seed(seed)

        def weight(k, n):
            return (torch.randn(k, n, generator=g) * k ** -0.5).half().cuda()

        self.heads, self.kv_heads, self.page = heads, kv_heads, page
        self.qkv = Linear4(weight(hidden, (heads + 2 * kv_heads) * HEAD_DIM), random_signs(hidden, g))
        self.out = Linear4(weight(heads * HEAD_DIM, hidden), random_signs(heads * HEAD_DIM, g))
        turn = random_signs(HEAD_DIM, g)
        self.cache = qlin.KVCache.empty(pages, kv_heads, HEAD_DIM, page, bits, signs=turn if bits < 16 else None)
        self.freq, self.amplitude = qlin.qlin_rope_freqs(HEAD_DIM, scaling=scaling, factor=factor,
                                                         original_len=original_len)
        self.table = torch.full((rows, max_pages), -1, dtype=torch.int32, device="cuda")
        self.held, self.lens = (torch.zeros(rows, dtype=torch.int32, device="cuda") for _ in range(2))
        self.ring = torch.randperm(pages, generator=g, dtype=torch.int32).cuda()
        self.state = torch.tensor([0, pages], dtype=torch.int32, device="cuda")
        self.capacity = max_pages * page

    def _turned(self, x, position):
        """q, k, v of rows x [T, hidden], q and k turned by their positions in place."""
        y = self.qkv(x).view(x.shape[0], self.heads + 2 * self.kv_heads, HEAD_DIM)
        q, k, v = y.split([self.heads, self.kv_heads, self.kv_heads], dim=1)
        qlin.qlin_rope(q, k, position, self.freq, amplitude=self.amplitude, q_out=q, k_out=k)
        return q, k, v

    def _place(self, add, T):
        """Pages and places for add int32 [rows] new tokens of every request: (cu, row, slot, position, missing)."""
        cu, row, slot, position, lens = qlin.qlin_kv_slots(self.lens, add, T)
        missing = qlin.qlin_kv_pages(lens, self.page, self.table, self.held, self.ring, self.state)[3]
        self.lens = lens
        return cu, row, slot, position, missing

    def prefill(self, x, add):
        """Prompts of empty rows: x [sum(add), hidden], a prompt after another, add int32 [rows] (0: no new
        request).  The layer's output for every token, and the pages that were missing."""
        cu, row, slot, position, missing = self._place(add, x.shape[0])
        q, k, v = self._turned(x, position)
        qlin.qlin_kv_append(self.cache, k, v, self.table, slot, row)
        o, _ = qlin.qlin_attn_prompt(q, k, v, cu)
        return self.out(o.view(x.shape[0], -1)), missing

    def step(self, x, running):
        """One token of every running request (int32 [rows], 1 or 0): x [rows, hidden] -> [rows, hidden], and the
        pages that were missing.  Rows without a request give what an empty cache gives;
        a request that pauses stores nothing."""
        rows = x.shape[0]
        slot = torch.where(running > 0, self.lens, -1)
        missing = qlin.qlin_kv_pages(self.lens + running, self.page, self.table, self.held, self.ring, self.state)[3]
        q, k, v = self._turned(x, slot)
        qlin.qlin_kv_append(self.cache, k, v, self.table, slot)
        self.lens = self.lens + running
        o, _ = qlin.qlin_attn_decode(self.cache, q, self.table, self.lens, self.capacity)
        return self.out(o.view(rows, -1)), missing

    def end(self, going):
        """Requests going int32 [rows] (1: ends) give their pages back."""
        self.lens = torch.where(going > 0, 0, self.lens)
        qlin.qlin_kv_pages(self.lens, self.page, self.table, self.held, self.ring, self.state)


def normed(y):
    return y * torch.rsqrt(y.float().pow(2).mean(-1, keepdim=True) + 1e-6).half()


def serve(server, hidden, rows, steps, prompt, new_tokens, seed=1):
    """Requests of random lengths, one beginning wherever a row is free; (tokens made, requests ended, states)."""
    host = torch.Generator().manual_seed(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    left = [0] * rows  # tokens that a row's request still makes: all that the host decides by
    state = torch.zeros(rows, hidden, dtype=torch.float16, device="cuda")
    made = ended = 0
    for _ in range(steps):
        add = [0] * rows
        for b in range(rows):
            if left[b] == 0 and torch.rand((), generator=host) < 0.5:
                add[b] = int(torch.randint(1, prompt + 1, (), generator=host))
                left[b] = int(torch.randint(1, new_tokens + 1, (), generator=host))
        if sum(add):
            x = torch.randn(sum(add), hidden, generator=g, device="cuda", dtype=torch.float16)
            y, missing = server.prefill(x, torch.tensor(add, dtype=torch.int32).cuda())
            last, at = [], 0
            for n in add:
                at += n
                last.append(at - 1)
            new = torch.tensor(add).cuda() > 0
            state = torch.where(new[:, None], normed(y)[torch.tensor(last).clamp(min=0).cuda()], state)
        running = torch.tensor([int(n > 0) for n in left], dtype=torch.int32).cuda()
        y, missing = server.step(state, running)
        state = normed(y)
        made += sum(n > 0 for n in left)
        going = [int(n == 1) for n in left]
        left = [max(0, n - 1) for n in left]
        if any(going):
            server.end(torch.tensor(going, dtype=torch.int32).cuda())
            ended += sum(going)
    return made, ended, state


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    p.add_argument("--hidden", type=int, default=4096)
    p.add_argument("--heads", type=int, default=32)
    p.add_argument("--kv-heads", type=int, default=8)
    p.add_argument("--rows", type=int, default=16, help="requests at a time")
    p.add_argument("--prompt", type=int, default=2000, help="tokens of the longest prompt")
    p.add_argument("--new-tokens", type=int, default=64, help="tokens of the longest answer")
    p.add_argument("--steps", type=int, default=128)
    p.add_argument("--bits", type=int, default=4, choices=(4, 8, 16))
    a = p.parse_args(argv)
    max_pages = -(-(a.prompt + a.new_tokens) // 64)
    server = Server4(a.hidden, a.heads, a.kv_heads, a.rows, a.rows * max_pages, max_pages, a.bits)
    serve(server, a.hidden, a.rows, 2, a.prompt, 1)  # first launches
    server = Server4(a.hidden, a.heads, a.kv_heads, a.rows, a.rows * max_pages, max_pages, a.bits)
    torch.cuda.synchronize()
    t = time.perf_counter()
    made, ended, x = serve(server, a.hidden, a.rows, a.steps, a.prompt, a.new_tokens)
    torch.cuda.synchronize()
    t = time.perf_counter() - t
    print(f"{a.steps} steps, {made} tokens, {ended} requests ended, {t / a.steps * 1e6:.0f} us a step")
    print(f"free pages {int(server.state[1])} of {server.ring.numel()}, last states finite: "
          f"{bool(torch.isfinite(x).all())}")
    return server, x


if __name__ == "__main__":
    main()
