"""Packed prompts for the GPU tests, the oracle's answers for them, and how far
the kernels' may be off, term by term (no method arithmetic of the library)."""
import numpy as np

from oracle import prompt

HALF = 2.0 ** -11  # one rounding to fp16, relative
TINY = 2.0 ** -25  # and among its smallest numbers
ADD = 2.0 ** -23   # one fp32 operation of a matrix instruction's sum, rounded or cut off


class Packed:
    """fp16 q, k, v (and dout) of sequences with nq[b] queries and nk[b] keys."""

    def __init__(self, seed, nq, nk, heads, kv_heads, D, causal=True, window=0, scale=None, gap=0):
        rng = np.random.default_rng(seed)
        self.nq, self.nk, self.heads, self.kv_heads, self.D = list(nq), list(nk), heads, kv_heads, D
        self.causal, self.window, self.scale = causal, window, D ** -0.5 if scale is None else scale
        self.cu_q, self.cu_k = (np.concatenate([[0], np.cumsum(n)]).astype(np.int32) + gap for n in (nq, nk))
        Tq, Tk = int(self.cu_q[-1]) + gap, int(self.cu_k[-1]) + gap
        self.q, self.k, self.v, self.dout = (rng.standard_normal((n, h, D)).astype(np.float16)
                                             for n, h in ((Tq, heads), (Tk, kv_heads), (Tk, kv_heads), (Tq, heads)))
        self.k[..., 3] += 4.0  # a channel with an offset, as keys have

    def each(self):
        """(rows of q, rows of k, head, kv head, visible) of every sequence and query head."""
        for b, (m, n) in enumerate(zip(self.nq, self.nk)):
            see = prompt.visible(m, n, self.causal, self.window)
            i, j = slice(self.cu_q[b], self.cu_q[b] + m), slice(self.cu_k[b], self.cu_k[b] + n)
            for h in range(self.heads):
                yield i, j, h, h * self.kv_heads // self.heads, see

    def score_error(self, q, k):
        """Of scale q.k as the kernels have it: D products, exact, added in fp32; one
        more rounding for the product with the scale, one in the exponent, and one
        of a reference of the scores' size taken off."""
        a = abs(self.scale) * (np.abs(q) @ np.abs(k).T)
        return a * ADD * (self.D + 3)

    def forward(self):
        """(out, lse) and their bounds; rows of no sequence are NaN."""
        out, tol = (np.full(self.q.shape, np.nan) for _ in range(2))
        lse, lse_tol = (np.full((self.heads, self.q.shape[0]), np.nan) for _ in range(2))
        for i, j, h, g, see in self.each():
            q, k, v = (x.astype(np.float64) for x in (self.q[i, h], self.k[j, g], self.v[j, g]))
            o, e, p = prompt.attend(q, k, v, self.scale, see)
            err = np.where(see, self.score_error(q, k), 0.0).max(1, initial=0.0)
            # p: the scores of a row are off by err each, the exponential by 2^-21;
            # rounded to fp16 for the product (the smallest to 2^-32 of the largest);
            # its sum, the products' and the division in fp32.
            n = see.sum(1)
            rel = 2.0 * err + 2.0 ** -21 + 4 * ADD + n * ADD
            out[i, h] = o
            tol[i, h] = HALF * np.abs(o) + TINY + (p @ np.abs(v)) * (HALF + rel)[:, None] * 1.01 + \
                2.0 ** -31 * np.where(see[..., None], np.abs(v)[None], 0.0).sum(1)
            lse[h, i], lse_tol[h, i] = e, rel + 2.0 ** -21 * np.where(np.isfinite(e), np.abs(e), 0.0)
        return out, tol, lse, lse_tol

    def backward(self):
        """(dq, dk, dv) and their bounds, for a backward pass that is given out
        rounded to fp16 and lse to fp32."""
        shapes = (self.q.shape, self.k.shape, self.k.shape)
        grads, tols = [np.zeros(s) for s in shapes], [np.zeros(s) for s in shapes]
        for i, j, h, g, see in self.each():
            q, k, v, do = (x.astype(np.float64) for x in (self.q[i, h], self.k[j, g], self.v[j, g], self.dout[i, h]))
            o, e, p = prompt.attend(q, k, v, self.scale, see)
            dp = do @ v.T
            ds = p * (dp - (do * o).sum(1, keepdims=True))
            dq, dk, dv = prompt.attend_grad(do, q, k, v, self.scale, see)
            e = np.where(np.isfinite(e), np.abs(e), 0.0)[:, None]
            rel = 2.0 * self.score_error(q, k) + 2.0 ** -21 * (1.0 + e)
            # delta: out is off by a rounding, and D products are added in fp32.
            off = ((np.abs(do) @ np.abs(v).T) + (np.abs(do) * np.abs(o)).sum(1, keepdims=True)) * ADD * (self.D + 2) + \
                (np.abs(do) * (np.abs(o) * HALF + TINY)).sum(1, keepdims=True)
            n = see.shape[0] * self.heads // self.kv_heads + see.shape[1]
            # ds: those two, one rounding to fp16 and (far below the largest) 2^-35 of it.
            dse = p * off + np.abs(ds) * (rel + HALF * 1.01 + 2 * ADD) + 2.0 ** -35 * np.abs(ds).max(initial=0.0) * see
            add = n * ADD
            for x, want, t in ((0, dq, abs(self.scale) * (dse + add * np.abs(ds)) @ np.abs(k)),
                               (1, dk, abs(self.scale) * (dse + add * np.abs(ds)).T @ np.abs(q)),
                               (2, dv, (p * (rel + HALF * 1.01 + add) + 2.0 ** -38 * see).T @ np.abs(do))):
                rows, head = (i, h) if x == 0 else (j, g)
                grads[x][rows, head] += want
                tols[x][rows, head] += t
        return grads, [t + HALF * np.abs(g) + TINY for g, t in zip(grads, tols)]


def within(got, want, tol, what):
    got = np.asarray(got, np.float64)
    here = ~np.isnan(want)
    assert np.array_equal(np.isneginf(got[here]), np.isneginf(want[here])), what
    here &= np.isfinite(want)
    off = np.abs(got[here] - want[here])
    assert np.all(off <= tol[here]), f"{what}: {float(np.nanmax(off / tol[here])):.3g} of what it may be off"


def strided(x, pad=16):
    """A GPU copy of x [T, heads, D] whose tokens lie apart, other values between them."""
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    room = torch.full((t.shape[0], t.shape[1] * t.shape[2] + pad), 7.0, dtype=t.dtype, device="cuda")
    view = room[:, 8:8 + t.shape[1] * t.shape[2]].unflatten(1, t.shape[1:])
    view.copy_(t)
    return view
