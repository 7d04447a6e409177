"""Around the paged cache's decoding step: rotary positions, attention over whole
prompts with its gradients, slot maps and page tables (test infrastructure only).

OffQ ("OffQ: Taming Structured Outliers in LLM Quantization by Offsetting",
core contributions) serves models as W4A4KV4 and Quaff ("Quaff: Quantized
Parameter-Efficient Fine-Tuning under Outlier Spatial Stability Hypothesis",
method) trains them; both take the attention between the layers as given.

Everything is float64 or Python integers.
"""
from __future__ import annotations

import math

import numpy as np


# ---------------------------------------------------------------- rotary positions
def rope_freqs(rot: int, base: float = 10000.0, scaling: str = "plain", factor: float = 1.0, original_len: int = 0,
               fast: float = 32.0, slow: float = 1.0):
    """Radians per position of each pair, and the amplitude."""
    if scaling == "base":
        base = base * factor ** (rot / (rot - 2))
    freq = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if scaling == "linear":
        freq = [f / factor for f in freq]
    if scaling != "ramp":
        return np.array(freq), 1.0

    def pair(turns):  # that turns so often within original_len positions
        return rot * math.log(original_len / (2.0 * math.pi * turns)) / (2.0 * math.log(base))

    lo, hi = max(math.floor(pair(fast)), 0), min(math.ceil(pair(slow)), rot - 1)
    for i, f in enumerate(freq):
        part = min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
        freq[i] = f * (1.0 - part) + f / factor * part
    return np.array(freq), 0.1 * math.log(factor) + 1.0


def rope(x: np.ndarray, position: np.ndarray, freq: np.ndarray, interleaved: bool = False, inverse: bool = False,
         amplitude: float = 1.0) -> np.ndarray:
    """x [T, heads, D] turned; tokens at negative positions as they are."""
    x = np.asarray(x, np.float64).copy()
    half = len(freq)
    a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    for t, p in enumerate(position):
        if p < 0:
            continue
        w = (-float(p) if inverse else float(p)) * np.asarray(freq, np.float64)
        c, s = amplitude * np.cos(w), amplitude * np.sin(w)
        u, v = x[t][:, a].copy(), x[t][:, b].copy()
        x[t][:, a], x[t][:, b] = u * c - v * s, u * s + v * c
    return x


# ---------------------------------------------------------------- attention over a prompt
def visible(nq: int, nk: int, causal: bool = True, window: int = 0) -> np.ndarray:
    """[nq, nk]: whether query i sees key j."""
    if not causal:
        return np.ones((nq, nk), bool)
    p, j = np.arange(nq)[:, None] + nk - nq, np.arange(nk)[None, :]
    return (j <= p) & ((j > p - window) if window else True)


def attend(q: np.ndarray, k: np.ndarray, v: np.ndarray, scale: float, see: np.ndarray):
    """One head: q [nq, D], k and v [nk, D] -> (out, lse, p).  Hidden keys take no
    part at all, whatever they hold."""
    nq, nk = see.shape
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    out, lse, p = np.zeros((nq, q.shape[1])), np.full(nq, -np.inf), np.zeros((nq, nk))
    for i in range(nq):
        j = np.flatnonzero(see[i])
        if len(j) == 0:
            continue
        s = scale * (k[j] @ q[i])
        top = s.max()
        if top == -np.inf:
            continue
        e = np.exp(s - top)
        p[i, j] = e / e.sum()
        out[i], lse[i] = p[i, j] @ v[j], top + math.log(e.sum())
    return out, lse, p


def attend_grad(dout: np.ndarray, q: np.ndarray, k: np.ndarray, v: np.ndarray, scale: float, see: np.ndarray):
    """(dq, dk, dv) of one head by the formula."""
    dout, q, k, v = (np.asarray(x, np.float64) for x in (dout, q, k, v))
    out, _, p = attend(q, k, v, scale, see)
    dp = dout @ v.T
    ds = p * (dp - (dout * out).sum(1, keepdims=True))
    return scale * ds @ k, scale * ds.T @ q, p.T @ dout


# ---------------------------------------------------------------- slots and pages
def slots(lens, add, T: int, first=None):
    """(cu, row, slot, position, lens_out) as lists."""
    first = lens if first is None else first
    cu, row, slot, position, lens_out = [0], [], [], [], []
    for b, n in enumerate(add):
        here = 0
        for i in range(max(0, n)):
            if len(row) < T:
                row.append(b)
                slot.append(max(0, lens[b]) + i)
                position.append((max(0, lens[b]) if first is lens else first[b]) + i)
                here += 1
        cu.append(len(row))
        lens_out.append(max(0, lens[b]) + here)
    fill = [-1] * (T - len(row))
    return cu, row + fill, slot + fill, position + fill, lens_out


def pages(want, page: int, table, held, ring, head: int, count: int):
    """(table, held, ring, head, count, missing): rows that lack pages take them
    from the ring's head, in order, until one finds too few; surplus pages go to
    its tail."""
    table, held, ring = [list(r) for r in table], list(held), list(ring)
    size, most = len(ring), len(table[0]) if table else 0
    free = [ring[(head + i) % size] for i in range(count)]
    taken, back, missing, stopped = 0, [], 0, False
    for b, n in enumerate(want):
        need = -(-max(0, n) // page)
        if need > most:
            missing += need - held[b]
            continue
        if need > held[b]:
            grow = need - held[b]
            if stopped or taken + grow > count:
                stopped = True
                missing += grow
                continue
            table[b][held[b]:need] = free[taken:taken + grow]
            taken += grow
        else:
            back += table[b][need:held[b]]
            table[b][need:held[b]] = [-1] * (held[b] - need)
        held[b] = need
    for i, p in enumerate(back):
        ring[(head + count + i) % size] = p
    return table, held, ring, (head + taken) % size, count - taken + len(back), missing
