"""Paged key/value cache: row quantization, attention of one new token, and
eviction by accumulated attention weight (test infrastructure only).

OffQ ("OffQ: Taming Structured Outliers in LLM Quantization by Offsetting",
core contributions) serves models as W4A4KV4; methodology: standard uniform
asymmetric quantization, after a Hadamard whose all-ones first row turns an
outlier channel into an offset.

The codes of a row are decided in IEEE float32, one rounding per operation;
everything computed from them is float64.
"""
from __future__ import annotations

import numpy as np


def butterfly128(x: np.ndarray, signs: np.ndarray) -> np.ndarray:
    """(x * signs) H_128 of rows [.., 128], in float32, spans 1, 2, .., 64."""
    u = np.asarray(x, np.float32) * np.asarray(signs, np.float32)
    h = 1
    while h < 128:
        w = u.reshape(u.shape[:-1] + (128 // (2 * h), 2, h))
        u = np.stack([w[..., 0, :] + w[..., 1, :], w[..., 0, :] - w[..., 1, :]], axis=-2).reshape(u.shape)
        h *= 2
    return u


def quant_rows(t: np.ndarray, bits: int):
    """Codes (uint8) and (step, lo) float16 [.., 2] of float32 rows [.., D]."""
    f = np.float32
    qmax = f(2 ** bits - 1)
    t = np.asarray(t, f)
    lo = t.min(-1).astype(np.float16)
    step = ((t.max(-1) - lo.astype(f)) * (f(1) / qmax)).astype(np.float16)
    s = step.astype(f)
    inv = np.where(s == 0, f(0), f(1) / np.where(s == 0, f(1), s)).astype(f)
    codes = np.clip(np.rint((t - lo.astype(f)[..., None]) * inv[..., None]), f(0), qmax).astype(np.uint8)
    return codes, np.stack([step, lo], -1)


def dequant_rows(codes: np.ndarray, meta: np.ndarray) -> np.ndarray:
    """lo + step * code in float64."""
    m = np.asarray(meta, np.float64)
    return m[..., 1:] + m[..., :1] * np.asarray(codes, np.float64)


def pack4(codes: np.ndarray) -> np.ndarray:
    """Two codes per byte, low nibble = even index."""
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def unpack4(packed: np.ndarray) -> np.ndarray:
    out = np.empty(packed.shape[:-1] + (2 * packed.shape[-1],), np.uint8)
    out[..., 0::2] = packed & 15
    out[..., 1::2] = packed >> 4
    return out


def attend(q: np.ndarray, k: np.ndarray, v: np.ndarray, scale: float, use: np.ndarray | None = None):
    """Softmax attention of queries [G, D] over rows k, v [n, D] in float64, over
    the slots where ``use`` is true: (out [G, D], weights [G, n]).  Without a
    slot of finite logit the output is zero."""
    q, k, v = (np.asarray(a, np.float64) for a in (q, k, v))
    n = k.shape[0]
    use = np.ones(n, bool) if use is None else np.asarray(use, bool)
    p = np.zeros((q.shape[0], n))
    if use.any():
        s = (q @ k[use].T) * scale
        top = s.max(1, keepdims=True)
        e = np.exp(s - np.where(np.isneginf(top), 0.0, top))
        total = e.sum(1, keepdims=True)
        p[:, use] = e / np.where(total == 0, 1.0, total)
    return p[:, use] @ v[use], p


def evict(mass: np.ndarray, pos: np.ndarray, budget: int, recent: int, there=None):
    """Which slots of one row stay: (left, src [left]) with src[j] the old slot
    of new slot j.  The ``recent`` newest positions first, then the others, each
    by mass, the largest first, a NaN least, ties to the lowest slot; slots that
    stay past ``left`` fill the freed ones before it, both in ascending order.
    Slots where ``there`` is false do not exist: one before ``left`` keeps its
    place, one past it goes, and their mass and position decide nothing."""
    n = len(mass)
    left = min(n, budget)
    there = [True] * n if there is None else there
    newest = max((int(p) for p, t in zip(pos, there) if t), default=0)

    def rank(i):
        if not there[i]:
            return (0 if i < left else 3, False, 0.0, i)
        m = float(mass[i])
        late = int(pos[i]) > newest - recent
        return (1 if late else 2, np.isnan(m), 0.0 if np.isnan(m) else -m, i)
    stay = sorted(sorted(range(n), key=rank)[:left])
    src = list(range(left))
    kept = set(stay)
    holes = [j for j in range(left) if j not in kept]
    for j, i in zip(holes, [i for i in stay if i >= left]):
        src[j] = i
    return left, np.array(src, np.int64)
