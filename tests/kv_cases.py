"""Inputs of qlin_attn_decode that show one of its roundings each."""
import numpy as np

from oracle import kv


def put_codes(c, b, name, codes, step, lo):
    """Rows of slots 0 .. n - 1 of sequence b as codes [heads, n, D] with one
    step and lo (numbers, or one per slot); fp16 caches take their values."""
    n = codes.shape[1]
    slot = np.arange(n)
    page, line = c.table[b, slot // c.page], slot % c.page
    step, lo = (np.broadcast_to(np.asarray(a, np.float16), (n,)) for a in (step, lo))
    if c.bits == 16:
        rows = (lo[:, None].astype(np.float64) + step[:, None].astype(np.float64) * codes).astype(np.float16)
    else:
        rows = codes.astype(np.uint8)
        rows = kv.pack4(rows) if c.bits == 4 else rows
        getattr(c, name + "meta")[page, :, line] = np.stack([step, lo], -1)[:, None]
    getattr(c, name)[page, :, line] = rows.transpose(1, 0, 2)


def cancelling_v(rng, c, b, n, step):
    """V whose slots come in pairs that cancel, so that the output is small
    against its terms and its fp16 rounding hides little."""
    qmax = 15 if c.bits == 4 else 255
    half = rng.integers(0, qmax + 1, (c.heads, n // 2, c.D))
    codes = np.empty((c.heads, n // 2 * 2, c.D), np.int64)
    codes[:, 0::2], codes[:, 1::2] = half, qmax - half
    put_codes(c, b, "v", codes, step, -qmax * step / 2)


def shifted_k(rng, c, b, n, channel, size):
    """K rows N(0, 1) whose channel `channel` holds `size`: a query of c0 there
    moves every logit by scale c0 size."""
    rows = rng.standard_normal((c.heads, n, c.D)).astype(np.float16)
    rows[..., channel] = size
    c._put(b, "k", rows)
