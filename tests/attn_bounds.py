"""Error bounds of qlin_attn_decode, term by term from its arithmetic, and that
arithmetic on the host, for inputs that show each of its roundings.

Per query head and slot, with |q| the query as it meets the stored rows and
(step, lo, code) the row (fp16 rows: step 1, lo 0, code the value):
* a logit is fp32 sums of D products: 2^-23 (sqrt(D) + 8) of the sum of the
  terms' magnitudes, scale (sum_d |q_d| step |code_d| + |lo| sum_d |q_d|), q's
  own two fp16 parts (2^-22) among them; and, with the reference taken off and
  a few roundings of numbers below 64, 2^-19;
* a weight is off by that, by the largest such error of the slots that it is
  normalised by, and by 2^-20 for exp2, the sum and the division;
* in the output each term p_i v_i takes, besides, 2^-21 for p in two fp16 parts
  and 2^-23 (sqrt(n) + 8) for the fp32 sums, on |v_i| as step code + |lo|;
  weights below 2^-31 of the largest may vanish;
* the output is rounded once to fp16: 2^-11 |o| + 2^-25.
"""
import numpy as np


class Rows:
    """k or v of one kv head as stored: code [n, D], step and lo [n], float64."""

    def __init__(self, code, step, lo):
        self.code, self.step, self.lo = (np.asarray(a, np.float64) for a in (code, step, lo))

    @classmethod
    def of(cls, c, name, b, h, n):
        """Slots 0 .. n - 1 of a tests.kv_helpers.HostCache."""
        from oracle import kv
        slot = np.arange(n)
        page, line = c.table[b, slot // c.page], slot % c.page
        code = getattr(c, name)[page, h, line]
        if c.bits == 16:
            return cls(code, np.ones(n), np.zeros(n))
        meta = getattr(c, name + "meta")[page, h, line].astype(np.float64)
        return cls(kv.unpack4(code) if c.bits == 4 else code, meta[:, 0], meta[:, 1])

    def values(self):
        return self.lo[:, None] + self.step[:, None] * self.code

    def size(self):
        """step |code| + |lo|."""
        return np.abs(self.step[:, None] * self.code) + np.abs(self.lo)[:, None]


def attend(qt, k, v, scale, use=None):
    """float64 attention of turned queries qt [G, D]: (out, p)."""
    from oracle import kv
    return kv.attend(qt, k.values(), v.values(), scale, use)


def bounds(qt, k, v, scale, out, p, use=None):
    """(bound of out [G, D], bound of the weights p [G, n])."""
    n, D = k.code.shape
    use = np.ones(n, bool) if use is None else use
    terms = np.abs(qt) @ np.abs(k.step[:, None] * k.code).T + np.abs(qt).sum(1)[:, None] * np.abs(k.lo)[None, :]
    ds = abs(scale) * terms * (D ** 0.5 + 8) * 2.0 ** -23 + 2.0 ** -19
    rel = ds + np.where(use, ds, 0).max(1, keepdims=True, initial=0) + 2.0 ** -20
    size = v.size()
    each = p * (rel + 2.0 ** -21 + (n ** 0.5 + 8) * 2.0 ** -23)
    tol = each @ size + n * 2.0 ** -31 * p.max(1, keepdims=True, initial=0) * size.max(0, initial=0)[None, :]
    return tol + 2.0 ** -11 * np.abs(out) + 2.0 ** -25, p * rel


def emulate(qh, qt, k, v, scale, bits, turned, p_parts=2, q_parts=2, q_scaled=True, reference=True, inf_steps=False):
    """What the kernel computes, its roundings to fp16 and the reference
    exponent in their places and its sums in float64: (out, p).  Each argument
    after `turned` takes one of its measures away."""
    f16, f32, f64 = np.float16, np.float32, np.float64
    G, D = qt.shape
    q = np.asarray(qt if turned else qh, f64)
    s = np.ones((G, 1))
    if q_scaled and (turned or bits == 4):
        top = np.abs(q).max(1, keepdims=True)
        s = 2.0 ** (14 - np.floor(np.log2(np.where(top > 0, top, 2.0 ** 14))))
    # Every other pair of an int4 row's channels meets codes four bits higher.
    down = np.where((np.arange(D) & 1) == 1, 1 / 16, 1.0) if bits == 4 else np.ones(D)
    x = q * s * down
    hi = x.astype(f16).astype(f64)
    rem = (x - hi).astype(f16).astype(f64) if (turned and q_parts == 2) else 0.0
    qr = (hi + rem) / down / s
    unit = np.log2(np.e) * scale
    logit = (unit * ((qr @ k.code.T) * k.step[None, :] + q.sum(1)[:, None] * k.lo[None, :])).astype(f32).astype(f64)
    with np.errstate(divide="ignore"):
        step = v.step if bits < 16 else np.ones_like(v.step)
        ok = (step > 0) & (np.isfinite(step) | inf_steps)
        up = np.maximum(logit - 30, np.where(ok, logit + np.log2(np.where(ok, step, 1.0)) - 7, -np.inf))
    m = up.max(1, keepdims=True) if reference else np.zeros((G, 1))
    with np.errstate(invalid="ignore", over="ignore"):
        e = np.exp2(logit - m).astype(f32).astype(f64)
        w = (e * step).astype(f32)
        ph = w.astype(f16)
        pr = (w - ph.astype(f32)).astype(f16).astype(f64) if p_parts == 2 else 0.0
        total = e.sum(1, keepdims=True)
        o = (ph.astype(f64) + pr) @ v.code + e @ v.lo[:, None]
        out = np.where(total == 0, 0.0, o / np.where(total == 0, 1.0, total)).astype(f16)
    return out.astype(f64), e / np.where(total == 0, 1.0, total)
