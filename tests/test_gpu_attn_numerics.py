"""Attention of one new token over the paged cache (qlin_attn_decode) where its
arithmetic is put to the test, against float64 within bounds that let it pass
and reject it with any one of its measures taken away."""
import numpy as np
import pytest

from tests import attn_bounds, kv_cases
from tests.gpu_helpers import dev, host, log
from tests.kv_helpers import HostCache

pytestmark = pytest.mark.gpu

FORMS = [(16, 64, False), (16, 128, False), (16, 256, False), (8, 64, False), (8, 128, False), (8, 128, True),
         (8, 256, False), (4, 64, False), (4, 128, False), (4, 128, True), (4, 256, False)]


@pytest.fixture(scope="module")
def q():
    import torch
    assert torch.cuda.is_available()
    from outlier_aware_bit_amd import qlin
    return qlin


def _run(q, c, qh, scale, max_len=None):
    """(out, mass) in float64, mass from nothing."""
    import torch
    max_len = c.max_pages * c.page if max_len is None else max_len
    mass = torch.zeros((len(c.lens), c.heads, max_len), device="cuda")
    out, mass = q.qlin_attn_decode(c.device(q), dev(qh), dev(c.table), dev(c.lens), max_len, scale=scale,
                                   mass_out=mass)
    return host(out).astype(np.float64), host(mass).astype(np.float64)


def _check(q, c, qh, scale, max_len=None, skip=()):
    """Every (sequence, kv head) within its bounds; the output of those in
    `skip` has no finite value."""
    got, mass = _run(q, c, qh, scale, max_len)
    G = qh.shape[1] // c.heads
    worst_o = worst_p = 0.0
    for b, n in enumerate(int(x) for x in c.lens):
        for h in range(c.heads):
            qs = slice(h * G, (h + 1) * G)
            k, v = (attn_bounds.Rows.of(c, name, b, h, n) for name in "kv")
            qt = c.turn(qh[b, qs])
            if (b, h) in skip:
                v.step[~np.isfinite(v.step)], v.lo[~np.isfinite(v.lo)] = 0, 0
            out, p = attn_bounds.attend(qt, k, v, scale)
            tol_o, tol_p = attn_bounds.bounds(qt, k, v, scale, out, p)
            if (b, h) in skip:
                assert not np.isfinite(got[b, qs]).any(), (b, h)
            elif n == 0:
                assert not got[b, qs].any(), (b, h)
            else:
                ratio = np.abs(got[b, qs] - out) / tol_o
                assert np.all(ratio <= 1), (b, h, "out", float(np.nanmax(ratio)))
                worst_o = max(worst_o, float(ratio.max()))
            if n:
                ratio = np.abs(mass[b, h, :n] - p.sum(0)) / (tol_p.sum(0) + 2.0 ** -30)
                assert np.all(ratio <= 1), (b, h, "mass", float(np.nanmax(ratio)))
                worst_p = max(worst_p, float(ratio.max()))
    log(f"  worst {worst_o:.3f} of the output's bound, {worst_p:.3f} of the mass's")


@pytest.mark.parametrize("bits,D,rotate", FORMS)
@pytest.mark.parametrize("shift", [-16.0, -60.0, 60.0])
def test_logits_that_all_lie_far_from_zero(q, bits, D, rotate, shift):
    # One channel of K holds 8 and one of q what moves every logit by `shift`;
    # softmax does not see it.  A short row, and one in several parts.
    log(f"attend shifted by {shift} bits={bits} D={D} rotate={rotate}")
    rng = np.random.default_rng(bits + D + rotate)
    lens = [20, 700, 1]
    c = HostCache(rng, lens, 700, 2, D, 32, bits, rotate, outliers=False)
    for b, n in enumerate(lens):
        kv_cases.shifted_k(rng, c, b, n, 5, 8.0)
    scale = D ** -0.5
    qh = rng.standard_normal((3, 4, D)).astype(np.float16)
    qh[..., 5] = shift / (8.0 * scale)
    _check(q, c, qh, scale)


@pytest.mark.parametrize("bits,rotate", [(16, False), (8, False), (4, True)])
def test_logits_that_fall_and_rise_along_a_row(q, bits, rotate):
    # The reference follows: far below zero at first, then hundreds higher, and
    # back; the weights of what came before vanish.
    log(f"attend a row of steps, bits={bits}")
    rng = np.random.default_rng(bits)
    n, D = 400, 128
    c = HostCache(rng, [n, n], n, 1, D, 16, bits, rotate, outliers=False)
    for b, sign in enumerate((1, -1)):
        rows = rng.standard_normal((1, n, D)).astype(np.float16)
        rows[0, :, 5] = sign * np.linspace(-8, 8, n)
        c._put(b, "k", rows)
    qh = rng.standard_normal((2, 4, D)).astype(np.float16)
    qh[..., 5] = [1, 10, 100, 1000]
    _check(q, c, qh, D ** -0.5)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("step,lo", [(np.inf, -1.0), (np.inf, -np.inf), (np.nan, np.nan)])
@pytest.mark.parametrize("n,group", [(20, 2), (33, 2), (600, 2), (600, 20), (900, 40)])
def test_a_v_row_that_is_not_finite(q, bits, step, lo, n, group):
    # Rows of an infinity or a NaN have no finite step; their heads' output is
    # not finite, and the weights, which do not depend on V, are what they are.
    log(f"attend V row step={step} lo={lo} bits={bits} n={n} group={group}")
    rng = np.random.default_rng(n + group)
    c = HostCache(rng, [n, 40], max(n, 40), 2, 128, 16, bits, bits == 4, outliers=False)
    for slot in (7, n - 1):
        c.vmeta[c.table[0, slot // 16], 1, slot % 16] = step, lo
    qh = rng.standard_normal((2, 2 * group, 128)).astype(np.float16)
    _check(q, c, qh, 128 ** -0.5, skip={(0, 1)})


@pytest.mark.parametrize("bits,D,rotate", FORMS)
@pytest.mark.parametrize("std", [1e4, 1.0, 1e-1, 1e-2, 1e-3, 1e-4])
def test_queries_of_any_size(q, bits, D, rotate, std):
    # Logits of the same size from large and small queries, one head a
    # thousandth of the others, one all zeros.
    log(f"attend q of {std} bits={bits} D={D} rotate={rotate}")
    rng = np.random.default_rng(bits + D)
    c = HostCache(rng, [100, 530], 530, 2, D, 16, bits, rotate, outliers=False)
    qh = rng.standard_normal((2, 10, D)) * std
    qh[:, 1] *= 1e-3
    qh[:, 2] = 0
    qh = np.clip(qh, -65504, 65504).astype(np.float16)
    _check(q, c, qh, D ** -0.5 / std)


@pytest.mark.parametrize("bits,D,rotate", [f for f in FORMS if f[0] < 16])
def test_one_large_channel_of_the_query(q, bits, D, rotate):
    # What a head's largest channel leaves to the others.
    log(f"attend one large channel bits={bits} D={D} rotate={rotate}")
    rng = np.random.default_rng(bits + D)
    c = HostCache(rng, [100], 100, 1, D, 16, bits, rotate, outliers=False)
    qh = rng.standard_normal((1, 3, D)).astype(np.float16)
    qh[:, 0, 6], qh[:, 1, 7], qh[:, 2, D - 1] = 3000, -65504, 60000
    _check(q, c, qh, D ** -0.5 / 100)


@pytest.mark.parametrize("bits,D,rotate", FORMS)
@pytest.mark.parametrize("step", [2.0 ** -3, 2.0 ** -7])
def test_weights_in_two_parts(q, bits, D, rotate, step):
    # V in pairs that cancel, weights nearly equal: the output's rounding hides
    # little of what the weights lose.
    log(f"attend cancelling V bits={bits} D={D} rotate={rotate} step={step}")
    rng = np.random.default_rng(bits + D)
    c = HostCache(rng, [20, 200], 200, 2, D, 16, bits, rotate, outliers=False)
    for b, n in enumerate((20, 200)):
        kv_cases.cancelling_v(rng, c, b, n, step)
    qh = rng.standard_normal((2, 8, D)).astype(np.float16)
    _check(q, c, qh, D ** -0.5 / 64)


@pytest.mark.parametrize("bits,D,rotate", FORMS)
def test_rows_of_one_workgroup_and_of_several(q, bits, D, rotate):
    # Both sides of the length from which rows are divided, and outliers in K.
    log(f"attend 512 and 513 slots bits={bits} D={D} rotate={rotate}")
    for n in (511, 512, 513):
        rng = np.random.default_rng(n)
        c = HostCache(rng, [n, 3, 0, 480], n, 2, D, 32, bits, rotate)
        qh = rng.standard_normal((4, 6, D)).astype(np.float16)
        _check(q, c, qh, D ** -0.5, max_len=n)
