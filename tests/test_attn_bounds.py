"""The bounds that qlin_attn_decode is held to let its arithmetic pass and
reject it with any one of its measures taken away (CPU: the mistakes are planted
in an emulation on the host)."""
import numpy as np
import pytest

from tests import attn_bounds, kv_cases
from tests.kv_helpers import HostCache

FORMS = [(16, False), (8, False), (8, True), (4, False), (4, True)]


def _worst(c, qh, scale, n, **missing):
    """Largest error over its bound: (out, weights)."""
    k, v = (attn_bounds.Rows.of(c, name, 0, 0, n) for name in "kv")
    qt = c.turn(qh)
    out, p = attn_bounds.attend(qt, k, v, scale)
    tol_o, tol_p = attn_bounds.bounds(qt, k, v, scale, out, p)
    got, got_p = attn_bounds.emulate(qh, qt, k, v, scale, c.bits, c.signs is not None, **missing)
    return float((np.abs(got - out) / tol_o).max()), float((np.abs(got_p - p) / tol_p).max())


def _cache(rng, n, bits, rotate):
    return HostCache(rng, [n], n, 1, 128, 16, bits, rotate, outliers=False)


@pytest.mark.parametrize("bits,rotate", FORMS)
@pytest.mark.parametrize("step", [2.0 ** -3, 2.0 ** -7])
def test_weights_in_one_part_are_seen(bits, rotate, step):
    rng = np.random.default_rng(bits + rotate)
    c = _cache(rng, 20, bits, rotate)
    kv_cases.cancelling_v(rng, c, 0, 20, step)
    qh = rng.standard_normal((4, 128)).astype(np.float16)
    scale = 128 ** -0.5 / 64  # nearly equal weights: the logits' own bound, which grows with them, is small
    assert max(_worst(c, qh, scale, 20)) < 1
    assert _worst(c, qh, scale, 20, p_parts=1)[0] > 2


@pytest.mark.parametrize("bits", [8, 4])
def test_a_turned_query_in_one_part_is_seen(bits):
    rng = np.random.default_rng(bits)
    c = _cache(rng, 200, bits, True)
    qh = rng.standard_normal((4, 128)).astype(np.float16)
    assert max(_worst(c, qh, 128 ** -0.5, 200)) < 1
    assert _worst(c, qh, 128 ** -0.5, 200, q_parts=1)[1] > 2


@pytest.mark.parametrize("bits,rotate", [(8, True), (4, False), (4, True)])
def test_a_small_query_rounded_to_an_absolute_grain_is_seen(bits, rotate):
    for std in (1e-3, 1e-4):
        rng = np.random.default_rng(bits)
        c = _cache(rng, 200, bits, rotate)
        qh = (rng.standard_normal((4, 128)) * std).astype(np.float16)
        scale = 128 ** -0.5 / std
        assert max(_worst(c, qh, scale, 200)) < 1
        assert _worst(c, qh, scale, 200, q_scaled=False)[1] > 2


@pytest.mark.parametrize("bits,rotate", FORMS)
@pytest.mark.parametrize("shift", [-16.0, -60.0])
def test_a_missing_reference_is_seen(bits, rotate, shift):
    rng = np.random.default_rng(bits)
    c = _cache(rng, 100, bits, rotate)
    kv_cases.shifted_k(rng, c, 0, 100, 5, 8.0)
    qh = rng.standard_normal((4, 128)).astype(np.float16)
    qh[:, 5] = shift / (8.0 * 128 ** -0.5)
    assert max(_worst(c, qh, 128 ** -0.5, 100)) < 1
    assert _worst(c, qh, 128 ** -0.5, 100, reference=False)[0] > 2


@pytest.mark.parametrize("bits", [8, 4])
def test_a_reference_that_follows_an_infinite_step_is_seen(bits):
    rng = np.random.default_rng(bits)
    c = _cache(rng, 40, bits, False)
    c.vmeta[c.table[0, 0], 0, 7, 0] = np.inf
    qh = rng.standard_normal((2, 128)).astype(np.float16)
    k, v = (attn_bounds.Rows.of(c, name, 0, 0, 40) for name in "kv")
    qt = c.turn(qh)
    s = qt @ k.values().T * 0.1
    p = np.exp(s - s.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    out, got = attn_bounds.emulate(qh, qt, k, v, 0.1, bits, False)
    assert not np.isfinite(out).any() and np.allclose(got, p, rtol=1e-4)
    out, got = attn_bounds.emulate(qh, qt, k, v, 0.1, bits, False, inf_steps=True)
    assert not out.any() and not got.any()
