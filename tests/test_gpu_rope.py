"""qlin_rope against the float64 oracle: layouts, parts of heads, far positions,
strides, in place, padding and refusals."""
import numpy as np
import pytest

from oracle import prompt
from tests.gpu_helpers import dev, host, log
from tests.prompt_helpers import HALF, TINY, strided

pytestmark = pytest.mark.gpu


def _inputs(seed, T, heads, kv_heads, D, far):
    rng = np.random.default_rng(seed)
    q, k = (rng.standard_normal((T, h, D)).astype(np.float16) for h in (heads, kv_heads))
    return q, k, rng.integers(0, far, T).astype(np.int32)


def _check(got, x, position, freq, interleaved, inverse, amplitude, what):
    want = prompt.rope(x, position, freq, interleaved, inverse, amplitude)
    # The sine and cosine are good to 2^-22; two fp32 products and their sum; one rounding.
    half, size = len(freq), np.zeros(x.shape)
    a = np.abs(x.astype(np.float64))
    i, j = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    size[..., i] = size[..., j] = (a[..., i] + a[..., j]) * amplitude
    tol = np.where(size > 0, HALF * np.abs(want) + TINY + size * 2.0 ** -20, 0.0)
    tol[position < 0] = 0.0
    off = np.abs(host(got).astype(np.float64) - want)
    assert np.all(off <= tol), f"{what}: off by {off.max():.3g}"


@pytest.mark.parametrize("D,rot", [(64, 64), (64, 16), (128, 128), (128, 32), (128, 48), (256, 256), (256, 64)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
def test_turns(D, rot, interleaved, inverse):
    from outlier_aware_bit_amd import qlin as q
    log(f"rope D={D} rot={rot} interleaved={interleaved} inverse={inverse}")
    for T, heads, kv_heads in ((1, 8, 2), (5, 1, 1), (67, 7, 3), (300, 32, 8)):
        x, y, p = _inputs(rot + T, T, heads, kv_heads, D, 100000)
        freq, amp = q.qlin_rope_freqs(rot, scaling="ramp", factor=4.0, original_len=4096)
        a, b = q.qlin_rope(strided(x), strided(y, 24), dev(p), freq, interleaved, inverse, amp)
        _check(a, x, p, host(freq), interleaved, inverse, amp, "q")
        _check(b, y, p, host(freq), interleaved, inverse, amp, "k")


def test_far_positions_and_any_frequency():
    from outlier_aware_bit_amd import qlin as q
    log("rope, positions up to 2^31 - 1")
    x, _, p = _inputs(1, 200, 2, 1, 128, 2 ** 31 - 1)
    p[:3] = [0, 2 ** 31 - 1, 2 ** 30]
    freq = np.random.default_rng(2).uniform(-7.0, 7.0, 64)
    freq[:3] = [0.0, np.pi, 2.0 ** 20]
    # The angle in turns is good to 2^-53 of itself: the oracle's own float64 angle has no more bits, so it is
    # compared where those are enough.
    near = np.abs(p[:, None].astype(np.float64) * freq).max(1) < 2.0 ** 30
    got, none = q.qlin_rope(dev(x), None, dev(p), dev(freq))
    assert none is None
    near[:3] = False
    freq_ok = np.abs(freq) < 8.0
    got = host(got)
    far = prompt.rope(x, p, freq)
    a = np.abs(x.astype(np.float64))
    for i in np.flatnonzero(freq_ok):
        # 2^31 * 7 radians: 2^-53 of them is 2^-19.
        tol = HALF * np.abs(far[:, :, [i, i + 64]]) + TINY + (a[:, :, [i]] + a[:, :, [i + 64]]) * 2.0 ** -17
        assert np.all(np.abs(got[:, :, [i, i + 64]].astype(np.float64) - far[:, :, [i, i + 64]]) <= tol), i
    assert np.isfinite(got.astype(np.float64)).all()


def test_quadrants():
    # Angles at and around every multiple of an eighth of a turn.
    from outlier_aware_bit_amd import qlin as q
    log("rope, eighths of a turn")
    p = np.arange(64, dtype=np.int32)
    for nudge in (-1e-9, 0.0, 1e-9):
        freq = np.full(32, np.pi / 4.0 + nudge) * np.where(np.arange(32) % 2, -1.0, 1.0)
        x = np.random.default_rng(3).standard_normal((64, 1, 64)).astype(np.float16)
        got, _ = q.qlin_rope(dev(x), None, dev(p), dev(freq))
        _check(got, x, p, freq, False, False, 1.0, f"nudge {nudge}")


def test_in_place_and_padding():
    import torch
    from outlier_aware_bit_amd import qlin as q
    log("rope, in place, with padded tokens")
    x, y, p = _inputs(4, 90, 4, 2, 128, 5000)
    p[[0, 17, 89]] = -1
    freq, _ = q.qlin_rope_freqs(64)
    qkv = torch.zeros((90, 8, 128), dtype=torch.float16, device="cuda")
    qkv[:, :4], qkv[:, 4:6], qkv[:, 6:] = dev(x), dev(y), 5.0
    a, b = qkv[:, :4], qkv[:, 4:6]
    got = q.qlin_rope(a, b, dev(p), freq, q_out=a, k_out=b)
    assert got[0].data_ptr() == a.data_ptr()
    _check(a, x, p, host(freq), False, False, 1.0, "q")
    _check(b, y, p, host(freq), False, False, 1.0, "k")
    assert torch.all(qkv[:, 6:] == 5.0)
    # Elsewhere, padded tokens' rows are not written.
    out = torch.full((90, 4, 128), 9.0, dtype=torch.float16, device="cuda")
    q.qlin_rope(dev(x), None, dev(p), freq, q_out=out)
    assert torch.all(out[[0, 17, 89]] == 9.0)
    # There and back.
    q.qlin_rope(a, b, dev(p), freq, inverse=True, q_out=a, k_out=b)
    assert np.all(np.abs(host(a).astype(np.float64) - x) <= 4 * HALF * np.abs(x).max())


def test_values_that_are_not_finite_stay_in_their_pair():
    from outlier_aware_bit_amd import qlin as q
    log("rope, NaN")
    x, _, p = _inputs(5, 3, 2, 1, 64, 50)
    freq, _ = q.qlin_rope_freqs(32)
    want = host(q.qlin_rope(dev(x), None, dev(p), freq)[0])
    x[1, 1, 2] = np.nan
    got = host(q.qlin_rope(dev(x), None, dev(p), freq)[0])
    bad = np.zeros(x.shape, bool)
    bad[1, 1, [2, 18]] = True
    assert np.array_equal(got[~bad], want[~bad]) and np.isnan(got[bad]).all()


def test_refusals():
    import torch
    from outlier_aware_bit_amd import qlin as q
    log("rope, refusals")
    x, y, p = (dev(t) for t in _inputs(6, 10, 4, 2, 64, 50))
    freq, _ = q.qlin_rope_freqs(64)
    for err, kw in ((TypeError, dict(q=x.float())), (ValueError, dict(q=x.cpu())), (ValueError, dict(k=y[:5])),
                    (ValueError, dict(position=p[:5])), (TypeError, dict(position=p.long())),
                    (TypeError, dict(freq=freq.float())), (ValueError, dict(freq=freq[:, None])),
                    (q.QlinError, dict(freq=freq[:20].contiguous())), (ValueError, dict(q_out=x[:5])),
                    (ValueError, dict(k=None, k_out=y)), (q.QlinError, dict(q=x.repeat(1, 1, 2)[..., :96].contiguous(), k=None)),
                    (ValueError, dict(q=x[:, :, ::2])), (q.QlinError, dict(q=x[:1].expand(10, 4, 64)))):
        a = dict(q=x, k=y, position=p, freq=freq)
        a.update(kw)
        with pytest.raises(err):
            q.qlin_rope(**a)
    assert q.qlin_rope(x[:0], y[:0], p[:0], freq)[0].shape == (0, 4, 64)
    assert torch.cuda.current_device() == 0
