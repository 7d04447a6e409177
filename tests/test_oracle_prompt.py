"""The oracle's rotary positions, prompt attention, slot maps and page tables,
against closed forms, hand-worked cases and differences."""
import math

import numpy as np
import pytest

from oracle import prompt


def test_a_quarter_turn_by_hand():
    x = np.array([[[1.0, 2.0, 3.0, 4.0, 5.0]]])
    freq = np.array([math.pi / 2, 0.0])
    half = prompt.rope(x, [1], freq)
    assert np.allclose(half, [[[-3.0, 2.0, 1.0, 4.0, 5.0]]], atol=1e-15)
    pairs = prompt.rope(x, [1], freq, interleaved=True)
    assert np.allclose(pairs, [[[-2.0, 1.0, 3.0, 4.0, 5.0]]], atol=1e-15)
    assert np.array_equal(prompt.rope(x, [-1], freq), x)


@pytest.mark.parametrize("interleaved", [False, True])
def test_turning_back_and_scores_by_distance(interleaved):
    rng = np.random.default_rng(0)
    freq, _ = prompt.rope_freqs(16)
    q, k = rng.standard_normal((2, 1, 1, 32))

    def turned(x, p, **kw):
        return prompt.rope(x, [p], freq, interleaved, **kw)

    assert np.allclose(turned(turned(q, 91), 91, inverse=True), q, atol=1e-13)
    a = (turned(q, 100) * turned(k, 70)).sum()
    assert abs(a - (turned(q, 30) * turned(k, 0)).sum()) < 1e-12
    # The inverse is the transposed map: <u, turn(x)> = <turn back(u), x>.
    u = rng.standard_normal((1, 1, 32))
    left = (u * turned(q, 77, amplitude=1.3)).sum()
    assert abs(left - (turned(u, 77, inverse=True, amplitude=1.3) * q).sum()) < 1e-12


def test_frequencies():
    f, amp = prompt.rope_freqs(8, base=16.0)
    assert np.allclose(f, [1.0, 0.5, 0.25, 0.125]) and amp == 1.0
    assert np.allclose(prompt.rope_freqs(8, base=16.0, scaling="linear", factor=4.0)[0], f / 4.0)
    g, _ = prompt.rope_freqs(8, base=16.0, scaling="base", factor=4.0)
    assert g[0] == 1.0 and math.isclose(g[-1], f[-1] / 4.0)
    g, amp = prompt.rope_freqs(128, scaling="ramp", factor=16.0, original_len=8192)
    f, _ = prompt.rope_freqs(128)
    assert g[0] == f[0] and math.isclose(g[-1], f[-1] / 16.0) and math.isclose(amp, 0.1 * math.log(16.0) + 1.0)
    assert np.all(np.diff(g / f) <= 1e-15)


def test_visible_by_hand():
    assert prompt.visible(2, 4).tolist() == [[True, True, True, False], [True] * 4]
    assert prompt.visible(2, 4, window=2).tolist() == [[False, True, True, False], [False, False, True, True]]
    assert prompt.visible(3, 2).tolist() == [[False, False], [True, False], [True, True]]  # a row sees nothing
    assert prompt.visible(1, 0).shape == (1, 0)


@pytest.mark.parametrize("nq,nk,window", [(5, 5, 0), (3, 7, 0), (6, 4, 0), (5, 5, 2), (1, 1, 0)])
def test_attention_against_the_sum_itself(nq, nk, window):
    rng = np.random.default_rng(nq)
    q, k, v = rng.standard_normal((nq, 4)), rng.standard_normal((nk, 4)), rng.standard_normal((nk, 4))
    see = prompt.visible(nq, nk, True, window)
    out, lse, _ = prompt.attend(q, k, v, 0.7, see)
    for i in range(nq):
        w = [math.exp(0.7 * float(q[i] @ k[j])) if see[i, j] else 0.0 for j in range(nk)]
        if sum(w) == 0.0:
            assert np.all(out[i] == 0.0) and lse[i] == -np.inf
        else:
            assert np.allclose(out[i], sum(a * b for a, b in zip(w, v)) / sum(w)) and math.isclose(lse[i], math.log(sum(w)))


def test_hidden_keys_take_no_part():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((3, 4, 4))
    see = prompt.visible(4, 4)
    out = prompt.attend(q, k, v, 1.0, see)[0]
    k[3], v[3] = np.nan, np.inf
    assert np.array_equal(prompt.attend(q, k, v, 1.0, see)[0][:3], out[:3])


@pytest.mark.parametrize("nq,nk,window", [(4, 4, 0), (3, 6, 0), (5, 3, 0), (6, 6, 3)])
def test_gradients_against_differences(nq, nk, window):
    rng = np.random.default_rng(nk)
    x = [rng.standard_normal((n, 4)) for n in (nq, nk, nk)]
    dout, see = rng.standard_normal((nq, 4)), prompt.visible(nq, nk, True, window)
    grads = prompt.attend_grad(dout, *x, 0.6, see)
    h = 1e-5
    for n in range(3):
        for at in np.ndindex(x[n].shape):
            was = x[n][at]
            loss = []
            for s in (h, -h):
                x[n][at] = was + s
                loss.append((prompt.attend(*x, 0.6, see)[0] * dout).sum())
            x[n][at] = was
            assert abs((loss[0] - loss[1]) / (2 * h) - grads[n][at]) < 1e-8, (n, at)


def test_slots_by_hand():
    cu, row, slot, pos, lens = prompt.slots([5, 0, 2], [2, 0, 3], 7, [9, 1, 4])
    assert (cu, row, slot) == ([0, 2, 2, 5], [0, 0, 2, 2, 2, -1, -1], [5, 6, 2, 3, 4, -1, -1])
    assert (pos, lens) == ([9, 10, 4, 5, 6, -1, -1], [7, 0, 5])
    cu, row, slot, pos, lens = prompt.slots([5, -3], [2, 4], 3)  # no room behind three tokens
    assert (cu, row, slot, pos, lens) == ([0, 2, 3], [0, 0, 1], [5, 6, 0], [5, 6, 0], [7, 1])


def test_pages_by_hand():
    table = [[7, -1, -1], [1, 2, 3], [4, -1, -1], [-1, -1, -1]]
    ring = [10, -1, -1, 8, 9]  # 8, 9, 10 are free, from 3 on around the end
    got = prompt.pages([33, 10, 0, 100], 16, table, [1, 3, 1, 0], ring, 3, 3)
    # Row 0 takes 8 and 9; rows 1 and 2 give 2, 3 and 4 back; row 3 would need seven of three entries.
    assert got == ([[7, 8, 9], [1, -1, -1], [-1, -1, -1], [-1, -1, -1]], [3, 1, 0, 0], [10, 2, 3, 4, 9], 0, 4, 7)
    # The first row that finds too few stops the later ones.
    got = prompt.pages([48, 48, 16], 16, [[-1] * 3] * 3, [0, 0, 0], [5, 6, 7, 8], 0, 4)
    assert got == ([[5, 6, 7], [-1] * 3, [-1] * 3], [3, 0, 0], [5, 6, 7, 8], 3, 1, 4)
