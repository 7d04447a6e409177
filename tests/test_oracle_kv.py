"""The key/value cache oracle against closed forms, exact rationals and brute
force (CPU)."""
import math
from fractions import Fraction

import numpy as np
import pytest

from oracle import hadamard, kv
from tests.exact import f16, f32, rint_half_even


def test_butterfly_is_the_sylvester_product_on_integers():
    rng = np.random.default_rng(0)
    x = rng.integers(-50, 50, (5, 128)).astype(np.float16)
    d = rng.choice([-1, 1], 128).astype(np.int8)
    d[0] = 1
    want = x.astype(np.int64) @ hadamard.partial_random(d)
    assert np.array_equal(kv.butterfly128(x, d), want.astype(np.float32))
    # A lone outlier in channel 0 becomes the same offset everywhere.
    e = np.zeros((1, 128), np.float16)
    e[0, 0] = 300
    assert np.array_equal(kv.butterfly128(e, d), np.full((1, 128), 300, np.float32))


@pytest.mark.parametrize("bits", [4, 8])
def test_row_codes_in_exact_arithmetic(bits):
    rng = np.random.default_rng(bits)
    rows = np.concatenate([rng.standard_normal((6, 16)), 100 * rng.standard_normal((2, 16)),
                           np.full((1, 16), 0.3)]).astype(np.float16).astype(np.float32)
    codes, meta = kv.quant_rows(rows, bits)
    qmax = 2 ** bits - 1
    for r, c, m in zip(rows, codes, meta):
        t = [Fraction(float(v)) for v in r]
        lo = f16(min(t))
        step = f16(f32(f32(max(t) - lo) * f32(Fraction(1, qmax))))
        assert Fraction(float(m[0])) == step and Fraction(float(m[1])) == lo
        for v, got in zip(t, c):
            want = 0
            if step != 0:
                want = min(qmax, max(0, rint_half_even(f32(f32(v - lo) * f32(1 / step)))))
            assert got == want


@pytest.mark.parametrize("bits", [4, 8])
def test_a_code_stands_within_half_a_step_of_its_value(bits):
    rows = np.random.default_rng(3).standard_normal((50, 64)).astype(np.float16).astype(np.float32)
    codes, meta = kv.quant_rows(rows, bits)
    err = np.abs(kv.dequant_rows(codes, meta) - rows)
    step = meta[..., :1].astype(np.float64)
    # Half a step, plus what rounding the step to fp16 loses over the range.
    assert np.all(err <= step * (0.5 + (2 ** bits - 1) * 2.0 ** -11 + 1e-4))
    assert np.array_equal(kv.unpack4(kv.pack4(codes & 15)), codes & 15)


def test_attend_against_a_loop():
    rng = np.random.default_rng(4)
    q, k, v = rng.standard_normal((2, 8)), rng.standard_normal((7, 8)), rng.standard_normal((7, 8))
    use = np.array([1, 1, 0, 1, 0, 1, 1], bool)
    out, p = kv.attend(q, k, v, 0.5, use)
    for g in range(2):
        w = [math.exp(0.5 * sum(q[g, d] * k[i, d] for d in range(8))) if use[i] else 0.0 for i in range(7)]
        assert np.allclose(p[g], np.array(w) / sum(w), rtol=1e-12)
        assert np.allclose(out[g], sum(w[i] * v[i] for i in range(7)) / sum(w), rtol=1e-12)
    out, p = kv.attend(q, k, v, 0.5, np.zeros(7, bool))
    assert not out.any() and not p.any()
    k[:, 0] = -np.inf  # every logit -inf
    out, p = kv.attend(np.abs(q), k, v, 0.5)
    assert not out.any() and not p.any()


def test_evict_small_cases_by_hand():
    m = np.array([5, 1, 9, 3, 7], np.float32)
    p = np.arange(5)
    assert kv.evict(m, p, 3, 0)[1].tolist() == [0, 4, 2]      # 1 and 3 go, 4 fills 1
    assert kv.evict(m, p, 3, 2)[1].tolist() == [3, 4, 2]      # 3 and 4 are newest, then 2
    assert kv.evict(m, p, 5, 2)[1].tolist() == [0, 1, 2, 3, 4]
    assert kv.evict(m, p, 8, 2)[0] == 5
    ties = np.array([2, 2, 2, 2], np.float32)
    assert kv.evict(ties, np.arange(4), 2, 0)[1].tolist() == [0, 1]
    assert kv.evict(ties, np.arange(4)[::-1], 2, 1)[1].tolist() == [0, 1]
    bad = np.array([np.nan, -np.inf, 0, -1], np.float32)
    assert kv.evict(bad, np.arange(4), 3, 0)[1].tolist() == [3, 1, 2]
    assert kv.evict(m[:0], p[:0], 3, 1)[0] == 0


def test_evict_keeps_the_largest_total():
    rng = np.random.default_rng(5)
    for _ in range(20):
        n = int(rng.integers(1, 30))
        budget, m = int(rng.integers(1, 30)), rng.random(n).astype(np.float32)
        recent = int(rng.integers(0, budget + 1))
        pos = rng.permutation(n)
        left, src = kv.evict(m, pos, budget, recent)
        assert left == min(n, budget) and len(set(src.tolist())) == left
        late = [i for i in range(n) if pos[i] >= n - recent]
        assert len(late) > left or set(late) <= set(src.tolist())
        rest = sorted((m[i] for i in range(n) if i not in late), reverse=True)
        got = sorted((m[i] for i in src if i not in late), reverse=True)
        assert got == rest[:len(got)]
        moved = [(j, s) for j, s in enumerate(src) if s != j]
        assert all(s >= left for _, s in moved)
        assert [s for _, s in moved] == sorted(s for _, s in moved)
