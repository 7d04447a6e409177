"""qlin_attn_prompt and its backward pass against the float64 oracle: types of
lengths, heads, windows, rows that see nothing, strides, values that are not
finite in places that a row does not see, gradients of every size, and that the
same call gives the same bits."""
import numpy as np
import pytest
import torch

from tests.gpu_helpers import dev, host, log
from tests.prompt_helpers import Packed, strided, within

pytestmark = pytest.mark.gpu

# nq, nk (None: the same), heads, kv heads, D, causal, window
CASES = [
    ([1], None, 1, 1, 64, True, 0), ([1], None, 4, 1, 128, True, 0), ([2], None, 2, 2, 256, True, 1),
    ([5], [9], 4, 2, 128, True, 0), ([9], [5], 4, 2, 128, True, 0),  # rows that see nothing
    ([63, 64, 65], None, 4, 2, 64, True, 0), ([127, 1, 128, 129], None, 2, 1, 128, True, 0),
    ([31, 32, 33, 200], None, 6, 2, 256, True, 0), ([300], None, 5, 1, 64, True, 37), ([150, 260], None, 2, 2, 128, True, 100),
    ([140], [400], 2, 1, 256, True, 150), ([40, 77], None, 4, 4, 128, False, 0), ([33], [190], 2, 1, 64, False, 0),
    ([10, 0, 20], [10, 30, 0], 4, 2, 128, True, 0),  # without queries, without keys
    ([10, 0, 20], [10, 30, 0], 2, 1, 64, False, 0), ([0, 0], None, 2, 1, 128, True, 0),
    ([3] * 70 + [40], None, 2, 1, 64, True, 0),  # more sequences than a search step looks at
    ([60], [1000], 2, 1, 64, True, 3), ([300], [290], 8, 8, 128, True, 64),
]


def _run(q, c, rows=strided, want_lse=True, **kw):
    x = [rows(t) for t in (c.q, c.k, c.v)]
    return x, q.qlin_attn_prompt(*x, dev(c.cu_q), dev(c.cu_k), scale=c.scale, causal=c.causal, window=c.window,
                                 want_lse=want_lse, **kw)


def _case(n, seed=0, **kw):
    nq, nk, heads, kv, D, causal, window = CASES[n]
    return Packed(n + seed, nq, nq if nk is None else nk, heads, kv, D, causal, window, **kw)


@pytest.mark.parametrize("n", range(len(CASES)))
def test_forward(n):
    from outlier_aware_bit_amd import qlin as q
    log(f"prompt attention {CASES[n]}")
    c = _case(n)
    _, (out, lse) = _run(q, c)
    want, tol, want_lse, lse_tol = c.forward()
    within(host(out), want, tol, "out")
    within(host(lse), want_lse, lse_tol, "lse")


@pytest.mark.parametrize("n", range(len(CASES)))
def test_backward(n):
    from outlier_aware_bit_amd import qlin as q
    log(f"prompt attention's gradients {CASES[n]}")
    c = _case(n)
    x, (out, lse) = _run(q, c)
    got = q.qlin_attn_prompt_backward(strided(c.dout), *x, out, lse, dev(c.cu_q), dev(c.cu_k), scale=c.scale,
                                      causal=c.causal, window=c.window)
    want, tol = c.backward()
    for name, g, w, t in zip(("dq", "dk", "dv"), got, want, tol):
        within(host(g), w, t, name)


@pytest.mark.parametrize("heads,kv,D,nq,nk,causal,window", [
    (8, 1, 64, [700], [700], True, 0), (8, 1, 128, [600, 0, 90], [900, 50, 0], True, 0), (4, 1, 256, [700], [700], False, 0),
    (8, 2, 128, [1100], [1100], True, 300), (6, 1, 128, [900], [300], True, 0), (5, 1, 256, [640, 3], [700, 200], True, 70)])
def test_gradients_of_few_keys(heads, kv, D, nq, nk, causal, window):
    # The queries of a key are divided among workgroups; rows of no sequence stay.
    from outlier_aware_bit_amd import qlin as q
    log(f"prompt attention's gradients, divided {heads} {kv} {D} {nq} {nk} {causal} {window}")
    c = Packed(31, nq, nk, heads, kv, D, causal, window, gap=3)
    x, (out, lse) = _run(q, c)
    Tq, Tk = c.q.shape[0], c.k.shape[0]
    need = q.qlin_attn_prompt_backward_work_bytes(heads, kv, D, len(nq), Tq, Tk, causal, window)
    assert need >= 2 * Tk * kv * D * 8
    runs = []
    for _ in range(2):
        dkv = torch.full((Tk, 2 * kv, D), 7.0, dtype=torch.float16, device="cuda")
        work = torch.full((need,), 255, dtype=torch.uint8, device="cuda")  # NaN, if it were read
        runs.append(q.qlin_attn_prompt_backward(strided(c.dout), *x, out, lse, dev(c.cu_q), dev(c.cu_k), scale=c.scale,
                                                causal=causal, window=window, dk=dkv[:, :kv], dv=dkv[:, kv:], work=work))
    want, tol = c.backward()
    for name, g, again, w, t, cu in zip(("dq", "dk", "dv"), *runs, want, tol, (c.cu_q, c.cu_k, c.cu_k)):
        assert torch.equal(g[cu[0]:cu[-1]], again[cu[0]:cu[-1]])
        within(host(g)[cu[0]:cu[-1]], w[cu[0]:cu[-1]], t[cu[0]:cu[-1]], name)
        if name != "dq":
            assert bool((g[:cu[0]] == 7.0).all()) and bool((g[cu[-1]:] == 7.0).all())


@pytest.mark.parametrize("D,nq,nk", [(256, [50], [6000]), (128, [1], [9000]), (64, [130, 7], [5000, 3001])])
def test_long_axis_of_few_rows(D, nq, nk):
    from outlier_aware_bit_amd import qlin as q
    log(f"prompt attention, {nq} queries of {nk} keys")
    c = Packed(D, nq, nk, 2, 1, D)
    assert q.qlin_attn_prompt_work_bytes(2, 1, D, len(nq), sum(nq), sum(nk)) > 0
    _, (out, lse) = _run(q, c)
    want, tol, want_lse, lse_tol = c.forward()
    within(host(out), want, tol, "out")
    within(host(lse), want_lse, lse_tol, "lse")


@pytest.mark.parametrize("scale", [0.0, -0.3, 1.0, 40.0])
def test_scales(scale):
    from outlier_aware_bit_amd import qlin as q
    log(f"prompt attention, scale {scale}")
    c = Packed(5, [90], [90], 2, 1, 64, scale=scale)
    x, (out, lse) = _run(q, c)
    want, tol, want_lse, lse_tol = c.forward()
    within(host(out), want, tol, "out")
    within(host(lse), want_lse, lse_tol, "lse")
    if abs(scale) <= 1.0:
        got = q.qlin_attn_prompt_backward(strided(c.dout), *x, out, lse, dev(c.cu_q), scale=scale)
        for name, g, w, t in zip(("dq", "dk", "dv"), got, *c.backward()):
            within(host(g), w, t, name)


def test_logits_far_apart_and_far_below_zero():
    # The running maximum moves by thousands, up and down; weights of the first keys vanish, or all but theirs.
    from outlier_aware_bit_amd import qlin as q
    log("prompt attention, logits of thousands")
    for sign in (1.0, -1.0):
        c = Packed(6, [400], [400], 2, 1, 128, scale=1.0)
        c.k[:] = (c.k.astype(np.float64) * 0.2).astype(np.float16)
        c.q[..., 7] = 60.0
        c.k[..., 7] = (sign * np.linspace(-50.0, 50.0, 400)[:, None]).astype(np.float16)
        _, (out, lse) = _run(q, c)
        want, tol, want_lse, lse_tol = c.forward()
        within(host(out), want, tol, "out")
        within(host(lse), want_lse, lse_tol, "lse")


@pytest.mark.parametrize("power", [-20, -12, 6])
def test_gradients_of_every_size(power):
    # dout of one row in eight is 2^14 larger still: ds of the others is small beside it.
    from outlier_aware_bit_amd import qlin as q
    log(f"prompt attention's gradients, dout times 2^{power}")
    c = Packed(8, [150], [150], 2, 1, 128)
    size = np.where(np.arange(150) % 8 == 5, 2.0 ** (power + 14 if power < 0 else power), 2.0 ** power)
    c.dout[:] = (c.dout.astype(np.float64) * size[:, None, None]).astype(np.float16)
    x, (out, lse) = _run(q, c)
    got = q.qlin_attn_prompt_backward(strided(c.dout), *x, out, lse, dev(c.cu_q))
    for name, g, w, t in zip(("dq", "dk", "dv"), got, *c.backward()):
        within(host(g), w, t, name)


def test_gradients_against_differences():
    from outlier_aware_bit_amd import qlin as q
    log("prompt attention's gradients against differences")
    c = Packed(9, [70, 33], [70, 33], 4, 2, 64, window=20)
    x, (out, lse) = _run(q, c)
    grads = [host(g).astype(np.float64) for g in q.qlin_attn_prompt_backward(strided(c.dout), *x, out, lse, dev(c.cu_q),
                                                                              window=20)]
    tols = c.backward()[1]
    rng = np.random.default_rng(0)
    for n, name in enumerate(("q", "k", "v")):
        base = getattr(c, name)
        u, h, loss = rng.standard_normal(base.shape), 1e-4, []
        for s in (h, -h):
            setattr(c, name, base.astype(np.float64) + s * u)
            loss.append(np.nansum(c.forward()[0] * c.dout.astype(np.float64)))
        setattr(c, name, base)
        # Central differences of a smooth function: off by h^2 times its third derivative, far below the rest.
        slope = (loss[0] - loss[1]) / (2 * h)
        assert abs(slope - (grads[n] * u).sum()) <= (tols[n] * np.abs(u)).sum() + 1e-4 * abs(slope), name


@pytest.mark.parametrize("D,window", [(64, 0), (128, 0), (128, 40), (256, 70)])
def test_values_that_are_not_finite_reach_only_rows_that_see_them(D, window):
    import torch
    from outlier_aware_bit_amd import qlin as q
    log(f"prompt attention, NaN and infinities, D={D}, window={window}")
    c = Packed(10, [150, 1, 300, 77], [150, 1, 300, 77], 4, 2, D, window=window)
    x, (out, _) = _run(q, c)
    want = host(out)
    for which in (1, 2):
        for value in (np.nan, np.inf, -np.inf):
            for at in (0, 60, 149, 150, 151, 280, 450, 527):
                y = list(x)
                y[which] = x[which].clone()
                y[which][at, 1, 3] = value
                got = host(q.qlin_attn_prompt(*y, dev(c.cu_q), window=window)[0])
                b = int((c.cu_q <= at).sum()) - 1
                sees = np.zeros(len(want), bool)
                sees[at:min(int(c.cu_q[b + 1]), at + window) if window else int(c.cu_q[b + 1])] = True
                assert np.array_equal(got[~sees], want[~sees]), (which, value, at)
                assert np.array_equal(got[:, :2], want[:, :2]), (which, value, at)
                if which == 2:
                    assert not np.isfinite(got[sees][:, 2:, 3]).any(), (value, at)
                    assert np.array_equal(np.delete(got, 3, 2), np.delete(want, 3, 2)), (value, at)
                elif np.isnan(value):
                    assert not np.isfinite(got[sees][:, 2:]).any(), at
    torch.cuda.synchronize()


def test_logits_of_minus_infinity_give_zeros():
    from outlier_aware_bit_amd import qlin as q
    log("prompt attention, logits of -inf")
    c = Packed(11, [40], [40], 2, 1, 64)
    c.q[...] = np.abs(c.q) + 1
    c.k[:20, :, 0] = -np.inf
    x, (out, lse) = _run(q, c)
    assert np.all(host(out)[:20] == 0.0) and np.all(np.isneginf(host(lse)[:, :20]))
    assert np.isfinite(host(out)[20:]).all() and np.isfinite(host(lse)[:, 20:]).all()


def test_a_value_that_is_not_finite_stays_in_its_sequence_backwards():
    from outlier_aware_bit_amd import qlin as q
    log("prompt attention's gradients, NaN in one sequence")
    c = Packed(12, [70, 90, 40], [70, 90, 40], 4, 2, 128)
    x, (out, lse) = _run(q, c)
    do = strided(c.dout)
    want = [host(g) for g in q.qlin_attn_prompt_backward(do, *x, out, lse, dev(c.cu_q))]
    for which in range(4):
        y = [t.clone() for t in (do, *x)]
        y[which][100, 1, 5] = np.nan
        got = [host(g) for g in q.qlin_attn_prompt_backward(y[0], *y[1:], out, lse, dev(c.cu_q))]
        for g, w in zip(got, want):
            assert np.array_equal(g[:70], w[:70]) and np.array_equal(g[160:], w[160:]), which
        assert not all(np.isfinite(g[70:160]).all() for g in got), which


def test_rows_of_no_sequence_are_left():
    import torch
    from outlier_aware_bit_amd import qlin as q
    log("prompt attention, rows before and behind the sequences")
    c = Packed(13, [50, 20], [60, 20], 2, 1, 64, gap=9)
    out = torch.full(c.q.shape, 3.0, dtype=torch.float16, device="cuda")
    lse = torch.full((2, len(c.q)), 5.0, device="cuda")
    x, _ = _run(q, c, out=out, lse=lse, want_lse=False)
    want, tol, want_lse, lse_tol = c.forward()
    within(host(out), want, tol, "out")
    within(host(lse), want_lse, lse_tol, "lse")
    for t in (host(out), host(lse).T):
        assert np.all(t[:9] == t[0]) and np.all(t[79:] == t[0])
    qkv = torch.full((len(c.k), 4, 64), 2.0, dtype=torch.float16, device="cuda")  # dk and dv as slices, a gap behind them
    dq = torch.full(c.q.shape, 2.0, dtype=torch.float16, device="cuda")
    q.qlin_attn_prompt_backward(strided(c.dout), *x, out, lse, dev(c.cu_q), dev(c.cu_k), dq=dq, dk=qkv[:, 1:2],
                                dv=qkv[:, 2:3])
    grads, tol = c.backward()
    for name, g, w, t, n in zip(("dq", "dk", "dv"), (dq, qkv[:, 1:2], qkv[:, 2:3]), grads, tol, (70, 80, 80)):
        within(host(g)[9:9 + n], w[9:9 + n], t[9:9 + n], name)
        assert np.all(host(g)[:9] == 2.0) and np.all(host(g)[9 + n:] == 2.0)
    assert np.all(host(qkv)[:, [0, 3]] == 2.0)


def test_the_same_call_gives_the_same_bits_whatever_stands_beside_it():
    import torch
    from outlier_aware_bit_amd import qlin as q
    log("prompt attention, bits")
    c = Packed(14, [200, 333, 5], [200, 333, 5], 4, 2, 128)
    x, (out, lse) = _run(q, c)
    do = strided(c.dout)
    cu = dev(c.cu_q)
    first = [out, lse, *q.qlin_attn_prompt_backward(do, *x, out, lse, cu)]
    for _ in range(3):
        out2, lse2 = q.qlin_attn_prompt(*x, cu, want_lse=True)
        again = [out2, lse2, *q.qlin_attn_prompt_backward(do, *x, out2, lse2, cu)]
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    # Another sequence in front: the others' rows keep their bits.
    y = [strided(np.concatenate([t[:200] * np.float16(9), t])) for t in (c.q, c.k, c.v)]
    cu2 = dev(np.concatenate([[0], c.cu_q + 200]).astype(np.int32))
    got, _ = q.qlin_attn_prompt(*y, cu2)
    assert torch.equal(got[200:], out)


def test_borders_past_the_arrays_stay_inside_them():
    import torch
    from outlier_aware_bit_amd import qlin as q
    log("prompt attention, borders past the arrays")
    c = Packed(15, [60], [60], 2, 1, 64)
    x, (out, lse) = _run(q, c)
    for cu in ([0, 1000], [-5, 60], [0, 60]):
        got, _ = q.qlin_attn_prompt(*x, dev(np.array(cu, np.int32)), want_lse=True)
        assert torch.equal(got, out)
        grads = q.qlin_attn_prompt_backward(strided(c.dout), *x, out, lse, dev(np.array(cu, np.int32)))
        assert all(torch.isfinite(g).all() for g in grads)


def test_refusals():
    import torch
    from outlier_aware_bit_amd import qlin as q
    log("prompt attention, refusals")
    c = Packed(16, [20], [20], 4, 2, 64)
    x, (out, lse) = _run(q, c)
    cu, do = dev(c.cu_q), strided(c.dout)
    bad = [(TypeError, dict(q=x[0].float())), (ValueError, dict(k=x[1][:, :1, :])), (ValueError, dict(v=x[2][:10])),
           (ValueError, dict(q=x[0].cpu())), (ValueError, dict(k=x[1].cpu())), (TypeError, dict(cu_q=cu.long())),
           (ValueError, dict(cu_k=dev(np.array([0, 10, 20], np.int32)))), (ValueError, dict(out=out[:10])),
           (q.QlinError, dict(window=-1)), (q.QlinError, dict(window=3, causal=False)),
           (q.QlinError, dict(scale=float("nan"))), (ValueError, dict(q=x[0].transpose(0, 1))),
           (TypeError, dict(lse=lse.double()))]
    for err, kw in bad:
        a = dict(q=x[0], k=x[1], v=x[2], cu_q=cu)
        a.update(kw)
        with pytest.raises(err):
            q.qlin_attn_prompt(**a)
    with pytest.raises(ValueError, match="workspace|work"):
        y = Packed(17, [1], [9000], 2, 1, 64)
        q.qlin_attn_prompt(*(dev(t) for t in (y.q, y.k, y.v)), dev(y.cu_q), dev(y.cu_k),
                           work=torch.empty(16, dtype=torch.uint8, device="cuda"))
    for err, kw in ((ValueError, dict(dout=do[:5])), (TypeError, dict(lse=lse.half())), (ValueError, dict(out=out[:, :2])),
                    (ValueError, dict(dq=out[:3])), (TypeError, dict(dv=x[2].float())),
                    (ValueError, dict(work=torch.empty(8, dtype=torch.uint8, device="cuda")))):
        a = dict(dout=do, q=x[0], k=x[1], v=x[2], out=out, lse=lse, cu_q=cu)
        a.update(kw)
        with pytest.raises(err):
            q.qlin_attn_prompt_backward(**a)


def test_empty_calls():
    import torch
    from outlier_aware_bit_amd import qlin as q
    log("prompt attention, nothing to do")
    c = Packed(18, [], [], 2, 1, 64, gap=3)
    x, (out, _) = _run(q, c, out=torch.full(c.q.shape, 3.0, dtype=torch.float16, device="cuda"))
    assert torch.all(out == 3.0)
    e = torch.empty(0, 2, 64, dtype=torch.float16, device="cuda")
    cu = torch.zeros(2, dtype=torch.int32, device="cuda")
    assert q.qlin_attn_prompt(e, e, e, cu)[0].shape == (0, 2, 64)
    # Queries without any key, and keys without any query.
    y = torch.ones(5, 2, 64, dtype=torch.float16, device="cuda")
    five = torch.tensor([0, 5], dtype=torch.int32, device="cuda")
    out, lse = q.qlin_attn_prompt(y, e, e, five, cu, want_lse=True)
    assert torch.all(out == 0.0) and torch.all(torch.isneginf(lse))
    dq, dk, _ = q.qlin_attn_prompt_backward(y, y, e, e, out, lse, five, cu)
    assert torch.all(dq == 0.0) and dk.shape == (0, 2, 64)
    none = torch.empty(2, 0, device="cuda")
    dq, dk, dv = q.qlin_attn_prompt_backward(e, e, y, y, e, none, cu, five)
    assert torch.all(dk == 0.0) and torch.all(dv == 0.0) and dq.shape == (0, 2, 64)


def test_offsets_past_32_bits():
    # Tokens 2^22 elements apart: 700 of them pass 2^31 elements, in every tensor that may be strided.
    import torch
    from outlier_aware_bit_amd import qlin as q
    log("prompt attention, offsets past 2^31")
    c = Packed(19, [500, 200], [500, 200], 2, 1, 64)
    ld, T = 1 << 22, 700
    room = torch.empty((T, ld), dtype=torch.float16, device="cuda")
    at = [0]

    def far(x):
        n = x.shape[1] * x.shape[2]
        view = room[:, at[0]:at[0] + n].unflatten(1, x.shape[1:])
        at[0] += n
        view.copy_(dev(x) if isinstance(x, np.ndarray) else x)
        return view

    x = [far(t) for t in (c.q, c.k, c.v)]
    out, lse = q.qlin_attn_prompt(*x, dev(c.cu_q), want_lse=True)
    want, tol, want_lse, lse_tol = c.forward()
    within(host(out), want, tol, "out")
    within(host(lse), want_lse, lse_tol, "lse")
    grads = [far(torch.zeros(t.shape, dtype=torch.float16, device="cuda")) for t in x]
    q.qlin_attn_prompt_backward(far(c.dout), *x, out, lse, dev(c.cu_q), dq=grads[0], dk=grads[1], dv=grads[2])
    for name, g, w, t in zip(("dq", "dk", "dv"), grads, *c.backward()):
        within(host(g), w, t, name)
    freq, _ = q.qlin_rope_freqs(64)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    near = q.qlin_rope(x[0].contiguous(), x[1].contiguous(), pos, freq)
    got = q.qlin_rope(x[0], x[1], pos, freq, q_out=x[0], k_out=x[1])
    assert all(torch.equal(a, b) for a, b in zip(near, got))
