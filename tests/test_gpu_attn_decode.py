"""Attention of one new token over the paged key/value cache
(qlin_attn_decode) against the float64 oracle.

Bounds, from the arithmetic the header states (all elementwise):
* a logit is an fp32 sum of D exact fp16 products (and the row's lo term): off
  by at most ds = (D + 8) 2^-23 scale sum_d |q_d| |k_d|, plus, with the
  Hadamard, 2^-20 of that sum for q in two fp16 parts;
* a weight is then off by a factor e^(2 ds) - 1 <= 4 ds, and by 2^-18 for exp2,
  the fp32 sums over the slots and P in two fp16 parts;
* weights below 2^-31 of the largest may vanish: n 2^-31 max|v|;
* the output is rounded once to fp16: 2^-11 |o| + 2^-25.
"""
import numpy as np
import pytest

from oracle import kv
from tests.gpu_helpers import assert_equal, dev, host, log
from tests.kv_helpers import HostCache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    import torch
    assert torch.cuda.is_available()
    from outlier_aware_bit_amd import qlin
    return qlin


def _use(n, window):
    use = np.ones(n, bool)
    if window:
        use[:max(0, n - window)] = False
    return use


def _bounds(c, b, h, qs, scale, use, out, p):
    """(elementwise bound of out [G, D], of the weights [G, n])."""
    k, v = c.values[b][0][h], c.values[b][1][h]
    prods = np.abs(qs) @ np.abs(k).T
    if c.bits < 16:
        # lo * sum q and step * code . q are separate terms.
        m = np.abs(c.values[b][0][h]).max(1)[None, :] * np.abs(qs).sum(1)[:, None]
        prods = prods + 2 * m
    ds = ((c.D + 8) * 2.0 ** -23 + (2.0 ** -20 if c.signs is not None else 0)) * scale * prods
    ds = np.where(use[None, :], ds, 0).max(1, initial=0)[:, None]
    rel = 4 * ds + 2.0 ** -18
    vmag = np.abs(v) + (2 * np.abs(v).max(1, initial=0)[:, None] if c.bits < 16 else 0)
    vmax = vmag[use].max(initial=0)
    tol_o = 2.0 ** -11 * np.abs(out) + rel * (p @ vmag) + len(v) * 2.0 ** -31 * vmax + 2.0 ** -25
    return tol_o, rel * p + 2.0 ** -31


def _check(q, c, group, window=0, max_len=None, ld_pad=0, mass=True, scale=None, seed=0, qstd=1.0, out_only=False):
    import torch
    rng = np.random.default_rng(seed)
    B, heads = len(c.lens), c.heads * group
    scale = c.D ** -0.5 if scale is None else scale
    qh = (rng.standard_normal((B, heads, c.D)) * qstd).astype(np.float16)
    wide = np.concatenate([qh, rng.standard_normal((B, 2, c.D)).astype(np.float16)], 1) if ld_pad else qh
    qd = dev(wide)[:, :heads]
    max_len = c.max_pages * c.page if max_len is None else max_len
    ld = c.max_pages * c.page + 3
    m_in = rng.random((B, c.heads, ld)).astype(np.float32)
    m_out = torch.full((B, c.heads, ld), -7.0, device="cuda") if mass else None
    cache, table, lens = c.device(q), dev(c.table), dev(c.lens)
    out, got_mass = q.qlin_attn_decode(cache, qd, table, lens, max_len, scale=scale, window=window,
                                       mass=dev(m_in) if mass else None, mass_out=m_out)
    got = host(out).astype(np.float64)
    assert got.shape == (B, heads, c.D)
    worst = 0.0
    for b in range(B):
        n = int(min(max(c.lens[b], 0), max_len))
        for h in range(c.heads):
            qs = c.turn(qh[b, h * group:(h + 1) * group])
            k, v = c.values[b][0][h][:n], c.values[b][1][h][:n]
            use = _use(n, window)
            ref, p = kv.attend(qs, k, v, scale, use)
            sub = HostView(c, b, n)
            tol_o, tol_p = _bounds(sub, 0, h, qs, scale, use, ref, p)
            err = np.abs(got[b, h * group:(h + 1) * group] - ref)
            assert np.all(err <= tol_o), (b, h, float((err / tol_o).max()))
            worst = max(worst, float((err / tol_o).max(initial=0)))
            if mass:
                gm = host(got_mass[b, h]).astype(np.float64)
                want = m_in[b, h, :n].astype(np.float64) + p.sum(0)
                tol = tol_p.sum(0) + 2.0 ** -22 * want
                assert np.all(np.abs(gm[:n] - want) <= tol), (b, h, "mass")
                assert np.all(gm[n:] == -7.0), (b, h, "mass past the length")
    # Without mass, and again: the same bits.
    again, none = q.qlin_attn_decode(cache, qd, table, lens, max_len, scale=scale, window=window)
    assert none is None
    assert_equal(host(again).view(np.uint16), host(out).view(np.uint16), "a second call")
    return worst


class HostView:
    """One row of a cache, cut to n slots."""

    def __init__(self, c, b, n):
        self.D, self.bits, self.signs = c.D, c.bits, c.signs
        self.values = [tuple(x[:, :n] for x in c.values[b])]


SHAPES = [(16, 64, False), (16, 128, False), (16, 256, False), (8, 64, False), (8, 128, False), (8, 128, True),
          (8, 256, False), (4, 64, False), (4, 128, False), (4, 128, True), (4, 256, False)]


@pytest.mark.parametrize("bits,D,rotate", SHAPES)
def test_lengths_and_pages(q, bits, D, rotate):
    for page, group, heads in [(16, 1, 3), (32, 4, 2), (64, 5, 1)]:
        rng = np.random.default_rng(page + D + bits)
        lens = [0, 1, 7, 8, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 129, 200]
        log(f"attend lengths bits={bits} D={D} rotate={rotate} page={page} group={group}")
        c = HostCache(rng, lens, 200, heads, D, page, bits, rotate)
        log(f"  worst {_check(q, c, group, ld_pad=2, seed=page):.3f} of the bound")


@pytest.mark.parametrize("bits,D,rotate", SHAPES)
def test_long_rows_are_split_and_joined(q, bits, D, rotate):
    rng = np.random.default_rng(1000 + D + bits)
    log(f"attend long bits={bits} D={D} rotate={rotate}")
    c = HostCache(rng, [2049, 513, 0, 5000], 5000, 2, D, 128, bits, rotate)
    log(f"  worst {_check(q, c, 4, seed=1):.3f} of the bound")


@pytest.mark.parametrize("group", [1, 2, 3, 7, 8, 9, 16, 20])
def test_groups(q, group):
    for bits in (16, 8, 4):
        log(f"attend group={group} bits={bits}")
        rng = np.random.default_rng(group)
        c = HostCache(rng, [70, 600, 3], 600, 2, 128, 16, bits, bits == 4)
        _check(q, c, group, seed=group)


def test_more_query_heads_than_a_workgroup_takes(q):
    for group in (33, 40, 64):
        rng = np.random.default_rng(group)
        log(f"attend group={group}")
        c = HostCache(rng, [5, 700, 0, 300], 700, 2, 64, 16, 8)
        _check(q, c, group, seed=group)
        c = HostCache(rng, [5, 100], 100, 1, 64, 16, 8)  # one workgroup a row
        _check(q, c, group, seed=group)


@pytest.mark.parametrize("B", [63, 65, 200])
def test_many_ragged_sequences(q, B):
    # Runs of tiles that begin and end anywhere, idle rows at both ends and
    # between, and more sequences than a wave has lanes.
    rng = np.random.default_rng(B)
    lens = rng.integers(0, 900, B)
    lens[rng.random(B) < 0.3] = 0
    lens[:2], lens[-2:] = 0, 0
    log(f"attend B={B}")
    _check(q, HostCache(rng, lens, 900, 1, 64, 32, 4), 2, seed=B)
    lens[:] = 0
    lens[B // 2] = 600
    _check(q, HostCache(rng, lens, 900, 3, 64, 16, 16), 1, seed=B)
    lens[:] = 0
    _check(q, HostCache(rng, lens, 900, 1, 64, 16, 16), 1, seed=B)


@pytest.mark.parametrize("window", [1, 31, 32, 100, 511, 5000])
def test_windows(q, window):
    for bits in (16, 8, 4):
        log(f"attend window={window} bits={bits}")
        rng = np.random.default_rng(window)
        c = HostCache(rng, [0, 1, 33, 100, 101, 1300], 1300, 2, 64 if bits == 8 else 128, 32, bits)
        _check(q, c, 2, window=window, seed=window)


def test_lengths_beyond_the_bounds_are_cut(q):
    rng = np.random.default_rng(5)
    c = HostCache(rng, [100, 64, 30], 100, 2, 128, 16, 4)
    _check(q, c, 2, max_len=64)  # lens above max_len
    c.lens = np.array([100, -5, 30], np.int32)
    _check(q, c, 2)


def test_large_logits_and_weights_that_vanish(q):
    for bits in (16, 8, 4):
        rng = np.random.default_rng(6 + bits)
        c = HostCache(rng, [300, 65], 300, 2, 128, 16, bits, False)
        log(f"attend sharp bits={bits}")
        _check(q, c, 4, scale=4.0, qstd=2.0, seed=6)
        _check(q, c, 4, scale=0.0, seed=7)      # every slot the same weight
        _check(q, c, 4, scale=-0.05, seed=8)


def test_steps_of_very_different_size(q):
    # Rows of V whose steps span fp16's range, the large ones last.
    for bits in (8, 4):
        rng = np.random.default_rng(9)
        c = HostCache(rng, [700], 700, 1, 128, 16, bits)
        k, v = c.values[0]
        mag = 10.0 ** np.linspace(-4, 3, 700)
        rows = (rng.standard_normal((1, 700, 128)) * mag[None, :, None]).astype(np.float16)
        c.values[0] = (k, c._put(0, "v", rows))
        _check(q, c, 4, seed=9, scale=0.01)


def test_unmapped_pages_have_no_weight(q):
    for bits in (16, 4):
        rng = np.random.default_rng(11)
        c = HostCache(rng, [100, 100], 100, 2, 128, 16, bits)
        for bad in (-1, c.pages, 2147483647, -2147483648):
            c2 = HostCache(np.random.default_rng(11), [100, 100], 100, 2, 128, 16, bits)
            c2.table[0, 2] = bad      # slots 32 .. 47 do not exist
            c2.table[1, :] = bad      # nothing does
            cache, table, lens = c2.device(q), dev(c2.table), dev(c2.lens)
            qh = rng.standard_normal((2, 4, 128)).astype(np.float16)
            out, _ = q.qlin_attn_decode(cache, dev(qh), table, lens, 112, scale=0.1)
            got = host(out).astype(np.float64)
            use = np.ones(100, bool)
            use[32:48] = False
            for h in range(2):
                qs = qh[0, 2 * h:2 * h + 2].astype(np.float64)
                ref, p = kv.attend(qs, c2.values[0][0][h], c2.values[0][1][h], 0.1, use)
                tol, _ = _bounds(HostView(c2, 0, 100), 0, h, qs, 0.1, use, ref, p)
                assert np.all(np.abs(got[0, 2 * h:2 * h + 2] - ref) <= tol)
            assert not got[1].any()


def test_infinite_logits_and_values(q):
    rng = np.random.default_rng(12)
    c = HostCache(rng, [50, 50, 50, 50], 50, 1, 128, 16, 16, outliers=False)
    for b in range(4):
        k, v = c.values[b]
        kf, vf = k.astype(np.float16), v.astype(np.float16)
        if b == 0:
            kf[0, :, 0] = -np.inf      # with q[0] > 0 every logit is -inf: zero
        if b == 1:
            kf[0, 10:, 0] = -np.inf    # only ten slots have weight
        if b == 2:
            vf[0, 20, 3] = np.inf      # one infinite channel of V
        if b == 3:
            vf[0, 20, 3] = np.nan
        c.values[b] = (c._put(b, "k", kf), c._put(b, "v", vf))
    qh = np.abs(rng.standard_normal((4, 1, 128))).astype(np.float16)
    out, _ = q.qlin_attn_decode(c.device(q), dev(qh), dev(c.table), dev(c.lens), 64, scale=0.02)
    got = host(out).astype(np.float64)
    assert not got[0].any()
    use = np.arange(50) < 10
    ref, p = kv.attend(qh[1].astype(np.float64), c.values[1][0][0], c.values[1][1][0], 0.02, use)
    assert np.allclose(got[1], ref, rtol=2 ** -9, atol=1e-3)
    assert np.isposinf(got[2, 0, 3]) and np.isfinite(np.delete(got[2, 0], 3)).all()
    assert np.isnan(got[3, 0, 3]) and np.isfinite(np.delete(got[3, 0], 3)).all()


def test_mass_in_place_and_without_input(q):
    import torch
    rng = np.random.default_rng(13)
    c = HostCache(rng, [40, 300], 300, 2, 128, 16, 4, True)
    qd = dev(rng.standard_normal((2, 8, 128)).astype(np.float16))
    args = (c.device(q), qd, dev(c.table), dev(c.lens), 300)
    zero = torch.zeros((2, 2, 304), device="cuda")
    _, first = q.qlin_attn_decode(*args, mass_out=torch.zeros_like(zero))
    _, same = q.qlin_attn_decode(*args, mass=zero, mass_out=torch.zeros_like(zero))
    assert_equal(host(first), host(same), "mass without input")
    m = dev(rng.random((2, 2, 304)).astype(np.float32))
    _, apart = q.qlin_attn_decode(*args, mass=m, mass_out=m.clone())
    q.qlin_attn_decode(*args, mass=m, mass_out=m)
    assert_equal(host(m), host(apart), "mass in place")
    # A sequence's weights sum to its query heads.
    assert np.allclose(host(first).sum(2), 4.0, rtol=1e-5)


def test_another_stream_and_own_workspace(q):
    import torch
    rng = np.random.default_rng(14)
    c = HostCache(rng, [1000, 20], 1000, 2, 128, 16, 8)
    cache, table, lens = c.device(q), dev(c.table), dev(c.lens)
    qd = dev(rng.standard_normal((2, 4, 128)).astype(np.float16))
    want, _ = q.qlin_attn_decode(cache, qd, table, lens, 1000)
    need = q.qlin_attn_decode_work_bytes(cache, 4, 2, 1000)
    work = torch.full((need,), 255, dtype=torch.uint8, device="cuda")  # NaN in every word
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got, _ = q.qlin_attn_decode(cache, qd, table, lens, 1000, work=work)
    st.synchronize()
    assert_equal(host(got).view(np.uint16), host(want).view(np.uint16), "another stream")


def test_offsets_past_32_bits(q):
    import torch
    # 5 GiB of rows per array; the sequence lives in the first and last pages.
    pages, heads, page, D = 5 * 1024, 8, 128, 256
    k = torch.empty((pages, heads, page, D), dtype=torch.float16, device="cuda")
    v = torch.empty_like(k)
    rng = np.random.default_rng(15)
    ids = [pages - 1, 0, pages - 2]
    rows = rng.standard_normal((2, 3, heads, page, D)).astype(np.float16)
    for i, p in enumerate(ids):
        k[p].copy_(dev(rows[0, i]))
        v[p].copy_(dev(rows[1, i]))
    qh = rng.standard_normal((1, heads, D)).astype(np.float16)
    out, _ = q.qlin_attn_decode(q.KVCache(k, v, D, 16), dev(qh), dev(np.array([ids], np.int32)),
                                dev(np.array([300], np.int32)), 384)
    got = host(out).astype(np.float64)
    for h in range(heads):
        kk, vv = (rows[i, :, h].reshape(384, D)[:300].astype(np.float64) for i in (0, 1))
        ref, _ = kv.attend(qh[0, h:h + 1], kk, vv, D ** -0.5)
        assert np.allclose(got[0, h], ref[0], rtol=2 ** -9, atol=2e-4)


def test_graph_replays_match_eager(q):
    import torch
    rng = np.random.default_rng(16)
    c = HostCache(rng, [900, 33], 900, 2, 128, 16, 4, True)
    cache, table, lens = c.device(q), dev(c.table), dev(c.lens)
    qd = dev(rng.standard_normal((2, 8, 128)).astype(np.float16))
    work = torch.empty(q.qlin_attn_decode_work_bytes(cache, 8, 2, 900, mass=True), dtype=torch.uint8, device="cuda")
    out = torch.empty((2, 8, 128), dtype=torch.float16, device="cuda")
    mass = torch.zeros((2, 2, 912), device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q.qlin_attn_decode(cache, qd, table, lens, 900, mass=mass, mass_out=mass, out=out, work=work)
    ref_mass = torch.zeros_like(mass)
    for t in range(5):
        lens.copy_(dev(np.array([900 - 37 * t, 33 + t], np.int32)))
        # Slots of row 1 past its first 33 were never written: give it row 0's pages.
        table[1, :3] = table[0, :3]
        qd.mul_(1.03)
        work.fill_(255)
        torch.cuda.synchronize()
        want, _ = q.qlin_attn_decode(cache, qd, table, lens, 900, mass=ref_mass, mass_out=ref_mass)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert_equal(host(out).view(np.uint16), host(want).view(np.uint16), f"replay {t}")
        assert_equal(host(mass), host(ref_mass), f"mass, replay {t}")


def test_empty_batch_and_refusals(q):
    import torch
    rng = np.random.default_rng(17)
    c = HostCache(rng, [20], 20, 2, 128, 16, 4)
    cache, table, lens = c.device(q), dev(c.table), dev(c.lens)
    qd = torch.zeros((1, 4, 128), dtype=torch.float16, device="cuda")
    out, _ = q.qlin_attn_decode(cache, qd[:0], table[:0], lens[:0], 20)
    assert out.shape == (0, 4, 128)
    out, _ = q.qlin_attn_decode(cache, qd, table, lens, 0)  # max_len 0: nothing to attend to
    assert not host(out).any()
    with pytest.raises(q.QlinError):
        q.qlin_attn_decode(cache, qd[:, :3].contiguous(), table, lens, 20)     # heads % kv_heads
    with pytest.raises(q.QlinError):
        q.qlin_attn_decode(cache, qd, table, lens, 33)                         # past the table
    with pytest.raises(q.QlinError):
        q.qlin_attn_decode(cache, qd, table, lens, -1)
    with pytest.raises(q.QlinError):
        q.qlin_attn_decode(cache, qd, table, lens, 20, window=-1)
    with pytest.raises(q.QlinError):
        q.qlin_attn_decode(cache, qd, table, lens, 20, scale=float("nan"))
    with pytest.raises(ValueError):
        q.qlin_attn_decode(cache, qd, table, lens, 20, mass=torch.zeros((1, 2, 32), device="cuda"))
    with pytest.raises(q.QlinError):
        q.qlin_attn_decode(cache, qd, table, lens, 20, mass_out=torch.zeros((1, 2, 19), device="cuda"))
    with pytest.raises(TypeError):
        q.qlin_attn_decode(cache, qd.float(), table, lens, 20)
    with pytest.raises(TypeError):
        q.qlin_attn_decode(cache, qd, table, lens.long(), 20)
    with pytest.raises(ValueError):
        q.qlin_attn_decode(cache, qd, table, lens, 20, mass_out=torch.zeros((1, 2, 32), device="cuda"),
                           work=torch.zeros(16, dtype=torch.uint8, device="cuda"))
