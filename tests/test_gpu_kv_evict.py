"""Eviction from the paged key/value cache (qlin_kv_evict), bit for bit against
the oracle: which slots stay, where they go, their rows, masses and positions,
and every byte that the call must leave alone."""
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


def _masses(rng, shape, kind):
    if kind == "spread":
        m = np.exp(2 * rng.standard_normal(shape))
        m[m < 0.3] = 0
        return m.astype(np.float32)
    if kind == "ties":
        return rng.integers(0, 3, shape).astype(np.float32)
    if kind == "close":  # equal but for the last bits
        return (np.float32(1.5).view(np.uint32) + rng.integers(0, 40, shape).astype(np.uint32)).view(np.float32)
    m = rng.standard_normal(shape).astype(np.float32)  # "odd": signs, zeros of both signs, what is not finite
    for v in (0.0, -0.0, np.nan, np.inf, -np.inf):
        m[rng.random(shape) < 0.08] = v
    return m


def _check(q, rng, c, budget, recent, kind="spread", scrambled=True, max_len=None, in_place=False):
    import torch
    B, heads = len(c.lens), c.heads
    max_len = c.max_pages * c.page if max_len is None else max_len
    ld = max(max_len, c.max_pages * c.page) + 1
    mass = _masses(rng, (B, heads, ld), kind)
    pos = np.stack([rng.permutation(ld) if scrambled else np.arange(ld) for _ in range(B * heads)])
    pos = (pos.reshape(B, heads, ld) + 5).astype(np.int32)
    cache, md, pd, lens = c.device(q), dev(mass), dev(pos), dev(c.lens)
    want = {n: getattr(c, n).copy() for n in ("k", "v", "kmeta", "vmeta") if getattr(c, n) is not None}
    mo = md if in_place else torch.full_like(md, -3.0)
    po = pd if in_place else torch.full_like(pd, -3)
    lens_out, kept, mo, po = q.qlin_kv_evict(cache, dev(c.table), lens, max_len, budget, recent, md, pd, mass_out=mo,
                                             pos_out=po)
    want_m = mass.copy() if in_place else np.full_like(mass, -3)
    want_p = pos.copy() if in_place else np.full_like(pos, -3)
    want_kept = np.full((B, heads, budget), -1, np.int32)
    want_len = np.zeros(B, np.int32)
    for b in range(B):
        n = int(min(max(c.lens[b], 0), max_len))
        for h in range(heads):
            left, src = kv.evict(mass[b, h, :n], pos[b, h, :n], budget, recent)
            want_len[b] = left
            want_kept[b, h, :left] = src
            want_m[b, h, :left], want_p[b, h, :left] = mass[b, h, src], pos[b, h, src]
            for j in np.nonzero(src != np.arange(left))[0]:
                i = int(src[j])
                pj, pi = c.table[b, j // c.page], c.table[b, i // c.page]
                for a in want.values():
                    a[pj, h, j % c.page] = a[pi, h, i % c.page]
    assert_equal(host(lens_out), want_len, "lens_out")
    assert_equal(host(kept), want_kept, "kept")
    assert_equal(host(mo).view(np.uint32), want_m.view(np.uint32), "mass")
    assert_equal(host(po), want_p, "pos")
    for n, w in want.items():
        assert_equal(host(getattr(cache, n)).view(np.uint8), w.view(np.uint8), n)
    assert_equal(host(lens), c.lens, "lens")


@pytest.mark.parametrize("bits,D", [(16, 64), (16, 128), (16, 256), (8, 64), (8, 128), (8, 256), (4, 64), (4, 128),
                                    (4, 256)])
def test_rows_of_every_width(q, bits, D):
    log(f"evict bits={bits} D={D}")
    rng = np.random.default_rng(bits + D)
    c = HostCache(rng, [0, 1, 40, 41, 100, 300], 300, 3, D, 16, bits)
    _check(q, rng, c, 40, 10)


@pytest.mark.parametrize("kind", ["spread", "ties", "close", "odd"])
@pytest.mark.parametrize("budget,recent", [(1, 0), (1, 1), (63, 0), (64, 64), (100, 31), (1000, 3), (4000, 100)])
def test_masses_and_budgets(q, kind, budget, recent):
    log(f"evict {kind} budget={budget} recent={recent}")
    rng = np.random.default_rng(budget + recent)
    c = HostCache(rng, [1, 64, 65, 1001, 3000], 3000, 2, 64, 32, 4)
    for scrambled in (False, True):
        _check(q, rng, c, budget, recent, kind, scrambled)
    _check(q, rng, c, budget, recent, kind, in_place=True)


def test_one_slot_over(q):
    rng = np.random.default_rng(1)
    c = HostCache(rng, [1025] * 4, 1025, 8, 128, 16, 4)
    for kind in ("spread", "ties"):
        _check(q, rng, c, 1024, 256, kind)
        _check(q, rng, c, 1024, 0, kind, in_place=True)


@pytest.mark.parametrize("n", [2048, 2049, 8192, 8193, 20480, 20481, 24576, 24577, 60000])
def test_long_rows(q, n):
    log(f"evict long n={n}")
    rng = np.random.default_rng(n)
    c = HostCache(rng, [n, 5], n, 1, 64, 128, 4)
    _check(q, rng, c, 2000, 500, max_len=n)
    _check(q, rng, c, n // 3, 0, "ties", max_len=n, in_place=True)
    _check(q, rng, c, n - 3, n // 2, "close", max_len=n, in_place=True)


def test_lengths_beyond_the_bounds_are_cut(q):
    rng = np.random.default_rng(2)
    c = HostCache(rng, [100, 64, 30], 100, 2, 128, 16, 8)
    _check(q, rng, c, 20, 5, max_len=64)
    c.lens = np.array([100, -5, 30], np.int32)
    _check(q, rng, c, 20, 5)


def test_positions_of_the_whole_int_range(q):
    import torch
    pos = np.array([[[2147483647, -2147483648, 0, 5, 2147483646, -7, 100, 3]]], np.int32)
    mass = np.array([[[1, 9, 2, 3, 1, 8, 7, 4]]], np.float32)
    cache = q.KVCache.empty(1, 1, 64, 16, 16)
    lens = dev(np.array([8], np.int32))
    for budget, recent in ((4, 2), (3, 0), (3, 3)):
        left, src = kv.evict(mass[0, 0], pos[0, 0].astype(np.int64), budget, recent)
        _, kept, _, _ = q.qlin_kv_evict(cache, dev(np.zeros((1, 1), np.int32)), lens, 8, budget, recent, dev(mass),
                                        dev(pos))
        assert_equal(host(kept)[0, 0], src.astype(np.int32), f"budget {budget} recent {recent}")
    torch.cuda.synchronize()


def test_attention_is_the_same_over_what_stays(q):
    # Keep every slot but the last few, which get a mass of nothing: attention
    # over the evicted cache is attention over the kept slots.
    rng = np.random.default_rng(3)
    c = HostCache(rng, [500], 500, 2, 128, 16, 4, True)
    cache, table = c.device(q), dev(c.table)
    ld = c.max_pages * c.page
    mass = rng.random((1, 2, ld)).astype(np.float32)
    pos = np.broadcast_to(np.arange(ld, dtype=np.int32), (1, 2, ld)).copy()
    lens_out, kept, _, _ = q.qlin_kv_evict(cache, table, dev(c.lens), 500, 200, 20, dev(mass), dev(pos))
    qh = rng.standard_normal((1, 8, 128)).astype(np.float16)
    out, _ = q.qlin_attn_decode(cache, dev(qh), table, lens_out, 500)
    got = host(out).astype(np.float64)
    for h in range(2):
        src = host(kept)[0, h]
        qs = c.turn(qh[0, 4 * h:4 * h + 4])
        ref, _ = kv.attend(qs, c.values[0][0][h][src], c.values[0][1][h][src], 128 ** -0.5)
        assert np.allclose(got[0, 4 * h:4 * h + 4], ref, rtol=2 ** -9, atol=2e-4)


def test_unmapped_pages_do_not_move(q):
    rng = np.random.default_rng(4)
    c = HostCache(rng, [64], 64, 1, 64, 16, 16)
    k0 = np.nan_to_num(c.k.copy())
    c.k[:], c.v[:] = k0, np.nan_to_num(c.v)
    c.table[0, 0], c.table[0, 3] = -1, c.pages + 4
    cache = c.device(q)
    mass, pos = dev(rng.random((1, 1, 64)).astype(np.float32)), dev(np.arange(64, dtype=np.int32).reshape(1, 1, 64))
    lens_out, kept, _, _ = q.qlin_kv_evict(cache, dev(c.table), dev(c.lens), 64, 20, 4, mass, pos)
    src, k = host(kept)[0, 0], host(cache.k)
    assert host(lens_out)[0] == 20
    # A move needs both of its pages: only 16 .. 19 can be filled, from 32 .. 47.
    want = k0.copy()
    for j in range(20):
        i = int(src[j])
        if i != j and j // 16 == 1 and i // 16 in (1, 2):
            want[c.table[0, 1], 0, j % 16] = k0[c.table[0, i // 16], 0, i % 16]
    assert_equal(k, want, "k")


def test_empty_batch_and_refusals(q):
    import torch
    rng = np.random.default_rng(5)
    c = HostCache(rng, [20], 20, 2, 128, 16, 4)
    cache, table, lens = c.device(q), dev(c.table), dev(c.lens)
    mass = torch.zeros((1, 2, 32), device="cuda")
    pos = torch.zeros((1, 2, 32), dtype=torch.int32, device="cuda")
    lo, kept, _, _ = q.qlin_kv_evict(cache, table[:0], lens[:0], 20, 4, 1, mass[:0], pos[:0])
    assert lo.shape == (0,) and kept.shape == (0, 2, 4)
    with pytest.raises(q.QlinError):
        q.qlin_kv_evict(cache, table, lens, 20, 0, 0, mass, pos)
    with pytest.raises(q.QlinError):
        q.qlin_kv_evict(cache, table, lens, 20, 4, 5, mass, pos)
    with pytest.raises(q.QlinError):
        q.qlin_kv_evict(cache, table, lens, 20, 4, -1, mass, pos)
    with pytest.raises(q.QlinError):
        q.qlin_kv_evict(cache, table, lens, 33, 4, 1, mass, pos)
    with pytest.raises(q.QlinError):
        q.qlin_kv_evict(cache, table, lens, 20, 4, 1, mass[..., :16].contiguous(), pos[..., :16].contiguous())
    with pytest.raises(ValueError):
        q.qlin_kv_evict(cache, table, lens, 20, 4, 1, mass, pos, lens_out=lens)
    with pytest.raises(TypeError):
        q.qlin_kv_evict(cache, table, lens, 20, 4, 1, mass, pos.long())
    with pytest.raises(ValueError):
        q.qlin_kv_evict(cache, table, lens, 20, 4, 1, mass, pos, work=torch.zeros(16, dtype=torch.uint8,
                                                                                  device="cuda"))
