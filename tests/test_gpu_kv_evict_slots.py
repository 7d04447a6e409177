"""Eviction from the paged cache (qlin_kv_evict) where slots do not exist,
positions repeat, or a row is as long as a kernel takes, bit for bit against the
oracle."""
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


def _check(q, c, mass, pos, budget, recent, max_len, in_place):
    import torch
    B, heads, ld = mass.shape
    cache, md, pd = c.device(q), dev(mass), dev(pos)
    mo, po = (md, pd) if in_place else (torch.full_like(md, -3.0), torch.full_like(pd, -3))
    want = {n: getattr(c, n).copy() for n in ("k", "v", "kmeta", "vmeta") if getattr(c, n) is not None}
    want_m, want_p = host(mo).copy(), host(po).copy()
    want_kept = np.full((B, heads, budget), -1, np.int32)
    lens_out, kept, mo, po = q.qlin_kv_evict(cache, dev(c.table), dev(c.lens), max_len, budget, recent, md, pd,
                                             mass_out=mo, pos_out=po)
    for b in range(B):
        n = int(c.lens[b])
        there = [0 <= c.table[b, i // c.page] < c.pages for i in range(n)]
        for h in range(heads):
            left, src = kv.evict(mass[b, h, :n], pos[b, h, :n], budget, recent, there)
            want_kept[b, h, :left] = src
            want_m[b, h, :left], want_p[b, h, :left] = mass[b, h, src], pos[b, h, src]
            for j in np.nonzero(src != np.arange(left))[0]:
                i = int(src[j])
                assert there[i] and there[j]
                pj, pi = c.table[b, j // c.page], c.table[b, i // c.page]
                for a in want.values():
                    a[pj, h, j % c.page] = a[pi, h, i % c.page]
    assert_equal(host(lens_out), np.minimum(c.lens, budget), "lens_out")
    assert_equal(host(kept), want_kept, "kept")
    assert_equal(host(mo).view(np.uint32), want_m.view(np.uint32), "mass")
    assert_equal(host(po), want_p, "pos")
    for n, w in want.items():
        assert_equal(host(getattr(cache, n)).view(np.uint8), w.view(np.uint8), n)


def _rows(rng, c, kind="spread"):
    shape = (len(c.lens), c.heads, c.max_pages * c.page)
    if kind == "odd":
        mass = rng.standard_normal(shape).astype(np.float32)
        for v in (0.0, -0.0, np.nan, np.inf, -np.inf):
            mass[rng.random(shape) < 0.08] = v
    else:
        mass = np.exp(2 * rng.standard_normal(shape)).astype(np.float32)
        mass[mass < 0.3] = 0
    pos = np.stack([rng.permutation(shape[2]) for _ in range(shape[0] * shape[1])]).reshape(shape).astype(np.int32)
    return mass, pos


# Rows of the kernel for short ones, of both for longer ones, and of the one
# that keeps no row in registers.
@pytest.mark.parametrize("n,bits,page", [(100, 16, 16), (1100, 4, 32), (5000, 8, 64), (12000, 4, 16), (21000, 4, 128)])
@pytest.mark.parametrize("share", [0.1, 0.6])
def test_slots_that_do_not_exist_neither_count_nor_move(q, n, bits, page, share):
    log(f"evict unmapped n={n} bits={bits} page={page} share={share}")
    rng = np.random.default_rng(n + bits)
    for in_place, kind in ((False, "spread"), (True, "odd")):
        c = HostCache(rng, [n, n - 3, n // 2], n, 2, 64, page, bits)
        for b in range(2):
            entries = -(-int(c.lens[b]) // page)
            gone = rng.random(entries) < share
            gone[rng.integers(entries)] = True
            c.table[b, :entries][gone] = rng.choice([-1, c.pages, 2147483647, -2147483648], int(gone.sum()))
        mass, pos = _rows(rng, c, kind)
        # What their entries hold decides nothing: the newest and the heaviest are among them.
        for b in range(2):
            slots = np.arange(int(c.lens[b]))
            gone = (c.table[b, slots // page] < 0) | (c.table[b, slots // page] >= c.pages)
            pos[b][:, slots[gone]] = 1 << 29
            mass[b][:, slots[gone]] = np.inf
        for budget, recent in ((1, 1), (n // 3, 0), (n // 2, n // 8), (n - 2, 5), (n, 3)):
            _check(q, c, mass, pos, budget, recent, n, in_place)


def test_attention_after_an_eviction_with_unmapped_pages(q):
    # What stays is what attention reads: each kept slot's own row.
    log("evict unmapped, then attend")
    rng = np.random.default_rng(3)
    c = HostCache(rng, [160], 160, 1, 64, 16, 16)
    c.table[0, [1, 6]] = -1
    mass, pos = _rows(rng, c)
    mass[0, 0, 16:32] = 50.0
    cache, table = c.device(q), dev(c.table)
    lens, kept, _, _ = q.qlin_kv_evict(cache, table, dev(c.lens), 160, 60, 10, dev(mass), dev(pos))
    qh = rng.standard_normal((1, 2, 64)).astype(np.float16)
    out, _ = q.qlin_attn_decode(cache, dev(qh), table, lens, 160, scale=0.125)
    src = host(kept)[0, 0]
    use = np.array([0 <= c.table[0, j // 16] < c.pages for j in range(60)])
    assert use.sum() == 44 and not set(src[use].tolist()) & set(range(16, 32))
    k, v = (x[0][src] for x in c.values[0])
    ref, _ = kv.attend(qh[0].astype(np.float64), k, v, 0.125, use)
    assert np.allclose(host(out)[0], ref, rtol=2 ** -9, atol=2e-4)


@pytest.mark.parametrize("n", [40, 1500, 3000, 15000, 21000])
@pytest.mark.parametrize("kind", ["spread", "odd"])
def test_more_newest_slots_than_fit(q, n, kind):
    # Positions repeat (the tokens of one image, say): of the newest, those of
    # largest mass stay.
    log(f"evict repeated positions n={n} {kind}")
    rng = np.random.default_rng(n)
    c = HostCache(rng, [n, n - 1, 7], n, 2, 64, 128, 4)
    mass, pos = _rows(rng, c, kind)
    for spread in (1, 3, n // 4 + 1):
        pos = rng.integers(0, spread, pos.shape).astype(np.int32) + 9
        for budget, recent in ((1, 1), (n // 3, 1), (n // 2, n // 2), (n - 2, 2)):
            _check(q, c, mass, pos, budget, min(recent, budget), n, False)
    # The same where slots that do not exist leave less room.
    c.table[0, 0] = -1
    _check(q, c, mass, np.zeros_like(pos), n // 2, 1, n, True)
    mass, pos = _rows(rng, c, kind)
    _check(q, c, mass, pos, n // 2, n // 2, n, False)


@pytest.mark.parametrize("n", [1535, 1536, 1537, 8191, 20479])
def test_rows_as_long_as_a_kernel_takes(q, n):
    # The lengths at which another kernel takes over: 1,536, 8,192 and 20,480.
    log(f"evict n={n}")
    rng = np.random.default_rng(n)
    c = HostCache(rng, [n, n - 1, 700], n, 1, 64, 64, 4)
    for kind in ("spread", "odd"):
        mass, pos = _rows(rng, c, kind)
        _check(q, c, mass, pos, n - 1, 9, n, False)
        _check(q, c, mass, pos, n // 2, 100, n, True)


@pytest.mark.parametrize("over", [63, 64, 65, 127, 128, 129])
def test_moves_by_the_selecting_workgroup_and_by_a_second_launch(q, over):
    # 16 KiB of moves: 64 slots of 128-byte rows.
    log(f"evict {over} over")
    rng = np.random.default_rng(over)
    for bits, D in ((4, 128), (8, 128), (4, 256)):
        c = HostCache(rng, [400 + over, 400, 399], 400 + over, 2, D, 16, bits)
        mass, pos = _rows(rng, c)
        _check(q, c, mass, pos, 400, 20, 400 + over, False)
