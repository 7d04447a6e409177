"""Appending rows to the paged key/value cache (qlin_kv_append), bit for bit
against the oracle: codes, steps, offsets, the slots' mass and position, and
every byte that the call must leave alone."""
import numpy as np
import pytest

from oracle import kv
from tests.gpu_helpers import assert_equal, dev, host, log
from tests.kv_helpers import signs128

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    import torch
    assert torch.cuda.is_available()
    from outlier_aware_bit_amd import qlin
    return qlin


def _stored(x, bits, signs):
    """fp16 rows [T, heads, D] as the cache holds them: (rows, meta or None)."""
    if bits == 16:
        return x, None
    t = x.astype(np.float32)
    codes, meta = kv.quant_rows(t if signs is None else kv.butterfly128(t, signs), bits)
    return (kv.pack4(codes) if bits == 4 else codes), meta


def _check(q, rng, T, heads, D, page, bits, rotate, track, row=None, slot=None, x=None, pad=0):
    import torch
    B, max_pages = 4, 3
    pages = B * max_pages + 2
    signs = signs128(rng) if rotate else None
    cache = q.KVCache.empty(pages, heads, D, page, bits, None if signs is None else dev(signs))
    for t in (cache.k, cache.v):  # what is not written has to stay
        t.view(torch.uint8).copy_(dev(rng.integers(0, 256, tuple(t.view(torch.uint8).shape)).astype(np.uint8)))
    want = {n: host(getattr(cache, n)).copy() for n in ("k", "v", "kmeta", "vmeta") if getattr(cache, n) is not None}
    table = rng.permutation(pages)[:B * max_pages].reshape(B, max_pages).astype(np.int32)
    if slot is None:
        free = rng.permutation(B * max_pages * page)[:T]
        row, slot = (free // (max_pages * page)).astype(np.int32), (free % (max_pages * page)).astype(np.int32)
    if x is None:
        x = rng.standard_normal((T, 2, heads, D)).astype(np.float16)
        x[:, 0, :, D // 2] *= 40
    wide = np.concatenate([x, rng.standard_normal((T, pad, heads, D)).astype(np.float16)], 1) if pad else x
    xd = dev(wide)
    ld = max_pages * page + 5
    mass = rng.random((B, heads, ld)).astype(np.float32)
    pos = rng.integers(0, 9999, (B, heads, ld)).astype(np.int32)
    position = rng.integers(0, 1 << 30, T).astype(np.int32)
    md, pd = dev(mass), dev(pos)
    kw = dict(position=dev(position), mass=md, pos=pd) if track else {}
    q.qlin_kv_append(cache, xd[:, 0], xd[:, 1], dev(table), dev(slot), row=None if row is None else dev(row), **kw)
    kr, km = _stored(x[:, 0], bits, signs)
    vr, vm = _stored(x[:, 1], bits, None)
    for t in range(T):
        r, s = (t if row is None else int(row[t])), int(slot[t])
        if not (0 <= r < B and 0 <= s < max_pages * page and 0 <= table[r, s // page] < pages):
            continue
        p, line = table[r, s // page], s % page
        want["k"][p, :, line], want["v"][p, :, line] = kr[t], vr[t]
        if bits < 16:
            want["kmeta"][p, :, line], want["vmeta"][p, :, line] = km[t], vm[t]
        if track:
            mass[r, :, s], pos[r, :, s] = 0, position[t]
    for n, w in want.items():
        assert_equal(host(getattr(cache, n)).view(np.uint8), w.view(np.uint8), n)
    assert_equal(host(md), mass, "mass")
    assert_equal(host(pd), pos, "pos")


@pytest.mark.parametrize("bits", [16, 8, 4])
@pytest.mark.parametrize("D,heads,page,T,pad", [(64, 1, 16, 1, 0), (64, 5, 32, 33, 1), (128, 8, 16, 17, 2),
                                                (128, 3, 64, 100, 0), (256, 2, 16, 9, 1), (256, 1, 128, 70, 0)])
def test_append(q, bits, D, heads, page, T, pad):
    log(f"append bits={bits} D={D} heads={heads} page={page} T={T} pad={pad}")
    rng = np.random.default_rng(bits + D + T)
    for track in (False, True):
        _check(q, rng, T, heads, D, page, bits, False, track, pad=pad)
        if D == 128 and bits < 16:
            _check(q, rng, T, heads, D, page, bits, True, track, pad=pad)


@pytest.mark.parametrize("bits", [16, 8, 4])
def test_append_without_rows_and_with_padding(q, bits):
    log(f"append padding bits={bits}")
    rng = np.random.default_rng(bits)
    _check(q, rng, 4, 2, 128, 16, bits, False, True, slot=np.array([0, 47, 16, 31], np.int32))
    _check(q, rng, 6, 2, 128, 16, bits, False, True, row=np.array([0, -1, 4, 2, 3, 1], np.int32),
           slot=np.array([5, 1, 1, -1, 48, 2147483647], np.int32))


@pytest.mark.parametrize("bits", [8, 4])
def test_append_rows_without_range_and_tiny_rows(q, bits):
    log(f"append flat rows bits={bits}")
    rng = np.random.default_rng(40 + bits)
    x = rng.standard_normal((5, 2, 1, 128)).astype(np.float16)
    x[0] = 0
    x[1] = -0.3
    x[2] = 65504
    x[3] *= 6e-8  # a step that rounds to nothing, or to one fp16 denormal
    x[4, :, :, 0], x[4, :, :, 1] = 65504, -65504
    for rotate in (False, True):
        # A constant 65504 or +-65504 leaves fp16's range when turned.
        y = x.copy()
        if rotate:
            y[2], y[4] = 1.0, x[3]
        _check(q, rng, 5, 1, 128, 16, bits, rotate, False, x=y)


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_a_row_that_is_not_finite_does_not_read_back_as_finite(q, bits, bad):
    log(f"append {bad} bits={bits}")
    rng = np.random.default_rng(50)
    for D in (64, 128, 256):
        cache = q.KVCache.empty(2, 1, D, 16, bits)
        x = rng.standard_normal((2, 2, 1, D)).astype(np.float16)
        x[0, :, 0, D - 3] = bad
        xd = dev(x)
        q.qlin_kv_append(cache, xd[:, 0], xd[:, 1], dev(np.array([[0], [1]], np.int32)),
                         dev(np.zeros(2, np.int32)))
        for codes, meta in ((cache.k, cache.kmeta), (cache.v, cache.vmeta)):
            c, m = host(codes), host(meta).astype(np.float64)
            with np.errstate(invalid="ignore"):
                vals = kv.dequant_rows(kv.unpack4(c) if bits == 4 else c, m)
            assert not np.isfinite(vals[0, 0, 0]).any()
            assert np.isfinite(vals[1, 0, 0]).all()


def test_append_nothing(q):
    import torch
    cache = q.KVCache.empty(2, 2, 64, 16, 4)
    x = torch.zeros((0, 2, 64), dtype=torch.float16, device="cuda")
    q.qlin_kv_append(cache, x, x, dev(np.zeros((1, 1), np.int32)), dev(np.zeros(0, np.int32)))
    assert not host(cache.k).any()


def test_append_beyond_32_bit_offsets(q):
    import torch
    # 5 GiB of K rows: the last page lies past 2^32 bytes and 2^31 elements.
    pages, heads, page, D = 5 * 1024, 8, 128, 512 // 2
    k = torch.empty((pages, heads, page, D), dtype=torch.float16, device="cuda")
    v = torch.empty_like(k)
    cache = q.KVCache(k, v, D, 16)
    rng = np.random.default_rng(60)
    x = rng.standard_normal((2, 2, heads, D)).astype(np.float16)
    xd = dev(x)
    q.qlin_kv_append(cache, xd[:, 0], xd[:, 1], dev(np.array([[pages - 1], [0]], np.int32)),
                     dev(np.array([127, 3], np.int32)))
    assert_equal(host(k[pages - 1, :, 127]), x[0, 0], "k at the end")
    assert_equal(host(v[pages - 1, :, 127]), x[0, 1], "v at the end")
    assert_equal(host(k[0, :, 3]), x[1, 0], "k at the start")


def test_append_refusals(q):
    import torch
    cache = q.KVCache.empty(2, 2, 128, 16, 4)
    x = torch.zeros((3, 2, 128), dtype=torch.float16, device="cuda")
    table = torch.zeros((3, 1), dtype=torch.int32, device="cuda")
    slot = torch.zeros(3, dtype=torch.int32, device="cuda")
    mass = torch.zeros((3, 2, 16), device="cuda")
    pos = torch.zeros((3, 2, 16), dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        q.qlin_kv_append(cache, x.float(), x, table, slot)
    with pytest.raises(ValueError):
        q.qlin_kv_append(cache, x, x[:2], table, slot)
    with pytest.raises(ValueError):
        q.qlin_kv_append(cache, x[..., ::2], x, table, slot)
    with pytest.raises(ValueError):
        q.qlin_kv_append(cache, x.transpose(0, 1).contiguous().transpose(0, 1), x, table, slot)
    with pytest.raises(ValueError):
        q.qlin_kv_append(cache, x, x, table, slot[:2])
    with pytest.raises(TypeError):
        q.qlin_kv_append(cache, x, x, table, slot.long())
    with pytest.raises(ValueError):
        q.qlin_kv_append(cache, x, x, table, slot, mass=mass, pos=pos)
    with pytest.raises(ValueError):
        q.qlin_kv_append(cache, x, x, table, slot, position=slot, mass=mass[:, :1], pos=pos)
    wide = torch.zeros((3, 2 * 128 + 4), dtype=torch.float16, device="cuda")[:, :256].unflatten(1, (2, 128))
    with pytest.raises(q.QlinError):  # tokens 260 elements apart
        q.qlin_kv_append(cache, wide, x, table, slot)
    with pytest.raises(q.QlinError):  # three tokens, two rows
        q.qlin_kv_append(cache, x, x, table[:2], slot)
    with pytest.raises(ValueError):
        q.KVCache.empty(2, 2, 128, 16, 5)
    with pytest.raises(ValueError):
        q.KVCache(cache.k, cache.v, 128, 4, cache.kmeta, None)
    with pytest.raises(q.QlinError):  # page of 24 slots
        c = q.KVCache.empty(2, 2, 128, 24, 4)
        q.qlin_kv_append(c, x, x, table, slot)
    with pytest.raises(q.QlinError):  # the Hadamard is 128 wide
        c = q.KVCache.empty(2, 2, 64, 16, 4, torch.ones(128, dtype=torch.int8, device="cuda"))
        q.qlin_kv_append(c, x[..., :64].contiguous(), x[..., :64].contiguous(), table, slot)
