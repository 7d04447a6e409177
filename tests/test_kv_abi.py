"""Host-side validation of the key/value cache's entry points (CPU only): every
case returns its documented status before any HIP call, and the workspace
sizes follow from the arguments alone."""
import ctypes as C

import pytest

from outlier_aware_bit_amd import _lib

# Fake but 16-byte aligned addresses: validation never dereferences them.
A, MIS = 0x10000, 0x10008
I, S, AL, U, OK = (_lib.QLIN_ERR_INVALID_ARG, _lib.QLIN_ERR_SHAPE, _lib.QLIN_ERR_ALIGN, _lib.QLIN_ERR_UNSUPPORTED,
                   _lib.QLIN_OK)


def cache(**kw):
    f = dict(k=A, v=A, kmeta=A, vmeta=A, signs=None, pages=8, page=16, kv_heads=2, head_dim=128, bits=4)
    f.update(kw)
    return _lib.KVCacheStruct(**f)


def append(c=None, k=A, ld_k=256, v=A, ld_v=256, T=3, row=A, slot=A, table=A, B=2, max_pages=4, position=None,
           mass=None, pos=None, ld=0):
    c = cache() if c is None else c
    return _lib.load().qlin_kv_append(C.addressof(c) if c else None, k, ld_k, v, ld_v, T, row, slot, table, B,
                                      max_pages, position, mass, pos, ld, None)


def attend(c=None, q=A, ld_q=512, heads=4, table=A, lens=A, B=2, max_pages=4, max_len=64, scale=1.0, window=0, out=A,
           mass_in=None, mass_out=None, ld=0, work=A):
    c = cache() if c is None else c
    return _lib.load().qlin_attn_decode(C.addressof(c) if c else None, q, ld_q, heads, table, lens, B, max_pages,
                                        max_len, scale, window, out, mass_in, mass_out, ld, work, None)


def evict(c=None, table=A, lens=A, B=2, max_pages=4, max_len=64, budget=16, recent=4, mass=A, pos=A, ld=64,
          mass_out=A, pos_out=A, lens_out=2 * A, kept=A, work=A):
    c = cache() if c is None else c
    return _lib.load().qlin_kv_evict(C.addressof(c) if c else None, table, lens, B, max_pages, max_len, budget, recent,
                                     mass, pos, ld, mass_out, pos_out, lens_out, kept, work, None)


BAD_CACHES = [(dict(bits=5), U), (dict(bits=0), U), (dict(head_dim=96), U), (dict(head_dim=0), U), (dict(page=8), U),
              (dict(page=24), U), (dict(page=2048), U), (dict(page=0), U), (dict(page=-16), U), (dict(kv_heads=0), S),
              (dict(kv_heads=65536), S), (dict(pages=0), S), (dict(pages=1 << 31), S),
              (dict(pages=(1 << 31) - 1, kv_heads=65535, page=1024), S), (dict(k=None), I), (dict(v=None), I),
              (dict(kmeta=None), I), (dict(vmeta=None), I), (dict(k=MIS), AL), (dict(vmeta=MIS), AL),
              (dict(signs=MIS), AL), (dict(signs=A, head_dim=64), U), (dict(bits=16), I),
              (dict(bits=16, kmeta=None, vmeta=None, signs=A), I)]


@pytest.mark.parametrize("fields,status", BAD_CACHES)
def test_cache_descriptions(fields, status):
    for call in (append, attend, evict):
        assert call(cache(**fields)) == status, _lib.load().qlin_last_error()
    assert b"" != _lib.load().qlin_last_error()


def test_no_cache():
    lib = _lib.load()
    assert lib.qlin_kv_append(None, *([A, 256] * 2), 1, A, A, A, 1, 1, None, None, None, 0, None) == I
    assert lib.qlin_attn_decode_work_bytes(None, 4, 2, 64, 0, 0) == 0
    assert lib.qlin_kv_evict_work_bytes(None, 2, 64, 16) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), I), (dict(B=-1), I), (dict(max_pages=0), S), (dict(max_pages=1 << 28), S), (dict(ld_k=255), S),
    (dict(ld_k=260), S), (dict(ld_v=248), S), (dict(T=1 << 31), S), (dict(T=1 << 30, ld_k=1 << 20), S),
    (dict(row=None, T=3), S), (dict(position=A), I), (dict(mass=A, pos=A), I), (dict(mass=A, position=A), I),
    (dict(mass=A, pos=A, position=A, ld=0), S), (dict(mass=A, pos=A, position=A, ld=1 << 31), S), (dict(k=None), I),
    (dict(v=MIS), AL), (dict(row=MIS), AL), (dict(slot=None), I), (dict(table=None), I),
    (dict(mass=MIS, pos=A, position=A, ld=8), AL), (dict(T=0, k=None), OK), (dict(B=0, table=None), OK)])
def test_append(kw, status):
    assert append(**kw) == status, _lib.load().qlin_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(heads=3), S), (dict(heads=0), S), (dict(heads=-2), S), (dict(ld_q=511), S), (dict(ld_q=516), S),
    (dict(max_len=-1), I), (dict(max_len=65), S), (dict(window=-1), I), (dict(scale=float("nan")), I),
    (dict(B=-1), I), (dict(B=1 << 31), S), (dict(B=1 << 30, ld_q=1024), S), (dict(mass_in=A), I),
    (dict(mass_out=A, ld=63), S), (dict(mass_out=A, ld=0), S), (dict(q=None), I), (dict(out=MIS), AL),
    (dict(lens=None), I), (dict(table=MIS), AL), (dict(mass_out=A, ld=64, work=None), I),
    (dict(mass_out=A, ld=64, work=MIS), AL), (dict(mass_out=MIS, ld=64), AL), (dict(B=0, q=None), OK)])
def test_attend(kw, status):
    assert attend(**kw) == status, _lib.load().qlin_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(budget=0), I), (dict(budget=-1), I), (dict(recent=17), I), (dict(recent=-1), I), (dict(max_len=65), S),
    (dict(max_len=-1), I), (dict(ld=63), S), (dict(ld=0), S), (dict(B=1 << 30), S), (dict(B=-1), I),
    (dict(mass=None), I), (dict(pos=MIS), AL), (dict(mass_out=None), I), (dict(pos_out=None), I),
    (dict(lens_out=None), I), (dict(kept=None), I), (dict(work=None), I), (dict(work=MIS), AL), (dict(lens=None), I),
    (dict(B=0, table=None), OK)])
def test_evict(kw, status):
    assert evict(**kw) == status, _lib.load().qlin_last_error()


def test_workspace_sizes():
    lib = _lib.load()
    held, wrong = cache(), cache(page=8)
    c = C.addressof(held)
    # One chunk: nothing to join.  The weights' sums need the logits.
    assert lib.qlin_attn_decode_work_bytes(c, 4, 2, 64, 0, 0) == 0
    assert lib.qlin_attn_decode_work_bytes(c, 4, 2, 64, 0, 1) >= 2 * 4 * 64 * 4
    long = lib.qlin_attn_decode_work_bytes(c, 4, 2, 100000, 0, 0)
    assert long > 2 * 4 * 128 * 4 * 2
    # A window bounds the chunks, whatever the length.
    assert lib.qlin_attn_decode_work_bytes(c, 4, 2, 100000, 64, 0) == 0
    for bad in ((3, 2, 64, 0, 0), (0, 2, 64, 0, 0), (4, 0, 64, 0, 0), (4, 2, -1, 0, 0), (4, 2, 64, -1, 0),
                (4, 1 << 31, 64, 0, 0), (4, 1 << 29, 1 << 20, 0, 1), (4, 2, 1 << 31, 0, 0)):
        assert lib.qlin_attn_decode_work_bytes(c, *bad) == 0
    assert lib.qlin_kv_evict_work_bytes(c, 2, 64, 16) >= 2 * 2 * (4 + 16 * 8)
    assert lib.qlin_kv_evict_work_bytes(c, 2, 64, 64) >= 2 * 2 * 4
    for bad in ((0, 64, 16), (2, -1, 16), (2, 64, -1), (1 << 31, 64, 16), (1 << 29, 1 << 20, 16)):
        assert lib.qlin_kv_evict_work_bytes(c, *bad) == 0
    assert lib.qlin_attn_decode_work_bytes(C.addressof(wrong), 4, 2, 64, 0, 1) == 0
