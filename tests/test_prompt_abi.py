"""Host-side validation of qlin_rope, qlin_attn_prompt, its backward pass,
qlin_kv_slots and qlin_kv_pages (CPU only): every case returns its documented
status before any HIP call; frequencies and workspace sizes."""
import ctypes as C

import numpy as np
import pytest

from oracle import prompt
from outlier_aware_bit_amd import _lib

# Fake but 16-byte aligned addresses: validation never dereferences them.
A, MIS = 0x10000, 0x10008
I, S, AL, U, OK = (_lib.QLIN_ERR_INVALID_ARG, _lib.QLIN_ERR_SHAPE, _lib.QLIN_ERR_ALIGN, _lib.QLIN_ERR_UNSUPPORTED,
                   _lib.QLIN_OK)


def rope(q=A, ld_q=512, heads=4, k=A, ld_k=256, kv_heads=2, T=3, D=128, rot=128, interleaved=0, position=A, freq=A,
         amplitude=1.0, inverse=0, q_out=2 * A, ld_qo=512, k_out=2 * A, ld_ko=256):
    return _lib.load().qlin_rope(q, ld_q, heads, k, ld_k, kv_heads, T, D, rot, interleaved, position, freq, amplitude,
                                 inverse, q_out, ld_qo, k_out, ld_ko, None)


def attend(q=A, ld_q=512, heads=4, k=A, ld_k=256, v=A, ld_v=256, kv_heads=2, D=128, cu_q=A, cu_k=A, B=2, Tq=40, Tk=50,
           scale=1.0, causal=1, window=0, out=4 * A, lse=None, work=None):
    return _lib.load().qlin_attn_prompt(q, ld_q, heads, k, ld_k, v, ld_v, kv_heads, D, cu_q, cu_k, B, Tq, Tk, scale,
                                        causal, window, out, lse, work, None)


def learn(dout=A, ld_do=512, q=A, ld_q=512, heads=4, k=A, ld_k=256, v=A, ld_v=256, kv_heads=2, D=128, out=A, lse=A,
          cu_q=A, cu_k=A, B=2, Tq=40, Tk=50, scale=1.0, causal=1, window=0, dq=5 * A, ld_dq=512, dk=6 * A, ld_dk=256, dv=7 * A,
          ld_dv=256, work=A):
    return _lib.load().qlin_attn_prompt_backward(dout, ld_do, q, ld_q, heads, k, ld_k, v, ld_v, kv_heads, D, out, lse,
                                                 cu_q, cu_k, B, Tq, Tk, scale, causal, window, dq, ld_dq, dk, ld_dk,
                                                 dv, ld_dv, work, None)


def slots(lens=A, add=A, first=None, B=2, T=5, cu=A, row=A, slot=A, position=A, lens_out=2 * A):
    return _lib.load().qlin_kv_slots(lens, add, first, B, T, cu, row, slot, position, lens_out, None)


def pages(want=A, B=2, max_pages=4, page=16, table=A, held=2 * A, ring=A, n=8, state=A, table_out=A, held_out=2 * A,
          state_out=A, missing=A):
    return _lib.load().qlin_kv_pages(want, B, max_pages, page, table, held, ring, n, state, table_out, held_out,
                                     state_out, missing, None)


@pytest.mark.parametrize("kw,status", [
    (dict(D=96), U), (dict(D=0), U), (dict(rot=8), U), (dict(rot=24), U), (dict(rot=144), U), (dict(rot=0), U),
    (dict(heads=0), S), (dict(heads=65536), S), (dict(kv_heads=-1), S), (dict(T=-1), I), (dict(ld_q=511), S),
    (dict(ld_q=516), S), (dict(ld_k=248), S), (dict(ld_qo=504), S), (dict(ld_ko=252), S), (dict(T=1 << 31), S),
    (dict(amplitude=float("nan")), I), (dict(k=None), I), (dict(k_out=None), I), (dict(kv_heads=0), I),
    (dict(q_out=A, ld_qo=520), S), (dict(k_out=A, ld_ko=264), S), (dict(q=None), I), (dict(q_out=None), I),
    (dict(position=None), I), (dict(freq=None), I), (dict(q=MIS), AL), (dict(k_out=MIS), AL), (dict(position=MIS), AL),
    (dict(freq=MIS), AL), (dict(T=0, q=None, q_out=None), OK), (dict(q=3 * A, q_out=A, k_out=4 * A), I),
    (dict(k=3 * A, k_out=A), I), (dict(k=3 * A), I)])
def test_rope(kw, status):
    assert rope(**kw) == status, _lib.load().qlin_last_error()


BOTH = [(dict(D=96), U), (dict(D=32), U), (dict(heads=3), S), (dict(heads=0), S), (dict(kv_heads=0), S),
        (dict(kv_heads=-2, heads=-4), S), (dict(heads=131072, kv_heads=1), S), (dict(B=-1), I), (dict(Tq=-1), I),
        (dict(Tk=-1), I), (dict(B=65536), S), (dict(Tq=(1 << 30) + 1), S), (dict(Tk=1 << 31), S),
        (dict(Tq=1 << 30, heads=128, ld_q=16384), S), (dict(B=65535, heads=130, ld_q=16640), S), (dict(scale=float("nan")), I), (dict(scale=float("inf")), I),
        (dict(scale=2.0 ** 41), I), (dict(scale=-2.0 ** 41), I),
        (dict(window=-1), I), (dict(window=5, causal=0), I), (dict(ld_q=504), S), (dict(ld_q=516), S),
        (dict(ld_k=0), S), (dict(ld_v=260), S), (dict(ld_v=(1 << 22) + 8), S), (dict(q=None), I), (dict(k=None), I),
        (dict(v=MIS), AL), (dict(out=None), I), (dict(out=MIS), AL), (dict(cu_q=None), I), (dict(cu_k=MIS), AL),
        (dict(B=0, q=None, cu_q=None), OK)]


@pytest.mark.parametrize("kw,status", BOTH + [(dict(lse=MIS), AL), (dict(work=MIS), AL), (dict(Tq=0, q=None), OK),
                                              (dict(Tq=40, Tk=100000), I),  # a long axis needs a workspace
                                              (dict(out=A), I), (dict(q=2 * A, k=2 * A, out=2 * A), I)])
def test_attention(kw, status):
    assert attend(**kw) == status, _lib.load().qlin_last_error()


@pytest.mark.parametrize("kw,status", BOTH + [
    (dict(dout=None), I), (dict(lse=None), I), (dict(lse=MIS), AL), (dict(dq=None), I), (dict(dk=MIS), AL),
    (dict(dv=None), I), (dict(work=None), I), (dict(work=MIS), AL), (dict(ld_do=256), S), (dict(ld_dq=508), S),
    (dict(ld_dk=8), S), (dict(ld_dv=(1 << 23)), S), (dict(Tq=0, Tk=0, q=None, k=None), OK), (dict(dq=A), I),
    (dict(dk=A), I), (dict(dv=A), I), (dict(dk=5 * A), I), (dict(dv=5 * A), I), (dict(dv=6 * A), I)])
def test_gradients(kw, status):
    assert learn(**kw) == status, _lib.load().qlin_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), I), (dict(T=-1), I), (dict(B=65536), S), (dict(T=1 << 31), S), (dict(lens=None), I),
    (dict(add=MIS), AL), (dict(first=MIS), AL), (dict(cu=None), I), (dict(row=None), I), (dict(slot=MIS), AL),
    (dict(position=None), I), (dict(lens_out=None), I), (dict(lens_out=A), I), (dict(first=2 * A), I),
    (dict(add=2 * A), I)])
def test_slots(kw, status):
    assert slots(**kw) == status, _lib.load().qlin_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(page=8), U), (dict(page=24), U), (dict(page=2048), U), (dict(page=0), U), (dict(B=-1), I),
    (dict(B=65536), S), (dict(max_pages=0), S), (dict(max_pages=1 << 28), S), (dict(n=0), S), (dict(n=1 << 31), S),
    (dict(want=None), I), (dict(want=2 * A), I), (dict(table=MIS), AL), (dict(held=None), I), (dict(ring=None), I),
    (dict(state=MIS), AL), (dict(table_out=None), I), (dict(held_out=MIS), AL), (dict(state_out=None), I),
    (dict(missing=None), I)])
def test_pages(kw, status):
    assert pages(**kw) == status, _lib.load().qlin_last_error()


@pytest.mark.parametrize("rot", [16, 64, 128, 256])
@pytest.mark.parametrize("scaling,kw", [("plain", {}), ("linear", dict(factor=4.0)), ("base", dict(factor=8.0)),
                                        ("ramp", dict(factor=16.0, original_len=8192)),
                                        ("ramp", dict(factor=2.0, original_len=50, fast=8.0, slow=0.5))])
def test_frequencies(rot, scaling, kw):
    from outlier_aware_bit_amd import qlin
    for base in (10000.0, 500000.0, 1.5):
        freq, amp = qlin.qlin_rope_freqs(rot, base, scaling, device="cpu", **kw)
        want, want_amp = prompt.rope_freqs(rot, base, scaling, **kw)
        assert np.allclose(freq.numpy(), want, rtol=1e-13, atol=0.0) and abs(amp - want_amp) <= 2.0 ** -23 * want_amp


@pytest.mark.parametrize("a,status", [
    ((8, 1e4, 0, 1.0, 0, 32.0, 1.0), U), ((24, 1e4, 0, 1.0, 0, 32.0, 1.0), U), ((272, 1e4, 0, 1.0, 0, 32.0, 1.0), U),
    ((64, 1.0, 0, 1.0, 0, 32.0, 1.0), I), ((64, float("nan"), 0, 1.0, 0, 32.0, 1.0), I),
    ((64, 1e4, 4, 1.0, 0, 32.0, 1.0), I), ((64, 1e4, -1, 1.0, 0, 32.0, 1.0), I),
    ((64, 1e4, 1, 0.5, 0, 32.0, 1.0), I), ((64, 1e4, 3, 2.0, 0, 32.0, 1.0), I), ((64, 1e4, 3, 2.0, 10, 1.0, 1.0), I),
    ((64, 1e4, 3, 2.0, 10, 2.0, 0.0), I), ((64, 1e4, 0, 0.0, 0, 0.0, 0.0), OK)])
def test_frequencies_refused(a, status):
    freq, amp = (C.c_double * 128)(), C.c_float()
    lib = _lib.load()
    assert lib.qlin_rope_freqs(*a, C.addressof(freq), C.addressof(amp)) == status
    assert lib.qlin_rope_freqs(*a, None, C.addressof(amp)) != OK
    assert lib.qlin_rope_freqs(*a, C.addressof(freq), None) != OK


def test_scaling_names():
    from outlier_aware_bit_amd import qlin
    with pytest.raises(ValueError, match="scaling"):
        qlin.qlin_rope_freqs(64, scaling="other", device="cpu")


def test_workspace_sizes():
    lib = _lib.load()
    # Rows enough to fill the GPU: nothing is divided.
    assert lib.qlin_attn_prompt_work_bytes(32, 8, 128, 1, 16384, 16384, 1, 0) == 0
    assert lib.qlin_attn_prompt_work_bytes(32, 8, 128, 1, 77, 77, 1, 0) == 0
    parts = lib.qlin_attn_prompt_work_bytes(16, 4, 256, 1, 500, 15500, 1, 0)
    assert parts >= 2 * 16 * 500 * (256 * 4 + 8) and parts % (16 * 500 * (256 * 4 + 8)) == 0
    # A window bounds the keys that there are to divide.
    assert lib.qlin_attn_prompt_work_bytes(16, 4, 256, 1, 500, 15500, 1, 64) == 0
    for bad in ((3, 2, 128, 1, 10, 10, 1, 0), (4, 2, 96, 1, 10, 10, 1, 0), (4, 2, 128, -1, 10, 10, 1, 0),
                (4, 2, 128, 0, 10, 10, 1, 0), (4, 2, 128, 1, -1, 10, 1, 0), (4, 2, 128, 1, 10, 1 << 31, 1, 0),
                (4, 2, 128, 1, 10, 10, 0, 5), (4, 2, 128, 1, 10, 10, 1, -5), (0, 0, 128, 1, 10, 10, 1, 0)):
        assert lib.qlin_attn_prompt_work_bytes(*bad) == 0
        assert lib.qlin_attn_prompt_backward_work_bytes(*bad) == 0
    # The gradients' statistics, and parts of dk and dv where the queries of a key are divided.
    assert 2 * 4 * 33 * 4 <= lib.qlin_attn_prompt_backward_work_bytes(4, 2, 128, 1, 33, 33, 1, 0) < 2 * 4 * 48 * 4
    assert lib.qlin_attn_prompt_backward_work_bytes(32, 8, 128, 4, 8192, 8192, 1, 0) == 2 * 32 * 8192 * 4
    parts = lib.qlin_attn_prompt_backward_work_bytes(8, 1, 64, 1, 1000, 1000, 1, 0) - 2 * 8 * 1000 * 4
    assert parts >= 2 * 1000 * 64 * 8 and parts % (1000 * 64 * 8) == 0
    for window in (0, 2 ** 31 - 1):
        assert lib.qlin_attn_prompt_backward_work_bytes(8, 1, 64, 1, 1000, 1000, 1, window) >= parts // 2
    assert lib.qlin_attn_prompt_backward_work_bytes(1, 1, 64, 1, 1000, 1000, 1, 8) == 2 * 1000 * 4
    assert lib.qlin_attn_prompt_work_bytes(16, 4, 256, 1, 500, 15500, 1, 2 ** 31 - 1) >= 2 * 16 * 500 * (256 * 4 + 8)
