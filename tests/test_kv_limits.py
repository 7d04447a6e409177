"""Sizes and aliases that the eviction's kernels cannot take are refused on the
host (CPU only)."""
import ctypes as C

import pytest

from outlier_aware_bit_amd import _lib
from tests.test_kv_abi import A, I, S, cache, evict

M = 1 << 30  # slots and budgets: kernels add up to a workgroup's reach in 32 bits


@pytest.mark.parametrize("kw", [dict(max_len=M + 1, ld=M + 1), dict(max_len=2 * M - 16, ld=2 * M - 16),
                                dict(budget=M + 1), dict(budget=2 * M - 1)])
def test_slots_and_budgets_beyond_2_to_30(kw):
    assert evict(max_pages=(2 * M - 1) // 16, B=1, **kw) == S, _lib.load().qlin_last_error()


def test_workspace_sizes_end_there():
    lib, held = _lib.load(), cache()
    c = C.addressof(held)
    assert lib.qlin_kv_evict_work_bytes(c, 1, M, M) > 0 and lib.qlin_kv_evict_work_bytes(c, 1, M, 16) > 0
    for max_len, budget in ((M + 1, 16), (2 * M - 2, 16), (64, M + 1), (64, 2 * M - 1)):
        assert lib.qlin_kv_evict_work_bytes(c, 1, max_len, budget) == 0


def test_lens_out_is_not_lens():
    # The kv heads of a sequence read lens while another writes lens_out.
    assert evict(lens=A, lens_out=A) == I, _lib.load().qlin_last_error()
    assert b"lens_out" in _lib.load().qlin_last_error()
