"""Appending rows to the paged cache (qlin_kv_append): more tokens than one
launch has workgroups for, rows at the edges of the quantizer's rule."""
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


def test_more_tokens_than_a_launch_has_workgroups(q):
    # 65,535 lots of eight tokens in the grid: the tokens past 524,280 are a
    # workgroup's second lot.
    import torch
    T, D, page, bits = 65535 * 8 + 21, 256, 1024, 4
    pages = -(-T // page)
    log(f"append {T} tokens")
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn((T, 1, D), generator=g, device="cuda", dtype=torch.float16) for _ in range(2))
    cache = q.KVCache.empty(pages, 1, D, page, bits)
    table = dev(np.arange(pages, dtype=np.int32)[::-1].copy().reshape(1, pages))
    slot = torch.arange(T, device="cuda", dtype=torch.int32)
    padded = [5, 65535 * 8 - 1, 65535 * 8 + 3]
    slot[torch.tensor(padded, device="cuda")] = -1
    q.qlin_kv_append(cache, k, v, table, slot, row=torch.zeros_like(slot))
    tokens = sorted({0, 7, 8, 65535 * 4, T - 1, *range(65535 * 8 - 9, T), *padded})
    for got, meta, x in ((cache.k, cache.kmeta, k), (cache.v, cache.vmeta, v)):
        codes, m = kv.quant_rows(host(x[tokens, 0]).astype(np.float32), bits)
        codes, m = kv.pack4(codes), m.copy()
        for i, t in enumerate(tokens):
            if t in padded:
                codes[i], m[i] = 0, 0
        p, line = pages - 1 - np.array(tokens) // page, np.array(tokens) % page
        at = torch.from_numpy(p).cuda(), 0, torch.from_numpy(line).cuda()
        assert_equal(host(got[at]), codes, "codes")
        assert_equal(host(meta[at]).view(np.uint16), m.view(np.uint16), "step and lo")
    # Every token arrived: no stored row is all zeros but the padded ones.
    stored = torch.flip(cache.kmeta[:, 0, :, 0], (0,)).reshape(-1)[:T]
    assert_equal(host((stored == 0).nonzero()[:, 0]), np.array(padded), "rows without a step")


@pytest.mark.parametrize("bits", [8, 4])
def test_the_step_is_a_product_with_the_reciprocal(q, bits):
    # Turned rows whose step differs between (max - lo) * fp32(1 / qmax), which
    # is the rule, and the division.
    f = np.float32
    qmax = f(2 ** bits - 1)
    rng = np.random.default_rng(bits)
    x = rng.standard_normal((200000, 128)).astype(np.float16)
    s = signs128(rng)
    t = kv.butterfly128(x, s)
    rng_of = t.max(-1) - t.min(-1).astype(np.float16).astype(f)
    differ = np.nonzero((rng_of * (f(1) / qmax)).astype(np.float16) != (rng_of / qmax).astype(np.float16))[0][:40]
    log(f"append {len(differ)} rows whose step depends on the rule, bits={bits}")
    assert len(differ) >= 4
    x = x[differ]
    T = len(x)
    cache = q.KVCache.empty(T, 1, 128, 16, bits, dev(s))
    xd = dev(x.reshape(T, 1, 128))
    q.qlin_kv_append(cache, xd, xd, dev(np.arange(T, dtype=np.int32).reshape(T, 1)), dev(np.zeros(T, np.int32)))
    codes, meta = kv.quant_rows(t[differ], bits)
    assert_equal(host(cache.kmeta)[:, 0, 0].view(np.uint16), meta.view(np.uint16), "step and lo")
    assert_equal(host(cache.k)[:, 0, 0], kv.pack4(codes) if bits == 4 else codes, "codes")


@pytest.mark.parametrize("bits", [8, 4])
def test_a_turned_row_beyond_fp16_does_not_read_back_as_finite(q, bits):
    # (k d) H of finite k may lie beyond fp16's range, which holds lo and step.
    log(f"append turned rows beyond fp16, bits={bits}")
    signs = np.ones(128, np.int8)
    x = np.zeros((3, 2, 1, 128), np.float16)
    x[0, 0, 0, :] = -1000       # turned: -128,000 in one channel
    x[1, 0, 0, :] = 1000        # 128,000: lo is 0, the step 128,000 / qmax
    x[2, 0, 0, 3] = 60000       # +-60,000 everywhere
    cache = q.KVCache.empty(3, 1, 128, 16, bits, dev(signs))
    xd = dev(x)
    q.qlin_kv_append(cache, xd[:, 0], xd[:, 1], dev(np.arange(3, dtype=np.int32).reshape(3, 1)),
                     dev(np.zeros(3, np.int32)))
    c, m = host(cache.k)[:, 0, 0], host(cache.kmeta)[:, 0, 0].astype(np.float64)
    with np.errstate(invalid="ignore"):
        vals = kv.dequant_rows(kv.unpack4(c) if bits == 4 else c, m)
    assert not np.isfinite(vals[0]).any()
    for i, t in ((1, kv.butterfly128(x[1, 0, 0], signs)), (2, kv.butterfly128(x[2, 0, 0], signs))):
        assert np.all(np.abs(vals[i] - t) <= m[i, 0] * (0.5 + (2 ** bits - 1) * 2.0 ** -11 + 1e-4))
