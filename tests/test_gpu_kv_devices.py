"""The key/value cache's calls take tensors of the cache's GPU, with that GPU the
current one.  One GPU is enough: the cache, or the current device, is said to be
another."""
import pytest

from tests.gpu_helpers import host

pytestmark = pytest.mark.gpu


@pytest.fixture
def calls():
    import torch
    from outlier_aware_bit_amd import qlin as q
    cache = q.KVCache.empty(2, 2, 128, 16, 4)
    table = torch.tensor([[0], [1]], dtype=torch.int32, device="cuda")
    x = torch.randn((2, 2, 128), device="cuda").half()
    slot, lens = (torch.full((2,), v, dtype=torch.int32, device="cuda") for v in (3, 4))
    mass, pos = torch.zeros((2, 2, 16), device="cuda"), torch.zeros((2, 2, 16), dtype=torch.int32, device="cuda")

    def append():
        q.qlin_kv_append(cache, x, x, table, slot)

    def attend():
        q.qlin_attn_decode(cache, x, table, lens, 16)

    def evict():
        q.qlin_kv_evict(cache, table, lens, 16, 2, 1, mass, pos)

    return q, cache, (append, attend, evict)


def test_tensors_of_another_gpu_are_refused(calls):
    q, cache, run = calls
    for f in run:
        f()
    before = host(cache.k)
    cache.index = 1
    for f in run:
        with pytest.raises(ValueError, match="cuda:0.*cuda:1"):
            f()
    assert (host(cache.k) == before).all()


def test_another_current_gpu_is_refused(calls, monkeypatch):
    q, cache, run = calls
    monkeypatch.setattr(q, "_current_device", lambda: 1)
    for f in run:
        with pytest.raises(ValueError, match="current"):
            f()
