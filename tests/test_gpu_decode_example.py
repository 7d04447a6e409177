"""examples/decode_kv4.py: a layer that decodes through qlin_kv_append,
qlin_attn_decode and qlin_kv_evict, every step's attention checked against the
float64 oracle over the rows that the oracle's own cache holds by then, and
every eviction against the oracle's choice."""
import importlib.util
import os
import types

import numpy as np
import pytest

from oracle import kv
from tests.gpu_helpers import assert_equal, host, log
from tests.kv_helpers import HostCache
from tests.test_gpu_attn_decode import _bounds

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode_kv4.py")


@pytest.fixture(scope="module")
def example():
    import torch
    assert torch.cuda.is_available()
    spec = importlib.util.spec_from_file_location("decode_kv4", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


class Mirror:
    """The layer's cache in float64, one list of (k, v) rows per sequence and kv head."""

    def __init__(self, layer):
        self.layer, self.bits, self.D = layer, layer.cache.bits, layer.cache.head_dim
        self.signs = None if layer.cache.signs is None else host(layer.cache.signs)
        self.rows = [[([], []) for _ in range(layer.kv_heads)] for _ in range(layer.table.shape[0])]

    def stored(self, t, turned):
        if self.bits == 16:
            return t.astype(np.float64)
        t = t.astype(np.float32)
        if turned and self.signs is not None:
            t = kv.butterfly128(t, self.signs)
        return kv.dequant_rows(*kv.quant_rows(t, self.bits))

    def append(self, b, k, v):
        for h, (ks, vs) in enumerate(self.rows[b]):
            ks.append(self.stored(k[h], True))
            vs.append(self.stored(v[h], False))

    def attend(self, b, q):
        """(out, its bound) [heads, D]."""
        G = self.layer.heads // self.layer.kv_heads
        outs, tols = [], []
        for h, (ks, vs) in enumerate(self.rows[b]):
            qs = HostCache.turn(self, q[h * G:(h + 1) * G])
            k, v = np.array(ks), np.array(vs)
            use, scale = np.ones(len(k), bool), self.D ** -0.5
            out, p = kv.attend(qs, k, v, scale)
            view = types.SimpleNamespace(D=self.D, bits=self.bits, signs=self.signs, values=[({h: k}, {h: v})])
            outs.append(out)
            tols.append(_bounds(view, 0, h, qs, scale, use, out, p)[0])
        return np.concatenate(outs), np.concatenate(tols)

    def evict(self, mass, pos, budget, recent):
        for b, heads in enumerate(self.rows):
            for h, (ks, vs) in enumerate(heads):
                n = len(ks)
                _, src = kv.evict(mass[b, h, :n], pos[b, h, :n], budget, recent)
                heads[h] = ([ks[i] for i in src], [vs[i] for i in src])


@pytest.mark.parametrize("bits", [4, 8, 16])
def test_every_step_against_the_oracle(example, bits):
    log(f"decoding example, {bits} bits")
    hidden, lens, steps = 512, [100, 1, 37], 90
    layer = example.Attention4(hidden, 8, 2, len(lens), capacity=128, budget=48, recent=16, bits=bits, seed=bits)
    mirror, seen = Mirror(layer), []
    rows, out, evict = layer._rows, layer.out, layer.evict

    def watched_rows(x):
        q, k, v = rows(x)
        seen.append(tuple(host(t) for t in (q, k, v)))
        if len(seen) == 1:  # the prompts
            at = 0
            for b, n in enumerate(lens):
                for t in range(at, at + n):
                    mirror.append(b, seen[0][1][t], seen[0][2][t])
                at += n
        return q, k, v

    def watched_out(o):
        q, k, v = seen[-1]
        got = host(o).reshape(q.shape).astype(np.float64)
        for b in range(len(lens)):
            mirror.append(b, k[b], v[b])
            want, tol = mirror.attend(b, q[b])
            assert np.all(np.abs(got[b] - want) <= tol), (len(seen), b, float((np.abs(got[b] - want) / tol).max()))
        return out(o)

    def watched_evict():
        mirror.evict(host(layer.mass), host(layer.pos), layer.budget, layer.recent)
        evict()
        assert_equal(host(layer.lens), np.array([len(r[0][0]) for r in mirror.rows], np.int32), "lens")

    layer._rows, layer.out, layer.evict = watched_rows, watched_out, watched_evict
    x = example.decode(layer, lens, steps, hidden)
    assert len(seen) == steps + 1
    assert layer.evictions == 1  # after 28 steps; 80 more fit
    assert np.all(np.isfinite(host(x)))


def test_command(example, capsys):
    log("decoding example, its command")
    layer, x = example.main(["--hidden", "512", "--heads", "4", "--kv-heads", "1", "--batch", "2", "--prompt", "60",
                             "--steps", "20", "--capacity", "64", "--budget", "32", "--recent", "8"])
    assert tuple(x.shape) == (2, 512) and layer.evictions == 1
    assert "last states finite: True" in capsys.readouterr().out


def test_refusals(example):
    log("decoding example, refusals")
    with pytest.raises(ValueError, match="budget"):
        example.Attention4(512, 4, 1, 1, capacity=64, budget=64, recent=8)
    layer = example.Attention4(512, 4, 1, 1, capacity=64, budget=32, recent=8)
    with pytest.raises(ValueError, match="prompt"):
        example.decode(layer, [65], 1, 512)
