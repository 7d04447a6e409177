"""A paged cache on the host and on the GPU, for the key/value cache tests."""
import numpy as np

from oracle import kv
from tests.gpu_helpers import dev


def signs128(rng):
    s = rng.choice([-1, 1], 128).astype(np.int8)
    s[0] = 1
    return s


class HostCache:
    """Rows of every slot, as they are stored, in NumPy; garbage wherever no
    sequence has a slot."""

    def __init__(self, rng, lens, max_len, heads, D, page, bits, rotate=False, extra_pages=3, outliers=True):
        self.heads, self.D, self.page, self.bits = heads, D, page, bits
        self.signs = signs128(rng) if rotate else None
        self.lens = np.asarray(lens, np.int32)
        B = len(lens)
        self.max_pages = max(1, -(-max_len // page))
        need = [-(-int(n) // page) for n in lens]
        self.pages = sum(need) + extra_pages
        ids = rng.permutation(self.pages).astype(np.int32)
        self.table = np.full((B, self.max_pages), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = ids[at:at + n]
            at += n
        shape = (self.pages, heads, page)
        if bits == 16:
            self.k, self.v = (np.full(shape + (D,), np.nan, np.float16) for _ in range(2))
            self.kmeta = self.vmeta = None
        else:
            self.k, self.v = (rng.integers(0, 256, shape + (D * bits // 8,)).astype(np.uint8) for _ in range(2))
            self.kmeta, self.vmeta = (np.full(shape + (2,), np.nan, np.float16) for _ in range(2))
        self.values = []  # per row: float64 (k, v) [heads, n, D], k as stored (turned with signs)
        for b in range(B):
            n = int(lens[b])
            kf, vf = (rng.standard_normal((heads, n, D)).astype(np.float16) for _ in range(2))
            if outliers:
                kf[..., D // 3] += np.float16(5)
            self.values.append((self._put(b, "k", kf), self._put(b, "v", vf)))

    def _put(self, b, name, rows):
        n = rows.shape[1]
        slot = np.arange(n)
        page, line = self.table[b, slot // self.page], slot % self.page
        if self.bits == 16:
            getattr(self, name)[page, :, line] = rows.transpose(1, 0, 2)
            return rows.astype(np.float64)
        t = rows.astype(np.float32)
        if name == "k" and self.signs is not None:
            t = kv.butterfly128(t, self.signs)
        codes, meta = kv.quant_rows(t, self.bits)
        stored = kv.pack4(codes) if self.bits == 4 else codes
        getattr(self, name)[page, :, line] = stored.transpose(1, 0, 2)
        getattr(self, name + "meta")[page, :, line] = meta.transpose(1, 0, 2)
        return kv.dequant_rows(codes, meta)

    def turn(self, q):
        """Queries as they meet the stored K rows, float64."""
        if self.signs is None:
            return q.astype(np.float64)
        from oracle import hadamard
        return (q.astype(np.float64) * self.signs) @ hadamard.sylvester(128) / 128.0

    def device(self, q):
        def put(a):
            return None if a is None else dev(a)
        return q.KVCache(put(self.k), put(self.v), self.D, self.bits, put(self.kmeta), put(self.vmeta),
                         put(self.signs))
