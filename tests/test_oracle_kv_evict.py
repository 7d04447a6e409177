"""The eviction oracle where slots do not exist or positions repeat (CPU)."""
import numpy as np

from oracle import kv


def test_slots_that_do_not_exist():
    m = np.array([5, 1, 9, 3, 7, 8], np.float32)
    p = np.arange(6)
    there = [True, False, True, True, False, True]
    # Slot 1 keeps its place and 4 goes; of 0, 2, 3 and 5 two stay.
    assert kv.evict(m, p, 3, 0, there)[1].tolist() == [5, 1, 2]
    # The newest that exists is 5, or 3 where 5 does not.
    assert kv.evict(m, p, 2, 1, there)[1].tolist() == [5, 1]
    assert kv.evict(m, p, 2, 1, there[:5] + [False])[1].tolist() == [3, 1]
    assert kv.evict(m, p, 3, 3, [False] * 6)[1].tolist() == [0, 1, 2]
    assert kv.evict(m, p, 3, 1)[1].tolist() == kv.evict(m, p, 3, 1, [True] * 6)[1].tolist() == [4, 5, 2]


def test_every_existing_slot_that_stays_has_a_place_of_its_own():
    rng = np.random.default_rng(0)
    for _ in range(200):
        n = int(rng.integers(1, 40))
        budget, there = int(rng.integers(1, 40)), rng.random(n) < rng.random()
        recent = int(rng.integers(0, budget + 1))
        mass, pos = rng.random(n).astype(np.float32), rng.permutation(n)
        left, src = kv.evict(mass, pos, budget, recent, there)
        assert left == min(n, budget) and len(set(src.tolist())) == left
        for j, i in enumerate(src):
            assert there[j] == there[i] and (there[j] or i == j)


def test_more_newest_slots_than_fit_stay_by_mass():
    m = np.array([1, 9, 5, 20, np.nan, 9], np.float32)
    p = np.array([7, 7, 7, 2, 7, 7])
    assert kv.evict(m, p, 1, 1)[1].tolist() == [1]
    assert kv.evict(m, p, 2, 2)[1].tolist() == [5, 1]
    assert kv.evict(m, p, 4, 3)[1].tolist() == [0, 1, 2, 5]
    assert kv.evict(m, p, 5, 1)[1].tolist() == [0, 1, 2, 5, 4]
