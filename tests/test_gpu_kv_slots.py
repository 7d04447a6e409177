"""qlin_kv_slots and qlin_kv_pages against the oracle's loops: every value."""
import numpy as np
import pytest

from oracle import prompt
from tests.gpu_helpers import assert_equal, dev, host, log

pytestmark = pytest.mark.gpu


def _i32(x):
    return np.asarray(x, np.int32)


@pytest.mark.parametrize("B,top,pad", [(1, 1, 0), (1, 5000, 3), (3, 0, 5), (7, 3, 0), (64, 1, 0), (65, 300, 1),
                                       (255, 4, 1030), (256, 9, 0), (257, 40, 7), (1000, 3, 0), (5000, 2, 11)])
def test_slots(B, top, pad):
    from outlier_aware_bit_amd import qlin as q
    log(f"slots of {B} sequences, up to {top} tokens, {pad} of padding")
    rng = np.random.default_rng(B)
    add, lens, first = (_i32(rng.integers(0, n + 1, B)) for n in (top, 900, 70000))
    add[rng.random(B) < 0.3] = 0
    T = int(add.sum()) + pad
    for f in (None, first):
        got = q.qlin_kv_slots(dev(lens), dev(add), T, first=None if f is None else dev(f))
        want = prompt.slots(lens.tolist(), add.tolist(), T, None if f is None else f.tolist())
        for n, g, w in zip(("cu", "row", "slot", "position", "lens_out"), got, want):
            assert_equal(host(g), _i32(w), n)


def test_slots_without_room_and_odd_lengths():
    from outlier_aware_bit_amd import qlin as q
    log("slots, no room, negative lengths")
    lens, add = _i32([5, -3, 7, 0, 2]), _i32([700, -9, 900, 0, 2000])
    for T in (0, 1, 3, 699, 700, 701, 1024, 1600, 1601, 3600, 3601):
        got = q.qlin_kv_slots(dev(lens), dev(add), T)
        for g, w in zip(got, prompt.slots(lens.tolist(), add.tolist(), T)):
            assert_equal(host(g), _i32(w), f"T={T}")
    # Lengths that add up past 2^31.
    got = q.qlin_kv_slots(dev(_i32([0, 0, 0])), dev(_i32([2 ** 31 - 1] * 3)), 1500)
    assert host(got[0]).tolist() == [0, 1500, 1500, 1500] and host(got[1]).tolist() == [0] * 1500
    assert host(got[2]).tolist() == list(range(1500)) and host(got[4]).tolist() == [1500, 0, 0]


def test_slots_of_no_sequence_and_given_outputs():
    import torch
    from outlier_aware_bit_amd import qlin as q
    log("slots, no sequence; outputs of one's own")
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    cu, row, slot, position, lens_out = q.qlin_kv_slots(e, e, 3)
    assert host(cu).tolist() == [0] and host(row).tolist() == host(slot).tolist() == host(position).tolist() == [-1] * 3
    assert host(q.qlin_kv_slots(e, e, 0)[0]).tolist() == [0]
    out = [torch.full((n,), 77, dtype=torch.int32, device="cuda") for n in (3, 6, 6, 6, 2)]
    got = q.qlin_kv_slots(dev(_i32([4, 0])), dev(_i32([1, 3])), 6, None, *out)
    assert all(a is b for a, b in zip(got, out))
    for g, w in zip(got, prompt.slots([4, 0], [1, 3], 6)):
        assert_equal(host(g), _i32(w), "given")


def _state(rng, B, max_pages, page, spare, fill):
    """A pool whose pages are dealt out at random, the free ones in a ring that begins anywhere."""
    held = rng.integers(0, max(1, int(max_pages * fill)) + 1, B)
    total = int(held.sum())
    size = total + spare
    ids = rng.permutation(size)
    table, at = np.full((B, max_pages), -1), 0
    for b in range(B):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    ring, head = np.full(size, -1), int(rng.integers(0, size))
    ring[(head + np.arange(spare)) % size] = ids[total:]
    return _i32(table), _i32(held), _i32(ring), head, spare


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,max_pages,page,spare", [(1, 1, 16, 1), (1, 9, 64, 5), (7, 5, 16, 9), (64, 40, 32, 300),
                                                    (300, 513, 16, 2000), (1024, 3, 16, 500), (1025, 7, 1024, 900),
                                                    (3000, 17, 128, 4000)])
def test_pages(B, max_pages, page, spare, in_place):
    import torch
    from outlier_aware_bit_amd import qlin as q
    log(f"pages of {B} sequences, {max_pages} each, {spare} free, in place: {in_place}")
    rng = np.random.default_rng(B + max_pages)
    table, held, ring, head, count = _state(rng, B, max_pages, page, spare, 0.5)
    d_table, d_held, d_ring, d_state = dev(table), dev(held), dev(ring), dev(_i32([head, count]))
    for step in range(6):
        # Some grow by a little or a lot, some end, some want more than the table has, some a negative length.
        want = held.astype(np.int64) * page - rng.integers(0, page, B) + rng.integers(0, 3 * page, B) * (rng.random(B) < 0.5)
        want[rng.random(B) < 0.2] = 0
        want[rng.random(B) < 0.05] = (max_pages + 2) * page
        want[rng.random(B) < 0.05] = -4
        want = _i32(np.maximum(want, -5))
        old = [t.clone() for t in (d_table, d_held, d_state)]
        out = {} if in_place else dict(table_out=torch.full_like(d_table, 99), held_out=torch.full_like(d_held, 99),
                                       state_out=torch.full_like(d_state, 99))
        got = q.qlin_kv_pages(dev(want), page, d_table, d_held, d_ring, d_state, **out)
        w = prompt.pages(want.tolist(), page, table.tolist(), held.tolist(), ring.tolist(), head, count)
        table, held, ring, (head, count) = _i32(w[0]), _i32(w[1]), _i32(w[2]), w[3:5]
        assert_equal(host(got[0]), table, f"table, step {step}")
        assert_equal(host(got[1]), held, f"held, step {step}")
        assert_equal(host(d_ring), ring, f"ring, step {step}")
        assert_equal(host(got[2]), _i32([head, count]), f"state, step {step}")
        assert host(got[3]).tolist() == [w[5]], step
        if not in_place:
            for was, t in zip(old, (d_table, d_held, d_state)):
                assert torch.equal(was, t)
            d_table, d_held, d_state = got[:3]
        free = ring[(head + np.arange(count)) % len(ring)]
        assert sorted(free.tolist() + table[table >= 0].tolist()) == list(range(len(ring)))  # every page once


def test_counts_that_contradict_each_other_stay_in_bounds():
    import torch
    from outlier_aware_bit_amd import qlin as q
    log("pages, counts out of range")
    ring = dev(_i32([3, 4, 5]))
    for state in ([-1, 2], [2 ** 31 - 1, 2 ** 31 - 1], [1, -7], [5, 9]):
        table, held = dev(_i32([[0, 1], [2, -1]])), dev(_i32([2 ** 31 - 1, -4]))
        out = q.qlin_kv_pages(dev(_i32([0, 20])), 16, table, held, ring, dev(_i32(state)))
        s = host(out[2])
        assert 0 <= s[0] < 3 and 0 <= s[1] <= 3 and np.all(host(out[1]) >= 0) and np.all(host(out[1]) <= 2)
    torch.cuda.synchronize()


def test_no_sequences():
    import torch
    from outlier_aware_bit_amd import qlin as q
    log("pages of no sequence")
    table = torch.empty((0, 4), dtype=torch.int32, device="cuda")
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    out = q.qlin_kv_pages(e, 16, table, e, dev(_i32([1, 0])), dev(_i32([1, 2])))
    assert host(out[2]).tolist() == [1, 2] and host(out[3]).tolist() == [0]


def test_refusals():
    from outlier_aware_bit_amd import qlin as q
    log("slots and pages, refusals")
    lens, add = dev(_i32([1, 2])), dev(_i32([1, 1]))
    for err, kw in ((TypeError, dict(lens=lens.long())), (ValueError, dict(add=add[:1])), (ValueError, dict(T=-1)),
                    (ValueError, dict(lens=lens.cpu())), (ValueError, dict(row=add)), (q.QlinError, dict(lens_out=lens)),
                    (ValueError, dict(first=add[:1])), (ValueError, dict(cu=add))):
        a = dict(lens=lens, add=add, T=5)
        a.update(kw)
        with pytest.raises(err):
            q.qlin_kv_slots(**a)
    table, ring, state = dev(_i32([[0, -1], [1, -1]])), dev(_i32([2, 3])), dev(_i32([0, 2]))
    for err, kw in ((q.QlinError, dict(page=20)), (TypeError, dict(table=table.long())), (ValueError, dict(held=add[:1])),
                    (ValueError, dict(state=ring[:1])), (ValueError, dict(table_out=table[:1])),
                    (ValueError, dict(ring=ring.cpu())), (ValueError, dict(missing=add)), (q.QlinError, dict(held_out=lens))):
        a = dict(want=lens, page=16, table=table, held=add, ring=ring, state=state)
        a.update(kw)
        with pytest.raises(err):
            q.qlin_kv_pages(**a)
