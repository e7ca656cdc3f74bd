"""The host rules of eviction by attention weight, on cases small enough to see."""
import numpy as np
import pytest

from oracle import compact as OC


def test_keep_first_recent_and_heaviest_with_ties():
    m = np.array([[0, 5, 1, 5, 5, 0, 2, 9.0]])
    idx, off = OC.keep_heavy(m, [8], [5], 1, 2)          # must: 0, 6, 7; two of the fives, the lower ones
    assert idx.tolist() == [0, 1, 3, 6, 7] and off.tolist() == [0, 5]


def test_keep_edges():
    m = np.arange(12.0).reshape(2, 6)
    assert OC.keep_heavy(m, [6, 0], [9, 9], 0, 0)[1].tolist() == [0, 6, 6]        # fewer than the budget; empty
    assert OC.keep_heavy(m, [6, 3], [0, 1], 2, 2)[0].tolist() == [0, 1, 4, 5, 0, 1, 2]   # protected beats the budget
    m[0] = [np.nan, -np.inf, -1, np.inf, -0.0, 0.0]
    assert OC.keep_heavy(m, [6, 0], [3, 0], 0, 0)[0].tolist() == [3, 4, 5]
    assert OC.keep_heavy(m, [6, 0], [5, 0], 0, 0)[0].tolist() == [1, 2, 3, 4, 5]


@pytest.mark.parametrize("shared", [False, True])
def test_compact_moves_rows(shared):
    block, cap = 4, 8
    slab = np.arange(cap * block, dtype=np.float64).reshape(cap, 1, block, 1)
    table, refs = np.array([[5, 2, 7]]), np.zeros(cap, np.int64)
    refs[[5, 2, 7]] = 2 if shared else 1
    keep = np.array([0, 1, 2, 3, 5, 9])
    s, t, ln, m, r, free, bad = OC.compact([slab], table, [11], keep, [0, 6], np.arange(12.0)[None], refs, [6, 4, 3, 1, 0], block)
    assert bad == [] and ln.tolist() == [6]
    assert t[0].tolist() == ([5, 0, -1] if shared else [5, 2, -1])
    where = t[0, 1]
    assert s[0][where, 0, :2, 0].tolist() == [2 * 4 + 1, 7 * 4 + 1]
    assert (s[0][where, 0, 2:] == slab[where, 0, 2:]).all()
    assert m[0].tolist() == [0, 1, 2, 3, 5, 9, 0, 0, 0, 0, 0, 11]
    assert free == ([6, 4, 3, 1] if shared else [6, 4, 3, 1, 0, 7])
    assert r.tolist() == ([1, 0, 1, 0, 0, 2, 0, 1] if shared else [0, 0, 1, 0, 0, 1, 0, 0])


def test_compact_leaves_what_it_cannot_do():
    slab = np.zeros((4, 1, 4, 1))
    args = dict(mass=None, refcount=np.array([2, 2, 0, 0]), block=4)
    for keep, free in (([1, 1], [3]), ([0, 9], [3]), ([1, 2], [])):
        _, t, ln, _, r, f, bad = OC.compact([slab], [[0, 1]], [8], np.array(keep), [0, 2], free=free, **args)
        assert bad == [0] and ln.tolist() == [8] and t.tolist() == [[0, 1]] and r.tolist() == [2, 2, 0, 0] and f == free
