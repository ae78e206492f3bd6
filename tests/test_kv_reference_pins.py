"""Pins of kv_reference.py, the plain forms the cache's and the attention's GPU
tests compare with: cases worked out by hand, closed forms and invariants."""

import math
import random

import numpy as np
import pytest

import kv_reference as ref


def test_reserve_by_hand():
    # pages of 4; row 0 has 5 tokens (pages 2, 0) and gets 4 more: 9 need a third page; row 1 is new
    table, lens, refs = [[2, 0, -1], [-1, -1, -1]], [5, 0], [1, 0, 1, 0, 0, 7]
    assert ref.reserve(table, lens, refs, 4, [4, 5]) == ([[2, 0, 1], [3, 4, -1]], [9, 5], [1, 1, 1, 1, 1, 7], [0, 3])
    assert ref.reserve(table, lens, refs, 4, [3, 0])[3] == [0, 0]  # 8 tokens still fit
    assert ref.reserve(table, lens, refs, 4, [4, 9]) == (table, lens, refs, [1, 4])  # three pages are free
    assert ref.reserve(table, lens, refs, 4, [8, 0])[3][0] == 2  # 13 tokens pass three pages
    assert table == [[2, 0, -1], [-1, -1, -1]] and refs == [1, 0, 1, 0, 0, 7]


def test_fork_by_hand():
    # row 0: a full page 1 and a partial page 3; both children of it share page 1, the second copies page 3 to page 0
    table, lens, refs = [[1, 3], [2, -1]], [6, 4], [0, 1, 1, 1, 0]
    out = ref.fork(table, lens, refs, 4, [0, 0])
    assert out == ([[1, 3], [1, 0]], [6, 6], [1, 2, 0, 1, 0], [0, 1], [(3, 0)])
    # somebody else holds page 3: the first child copies, too; row 1 is dropped and its page is free only afterwards
    out = ref.fork(table, lens, [0, 1, 1, 2, 0], 4, [0, -1, 0])
    assert out == ([[1, 0], [-1, -1], [1, 4]], [6, 0, 6], [1, 2, 0, 1, 1], [0, 2], [(3, 0), (3, 4)])


def test_trim_by_hand():
    # pages of 4, 15 tokens, window 5, 2 sinks: a query at 15 sees 0, 1 and 11 .. 15
    table, lens, refs = [[5, 4, 3, 2]], [15], [0, 0, 1, 1, 1, 1]
    assert ref.trim(table, lens, refs, 4, 5, 2) == ([[5, -1, 3, 2]], [15], [0, 0, 1, 1, 0, 1])
    assert ref.trim(table, lens, refs, 4, 4, 0) == ([[-1, -1, -1, 2]], [15], [0, 0, 1, 0, 0, 0])


def test_compact_by_hand():
    table, lens, refs = [[6, 1, -1]], [8], [0, 1, 0, 0, 2, 0, 1]
    assert ref.compact(table, lens, refs) == ([[2, 1, -1]], [8], [2, 1, 1, 0, 0, 0, 0], [-1, 1, -1, -1, 0, -1, 2], [3, 2],
                                              [(4, 0), (6, 2)])


@pytest.mark.parametrize("seed", range(5))
def test_counts_stay_those_of_the_tables(seed):
    """Whatever is done, a page's count is the number of entries that hold it."""
    rng = random.Random(seed)
    page, width, pages = 4, 6, 40
    table, lens, refs = [[-1] * width for _ in range(5)], [0] * 5, [0] * pages
    for _ in range(60):
        what = rng.randrange(4)
        if what == 0:
            table, lens, refs, _ = ref.reserve(table, lens, refs, page, [rng.randint(0, 6) for _ in table])
        elif what == 1:
            out = ref.fork(table, lens, refs, page, [rng.randint(-1, 4) for _ in range(5)])
            if out[3][0] == 0:
                table, lens, refs = out[:3]
        elif what == 2:
            table, lens, refs = ref.trim(table, lens, refs, page, rng.randint(1, 20), rng.randint(0, 5))
        else:
            table, lens, refs, _, info, _ = ref.compact(table, lens, refs)
            assert all(r > 0 for r in refs[:info[0]]) and not any(refs[info[0]:])
        count = [0] * pages
        for row in table:
            for p in row:
                if p >= 0:
                    count[p] += 1
        assert count == refs


def make(n, heads, dim, page, seed=0):
    rng = np.random.default_rng(seed)
    pages = -(-n // page) + 1
    pool = rng.standard_normal((pages, 1, 2, heads, page, dim))
    return pool, [pages - 1 - k for k in range(pages - 1)], rng


def test_attend_is_the_softmax_written_out():
    pool, row, rng = make(11, 2, 8, 4)
    q = rng.standard_normal((4, 8))
    out, bound, absum = ref.attend(q, 9, pool, 0, row, 0.3, 4, 2)
    for h in range(4):
        num, den = np.zeros(8), 0.0
        for j in (0, 1, 6, 7, 8, 9):  # two sinks, a window of four
            k, v = pool[row[j // 4], 0, :, h // 2, j % 4]
            w = math.exp(0.3 * sum(float(a) * float(b) for a, b in zip(q[h], k)))
            num, den = num + w * v, den + w
        assert np.allclose(out[h], num / den, rtol=1e-12, atol=1e-12)
    assert (bound > 0).all() and (absum >= np.abs(out)).all()


def test_attend_closed_forms():
    pool, row, rng = make(12, 1, 8, 4)
    v = np.concatenate([pool[p, 0, 1, 0] for p in row])
    q = rng.standard_normal((1, 8))
    assert np.allclose(ref.attend(q, 11, pool, 0, row, 0.0, 0, 0)[0][0], v[:12].mean(0))     # equal weights
    assert np.allclose(ref.attend(q, 7, pool, 0, row, 1.0, 1, 0)[0][0], v[7])                # itself alone
    assert np.allclose(ref.attend(q, 2, pool, 0, row, 0.0, 0, 0)[0][0], v[:3].mean(0))       # nothing after it
    assert not ref.attend(q, -1, pool, 0, row, 1.0, 0, 0)[0].any()                           # nothing visible
    holes = [row[0], -1, 99]
    assert np.allclose(ref.attend(q, 11, pool, 0, holes, 0.0, 0, 0)[0][0], v[:4].mean(0))    # entries that are no page
    pool[:, :, 1] = 2.5
    assert np.allclose(ref.attend(q, 11, pool, 0, row, 1.0, 0, 0)[0], 2.5)                   # weights sum to 1
