"""Pins of the oracle's prompts, forks and compaction: worked by hand, or against another of its
functions (CPU only)."""

import numpy as np

from oracle import paged_oracle as po


def test_attn_of_one_new_token_is_decode_and_rows_see_only_what_is_in_front():
    r = np.random.default_rng(0)
    page, num, Hkv, D, Hq = 4, 9, 2, 8, 6
    k, v = r.standard_normal((2, num, Hkv, page, D))
    table = r.permutation(num)[:8].reshape(2, 4)
    lens, new = [11, 6], [5, 6]
    cu = np.cumsum([0] + new)
    q = r.standard_normal((12, Hq, D))
    out, lse, absv, size = po.attn(q, k, v, table, lens, cu, 0.3)
    assert np.isnan(out[11]).all() and np.isnan(lse[11]).all()
    for b in range(2):
        for t in range(new[b]):
            n = [0, 0]
            n[b] = lens[b] - new[b] + t + 1
            qq = np.zeros((2, Hq, D))
            qq[b] = q[cu[b] + t]
            want = po.decode(qq, k, v, table, n, 0.3)
            for x, y in zip((out, lse, absv, size), want):
                np.testing.assert_allclose(x[cu[b] + t], y[b], rtol=1e-12)


def test_attn_by_hand():
    k, v = np.zeros((1, 1, 4, 1)), np.arange(4.0).reshape(1, 1, 4, 1)
    out, lse, _, _ = po.attn(np.ones((3, 1, 1)), k, v, np.array([[0]]), [4], [0, 3], 1.0)
    np.testing.assert_allclose(out[:, 0, 0], [0.5, 1.0, 1.5])
    np.testing.assert_allclose(np.exp(lse[:, 0]), [2, 3, 4])


def test_fork_by_hand():
    # two sequences of 6 and 4 tokens, pages of 4: pages 5, 2 and 7; page 5 has one more holder elsewhere
    table = np.array([[5, 2, 9], [7, -1, -1]])
    extra = np.zeros(10, int)
    extra[5] = 1
    free = np.array([-1, -1, -1, 3, 8, 0, 1])
    lens, to, ex, rest, head, moves = po.fork([0, -1, 0, 0], [6, 4], table, extra, free, 3, 4, 10)
    assert lens.tolist() == [6, 0, 6, 6]
    assert to.tolist() == [[5, 2, -1], [-1, -1, -1], [5, 3, -1], [5, 8, -1]]
    assert moves.tolist() == [[-1, -1, 0], [-1, -1, 0], [2, 3, 2], [2, 8, 2]]
    assert ex.tolist() == [0, 0, 0, 0, 0, 3, 0, 0, 0, 0]
    # page 7 is free again, in front of what is left
    assert head == 4 and rest == [7, 0, 1]
    # everything ends: page 5 stays with its other holder
    lens, to, ex, rest, head, moves = po.fork([-1], [6, 4], table, extra, free, 3, 4, 10)
    assert ex[5] == 0 and head == 1 and rest == [2, 7, 3, 8, 0, 1]


def test_fork_refuses():
    table, extra, free = np.array([[0, 1]]), np.zeros(4, int), np.array([-1, -1, 2])
    assert po.fork([0, 0], [6], table, extra, free, 2, 4, 4) is not None
    assert po.fork([0, 0, 0], [6], table, extra, free, 2, 4, 4) is None
    assert po.fork([1], [6], table, extra, free, 2, 4, 4) is None
    assert po.fork([0], [9], table, extra, free, 2, 4, 4) is None
    assert po.fork([0], [6], np.array([[0, 4]]), extra, free, 2, 4, 4) is None
    assert po.fork([-1], [6], table, extra, free, 1, 4, 4) is None  # two pages freed, room for one


def test_compact_by_hand():
    table, extra = np.array([[8, 1, 3], [8, 6, 0]]), np.array([0, 4, 0, 0, 0, 0, 2, 0, 1, 0])
    # pages 8, 1 (both), 6 are in use: 8 -> 0, 6 -> 2, 1 stays
    to, ex, free, head, moves = po.compact([7, 5], table, extra, 10, 5, 4, 10)
    assert moves.tolist() == [[8, 0, 4], [6, 2, 1], [-1, -1, 0], [-1, -1, 0], [-1, -1, 0]]
    assert to.tolist() == [[0, 1, 3], [0, 2, 0]]
    assert ex.tolist() == [1, 4, 2, 0, 0, 0, 0, 0, 0, 0]
    assert free == [3, 4, 5, 6, 7, 8, 9] and head == 3
    to, ex, free, head, moves = po.compact([7, 5], table, extra, 10, 1, 4, 10)
    assert moves.tolist() == [[8, 0, 4]] and free == [2, 3, 4, 5, 7, 8, 9]
    assert po.compact([7, 5], table, extra, 6, 1, 4, 10) is None


def test_copy_by_hand():
    k = np.arange(3 * 2 * 4.0).reshape(3, 1, 4, 2)
    v, mean = k + 100, np.arange(3.0)
    po.copy([(-1, -1, 0), (2, 0, 3)], k, v, mean)
    assert k[0, 0].tolist() == [[16, 17], [18, 19], [20, 21], [6, 7]] and (v == k + 100).all()
    assert mean.tolist() == [2, 1, 2]
