"""The fork's oracle on requests that cannot be (CPU)."""

import numpy as np
import pytest

from oracle import paged_oracle as po


@pytest.mark.parametrize("page,parents", [(0, [0, 0, 1]), (1, [0, 0, 1]), (2, [0]), (4, [-1]), (4, [0, 0, 0])])
def test_counts_below_zero_are_refused_wherever_they_stand(page, parents):
    """Of a page that gains holders, keeps or loses them, and of a free one."""
    table, extra = np.array([[0, 1, -1], [0, 2, -1]]), np.array([1, 0, 0, 0, 0, 0])
    args = (np.array([40 - 16, 30]), table)
    for head in (0, 3):  # without room in front of the free list, and with it
        free = np.array([9] * head + [3, 4, 5])
        extra[page] = int(page == 0)
        # an ended sequence frees its last page, both free the common one; a second child takes a page
        live = [x for x in parents if x >= 0]
        ended = 2 - len(set(live))
        room = head + len(live) - len(set(live)) - ended - (ended == 2)
        assert (po.fork(parents, *args, extra, free, head, 16, 6) is None) == (room < 0)
        for n in (-1, -5):
            extra[page] = n
            assert po.fork(parents, *args, extra, free, head, 16, 6) is None
