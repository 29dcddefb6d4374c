"""GPU tests of forks, compaction and page copies with requests at the edge of what they may hold."""

import numpy as np
import pytest
import torch

from tests import test_gpu_pages as tg
from tests import test_gpu_paged as tp
from token_sparse_attention_gb300 import build as mcs_build
from token_sparse_attention_gb300 import mcs

pytestmark = pytest.mark.gpu

_i32 = tp._i32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    mcs_build.build()
    mcs.lib()
    yield
    assert mcs.mcs_device_status() == 0


def test_copy_of_a_page_to_itself_is_checked_like_any_other():
    p = mcs.paged(1, 1, 1, 64, 16, 4, 1)
    k, v = (torch.arange(4 * 16 * 64, device="cuda").view(4, 1, 16, 64).to(torch.bfloat16) for _ in range(2))
    mean = torch.randn(4, 1, 64, device="cuda").to(torch.bfloat16)
    before = [x.clone() for x in (k, v, mean)]
    for row, status in (([2, 2, 16], 0), ([3, 3, 0], 0), ([-4, -4, 99], 0), ([4, 4, 3], 6), ([2 ** 31 - 1, 2 ** 31 - 1, 1], 6),
                        ([2, 2, 17], 6), ([0, 0, -1], 6)):
        mcs.mcs_paged_copy(p, _i32([row, [-1, -1, 0]]), k, v, mean)
        assert mcs.mcs_device_status() == status, row
        assert all(torch.equal(x, y) for x, y in zip((k, v, mean), before))


@pytest.mark.parametrize("count", [-1, -2, -2 ** 31])
@pytest.mark.parametrize("what", ["gains", "keeps", "loses", "free"])
def test_fork_refuses_counts_below_zero(what, count):
    """Of a page that gets more holders, one that keeps its holder, one that loses it, a free one."""
    s = tg.State(3, 2, 100, 90, 16, 9, seed=5, empty=0)
    b = next(b for b in range(6) if s.lens[b] >= 32)
    parents = {"gains": [b, b, b], "keeps": list(range(6)), "loses": [x for x in range(6) if x != b], "free": list(range(6))}[what]
    s.check_fork(parents, s.fork(parents), False)
    s.extra[s.free[-1] if what == "free" else s.table[b, 0]] = count
    for in_place in (False, True):
        lens, table, extra, free, head, moves = s.fork(parents, in_place)
        assert mcs.mcs_device_status() == 6
        assert (lens == -77).all() and (table == -77).all() and (moves == [-1, -1, 0]).all()
        assert (extra == (s.extra if in_place else -77)).all() and (free == (s.free if in_place else -77)).all()
        assert head.tolist() == [s.head if in_place else -77]
