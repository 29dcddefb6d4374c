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
