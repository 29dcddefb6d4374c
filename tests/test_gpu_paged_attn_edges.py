"""GPU parity of paged attention and shared decode where their kernels' bookkeeping is at its edges:
many short segments of which only some are looked through, keys that outweigh all others, batches on
either side of what is worth sharing, lengths and moves that cannot be."""

import numpy as np
import pytest
import torch

from tests import test_gpu_paged as tp
from tests import test_gpu_paged_attn as ta
from token_sparse_attention_gb300 import build as mcs_build
from token_sparse_attention_gb300 import mcs

pytestmark = pytest.mark.gpu

_i32, _f64 = tp._i32, tp._f64


@pytest.fixture(scope="module", autouse=True)
def _lib():
    mcs_build.build()
    mcs.lib()
    yield
    assert mcs.mcs_device_status() == 0


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("D,gap", [(64, 1), (64, 3), (128, 1), (128, 2)])
def test_infinite_values_of_many_short_segments(D, gap, e4m3):
    """One token each of thousands of sequences, a dozen and more to a block: those that end with a tile of
    128 keys have nothing to look through, those between them do, and hold infinite values there."""
    r = np.random.default_rng(D + gap)
    B = 2500
    lens = [int(r.integers(1, 4)) * 128 - (0 if b % (gap + 1) else int(r.integers(1, 100))) for b in range(B)]
    c = ta.Step(lens, [1] * B, 2, 1, D, 128, e4m3, seed=D)
    want, want_ls = c.attn()
    hit = torch.zeros(c.q.shape, dtype=torch.bool, device="cuda")
    at = [b for b in range(0, B, gap + 1) if r.random() < 0.6]
    cols = r.integers(0, D, (len(at), 3))
    for i in range(3):
        pos = np.array([int(r.integers(lens[b] // 128 * 128, lens[b])) for b in at])
        pid = torch.from_numpy(c.table[at, pos // 128]).cuda()
        col = torch.from_numpy(cols[:, i]).cuda()
        c.v[pid, 0, torch.from_numpy(pos % 128).cuda(), col] = 0x7F if e4m3 else [np.inf, -np.inf, np.nan][i]
        hit[torch.tensor(at, device="cuda"), :, col] = True
    for _ in range(5):
        out, ls = c.attn()
        assert not torch.isfinite(out.float()[hit]).any()
        assert torch.equal(out[~hit], want[~hit]) and torch.equal(ls, want_ls)
    assert mcs.mcs_device_status() == 0


@pytest.mark.parametrize("D,page", [(64, 16), (128, 128)])
def test_nan_values_in_every_tile_that_masks_cut(D, page):
    """E4M3 prompts of many tiles whose values hold NaN codes here and there, and nothing but NaN behind the
    sequences: slots in which tiles are looked through are loaded again and again."""
    lens, new = [1500, 1130, 70, 2049], [1500, 1000, 70, 300]
    r = np.random.default_rng(D)
    c = ta.Step(lens, new, 8, 4, D, page, True, seed=D)
    want, want_ls = c.attn()
    hit = torch.zeros(c.q.shape, dtype=torch.bool, device="cuda")
    for b, (n, m) in enumerate(zip(lens, new)):
        for t in range(int(r.integers(0, 60)), n, 61):
            h, col = int(r.integers(0, 4)), int(r.integers(0, D))
            c.v[int(c.table[b, t // page]), h, t % page, col] = 0x7F if t % 2 else 0xFF
            hit[int(c.cu[b]) + max(0, t - (n - m)):int(c.cu[b + 1]), 2 * h:2 * h + 2, col] = True
    for _ in range(3):
        out, ls = c.attn()
        assert torch.isnan(out.float()[hit]).all()
        assert torch.equal(out[~hit], want[~hit]) and torch.equal(ls, want_ls)
    assert mcs.mcs_device_status() == 0
