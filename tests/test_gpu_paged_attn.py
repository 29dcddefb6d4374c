"""GPU parity of the attention of several new tokens per sequence, and of sequences with a common
beginning, against the fp64 oracle.

Tolerances, taken before the first run (u = 2^-24): those of test_gpu_paged.py, with the weights
rounded once to bf16 (2^-8 of a weight) or f16 (2^-11) and the output normalised by the sum of the
rounded ones: numerator and denominator are each off by that times A = sum p |v|.  A weight's
smallest part: weights below 2^-24 of 2^15 times the row's reference maximum round in f16 by at most
2^-25, and the reference may lie 2^15 below the true maximum: 2^-25 per key of a sum of at least 1.
"""

import numpy as np
import pytest
import torch

from oracle import paged_oracle as po
from tests import test_gpu_paged as tp
from token_sparse_attention_gb300 import build as mcs_build
from token_sparse_attention_gb300 import mcs

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
_i32, _f64 = tp._i32, tp._f64


@pytest.fixture(scope="module", autouse=True)
def _lib():
    mcs_build.build()
    mcs.lib()
    yield
    assert mcs.mcs_device_status() == 0


def tolerance(want, lse, absv, size, D, n, e4m3, weight=None):
    """(of out, of lse)"""
    delta = (D + 8) * U * size
    weight = (2.0 ** -11 + n * 2.0 ** -25 if e4m3 else 2.0 ** -8) if weight is None else weight
    out = 2.0 ** -8 * np.abs(want) + absv * (2 * (2 * delta + 2.0 ** -21 + weight) + n * U)[..., None]
    return out, delta + 2.0 ** -20 + n * U + 2.0 ** -23 * np.abs(np.where(np.isfinite(lse), lse, 0))


class Step(tp.Cache):
    """A cache of `lens` tokens, of which the last new[b] of each sequence are asked about."""

    def __init__(self, lens, new, Hq, Hkv, D, page, e4m3=False, seed=0, behind=3, scale=0.0, q_stride=0, q_size=1.0, **kw):
        super().__init__(lens, Hq, Hkv, D, page, e4m3, seed=seed, scale=scale, **kw)
        g = torch.Generator(device="cuda").manual_seed(seed + 1)
        self.new, self.T = new, sum(new) + behind
        self.cu = np.concatenate([[0], np.cumsum(new)])
        rows = torch.randn(self.T, q_stride or Hq * D, generator=g, device="cuda").to(torch.bfloat16) * q_size
        self.q = rows[:, :Hq * D].view(self.T, Hq, D)
        self.p.q_stride = q_stride
        self.dcu = _i32(self.cu)
        self.ws = mcs.empty_workspace(mcs.mcs_paged_attn_workspace(self.p))

    def attn(self, lse=True, stream=None):
        out = torch.full(self.q.shape, 77.0, dtype=torch.bfloat16, device="cuda")
        ls = torch.full(self.q.shape[:2], 77.0, device="cuda")
        mcs.mcs_paged_attn(self.p, self.q, self.k, self.v, self.dtable, self.dlens, self.dcu, out, self.ws,
                           lse=ls if lse else None, stream=stream)
        return out, ls

    def check_attn(self, out, ls, skip=()):
        k, v = (_f64(x) * s for x, s in zip((self.k, self.v), self.scales))
        want, lse, absv, size = po.attn(_f64(self.q), k, v, self.table, self.lens, self.cu, self.scale)
        out, ls = _f64(out), _f64(ls)
        for b in skip:
            want[self.cu[b]:self.cu[b + 1]], lse[self.cu[b]:self.cu[b + 1]] = np.nan, np.nan
        none = np.isnan(lse)
        assert (out[none] == 77).all() and (ls[none] == 77).all()
        live = ~none
        tol, tol_lse = tolerance(want, lse, absv, size, self.D, max(self.lens), self.e4m3)
        bad = live[..., None] & ~(np.abs(out - want) <= tol)
        assert not bad.any(), (len(np.argwhere(bad)), np.argwhere(bad)[:5], out[bad][:5], want[bad][:5])
        empty = live & ~np.isfinite(lse)
        assert (ls[empty] == -np.inf).all()
        some = live & np.isfinite(lse)
        off = np.abs(ls[some] - lse[some])
        assert (off <= tol_lse[some]).all(), off.max()


SHAPES = [  # lens, new, Hq, Hkv, D, page
    ([1], [1], 1, 1, 128, 16), ([77], [77], 16, 16, 64, 16), ([128], [128], 4, 1, 128, 128),
    ([129, 5], [129, 5], 8, 2, 128, 16), ([300, 0, 17, 40], [2, 0, 17, 0], 5, 1, 64, 64),
    ([700], [260], 8, 8, 128, 32), ([1000, 64], [1, 64], 20, 1, 128, 64), ([513], [513], 2, 2, 64, 16),
    ([900, 333, 128, 1], [3, 333, 1, 1], 12, 4, 128, 128), ([2500], [4], 8, 2, 128, 16), ([300, 260], [7, 260], 130, 1, 64, 32)]


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("lens,new,Hq,Hkv,D,page", SHAPES)
def test_attn_matches_oracle(lens, new, Hq, Hkv, D, page, e4m3):
    c = Step(lens, new, Hq, Hkv, D, page, e4m3, seed=sum(lens) + Hq)
    got = c.attn()
    assert mcs.mcs_device_status() == 0
    c.check_attn(*got)


# ------------------------------------------------------------------ common beginnings

class Family(tp.Cache):
    """Groups of sequences: (pages in common, [tokens of each behind them; None: an empty sequence])."""

    def __init__(self, groups, Hq, Hkv, D, page, e4m3=False, seed=0, **kw):
        lens, self.starts, self.shared = [], [0], []
        for pages, own in groups:
            lens += [0 if x is None else pages * page + x for x in own]
            self.starts.append(len(lens))
            self.shared.append(pages)
        super().__init__(lens, Hq, Hkv, D, page, e4m3, seed=seed, **kw)
        for (pages, own), a in zip(groups, self.starts):
            first = next((b for b in range(a, a + len(own)) if lens[b]), a)
            for b in range(a, a + len(own)):
                if lens[b]:
                    self.table[b, :pages] = self.table[first, :pages]
        self.dtable = _i32(self.table)
        self.dstarts, self.dshared = _i32(self.starts), _i32(self.shared)
        self.ws = mcs.empty_workspace(mcs.mcs_paged_decode_shared_workspace(self.p))

    def run(self, lse=True, stream=None):
        B, Hq, D = self.q.shape
        out = torch.full((B + 1, Hq, D), 77.0, dtype=torch.bfloat16, device="cuda")
        ls = torch.full((B + 1, Hq), 77.0, device="cuda")
        mcs.mcs_paged_decode_shared(self.p, self.q, self.k, self.v, self.dtable, self.dlens, self.dstarts, self.dshared,
                                    out[:B], self.ws, lse=ls[:B] if lse else None, stream=stream)
        return out, ls

    def check(self, out, ls):
        B, Hq, D = self.q.shape
        k, v = (_f64(x) * s for x, s in zip((self.k, self.v), self.scales))
        want, lse, absv, size = po.decode(_f64(self.q), k, v, self.table, self.lens, self.scale)
        assert (_f64(out[B]) == 77).all() and (_f64(ls[B]) == 77).all()
        out, ls = _f64(out[:B]), _f64(ls[:B])
        tol, tol_lse = tolerance(want, lse, absv, size, D, max(self.lens), self.e4m3)
        bad = ~(np.abs(out - want) <= tol)
        assert not bad.any(), (len(np.argwhere(bad)), np.argwhere(bad)[:5], out[bad][:5], want[bad][:5])
        live = np.isfinite(lse)
        assert (ls[~live] == -np.inf).all()
        assert (np.abs(ls[live] - lse[live]) <= tol_lse[live]).all()


FAMILIES = [  # groups, Hq, Hkv, D, page
    ([(1, [1, 1])], 1, 1, 128, 16), ([(9, [0, 5, 40])], 8, 2, 128, 16), ([(3, [7, 1, None, 300])], 4, 4, 64, 64),
    ([(5, [3] * 9), (0, [17, 40]), (2, [None, 9, 0]), (4, [None, None]), (3, [11])], 5, 1, 128, 32),
    ([(20, list(range(1, 41)))], 8, 2, 128, 16), ([(2, [5] * 70), (1, [200] * 3)], 20, 2, 64, 128),
    ([(60, [1, 90, 3, 4])], 34, 2, 128, 16), ([(0, [0 + 5, 9])], 4, 2, 128, 16), ([(130, [33, 2])], 260, 2, 64, 16)]


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("groups,Hq,Hkv,D,page", FAMILIES)
def test_shared_decode_matches_oracle(groups, Hq, Hkv, D, page, e4m3):
    c = Family(groups, Hq, Hkv, D, page, e4m3, seed=Hq + page)
    got = c.run()
    assert mcs.mcs_device_status() == 0
    c.check(*got)
