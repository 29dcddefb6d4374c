"""GPU parity of the attention of several new tokens per sequence, and of sequences with a common
beginning, against the fp64 oracle.

Tolerances, taken before the first run (u = 2^-24): those of test_gpu_paged.py, with the weights
rounded once to bf16 (2^-8 of a weight) or f16 (2^-11) for the product: numerator and, where rounded
weights are summed, denominator are each off by that times A = sum p |v|.  A weight's
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


def test_shared_decode_of_enough_to_be_read_once():
    """Beginnings long enough for the attention over them (small ones are read again): several groups of
    unequal size, empty sequences, one whose first sequence is empty, sequences that end with the
    beginning, and units that are pairs and odd ones."""
    for groups, Hq, Hkv, D, page, e4m3 in (
            ([(75, [None, 0, 9, 300, 17, 1] * 3), (0, [40, 5]), (5, [77])], 40, 2, 128, 128, False),
            ([(145, [5, 0, 40, None] * 10), (3, [0] * 3)], 8, 4, 64, 64, True), ([(8, [1, 2, 3] * 7)], 16, 16, 128, 128, False),
            ([(60, [9, 1] * 13), (61, [2] * 12)], 20, 4, 128, 64, True)):
        c = Family(groups, Hq, Hkv, D, page, e4m3, seed=Hq)
        saved = sum(p * page * (sum(x is not None for x in own) - 1) for p, own in groups) * Hkv * D * (2 if e4m3 else 4)
        assert saved > 2 ** 27
        again = [c.run() for _ in range(3)]
        assert mcs.mcs_device_status() == 0
        c.check(*again[0])
        for x in again[1:]:
            assert torch.equal(x[0], again[0][0]) and torch.equal(x[1], again[0][1])
        assert torch.equal(c.run(lse=False)[0], again[0][0])


def big_family(e4m3=False, seed=3, **kw):
    return Family([(40, [5, 0, 40, None, 9, 100] * 3), (20, [7] * 20)], 16, 8, 128, 128, e4m3, seed=seed, **kw)


@pytest.mark.parametrize("what", ["descends", "starts", "ends", "negative", "too many", "short", "length", "negative length"])
def test_shared_decode_reports_and_reads_by_itself(what):
    """What the arrays may get wrong costs the sharing, not the result."""
    c = big_family()
    starts, shared, lens = list(c.starts), list(c.shared), list(c.lens)
    if what == "descends":
        starts[1] = -4
    elif what == "starts":
        starts[0] = 1
    elif what == "ends":
        starts[-1] -= 1
    elif what == "negative":
        shared[0] = -1
    elif what == "too many":
        shared[1] = c.p.max_pages + 1
    elif what == "short":
        lens[4] = 33  # shorter than its group's beginning
    elif what == "length":
        lens[1] = c.p.max_pages * 128 + 1
    else:
        lens[1] = -1
    c.dstarts, c.dshared, c.dlens = _i32(starts), _i32(shared), _i32(lens)
    c.lens = [x if 0 <= x <= c.p.max_pages * 128 else 0 for x in lens]
    got = c.run()
    assert mcs.mcs_device_status() == 6
    c.check(*got)


@pytest.mark.parametrize("extra", [2, 70000], ids=["small table", "wide table"])
@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_little_in_common_is_read_by_itself(e4m3, extra):
    """Beginnings too small to be worth it, in tables that cannot name larger ones and in tables that can:
    the same bits, which are those of a decode, and the same reports."""
    c = Family([(9, [0, 5, 40]), (0, [17, None]), (3, [7, 1])], 8, 2, 128, 16, e4m3, seed=5, extra=extra)
    out, ls = c.run()
    assert mcs.mcs_device_status() == 0
    c.check(out, ls)
    plain, plain_ls = torch.empty_like(out[:c.B]), torch.empty_like(ls[:c.B])
    mcs.mcs_paged_decode(c.p, c.q, c.k, c.v, c.dtable, c.dlens, plain, c.ws, lse=plain_ls)
    assert extra > 2 or (torch.equal(plain, out[:c.B]) and torch.equal(plain_ls, ls[:c.B]))
    for starts, shared, change in (([0, 3, 2, 7], c.shared, {}), ([1, 3, 5, 7], c.shared, {}), ([0, 3, 5, 6], c.shared, {}),
                                   (c.starts, [9, -1, 3], {}), (c.starts, [9, c.p.max_pages + 1, 3], {}),
                                   (c.starts, c.shared, {1: 30}), (c.starts, c.shared, {5: -2}),
                                   (c.starts, c.shared, {5: c.p.max_pages * 16 + 1})):
        lens = list(c.lens)
        for b, n in change.items():
            lens[b] = n
        d = Family([(9, [0, 5, 40]), (0, [17, None]), (3, [7, 1])], 8, 2, 128, 16, e4m3, seed=5, extra=extra)
        d.dstarts, d.dshared, d.dlens = _i32(starts), _i32(shared), _i32(lens)
        d.lens = [x if 0 <= x <= d.p.max_pages * 16 else 0 for x in lens]
        got = d.run()
        assert mcs.mcs_device_status() == 6
        d.check(*got)


# ------------------------------------------------------------------ what masks hide, and what they do not

@pytest.mark.parametrize("Hq,Hkv,D,page", [(4, 1, 128, 16), (1, 1, 64, 64), (10, 2, 128, 32)])
def test_values_behind_a_token_do_not_reach_it(Hq, Hkv, D, page):
    """Infinite and NaN keys and values at some positions: tokens in front of them are as if they were
    not there, tokens that attend to them get NaN or infinities in those columns."""
    lens, new = [300, 40, 700, 129], [300, 40, 90, 128]
    for e4m3 in (False, True):
        clean = Step(lens, new, Hq, Hkv, D, page, e4m3, seed=11)
        first = clean.attn()
        c = Step(lens, new, Hq, Hkv, D, page, e4m3, seed=11)
        spots = [(0, 37, 5), (0, 255, 0), (0, 256, D - 1), (1, 39, 7), (2, 611, 3), (2, 650, 3), (2, 699, 9), (3, 128, 1), (3, 1, 2)]
        values = [float("inf"), float("-inf"), float("nan")]
        for i, (b, t, col) in enumerate(spots):
            pid = int(c.table[b, t // page])
            for h in range(Hkv):
                c.v[pid, h, t % page, col] = 0x7F if e4m3 else values[i % 3]
        out, ls = c.attn()
        assert mcs.mcs_device_status() == 0
        assert torch.equal(ls, first[1])
        hit = torch.zeros(out.shape, dtype=torch.bool, device="cuda")
        for b, t, col in spots:
            # tokens at or behind position t
            lo = int(c.cu[b]) + max(0, t - (lens[b] - new[b]))
            hit[lo:int(c.cu[b + 1]), :, col] = True
        assert not torch.isfinite(out.float()[hit]).any()
        assert torch.equal(out[~hit], first[0][~hit])
        # keys: everything at and behind them becomes NaN, nothing in front
        c = Step(lens, new, Hq, Hkv, D, page, e4m3, seed=11)
        for b, t in ((0, 200), (2, 640)):
            c.k[int(c.table[b, t // page]), :, t % page, 3] = 0x7F if e4m3 else float("nan")
        out, ls = c.attn()
        hit = torch.zeros(ls.shape, dtype=torch.bool, device="cuda")
        for b, t in ((0, 200), (2, 640)):
            hit[int(c.cu[b]) + t - (lens[b] - new[b]):int(c.cu[b + 1])] = True
        assert torch.isnan(out.float()[hit]).all() and torch.isnan(ls[hit]).all()
        assert torch.equal(out[~hit], first[0][~hit]) and torch.equal(ls[~hit], first[1][~hit])


def test_rows_behind_the_last_token_and_gaps_in_q_may_hold_anything():
    c = Step([130, 3, 77], [130, 2, 5], 8, 2, 128, 16, seed=2, behind=200, q_stride=12 * 128)
    first = c.attn()
    c.check_attn(*first)
    c.q[int(c.cu[-1]):] = float("nan")
    again = c.attn()
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_attn_peaked_scores_and_own_scale(e4m3):
    # scores spread over about +-100: the running maximum moves and most weights vanish
    c = Step([400, 33, 700, 90], [100, 33, 6, 90], 8, 2, 128, 16, e4m3, seed=5, scale=0.25, q_size=8.0)
    got = c.attn()
    c.check_attn(*got)
    assert torch.equal(c.attn(lse=False)[0], got[0])
    f = big_family(e4m3, scale=0.25, q_size=8.0)
    f.check(*f.run())


@pytest.mark.parametrize("scale", [1e-38, 1e-45])
def test_attn_of_vanishing_scales_is_the_mean(scale):
    c = Step([300, 129], [300, 4], 4, 2, 64, 32, seed=4, scale=scale)
    c.check_attn(*c.attn())


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_attn_of_many_segments_per_block_and_long_shares(e4m3):
    """Blocks that walk over many short segments, over pairs and odd units of many sequences, and shares
    that cut long ones into many parts; the same bits again."""
    r = np.random.default_rng(3)
    for lens, new, Hq, Hkv, D, page in (
            ([int(x) for x in r.integers(0, 90, 300)], None, 4, 2, 64, 16), ([200] * 40, [200] * 40, 8, 8, 128, 32),
            ([20011, 5], [3, 5], 4, 1, 128, 64), ([9000], [700], 4, 1, 128, 16), ([1500] * 3, [1500] * 3, 2, 1, 128, 128)):
        new = [int(r.integers(0, x + 1)) for x in lens] if new is None else new
        c = Step(lens, new, Hq, Hkv, D, page, e4m3, seed=8)
        got = c.attn()
        assert mcs.mcs_device_status() == 0
        c.check_attn(*got)
        again = c.attn()
        assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_attn_skips_pages_outside_the_cache(e4m3):
    c = Step([300, 90, 700, 40], [10, 90, 90, 3], 4, 2, 128, 16, e4m3, seed=6)
    c.table[0, 3], c.table[1, 0], c.table[2, 40], c.table[2, 0] = -1, c.p.num_pages, 2 ** 31 - 1, -7
    c.table[3, :3] = -1  # nothing is left: zeros
    c.dtable = _i32(c.table)
    got = c.attn()
    assert mcs.mcs_device_status() == 6
    c.check_attn(*got)
    f = big_family(e4m3)
    f.table[:int(f.starts[1]), 7] = f.p.num_pages + 1
    f.dtable = _i32(f.table)
    out, ls = f.run()
    assert mcs.mcs_device_status() == 6
    sel = np.full((len(f.lens), 8, f.table.shape[1]), -1)
    for b, n in enumerate(f.lens):
        live = [j for j in range(-(-n // 128)) if 0 <= f.table[b, j] < f.p.num_pages]
        sel[b, :, :len(live)] = live
    k, v = (_f64(x) * s for x, s in zip((f.k, f.v), f.scales))
    want, lse, absv, size = po.decode(_f64(f.q), k, v, f.table, f.lens, f.scale, sel)
    tol, tol_lse = tolerance(want, lse, absv, size, 128, max(f.lens), e4m3)
    assert (np.abs(_f64(out[:-1]) - want) <= tol).all()
    live = np.isfinite(lse)
    assert (np.abs(_f64(ls[:-1])[live] - lse[live]) <= tol_lse[live]).all() and (_f64(ls[:-1])[~live] == -np.inf).all()


@pytest.mark.parametrize("what", ["length", "negative", "more new than there are", "rows", "descends"])
def test_attn_reports_sequences_that_cannot_be(what):
    c = Step([300, 90, 70, 40], [10, 90, 9, 3], 4, 2, 64, 16, seed=6)
    lens, cu, skip = list(c.lens), [int(x) for x in c.cu], (1,)
    if what == "length":
        lens[1] = c.p.max_pages * 16 + 1
    elif what == "negative":
        lens[1] = -3
    elif what == "more new than there are":
        lens[1] = 89
    elif what == "rows":
        cu[4], skip = c.T + 1, (3,)
    elif what == "descends":
        cu[2], skip = 5, (1, 2)
    c.dlens, c.dcu = _i32(lens), _i32(cu)
    out, ls = c.attn()
    assert mcs.mcs_device_status() == 6
    if what == "descends":  # rows 5 .. of the third sequence are more than it has tokens
        assert (out[10:100] == 77).all() and (out[109:112] != 77).any()
        return
    c.check_attn(out, ls, skip)


def test_no_rows_and_no_new_tokens():
    c = Step([30, 20], [0, 0], 4, 2, 64, 16, seed=1)
    out, ls = c.attn()
    assert (out == 77).all() and (ls == 77).all()
    mcs.mcs_paged_attn(c.p, c.q[:0], c.k, c.v, c.dtable, c.dlens, c.dcu, out[:0], c.ws)
    assert mcs.mcs_device_status() == 0


# ------------------------------------------------------------------ streams, graphs, bounded waits

@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_another_stream_and_graphs_of_new_lengths(e4m3):
    c = Step([300, 90, 700, 40], [10, 90, 90, 3], 4, 2, 128, 16, e4m3, seed=6)
    f = big_family(e4m3)
    want, wantf = c.attn(), f.run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = c.attn(stream=s), f.run(stream=s)
    s.synchronize()
    assert torch.equal(got[0][0], want[0]) and torch.equal(got[1][0], wantf[0]) and torch.equal(got[1][1], wantf[1])
    # captured once, replayed with other lengths and another batch
    out, ls = (torch.full_like(x, 77.0) for x in want)
    outf, lsf = (torch.zeros_like(x[:-1]) for x in wantf)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(2):  # two of each behind one another, in the same workspaces
            mcs.mcs_paged_attn(c.p, c.q, c.k, c.v, c.dtable, c.dlens, c.dcu, out, c.ws, lse=ls)
            mcs.mcs_paged_decode_shared(f.p, f.q, f.k, f.v, f.dtable, f.dlens, f.dstarts, f.dshared, outf, f.ws, lse=lsf)
    graph.replay()
    assert torch.equal(out, want[0]) and torch.equal(outf, wantf[0][:-1]) and torch.equal(lsf, wantf[1][:-1])
    c.lens, c.new = [280, 90, 0, 33], [3, 1, 0, 33]
    c.cu = np.concatenate([[0], np.cumsum(c.new)])
    c.dlens.copy_(_i32(c.lens))
    c.dcu.copy_(_i32(c.cu))
    out.fill_(77.0)
    ls.fill_(77.0)
    f.dshared.copy_(_i32([30, 0]))
    graph.replay()
    c.check_attn(out, ls)
    f.check(torch.cat([outf, wantf[0][-1:]]), torch.cat([lsf, wantf[1][-1:]]))
    assert mcs.mcs_device_status() == 0


def test_groups_without_sequences():
    groups = [(0, []), (40, [5, 0, 40, None, 9, 100] * 3), (3, []), (20, [7] * 20), (1, [])]
    for c in (Family(groups, 16, 8, 128, 128, seed=4), Family([(0, []), (9, [0, 5]), (4, [3])], 8, 2, 64, 16, seed=4)):
        got = c.run()
        assert mcs.mcs_device_status() == 0
        c.check(*got)


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_calls_at_once_on_two_streams(e4m3):
    c = Step([300, 9000, 700, 40], [10, 90, 300, 3], 8, 2, 128, 16, e4m3, seed=6)
    f = big_family(e4m3)
    want, wantf = c.attn(), f.run()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(6):
        got += [(c.attn(stream=streams[0]), want), (f.run(stream=streams[1]), wantf)]
    for s in streams:
        s.synchronize()
    assert mcs.mcs_device_status() == 0
    assert all(torch.equal(x, y) for pair in got for x, y in zip(*pair))


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_pages_whose_offsets_pass_32_bits(e4m3):
    """The same pages at the end of caches of 4.3 GB: the same bits, and copies between both ends."""
    for c in (Step([300, 90, 700, 40], [10, 90, 90, 3], 16, 8, 128, 128, e4m3, seed=6), big_family(e4m3)):
        run = c.attn if isinstance(c, Step) else c.run
        want, n = run(), c.k.shape[0]
        N = 2 ** 32 // c.k[0].nbytes + n
        far = [torch.empty((N,) + x.shape[1:], dtype=x.dtype, device="cuda") for x in (c.k, c.v)]
        for x, y in zip(far, (c.k, c.v)):
            x[N - n:] = y
        held = (c.table >= 0) & (c.table < n)
        c.dtable = _i32(np.where(held, c.table + (N - n), c.table))
        c.k, c.v, c.p.num_pages = *far, N
        got = run()
        assert mcs.mcs_device_status() == 0
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        moves = _i32([[N - 1 - i, i, c.page] for i in range(n)])
        mcs.mcs_paged_copy(c.p, moves, c.k, c.v)
        assert mcs.mcs_device_status() == 0
        for x in far:
            assert torch.equal(x[:n].flip(0).view(torch.uint8), x[N - n:].view(torch.uint8))
        del far, c


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_withheld_loads_time_out_and_the_context_survives(e4m3, monkeypatch):
    c = Step([700, 300], [90, 300], 4, 2, 128, 16, e4m3, seed=6)
    want = c.attn()
    monkeypatch.setenv("MCS_TEST_FAULT", "stall_load")
    c.attn()
    assert mcs.mcs_device_status() == 5
    monkeypatch.delenv("MCS_TEST_FAULT")
    got = c.attn()
    assert mcs.mcs_device_status() == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
