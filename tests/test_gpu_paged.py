"""GPU parity of the paged-cache entry points against the fp64 oracle.

Tolerances, taken before the first run (u = 2^-24, half a step of fp32):

* attention output: rounding to bf16 is off by at most 2^-8 |out|.  A score is
  a sum of D products in fp32, off by at most delta = (D + 8) u S with S the
  largest sum of |q k| scale of the row, and its exponential by 2 delta and
  2^-21 (the hardware's base-2 exponential and the argument's rounding); both
  change the weights, so the output by at most that times A = sum p |v|,
  numerator and denominator.  The weights enter the second product as two bf16
  parts (off by 2^-16) or one f16 (2^-11), again times A; sums of the products
  add (number of keys) u A.
* lse: delta + 2^-20 + 2^-23 |lse| + (number of keys) u.
* page means: 2^-8 |mean| for bf16, and (page + 2) u times the mean of |k|.
* codes, copied rows, slots, tables and selections: equal.
"""

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import mcs_oracle as orc
from oracle import paged_oracle as po
from token_sparse_attention_gb300 import build as mcs_build
from token_sparse_attention_gb300 import mcs

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
KS, VS = 3 / 256, 45 / 4096


@pytest.fixture(scope="module", autouse=True)
def _lib():
    mcs_build.build()
    mcs.lib()
    assert torch.cuda.is_available()
    yield
    assert mcs.mcs_device_status() == 0


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def _f64(t):
    if t.dtype == torch.uint8:
        return orc.e4m3_decode(t.cpu().numpy()).astype(np.float64)
    return t.cpu().double().numpy()


class Cache:
    """A paged cache of given lengths; rows without a token, spare pages and table entries
    past a sequence's end hold NaN or numbers outside the cache."""

    def __init__(self, lens, Hq, Hkv, D, page, e4m3=False, seed=0, level=0.8, extra=2, scale=0.0,
                 q_stride=0, q_size=1.0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = np.random.default_rng(seed)
        B, n = len(lens), [-(-x // page) for x in lens]
        total, P = sum(n) + 3, max(n) + extra
        self.lens, self.page, self.B, self.D, self.e4m3 = lens, page, B, D, e4m3
        self.table = np.full((B, P), 2 ** 31 - 1)
        order, at = r.permutation(total), 0
        shape = (total, Hkv, page, D)
        rand = lambda *s: torch.randn(*s, generator=g, device="cuda")
        k = level * rand(total, Hkv, 1, D) + 0.7 * rand(*shape)
        v = rand(*shape)
        hole = torch.ones(total, page, dtype=torch.bool, device="cuda")
        for b in range(B):
            for j in range(n[b]):
                self.table[b, j] = order[at]
                hole[order[at], :min(page, lens[b] - j * page)] = False
                at += 1
        self.scales = (KS, VS) if e4m3 else (1.0, 1.0)
        if e4m3:
            enc = lambda x, s: (x / s).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            k, v, nan = enc(k, KS), enc(v, VS), 0x7F
        else:
            k, v, nan = k.to(torch.bfloat16), v.to(torch.bfloat16), float("nan")
        self.k, self.v = (x.masked_fill(hole[:, None, :, None], nan) for x in (k, v))
        rows = rand(B, q_stride or Hq * D).to(torch.bfloat16) * q_size
        self.q = rows[:, :Hq * D].view(B, Hq, D)
        self.p = mcs.paged(B, Hq, Hkv, D, page, total, P, kv=int(e4m3), scale=scale,
                           k_scale=self.scales[0], v_scale=self.scales[1], q_stride=q_stride)
        self.scale = scale or D ** -0.5
        self.dtable, self.dlens = _i32(self.table), _i32(lens)
        self.ws = mcs.empty_workspace(mcs.mcs_paged_decode_workspace(self.p))

    def means(self):
        """bf16 means of the tokens in each page, NaN where there are none."""
        k = torch.from_numpy(_f64(self.k)) * self.scales[0]
        return torch.nanmean(k, 2).to(torch.bfloat16).cuda()

    def run(self, sel=None, lse=True, stream=None):
        # everything is written over, and one row behind the last sequence stays
        B, Hq, D = self.q.shape
        out = torch.full((B + 1, Hq, D), 77.0, dtype=torch.bfloat16, device="cuda")
        ls = torch.full((B + 1, Hq), 77.0, device="cuda")
        a = (self.dtable, self.dlens) if sel is None else (self.dtable, self.dlens, sel)
        f = mcs.mcs_paged_decode if sel is None else mcs.mcs_paged_decode_sparse
        f(self.p, self.q, self.k, self.v, *a, out[:B], self.ws, lse=ls[:B] if lse else None,
          stream=stream)
        return out, ls

    def check(self, out, ls, sel=None, terms=2 ** 31):
        B, Hq, D = self.q.shape
        k, v = (_f64(x) * s for x, s in zip((self.k, self.v), self.scales))
        q = self.q
        want, lse, absv, size = po.decode(_f64(q), k, v, self.table, self.lens, self.scale, sel)
        assert (_f64(out[B]) == 77).all() and (_f64(ls[B]) == 77).all()
        out, ls = _f64(out[:B]), _f64(ls[:B])
        n = min(max(self.lens), terms)
        delta = (D + 8) * U * size
        tol = 2.0 ** -8 * np.abs(want) + absv * (
            2 * (2 * delta + 2.0 ** -21) + (2.0 ** -11 if self.e4m3 else 2.0 ** -16) + n * U)[..., None]
        bad = ~(np.abs(out - want) <= tol)
        assert not bad.any(), (np.argwhere(bad)[:5], out[bad][:5], want[bad][:5])
        live = np.isfinite(lse)
        assert (ls[~live] == -np.inf).all()
        off = np.abs(ls[live] - lse[live])
        assert (off <= (delta + 2.0 ** -20 + n * U)[live] + 2.0 ** -23 * np.abs(lse[live])).all(), off.max()


SHAPES = [  # lens, Hq, Hkv, D, page
    ([1], 1, 1, 128, 16), ([1], 8, 1, 64, 128), ([16], 4, 4, 128, 16), ([17], 16, 2, 128, 16),
    ([0, 1, 15, 16, 33], 8, 2, 128, 16), ([129, 128, 0, 127], 5, 1, 64, 64),
    ([700, 3, 64], 20, 1, 128, 64), ([255, 1000], 34, 2, 64, 32), ([0, 0], 4, 2, 128, 128),
    ([513, 31, 2, 0, 260, 77, 1, 128], 6, 3, 128, 128), ([3001], 32, 8, 128, 16),
    ([1501, 40], 16, 16, 64, 32), ([2100], 40, 40, 128, 32)]


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("lens,Hq,Hkv,D,page", SHAPES)
def test_decode_matches_oracle(lens, Hq, Hkv, D, page, e4m3):
    c = Cache(lens, Hq, Hkv, D, page, e4m3, seed=sum(lens) + Hq)
    c.check(*c.run())
    assert mcs.mcs_device_status() == 0


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_decode_strided_queries_own_scale_and_peaks(e4m3):
    # q inside a fused projection; scores spread over about +-100, so that the running
    # maximum moves and most weights vanish
    c = Cache([400, 33, 0, 90], 8, 2, 128, 16, e4m3, seed=5, scale=0.25, q_stride=12 * 128, q_size=8.0)
    c.check(*c.run())
    # without lse
    out, ls = c.run(lse=False)
    assert torch.equal(out, c.run()[0]) and (ls == 77).all()


def test_decode_many_sequences_and_long_ones():
    c = Cache([int(x) for x in np.random.default_rng(0).integers(0, 90, 300)], 4, 2, 64, 16, seed=8)
    c.check(*c.run())
    c = Cache([20011, 5], 4, 1, 128, 64, seed=9)
    c.check(*c.run())


@pytest.mark.parametrize("B,Hq,Hkv,D,e4m3,most", [(26, 8, 8, 128, False, 9000), (84, 16, 16, 64, True, 4600),
                                                  (1, 10, 5, 128, False, 290000), (1, 18, 2, 128, False, 700000)])
def test_decode_of_lists_long_enough_for_the_last_blocks(B, Hq, Hkv, D, e4m3, most):
    # sequences of shared pages (a page may stand in many tables): lists so long that the
    # last part of them goes to blocks of its own, with empty and short sequences in it
    r = np.random.default_rng(most)
    c = Cache([30 * 128] + [0] * (B - 1), Hq, Hkv, D, 128, e4m3, seed=B, extra=-(-most // 128) - 30)
    live = c.table[0, :30].copy()
    c.lens = [int(x) for x in r.integers(most * 9 // 10, most, B)]
    for i, x in ((2, 0), (B // 2, 1), (B - 6, 0), (B - 4, 17), (B - 1, 128)):
        if B > 1:
            c.lens[i] = x
    c.table = live[r.integers(0, 30, c.table.shape)]
    c.dtable, c.dlens = _i32(c.table), _i32(c.lens)
    first = c.run()
    # no sum has more terms behind one another than a thread's of 80 tiles, 16 a tile, and
    # one per part of a segment, at most 608 blocks: below 2048
    c.check(*first, terms=2048)
    again = c.run()
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def _sel(c, select, seed, holes=False):
    r = np.random.default_rng(seed)
    Hkv = c.k.shape[1]
    sel = np.full((c.B, Hkv, select), -1)
    for b, x in enumerate(c.lens):
        n = -(-x // c.page)
        for h in range(Hkv):
            kept = np.sort(r.permutation(n)[:min(n, select)])
            sel[b, h, :len(kept)] = kept
            if holes and len(kept) > 1:
                sel[b, h, r.integers(0, len(kept))] = -1
    return sel


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("lens,Hq,Hkv,D,page,select", [
    ([1], 1, 1, 128, 16, 1), ([100, 0, 17], 8, 2, 128, 16, 3), ([1000, 33], 20, 1, 64, 32, 7),
    ([700, 64, 1], 16, 4, 128, 64, 5), ([3000, 2999], 8, 8, 128, 16, 40), ([500], 6, 2, 64, 128, 9)])
def test_sparse_decode_matches_oracle(lens, Hq, Hkv, D, page, select, e4m3):
    c = Cache(lens, Hq, Hkv, D, page, e4m3, seed=select)
    for holes in (False, True):
        sel = _sel(c, select, select, holes)
        c.check(*c.run(_i32(sel)), sel)
    # every page listed: the dense result up to summation order
    if select >= max(-(-x // page) for x in lens):
        c.check(*c.run(_i32(_sel(c, select, 0))))


@pytest.mark.parametrize("lens,Hq,Hkv,D,page,select,sink,recent", [
    ([1], 1, 1, 128, 16, 1, 0, 0), ([100, 0, 17, 16], 8, 2, 128, 16, 3, 1, 1),
    ([4000, 33], 20, 1, 64, 16, 100, 0, 2), ([2500, 64], 16, 4, 128, 32, 2, 2, 0),
    ([900, 800, 5], 32, 2, 64, 16, 30, 0, 0), ([20000], 2, 1, 128, 16, 333, 1, 3)])
def test_select_matches_oracle(lens, Hq, Hkv, D, page, select, sink, recent):
    c = Cache(lens, Hq, Hkv, D, page, seed=select)
    ws = mcs.empty_workspace(mcs.mcs_paged_select_workspace(c.p))
    mean = c.means()
    sel = torch.full((c.B, Hkv, select), -7, dtype=torch.int32, device="cuda")
    mcs.mcs_paged_select(c.p, c.q, mean, c.dtable, c.dlens, sel, ws, sink=sink, recent=recent)
    want = po.select(_f64(c.q), _f64(mean), c.table, lens, page, select, sink, recent)
    np.testing.assert_array_equal(sel.cpu().numpy(), want)


@pytest.mark.parametrize("n,select", [(5000, 1), (5000, 1234), (37, 36), (1025, 1024)])
def test_select_ties_go_to_the_lower_page(n, select):
    # three distinct scores, -0 among them, and whole rows of equal ones
    r = np.random.default_rng(n)
    page, D = 16, 64
    p = mcs.paged(2, 2, 1, D, page, n, n)
    mean = np.zeros((n, 1, D))
    mean[:, 0, 0] = r.integers(-1, 2, n)
    mean[::7, 0, 0] = -0.0
    table = np.stack([r.permutation(n), np.arange(n)])
    q = np.zeros((2, 2, D))
    q[0, :, 0] = 0.5
    lens = [n * page - 3, n * page]
    md, qd = (torch.from_numpy(x).cuda().to(torch.bfloat16) for x in (mean, q))
    sel = torch.empty(2, 1, select, dtype=torch.int32, device="cuda")
    ws = mcs.empty_workspace(mcs.mcs_paged_select_workspace(p))
    mcs.mcs_paged_select(p, qd, md, _i32(table), _i32(lens), sel, ws, sink=0, recent=0)
    want = po.select(q, mean, table, lens, page, select, 0, 0)
    np.testing.assert_array_equal(sel.cpu().numpy(), want)


def test_select_near_ties_follow_the_exact_sum():
    # scores that cancel: large parts of both signs leave differences at fp32's last bits
    r = np.random.default_rng(4)
    n, page, D, select = 600, 16, 128, 77
    p = mcs.paged(1, 4, 1, D, page, n, n)
    mean = np.zeros((n, 1, D))
    mean[:, 0, :63] = r.standard_normal((n, 63)) * 1000
    mean[:, 0, 64:127] = -mean[:, 0, :63]
    mean[:, 0, 127] = r.standard_normal(n) * 0.01
    md = torch.from_numpy(mean).cuda().to(torch.bfloat16)
    qd = torch.ones(1, 4, D, device="cuda", dtype=torch.bfloat16)
    qd[:, 1] = 2.0 ** -9
    sel = torch.empty(1, 1, select, dtype=torch.int32, device="cuda")
    ws = mcs.empty_workspace(mcs.mcs_paged_select_workspace(p))
    table = r.permutation(n)[None]
    mcs.mcs_paged_select(p, qd, md, _i32(table), _i32([n * page]), sel, ws, sink=0, recent=0)
    want = po.select(_f64(qd), _f64(md), table, [n * page], page, select, 0, 0)
    np.testing.assert_array_equal(sel.cpu().numpy(), want)


@pytest.mark.parametrize("n,m", [(600, 3), (600, 40), (5000, 200), (5000, 300), (9000, 7), (9000, 400)])
def test_select_inside_a_cluster_of_near_ties(n, m):
    # scores of any size, and m of them that agree to about fp32's last bits (some fully) at the
    # threshold; pages that are always kept, and one outside the cache
    r = np.random.default_rng(n + m)
    page, D = 32, 128
    mean = r.standard_normal((n, 1, D))
    mean[:, 0, 127] = 0
    cluster = r.permutation(n)[:m]
    mean[cluster] = mean[cluster[0]]
    mean[cluster, 0, 127] = r.integers(-3, 4, m) * 2.0 ** -7
    md = torch.from_numpy(mean).cuda().to(torch.bfloat16)
    q = r.standard_normal((1, 2, D))
    q[:, :, 127] = 2.0 ** -13
    qd = torch.from_numpy(q).cuda().to(torch.bfloat16)
    table = r.permutation(n)[None]
    score = (_f64(md)[table[0], 0] @ _f64(qd)[0].sum(0)).astype(np.float32)
    above = int((score > score[table[0] == cluster[0]].max() + 1e-3).sum())
    for select in (above + m // 2, above + m, above + 1):
        select = min(max(select, 5), n - 1)
        bad = table.copy()
        bad[0, np.argmin(score)] = n  # not among the kept ones
        p = mcs.paged(1, 2, 1, D, page, n, n)
        sel = torch.empty(1, 1, select, dtype=torch.int32, device="cuda")
        ws = mcs.empty_workspace(mcs.mcs_paged_select_workspace(p))
        mcs.mcs_paged_select(p, qd, md, _i32(bad), _i32([n * page]), sel, ws, sink=2, recent=3)
        assert mcs.mcs_device_status() != 0  # the page outside
        want = po.select(_f64(qd), _f64(md), table, [n * page], page, select, 2, 3)
        np.testing.assert_array_equal(sel.cpu().numpy(), want)


@pytest.mark.parametrize("scale", [1.0, 2.0 ** -80, 2.0 ** 100])
def test_select_follows_the_exact_sum_at_any_size(scale):
    """Means whose squares vanish or overflow in fp32, and infinite ones."""
    r = np.random.default_rng(6)
    n, page, D, select = 400, 16, 64, 60
    p = mcs.paged(1, 2, 2, D, page, n, n)
    md = torch.from_numpy(r.standard_normal((n, 2, D)) * scale).cuda().to(torch.bfloat16)
    if scale > 1:
        md[5, 0] = 0
        md[5, 0, 0], md[9, 1] = float("inf"), 0
        md[9, 1, 3] = float("-inf")
    qd = torch.from_numpy(r.standard_normal((1, 2, D)) + 0.01).cuda().to(torch.bfloat16)
    sel = torch.empty(1, 2, select, dtype=torch.int32, device="cuda")
    ws = mcs.empty_workspace(mcs.mcs_paged_select_workspace(p))
    table = r.permutation(n)[None]
    mcs.mcs_paged_select(p, qd, md, _i32(table), _i32([n * page]), sel, ws, sink=0, recent=0)
    m = _f64(md)
    with np.errstate(invalid="ignore", over="ignore"):
        q = _f64(qd)
        # (the infinite rows hold one value and zeros, and no query is zero: their sums are infinite)
        score = np.stack([np.where(m[:, h] == 0, 0.0, m[:, h] * q[0, h]).sum(1) for h in range(2)]).astype(np.float32)
    for h in range(2):
        s = score[h][table[0]]
        want = np.sort(np.lexsort((np.arange(n), -s))[:select])
        np.testing.assert_array_equal(sel[0, h].cpu().numpy(), want)


def test_tables_far_longer_than_their_sequences():
    c = Cache([500, 17, 0, 4000], 8, 2, 128, 16, seed=2, extra=60000)
    c.check(*c.run())
    mean, select = c.means(), 9
    ws = mcs.empty_workspace(mcs.mcs_paged_select_workspace(c.p))
    sel = torch.empty(4, 2, select, dtype=torch.int32, device="cuda")
    mcs.mcs_paged_select(c.p, c.q, mean, c.dtable, c.dlens, sel, ws, sink=1, recent=1)
    want = po.select(_f64(c.q), _f64(mean), c.table, c.lens, 16, select, 1, 1)
    np.testing.assert_array_equal(sel.cpu().numpy(), want)
    c.check(*c.run(sel), want)


def test_selection_of_a_long_sequence_takes_several_rounds():
    # more pages than all blocks of the score kernel look at in one round, for many pairs
    c = Cache([9000] * 40, 128, 64, 64, 16, seed=4)
    mean, select = c.means(), 5
    ws = mcs.empty_workspace(mcs.mcs_paged_select_workspace(c.p))
    sel = torch.empty(40, 64, select, dtype=torch.int32, device="cuda")
    mcs.mcs_paged_select(c.p, c.q, mean, c.dtable, c.dlens, sel, ws, sink=0, recent=1)
    q = c.q.double().view(40, 64, 2, 64).sum(2)
    score = torch.einsum("bhd,bphd->bhp", q, mean[c.dtable[:, :563].long()].double()).float()
    score[..., 562] = float("inf")
    want = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :select].sort(-1).values
    assert torch.equal(sel.long(), want)


def test_batches_of_the_largest_count():
    r = np.random.default_rng(1)
    c = Cache([int(x) for x in r.integers(0, 20, 4096)], 2, 1, 64, 16, seed=3, extra=0)
    c.check(*c.run())


# ------------------------------------------------------------------ plan and write

def _plan(p, new, lens, free, head, table, T, in_place=False):
    d = dict(lens=_i32(lens), head=_i32([head]), table=_i32(table))
    lo, ho = (d["lens"], d["head"]) if in_place else (_i32(lens) * 0 - 9, _i32([0]))
    cu = torch.full((p.B + 1,), -9, dtype=torch.int32, device="cuda")
    slots, pos = (torch.full((T,), -9, dtype=torch.int32, device="cuda") for _ in range(2))
    mcs.mcs_paged_plan(p, _i32(new), d["lens"], _i32(free), d["head"], d["table"], lo, ho, cu, slots, pos)
    return [x.cpu().numpy() for x in (lo, ho, d["table"], cu, slots, pos)]


@pytest.mark.parametrize("B,page,most,T_over,in_place", [
    (1, 16, 1, 0, False), (3, 16, 40, 5, True), (7, 64, 500, 0, False), (1500, 16, 9, 100, True),
    (4096, 32, 3, 0, False), (33, 128, 2000, 1, True)])
def test_plan_matches_oracle(B, page, most, T_over, in_place):
    r = np.random.default_rng(B + most)
    lens, new = r.integers(0, 300, B), r.integers(0, most + 1, B)
    lens[0] = 0
    new[-1] = most
    P = -(-(300 + most) // page) + 1
    num = 2 * int(sum(-(-(lens + new) // page))) + 7
    order = r.permutation(num)
    table, at = np.full((B, P), -1), 0
    for b in range(B):
        n = -(-lens[b] // page)
        table[b, :n] = order[at:at + n]
        at += n
    free, head, T = order[at:], 2, int(new.sum()) + T_over
    want = po.plan(new, lens, free, head, table, page, T, num)
    got = _plan(mcs.paged(B, 1, 1, 64, page, num, P), new, lens, free, head, table, T, in_place)
    for x, y in zip(got, want):
        np.testing.assert_array_equal(x, y)
    assert mcs.mcs_device_status() == 0


@pytest.mark.parametrize("what", ["tokens", "pages", "table", "negative", "free", "started", "head"])
def test_plan_refuses_and_takes_nothing(what):
    lens, new, free, head, T = [20, 0, 5], [3, 40, 12], [7, 8, 9, 4, 5], 1, 60
    table = np.array([[1, 2, -1, -1], [-1] * 4, [3, -1, -1, -1]])
    if what == "tokens":
        T = 54
    elif what == "pages":
        head = 2
    elif what == "table":
        new[1] = 65
    elif what == "negative":
        new[0] = -1
    elif what == "free":
        free[2] = 10
    elif what == "started":
        table[0, 1] = -1
    elif what == "head":
        head = -1
    p = mcs.paged(3, 1, 1, 64, 16, 10, 4)
    lo, ho, tab, cu, slots, pos = _plan(p, new, lens, free, head, table, T)
    assert mcs.mcs_device_status() == 6
    assert lo.tolist() == lens and ho.tolist() == [head] and (tab == table).all()
    assert not cu.any() and (slots == -1).all() and (pos == -1).all()


def test_plan_of_a_good_request_after_a_refused_one():
    lens, new, free = [20, 0, 5], [3, 40, 12], [7, 8, 9, 4, 5]
    table = np.array([[1, 2, -1, -1], [-1] * 4, [3, -1, -1, -1]])
    p = mcs.paged(3, 1, 1, 64, 16, 10, 4)
    got = _plan(p, new, lens, free, 1, table, 55)
    for x, y in zip(got, po.plan(new, lens, free, 1, table, 16, 55, 10)):
        np.testing.assert_array_equal(x, y)
    assert mcs.mcs_device_status() == 0


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("lens,new,Hkv,D,page,stride", [
    ([0], [1], 1, 128, 16, 0), ([15, 16, 17, 0], [1, 1, 0, 40], 2, 64, 16, 0),
    ([100, 3], [29, 300], 3, 128, 128, 8 * 128), ([31, 0, 64], [1, 7, 64], 8, 128, 32, 0)])
def test_write_matches_oracle(lens, new, Hkv, D, page, stride, e4m3):
    after = [a + n for a, n in zip(lens, new)]
    c = Cache(after, Hkv, Hkv, D, page, e4m3, seed=sum(after))
    c.p.kv_stride = stride
    free = np.concatenate([c.table[b, -(-a // page):-(-z // page)] for b, (a, z) in enumerate(zip(lens, after))])
    T = sum(new) + 3
    planned = po.plan(new, lens, free, 0, c.table, page, T, c.p.num_pages)
    slots = planned[4]
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn(T, stride or Hkv * D, generator=g, device="cuda").to(torch.bfloat16)[:, :Hkv * D]
            .view(T, Hkv, D) for _ in range(2))
    mean = c.means()
    before = [x.clone() for x in (c.k, c.v, mean)]
    mcs.mcs_paged_write(c.p, k, v, _i32(slots), c.k, c.v, mean)
    if e4m3:
        enc = lambda x, s: orc.e4m3_encode(x.float().cpu().numpy(), s)
        kn, vn, held = enc(k, KS), enc(v, VS), [x.cpu().numpy() for x in before[:2]]
        values = lambda x: orc.e4m3_decode(x).astype(np.float64) * KS
    else:
        bits = lambda x: x.contiguous().view(torch.int16).cpu().numpy()
        kn, vn, held = bits(k), bits(v), [bits(x) for x in before[:2]]
        values = lambda x: torch.from_numpy(np.ascontiguousarray(x)).view(torch.bfloat16).double().numpy()
    want_mean = _f64(before[2])
    touched = po.write(kn, vn, slots, *held, want_mean, values)
    for got, want in zip((c.k, c.v), held):
        got = got.cpu().numpy() if e4m3 else got.view(torch.int16).cpu().numpy()
        np.testing.assert_array_equal(got, want)
    got = _f64(mean)
    for pg in range(c.p.num_pages):
        if pg not in touched:
            np.testing.assert_array_equal(got[pg], _f64(before[2])[pg])
            continue
        size = np.abs(values(held[0][pg, :, :touched[pg]])).mean(1)
        assert (np.abs(got[pg] - want_mean[pg]) <= 2.0 ** -8 * np.abs(want_mean[pg]) + (page + 2) * U * size).all()
    # without means nothing else changes
    k2, v2 = before[0], before[1]
    mcs.mcs_paged_write(c.p, k, v, _i32(slots), k2, v2)
    eq = lambda a, b: torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert eq(k2, c.k) and eq(v2, c.v)


@pytest.mark.parametrize("D,Hkv,page,e4m3,means", [(128, 8, 64, False, True), (64, 5, 128, True, True),
                                                 (128, 7, 16, True, True), (64, 8, 32, False, False)])
def test_write_of_long_prompts(D, Hkv, page, e4m3, means):
    """Enough tokens for the widest windows; runs that begin in one block's window and end in the next's."""
    r = np.random.default_rng(page)
    B, P = 6, 100_000 // page
    lens = r.integers(0, 3 * page, B)
    new = r.integers(1, 2 * 152 * 8 * 4 * (256 // (D // 8)) // Hkv // B, B)
    new[-1] += max(0, 152 * 8 * 4 * (256 // (D // 8)) // Hkv + 1 - int(new.sum()))
    need = -(-(lens + new) // page)
    num = int(need.sum()) + 5
    order, table, at = r.permutation(num), np.full((B, P), -1), 0
    for b in range(B):
        table[b, :-(-lens[b] // page)] = order[at:at + -(-lens[b] // page)]
        at += -(-lens[b] // page)
    T = int(new.sum()) + 9
    slots = po.plan(new, lens, order[at:], 0, table, page, T, num)[4]
    g = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)
    k, v, s = rand(T, Hkv, D), rand(T, Hkv, D), _i32(slots)
    if e4m3:
        c = torch.randint(0, 0x78, (2, num, Hkv, page, D), generator=g, device="cuda").to(torch.uint8)
        codes = [torch.empty(x.shape, dtype=torch.uint8, device="cuda") for x in (k, v)]
        for x, y, f in zip((k, v), codes, (KS, VS)):
            mcs.mcs_quantize_e4m3(x, f, y)
        values = lambda x: x.view(torch.float8_e4m3fn).double() * KS
    else:
        c, codes, values = rand(2, num, Hkv, page, D), [k, v], lambda x: x.double()
    want = c.clone()
    live = s >= 0
    for i in range(2):
        want[i][s[live] // page, :, s[live] % page] = codes[i][live]
    p = mcs.paged(B, Hkv, Hkv, D, page, num, P, kv=int(e4m3), k_scale=KS, v_scale=VS)
    mean = rand(num, Hkv, D)
    before = mean.clone()
    mcs.mcs_paged_write(p, k, v, s, c[0], c[1], mean if means else None)
    assert mcs.mcs_device_status() == 0
    assert torch.equal(c.view(torch.uint8), want.view(torch.uint8))
    fill = torch.zeros(num, dtype=torch.int64, device="cuda")
    fill.scatter_reduce_(0, (s[live] // page).long(), (s[live] % page + 1).long(), "amax")
    touched = fill > 0
    assert torch.equal(mean[~touched], before[~touched])
    if not means:
        assert torch.equal(mean, before)
        return
    rows = torch.arange(page, device="cuda")[None] < fill[touched][:, None]
    x = torch.where(rows[:, None, :, None], values(want[0][touched]), 0.0)
    n = fill[touched][:, None, None]
    exact, size = x.sum(2) / n, x.abs().sum(2) / n
    assert ((mean[touched].double() - exact).abs() <= 2.0 ** -8 * exact.abs() + (page + 2) * U * size).all()


@pytest.mark.parametrize("ks,vs", [(KS, VS), (1.0, 3.0), (0.7131, 2.0 ** -20), (2.0 ** -90, 2.0 ** 70),
                                   (2.0 ** -60, 1.9999999), (1e-38, 3e38)])
def test_write_rounds_every_value_as_the_quantiser(ks, vs):
    """All 65536 bf16 patterns, infinities, NaN, zeros of both signs and denormals among them."""
    x = torch.arange(-32768, 32768, device="cuda", dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    p = mcs.paged(1, 4, 4, 128, 16, 8, 8, kv=mcs.KV_E4M3, k_scale=ks, v_scale=vs)
    rows = x.view(128, 4, 128)
    cache = torch.zeros(2, 8, 4, 16, 128, dtype=torch.uint8, device="cuda")
    mcs.mcs_paged_write(p, rows, rows, _i32(np.arange(128)), cache[0], cache[1])
    want = torch.empty(65536, dtype=torch.uint8, device="cuda")
    for got, scale in zip(cache, (ks, vs)):
        mcs.mcs_quantize_e4m3(x, scale, want)
        assert torch.equal(got.transpose(1, 2).reshape(-1), want)


def test_write_skips_padding_and_slots_past_the_cache():
    p = mcs.paged(1, 1, 1, 64, 16, 4, 4)
    cache, mean = torch.zeros(2, 4, 1, 16, 64, device="cuda").to(torch.bfloat16), None
    k = torch.ones(4, 1, 64, device="cuda", dtype=torch.bfloat16)
    mcs.mcs_paged_write(p, k, k, _i32([-1, 64, -5, 2 ** 31 - 1]), cache[0], cache[1], mean)
    assert mcs.mcs_device_status() == 6
    assert not cache.any()
    mcs.mcs_paged_write(p, k[:0], k[:0], _i32([]), cache[0], cache[1])
    assert mcs.mcs_device_status() == 0


# ------------------------------------------------------------------ what the arrays may get wrong

def test_decode_reports_and_skips_what_lies_outside():
    """A page outside the cache is skipped as if its tokens were not there; a length past the
    table counts as no tokens.  The checks stand in the kernels in front of each access."""
    c = Cache([40, 100, 33], 4, 2, 128, 16, seed=3)
    table = c.table.copy()
    table[1, 2], table[1, 4] = -1, c.p.num_pages
    c.dtable = _i32(table)
    out, ls = c.run()
    assert mcs.mcs_device_status() == 6
    sel = np.full((3, 2, 9), -1)
    for b, n in enumerate([3, 7, 3]):
        sel[b, :, :n] = np.arange(n)
    sel[1, :, 2] = sel[1, :, 4] = -1
    c.check(out, ls, sel)
    # the sparse form with logical pages outside the sequence
    bad = sel.copy()
    bad[0, 0, 1], bad[2, 1, 0] = 3, -2
    c.dtable = _i32(c.table)
    out, ls = c.run(_i32(bad))
    assert mcs.mcs_device_status() == 6
    sel[0, 0, 1] = sel[2, 1, 0] = -1
    c.check(out, ls, sel)
    # lengths outside the table
    c.dlens, c.lens = _i32([40, c.p.max_pages * 16 + 1, -3]), [40, 0, 0]
    out, ls = c.run()
    assert mcs.mcs_device_status() == 6
    c.check(out, ls)


def test_select_reports_and_ranks_bad_pages_last():
    c = Cache([100, 64], 4, 2, 64, 16, seed=3)
    mean, table = c.means(), c.table.copy()
    table[0, 3], table[1, 1] = -1, c.p.num_pages
    ws = mcs.empty_workspace(mcs.mcs_paged_select_workspace(c.p))
    sel = torch.empty(2, 2, 3, dtype=torch.int32, device="cuda")
    mcs.mcs_paged_select(c.p, c.q, mean, _i32(table), _i32([100, 64]), sel, ws, sink=0, recent=0)
    assert mcs.mcs_device_status() == 6
    got = sel.cpu().numpy()
    assert (got >= 0).all() and not (got[0] == 3).any() and not (got[1] == 1).any()
    mcs.mcs_paged_select(c.p, c.q, mean, _i32(c.table), _i32([-1, 10 ** 6]), sel, ws)
    assert mcs.mcs_device_status() == 6
    assert (sel == -1).all()


# ------------------------------------------------------------------ together, as they are used

@pytest.mark.parametrize("e4m3,Hq,Hkv,D,page", [(False, 8, 2, 128, 16), (True, 4, 4, 64, 32)])
def test_generation_steps_together(e4m3, Hq, Hkv, D, page):
    """Prompts, then tokens one at a time: normalise and rotate, plan, write, select, attend;
    the batch has an idle request.  Against the oracle over the whole sequences."""
    r = np.random.default_rng(D)
    B, rot, P, num, select = 3, D // 2, 12, 30, 3
    kv = mcs.KV_E4M3 if e4m3 else mcs.KV_BF16
    fused = (Hq + 2 * Hkv) * D
    g = torch.Generator(device="cuda").manual_seed(D)
    angle = np.arange(256)[:, None] * 100.0 ** -np.linspace(0, 1, rot // 2)
    cos, sin = (torch.from_numpy(f(angle)).float().cuda() for f in (np.cos, np.sin))
    w = [(1 + 0.1 * torch.randn(D, generator=g, device="cuda")) for _ in range(2)]
    p = mcs.paged(B, Hq, Hkv, D, page, num, P, kv=kv, k_scale=2.0 ** -6, v_scale=2.0 ** -6, kv_stride=0)
    dt = torch.uint8 if e4m3 else torch.bfloat16
    kc, vc = (torch.zeros(num, Hkv, page, D, dtype=dt, device="cuda") for _ in range(2))
    mean = torch.zeros(num, Hkv, D, dtype=torch.bfloat16, device="cuda")
    free, head = _i32(r.permutation(num)), _i32([0])
    lens, table = _i32([0] * B), _i32(np.full((B, P), -1))
    ws = mcs.empty_workspace(mcs.mcs_paged_decode_workspace(p))
    ws2 = mcs.empty_workspace(mcs.mcs_paged_select_workspace(p))
    seq_k, seq_v = [[] for _ in range(B)], [[] for _ in range(B)]
    for step, new in enumerate([[50, 0, 97], [1, 1, 1], [1, 0, 1], [1, 1, 1]]):
        T = sum(new) + 2
        x = torch.randn(T, fused, generator=g, device="cuda").to(torch.bfloat16)
        cu = torch.empty(B + 1, dtype=torch.int32, device="cuda")
        slots, pos = (torch.empty(T, dtype=torch.int32, device="cuda") for _ in range(2))
        mcs.mcs_paged_plan(p, _i32(new), lens, free, head, table, lens, head, cu, slots, pos)
        rp = mcs.rope_params(T, 1, Hq, Hkv, D, rot, 256, interleaved=e4m3, layout=mcs.LAYOUT_BNHD,
                             q_stride=fused, k_stride=fused)
        q, k = (torch.full((T, 1, h, D), 5.0, dtype=torch.bfloat16, device="cuda") for h in (Hq, Hkv))
        mcs.mcs_qk_norm_rope(rp, x[:, :Hq * D].view(T, 1, Hq, D), x[:, Hq * D:(Hq + Hkv) * D].view(T, 1, Hkv, D),
                             w[0], w[1], cos, sin, pos.view(T, 1), q, k)
        v = x[:, (Hq + Hkv) * D:].view(T, Hkv, D)
        mcs.mcs_paged_write(p, k.view(T, Hkv, D), v.contiguous(), slots, kc, vc, mean)
        # padding rows stay as they were
        assert (q[-2:] == 5).all() and (k[-2:] == 5).all()
        # the stored keys are the oracle's rotated ones
        c = cu.cpu().numpy()
        pn = pos.cpu().numpy()
        live = slice(0, c[-1])
        for h0, w0, got in ((0, w[0], q), (Hq, w[1], k)):
            n = Hq if h0 == 0 else Hkv
            xs = _f64(x[:, h0 * D:(h0 + n) * D]).reshape(T, 1, n, D)[live]
            want = po.norm_rope(xs, _f64(w0), _f64(cos), _f64(sin), pn[live, None], rot, e4m3, 1e-6)
            # bf16 rounding, and fp32 arithmetic on values below 2 max |y|
            assert (np.abs(_f64(got)[live] - want) <= 2.0 ** -8 * np.abs(want) + 2 * (D / 2 + 8) * U * np.abs(want).max()).all()
        for b in range(B):
            seq_k[b] += list(_f64(k)[c[b]:c[b + 1], 0])
            seq_v[b] += list(_f64(v)[c[b]:c[b + 1]])
        if step == 0:
            continue
        # one query per sequence, in batch order; the idle request asks nothing new
        # but still attends to what it has
        last = [max(c[b + 1] - 1, 0) for b in range(B)]
        qd = q[last, 0].contiguous()
        sel = torch.empty(B, Hkv, select, dtype=torch.int32, device="cuda")
        out, outs = (torch.empty(B, Hq, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        mcs.mcs_paged_decode(p, qd, kc, vc, table, lens, out, ws)
        mcs.mcs_paged_select(p, qd, mean, table, lens, sel, ws2, sink=1, recent=1)
        mcs.mcs_paged_decode_sparse(p, qd, kc, vc, table, lens, sel, outs, ws)
        assert mcs.mcs_device_status() == 0
        ln, tb = lens.cpu().numpy(), table.cpu().numpy()
        assert ln.tolist() == [len(x) for x in seq_k]
        np.testing.assert_array_equal(sel.cpu().numpy(), po.select(_f64(qd), _f64(mean), tb, ln, page, select, 1, 1))
        kd, vd = (_f64(x) * (2.0 ** -6 if e4m3 else 1) for x in (kc, vc))
        for b in range(B):  # the cache is the sequence
            for t in range(ln[b]):
                row = kd[tb[b, t // page], :, t % page]
                # E4M3: half a step, 2^-4 of the value or half the smallest step 2^-10 * scale
                assert (np.abs(row - seq_k[b][t]) <= (2.0 ** -4 * np.abs(seq_k[b][t]) + 2.0 ** -16 if e4m3 else 0)).all()
        for got, s in ((out, None), (outs, sel.cpu().numpy())):
            want, _, absv, size = po.decode(_f64(qd), kd, vd, tb, ln, D ** -0.5, s)
            tol = 2.0 ** -8 * np.abs(want) + absv * (4 * (D + 8) * U * size + 2.0 ** -20 + (2.0 ** -11 if e4m3 else 2.0 ** -16) + 100 * U)[..., None]
            assert (np.abs(_f64(got) - want) <= tol).all()


# ------------------------------------------------------------------ streams, graphs, repeats

def test_repeated_calls_give_the_same_bits():
    c = Cache([3000, 17, 900, 0], 16, 2, 128, 16, seed=1)
    a = c.run()
    for _ in range(5):
        b = c.run()
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_two_streams_with_workspaces_of_their_own():
    cs = [Cache([5000, 300], 8, 2, 128, 32, e, seed=i) for i, e in enumerate((False, True))]
    want = [c.run() for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    got = []
    for _ in range(10):
        for c, s in zip(cs, streams):
            with torch.cuda.stream(s):
                got.append(c.run())
    torch.cuda.synchronize()
    for i, (o, l) in enumerate(got):
        assert torch.equal(o, want[i % 2][0]) and torch.equal(l, want[i % 2][1])


def test_captured_step_follows_lengths_and_pages():
    """plan, write, select and both attentions in one graph, replayed while the state advances
    in place; a second graph shares the workspace on the same stream."""
    B, Hq, Hkv, D, page, P, num = 2, 8, 2, 128, 16, 8, 16
    p = mcs.paged(B, Hq, Hkv, D, page, num, P)
    g = torch.Generator(device="cuda").manual_seed(3)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)
    kc, vc, mean = rand(num, Hkv, page, D), rand(num, Hkv, page, D), rand(num, Hkv, D)
    lens, head, table = _i32([30, 0]), _i32([2]), _i32([[3, 9] + [-1] * 6, [-1] * 8])
    free = _i32([9, 3, 1, 0, 15, 7, 8, 2])
    new, cu = _i32([1, 1]), _i32([0] * 3)
    slots, pos = _i32([0, 0]), _i32([0, 0])
    q, k, v = rand(B, Hq, D), rand(B, Hkv, D), rand(B, Hkv, D)
    out, outs = (torch.empty(B, Hq, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    sel = torch.empty(B, Hkv, 2, dtype=torch.int32, device="cuda")
    ws = mcs.empty_workspace(mcs.mcs_paged_decode_workspace(p))
    ws2 = mcs.empty_workspace(mcs.mcs_paged_select_workspace(p))

    def attend(o):
        mcs.mcs_paged_decode(p, q, kc, vc, table, lens, o, ws)

    def step():
        mcs.mcs_paged_plan(p, new, lens, free, head, table, lens, head, cu, slots, pos)
        mcs.mcs_paged_write(p, k, v, slots, kc, vc, mean)
        mcs.mcs_paged_select(p, q, mean, table, lens, sel, ws2, sink=0, recent=1)
        mcs.mcs_paged_decode_sparse(p, q, kc, vc, table, lens, sel, outs, ws)
        attend(out)

    state = [x.clone() for x in (kc, vc, mean, lens, head, table)]
    step()  # first calls outside the capture
    for x, y in zip((kc, vc, mean, lens, head, table), state):
        x.copy_(y)
    s = torch.cuda.Stream()
    graph, other, out2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph(), torch.empty_like(out)
    with torch.cuda.graph(graph, stream=s):
        step()
    with torch.cuda.graph(other, stream=s):
        attend(out2)
    for x, y in zip((kc, vc, mean, lens, head, table), state):
        x.copy_(y)
    for i in range(4):
        k.copy_(rand(B, Hkv, D))
        graph.replay()
        other.replay()
        torch.cuda.synchronize()
        assert lens.tolist() == [31 + i, 1 + i]
        assert head.tolist() == [2 + 1 + (i >= 2)]
        assert torch.equal(out, out2)
        tb, ln = table.cpu().numpy(), lens.cpu().numpy()
        for o, sl in ((out, None), (outs, sel.cpu().numpy())):
            want, _, absv, size = po.decode(_f64(q), _f64(kc), _f64(vc), tb, ln, D ** -0.5, sl)
            tol = 2.0 ** -8 * np.abs(want) + absv * (4 * (D + 8) * U * size + 2.0 ** -15)[..., None]
            assert (np.abs(_f64(o) - want) <= tol).all()
    assert mcs.mcs_device_status() == 0


@pytest.mark.parametrize("B,page,D", [(5, 16, 128), (40, 32, 64)])
def test_steps_one_behind_another_see_their_own_lengths(B, page, D):
    # lengths that change from step to step, many steps in one graph with nothing between the
    # launches, against the same steps one at a time
    r = np.random.default_rng(B)
    steps, Hkv, Hq, P = 24, 2, 4, 24 * 40 // page + 2
    num = B * P
    p = mcs.paged(B, Hq, Hkv, D, page, num, P)
    g = torch.Generator(device="cuda").manual_seed(B)
    kc, vc, q = (torch.randn(*x, generator=g, device="cuda").to(torch.bfloat16)
                 for x in ((num, Hkv, page, D), (num, Hkv, page, D), (B, Hq, D)))
    mean = kc.float().mean(2).to(torch.bfloat16)
    new = _i32(r.integers(0, 40, (steps, B)) * (r.random((steps, B)) < 0.7))
    slots, cu, free = _i32(np.zeros(40 * B)), _i32(np.zeros(B + 1)), _i32(r.permutation(num))
    ws = mcs.empty_workspace(max(mcs.mcs_paged_decode_workspace(p), mcs.mcs_paged_select_workspace(p)))

    def run(between):
        lens, head, table = _i32(np.zeros(B)), _i32([0]), _i32(np.zeros((B, P)))
        outs = torch.zeros(steps, 2, B, Hq, D, dtype=torch.bfloat16, device="cuda")
        sels = torch.zeros(steps, B, Hkv, 5, dtype=torch.int32, device="cuda")
        def go():
            lens.zero_(), head.zero_()
            for i in range(steps):
                mcs.mcs_paged_plan(p, new[i], lens, free, head, table, lens, head, cu, slots)
                between()
                mcs.mcs_paged_decode(p, q, kc, vc, table, lens, outs[i, 0], ws)
                between()
                mcs.mcs_paged_select(p, q, mean, table, lens, sels[i], ws)
                between()
                mcs.mcs_paged_decode_sparse(p, q, kc, vc, table, lens, sels[i], outs[i, 1], ws)
                between()
        return go, outs, sels

    go, want, want_sel = run(torch.cuda.synchronize)
    go()
    go, outs, sels = run(lambda: None)
    go()
    torch.cuda.synchronize()
    assert torch.equal(outs, want) and torch.equal(sels, want_sel)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go()
    for _ in range(3):
        outs.zero_(), sels.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs, want) and torch.equal(sels, want_sel)
    assert mcs.mcs_device_status() == 0


def test_rows_past_two_gib_of_cache():
    """Pages whose byte offsets pass 32 bits: a 4.3 GB cache, the sequence's pages at its end."""
    page, Hkv, D, num = 64, 8, 128, 33000
    p = mcs.paged(1, 8, Hkv, D, page, num, 4)
    kc = torch.empty(num, Hkv, page, D, dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    last = num - 1
    tab = np.array([[last, last - 2, last - 1, 0]])
    k = torch.randn(150, Hkv, D, device="cuda").to(torch.bfloat16)
    slots = [tab[0, t // page] * page + t % page for t in range(150)]
    mcs.mcs_paged_write(p, k, -k, _i32(slots), kc, vc)
    q = torch.randn(1, 8, D, device="cuda").to(torch.bfloat16)
    out = torch.empty_like(q)
    ws = mcs.empty_workspace(mcs.mcs_paged_decode_workspace(p))
    mcs.mcs_paged_decode(p, q, kc, vc, _i32(tab), _i32([150]), out, ws)
    z = torch.einsum("hd,thd->ht", q[0].double(), k.double()) * D ** -0.5
    want = -torch.einsum("ht,thd->hd", torch.softmax(z, 1), k.double())
    absv = torch.einsum("ht,thd->hd", torch.softmax(z, 1), k.double().abs())
    # scores below about 10 in size: 2 (D + 8) u * 10 * 2 < 2^-13
    assert ((out[0].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -13 * absv).all()


def test_binding_refuses_what_does_not_fit():
    c = Cache([40], 4, 2, 128, 16, seed=0)
    out = torch.empty(1, 4, 128, dtype=torch.bfloat16, device="cuda")
    ok = (c.p, c.q, c.k, c.v, c.dtable, c.dlens, out, c.ws)
    for i, bad in [(1, c.q.float()), (2, c.k[:, :, :8]), (2, c.k.transpose(2, 3).contiguous().transpose(2, 3)),
                   (4, c.dtable[:, :2]), (5, c.dlens.long()), (6, out[:, :2]), (1, c.q.cpu())]:
        with pytest.raises(ValueError):
            mcs.mcs_paged_decode(*ok[:i], bad, *ok[i + 1:])
    with pytest.raises(ValueError, match="strides"):
        wide = torch.zeros(1, 4, 256, dtype=torch.bfloat16, device="cuda")[:, :, :128]
        mcs.mcs_paged_decode(ok[0], wide, *ok[2:])
    with pytest.raises(mcs.McsError, match="WORKSPACE"):
        mcs.mcs_paged_decode(*ok[:7], c.ws[:16])
    if torch.cuda.device_count() > 1:
        with pytest.raises(ValueError, match="cuda:1"):
            mcs.mcs_paged_decode(*ok[:1], c.q.to("cuda:1"), *ok[2:])


def test_caches_of_codes_come_as_bytes_or_as_what_they_stand_for():
    c = Cache([200, 33], 4, 2, 128, 16, True, seed=1)
    want = c.run()
    mean = torch.zeros(c.k.shape[0], 2, 128, dtype=torch.bfloat16, device="cuda")
    rows, slots = torch.ones(3, 2, 128, dtype=torch.bfloat16, device="cuda"), _i32([16, 17, 40])
    other = [x.clone() for x in (c.k, c.v, mean)]
    mcs.mcs_paged_write(c.p, rows, rows, slots, *other)
    c.k, c.v = c.k.view(torch.float8_e4m3fn), c.v.view(torch.float8_e4m3fn)
    assert all(torch.equal(a, b) for a, b in zip(c.run(), want))
    mcs.mcs_paged_write(c.p, rows, rows, slots, c.k, c.v, mean)
    assert all(torch.equal(a.view(b.dtype), b) for a, b in zip((c.k, c.v, mean), other))
    b = Cache([40], 4, 2, 128, 16, seed=0)
    out = torch.empty(1, 4, 128, dtype=torch.bfloat16, device="cuda")
    codes = b.k.to(torch.float8_e4m3fn)
    for bad in (codes, codes.view(torch.uint8)):
        with pytest.raises(ValueError, match="k_cache"):
            mcs.mcs_paged_decode(b.p, b.q, bad, b.v, b.dtable, b.dlens, out, b.ws)
    with pytest.raises(ValueError, match="ws"):
        mcs.mcs_paged_decode(b.p, b.q, b.k, b.v, b.dtable, b.dlens, out, b.ws.view(torch.float32))


@pytest.mark.parametrize("n,Hq,Hkv,D,page", [(48, 1, 1, 64, 16), (200, 12, 1, 128, 32), (200, 8, 8, 64, 16),
                                             (160, 6, 2, 128, 128)])
@pytest.mark.parametrize("off", [2.0 ** -13, -2.0 ** -14, 2.0 ** -12 * 0.7])
def test_e4m3_weights_keep_their_low_bits(n, Hq, Hkv, D, page, off):
    """Half of the keys have weight 1 and value -3/4, the others weight 3/4 (1 + off) and value 1, so
    that the output is 3/7 off and a bit: all of it lies below one f16's half step of the weight (2^-11).
    Two f16 parts are off by 2^-22, below the 2^-21 that is allowed here; the rest as above."""
    scale = -np.log(0.75 * (1 + off))
    c = Cache([n], Hq, Hkv, D, page, True, seed=1, scale=float(np.float32(scale)))
    c.scale = float(np.float32(scale))
    c.scales, c.p.k_scale, c.p.v_scale = (1.0, 1.0), 1.0, 1.0
    odd = torch.arange(page, device="cuda") % 2 == 1
    code = lambda x: int(torch.tensor(x).to(torch.float8_e4m3fn).view(torch.uint8))
    c.k.zero_()
    c.k[:, :, odd, 0] = code(-1.0)
    c.v[:, :, odd] = code(1.0)
    c.v[:, :, ~odd] = code(-0.75)
    c.q.zero_()
    c.q[:, :, 0] = 1
    out, ls = c.run()
    want, lse, absv, size = po.decode(_f64(c.q), _f64(c.k), _f64(c.v), c.table, c.lens, c.scale)
    tol = 2.0 ** -8 * np.abs(want) + absv * (2 * (2 * (D + 8) * U * size + 2.0 ** -21) + 2.0 ** -21 + n * U)[..., None]
    assert (tol < np.abs(want)).all()  # (that it would show)
    assert (np.abs(_f64(out[:1]) - want) <= tol).all(), (_f64(out[0, 0, 0]), want[0, 0, 0])
    c.check(out, ls)


def _plan_of_many(B):
    """A step of B sequences against the oracle."""
    r = np.random.default_rng(B)
    lens, new, page = r.integers(0, 40, B), r.integers(0, 3, B), 16
    need = int((-(-(lens + new) // page)).sum())
    order, table, at = r.permutation(need + 3), np.full((B, 3), -1), 0
    for b in range(B):
        n = -(-lens[b] // page)
        table[b, :n] = order[at:at + n]
        at += n
    p, T = mcs.paged(B, 1, 1, 64, page, need + 3, 3), int(new.sum()) + 1
    want = po.plan(new, lens, order[at:], 0, table, page, T, need + 3)
    for x, y in zip(_plan(p, new, lens, order[at:], 0, table, T), want):
        np.testing.assert_array_equal(x, y)
    assert mcs.mcs_device_status() == 0


def test_plan_of_every_count_that_is_documented():
    """Counts around the shared memory that a launch has without asking, in a process of its own: asking
    for one count holds for the process."""
    code = ("import sys; sys.path.insert(0, sys.argv[1]); from tests import test_gpu_paged as t; "
            "[t._plan_of_many(b) for b in (4051, 4052, 4060, 4095, 4096, 1)]")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code, root], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("e4m3,scale,k_scale", [(True, 1e-30, 1e-20), (True, 1e-45, 1e-45), (True, 0.0, 1e-45),
                                                (False, 1e-45, 1.0), (False, 1e-30, 1.0)])
def test_decode_of_scales_that_vanish_is_the_mean(e4m3, scale, k_scale):
    """Scales whose product is too small for a float, each of them accepted: all weights are equal."""
    c = Cache([700, 33, 0, 1, 16], 8, 2, 64, 16, e4m3, seed=2, scale=scale)
    if e4m3:
        c.p.k_scale = k_scale
        c.scales = (k_scale, VS)
    c.check(*c.run())
    sel = _sel(c, 3, 3)
    c.check(*c.run(_i32(sel)), sel)


@pytest.mark.parametrize("v_scale", [2.0 ** -122, 1.7 * 2.0 ** -126, 2.0 ** 100])
@pytest.mark.parametrize("lens", [[3000], [30, 2900, 0, 17]])
def test_value_scales_of_any_size(v_scale, lens):
    """The quotient of a small value scale and a sum of weights is far below the smallest normal
    float; the outputs are not.  (Half of bf16's smallest step is 2^-134.)"""
    c = Cache(lens, 4, 2, 128, 16, True, seed=7)
    c.p.v_scale = v_scale
    c.scales = (KS, v_scale)
    out, _ = c.run()
    want, _, absv, size = po.decode(_f64(c.q), _f64(c.k) * KS, _f64(c.v) * v_scale, c.table, lens, c.scale)
    tol = 2.0 ** -134 + 2.0 ** -8 * np.abs(want) + absv * (
        2 * (2 * (128 + 8) * U * size + 2.0 ** -21) + 2.0 ** -21 + max(lens) * U)[..., None]
    assert (np.abs(_f64(out[:len(lens)]) - want) <= tol).all()


@pytest.mark.parametrize("select", [2 ** 31 - 1, 2 ** 31 - 1000])
def test_select_rows_as_long_as_a_call_takes(select):
    """Far more places than pages: the rest of the row is -1 up to its end, and nothing else is written."""
    c = Cache([100], 2, 1, 64, 16, seed=1)
    row = torch.full((select + 1024,), 7, dtype=torch.int32, device="cuda")
    ws = mcs.empty_workspace(mcs.mcs_paged_select_workspace(c.p))
    mcs.mcs_paged_select(c.p, c.q, c.means(), c.dtable, c.dlens, row[:select].view(1, 1, select), ws)
    assert row[:7].tolist() == list(range(7)) and (row[select:] == 7).all()
    assert int(row[7:select].max()) == -1 and int(row[7:select].min()) == -1
    c.check(*c.run(row[:select].view(1, 1, select)))


@pytest.mark.parametrize("e4m3,means", [(False, True), (True, True), (False, False)])
@pytest.mark.parametrize("over", [-1, 0, 1])
def test_write_at_the_change_of_window(over, e4m3, means):
    """Tokens around the count from which windows are four times as wide: eight blocks for every SM
    that this device has.  The caches get the same rows either way, as the older tests check."""
    Hkv, D, page = 16, 128, 64
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    T = 8 * sms * 4 * (256 // (D // 8)) // Hkv + over
    num = -(-T // page) + 1
    g = torch.Generator(device="cuda").manual_seed(T)
    k, v = (torch.randn(T, Hkv, D, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    order = torch.randperm(num, generator=g, device="cuda")
    t = torch.arange(T, device="cuda")
    slots = (order[t // page] * page + t % page).to(torch.int32)
    p = mcs.paged(1, Hkv, Hkv, D, page, num, num, kv=int(e4m3), k_scale=KS, v_scale=VS)
    caches = torch.zeros(2, num, Hkv, page, D, dtype=torch.uint8 if e4m3 else torch.bfloat16, device="cuda")
    mean = torch.zeros(num, Hkv, D, dtype=torch.bfloat16, device="cuda")
    mcs.mcs_paged_write(p, k, v, slots, caches[0], caches[1], mean if means else None)
    values = None
    for x, scale, cache in ((k, KS, caches[0]), (v, VS, caches[1])):
        if e4m3:
            codes = torch.empty(x.shape, dtype=torch.uint8, device="cuda")
            mcs.mcs_quantize_e4m3(x, scale, codes)
            x = codes
        assert torch.equal(cache.transpose(1, 2).reshape(-1, Hkv, D)[slots.long()], x)
        values = x if values is None else values
    if means:
        values = values.view(torch.float8_e4m3fn).double() * KS if e4m3 else values.double()
        for j in (0, 1, num - 2):
            rows = values[j * page:(j + 1) * page]
            tol = 2.0 ** -8 * rows.mean(0).abs() + (page + 2) * U * rows.abs().mean(0)
            assert ((mean[order[j]].double() - rows.mean(0)).abs() <= tol).all()


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_steps_one_behind_another_see_their_own_rows(e4m3):
    """Keys normalised in place, written, averaged, scored and attended to, many steps with nothing
    between the launches (each kernel is set up while the one in front still writes what it reads),
    against the same steps one at a time."""
    B, Hq, Hkv, D, page, P, steps, most = 6, 16, 8, 128, 16, 40, 14, 45
    num = B * P
    r = np.random.default_rng(5)
    p = mcs.paged(B, Hq, Hkv, D, page, num, P, kv=int(e4m3), k_scale=KS, v_scale=VS)
    g = torch.Generator(device="cuda").manual_seed(5)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)
    new = r.integers(0, most, (steps, B))
    new[:, 0] = 1
    T = int(new.sum(1).max()) + 2
    ks, vs, qs = rand(steps, T, 1, Hkv, D), rand(steps, T, Hkv, D), rand(steps, B, Hq, D)
    angle = torch.rand(steps * most, D // 2, generator=g, device="cuda") * 6
    cos, sin = angle.cos(), angle.sin()
    rp = mcs.rope_params(T, 1, Hkv, 0, D, D, steps * most, layout=mcs.LAYOUT_BNHD)
    new, free = _i32(new), _i32(r.permutation(num))
    ws = mcs.empty_workspace(max(mcs.mcs_paged_decode_workspace(p), mcs.mcs_paged_select_workspace(p)))
    dt = torch.uint8 if e4m3 else torch.bfloat16
    caches = torch.zeros(2, num, Hkv, page, D, dtype=dt, device="cuda")
    mean = torch.zeros(num, Hkv, D, dtype=torch.bfloat16, device="cuda")
    lens, head, table, cu = _i32([0] * B), _i32([0]), _i32(np.zeros((B, P))), _i32([0] * (B + 1))
    slots, pos, k = _i32([0] * T), _i32([0] * T), torch.empty_like(ks[0])
    sels = torch.zeros(steps, B, Hkv, 4, dtype=torch.int32, device="cuda")
    outs = torch.zeros(steps, B, Hq, D, dtype=torch.bfloat16, device="cuda")

    def go(between):
        for x in (caches, mean, lens, head, table):
            x.zero_()
        for i in range(steps):
            k.copy_(ks[i])
            calls = [lambda: mcs.mcs_paged_plan(p, new[i], lens, free, head, table, lens, head, cu, slots, pos),
                     lambda: mcs.mcs_qk_norm_rope(rp, k, None, None, None, cos, sin, pos.view(T, 1), k, None),
                     lambda: mcs.mcs_paged_write(p, k.view(T, Hkv, D), vs[i], slots, caches[0], caches[1], mean),
                     lambda: mcs.mcs_paged_select(p, qs[i], mean, table, lens, sels[i], ws),
                     lambda: mcs.mcs_paged_decode_sparse(p, qs[i], caches[0], caches[1], table, lens, sels[i], outs[i], ws)]
            for call in calls:
                call()
                between()

    state = (caches, mean, lens, head, table, sels, outs)
    go(torch.cuda.synchronize)
    want = [x.clone() for x in state]
    assert mcs.mcs_device_status() == 0 and want[6].isfinite().all()
    same = lambda: all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(state, want))
    go(lambda: None)
    torch.cuda.synchronize()
    assert same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        go(lambda: None)
    for _ in range(4):
        sels.zero_(), outs.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert same()
    assert mcs.mcs_device_status() == 0


@pytest.mark.parametrize("B,Hq,Hkv,D,e4m3,page,select", [(20, 8, 8, 128, False, 128, 80), (48, 32, 16, 64, True, 64, 120)])
def test_sparse_lists_long_enough_for_the_last_blocks(B, Hq, Hkv, D, e4m3, page, select):
    # as the dense test above: pages stand in many tables; lists of every head are their own, some
    # with holes, some sequences short or empty
    r = np.random.default_rng(select)
    most = select * page * 5 // 4
    c = Cache([30 * page] + [0] * (B - 1), Hq, Hkv, D, page, e4m3, seed=B, extra=-(-most // page) - 30)
    live = c.table[0, :30].copy()
    c.lens = [int(x) for x in r.integers(most * 9 // 10, most, B)]
    for i, x in ((2, 0), (B // 2, 1), (B - 3, 17), (B - 1, page + 1)):
        c.lens[i] = x
    c.table = live[r.integers(0, 30, c.table.shape)]
    c.dtable, c.dlens = _i32(c.table), _i32(c.lens)
    sel = _sel(c, select, 3)
    sel[1, 0, ::3] = -1
    tiles = sum(Hkv * (min(-(-x // page), select) * page // (4096 // (D * (1 if e4m3 else 2)))) for x in c.lens)
    assert tiles >= 2 * torch.cuda.get_device_properties(0).multi_processor_count * 4 * 64
    first = c.run(_i32(sel))
    c.check(*first, sel, terms=2048)
    again = c.run(_i32(sel))
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_join_of_more_segments_than_its_blocks_take_at_once(e4m3):
    # 20480 segments, 32 to a block of the join and more blocks than are resident; long sequences
    # among short ones, so that some segments have parts
    r = np.random.default_rng(2)
    lens = [int(x) for x in r.integers(0, 4, 4096)]
    for i in (5, 6, 1999, 4095):
        lens[i] = 1900 + i % 7
    c = Cache(lens, 5, 5, 64, 16, e4m3, seed=3, extra=0)
    c.check(*c.run())
