"""GPU parity of paged attention and shared decode where their kernels' bookkeeping is at its edges:
many short segments of which only some are looked through, keys that outweigh all others, batches on
either side of what is worth sharing, lengths and moves that cannot be."""

import numpy as np
import pytest
import torch

from oracle import paged_oracle as po
from tests import test_gpu_paged as tp
from tests import test_gpu_paged_attn as ta
from tests import test_gpu_paged_sharing as ts
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


# ------------------------------------------------------------------ beginnings read once, whatever they save

LARGER = [  # groups, Hq, Hkv, D, page: odd numbers of rows, more than 16 and more than 128 heads per KV head
    ([(17, [1, None, 300, 0, 45])], 9, 1, 128, 16), ([(33, [5, 0, 7]), (70, [90] * 4)], 34, 2, 64, 16),
    ([(9, [130, 3, 40]), (0, [7]), (2, [1, 1])], 129, 1, 128, 32), ([(12, [0, 17, None, 9, 64])], 261, 1, 64, 64),
    ([(4, [55] * 33), (3, [1, 2])], 15, 3, 128, 128)]


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("groups,Hq,Hkv,D,page", ta.FAMILIES + LARGER)
def test_small_beginnings_read_once(groups, Hq, Hkv, D, page, e4m3, monkeypatch):
    monkeypatch.setenv("MCS_TEST_SHARED_WORTH", "0")
    c = ta.Family(groups, Hq, Hkv, D, page, e4m3, seed=Hq + page)
    first = c.run()
    assert mcs.mcs_device_status() == 0
    c.check(*first)
    again = c.run()
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    assert torch.equal(c.run(lse=False)[0], first[0])
    # the same read by themselves: another order of the sums, other roundings of the weights
    monkeypatch.setenv("MCS_TEST_SHARED_WORTH", str(1 << 60))
    c.check(*c.run())


def test_the_larger_families_are_read_by_themselves_too():
    for groups, Hq, Hkv, D, page in LARGER:
        for e4m3 in (False, True):
            c = ta.Family(groups, Hq, Hkv, D, page, e4m3, seed=Hq + page)
            c.check(*c.run())


@pytest.mark.parametrize("Hq,Hkv,D,page", [(8, 2, 128, 16), (18, 1, 64, 32)])
def test_infinite_values_in_a_common_beginning(Hq, Hkv, D, page, monkeypatch):
    """Beginnings that end inside a tile of 128 keys, and with one: columns with an infinite value or a NaN
    code come out so in the sequences that have it, and nowhere else."""
    monkeypatch.setenv("MCS_TEST_SHARED_WORTH", "0")
    tile = 128 // page
    groups = [(2 * tile + 1, [3, 0, 200]), (3 * tile, [1, 40, 0]), (3 * tile - 1, [9, 8])]
    for e4m3 in (False, True):
        clean = ta.Family(groups, Hq, Hkv, D, page, e4m3, seed=7)
        want, want_ls = clean.run()
        c = ta.Family(groups, Hq, Hkv, D, page, e4m3, seed=7)
        hit = torch.zeros(want.shape, dtype=torch.bool, device="cuda")
        group = Hq // Hkv
        for g, (t, h, col) in enumerate([((2 * tile + 1) * page - 1, 0, 5), (17, Hkv - 1, D - 1), ((3 * tile - 1) * page - 2, 0, 0)]):
            b = c.starts[g]
            c.v[int(c.table[b, t // page]), h, t % page, col] = 0x7F if e4m3 else [np.inf, -np.inf, np.nan][g]
            hit[c.starts[g]:c.starts[g + 1], h * group:(h + 1) * group, col] = True
        out, ls = c.run()
        assert mcs.mcs_device_status() == 0
        assert not torch.isfinite(out.float()[hit]).any()
        assert torch.equal(out[~hit], want[~hit]) and torch.equal(ls, want_ls)


@pytest.mark.parametrize("seed", range(24))
def test_read_once_of_random_shapes(seed, monkeypatch):
    monkeypatch.setenv("MCS_TEST_SHARED_WORTH", "0")
    r = np.random.default_rng(7000 + seed)
    Hkv = int(r.choice([1, 2, 3, 4]))
    Hq, D, page = Hkv * int(r.choice([1, 3, 4, 8, 9, 16, 17, 20, 33, 140])), int(r.choice([64, 128])), int(r.choice([16, 32, 64, 128]))
    groups = [(int(int(r.choice([1, 30, 400])) * r.random() * 16 / page) + int(r.integers(0, 2)),
               [int(200 ** r.random()) - 1 if r.random() > 0.1 else None for _ in range(int(r.integers(1, int(r.choice([2, 9, 40])))))])
              for _ in range(int(r.integers(1, 5)))]
    e4m3 = bool(seed // 2 % 2)
    c = ta.Family(groups, Hq, Hkv, D, page, e4m3, seed=seed, q_stride=int(r.choice([0, (Hq + 2 * Hkv) * D])))
    c.check(*c.run())
    # groups of empty sequences may name more pages than a table row has, which is reported
    assert mcs.mcs_device_status() == (6 if max(c.shared) > c.p.max_pages else 0)


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_batches_on_either_side_of_what_is_worth_it(e4m3):
    """Beginnings that save just enough to be read once and just too little: both as a decode says, and the
    bits are those of beginnings read once for the former alone."""
    Hq, Hkv, D, page, es = 8, 8, 128, 128, 2 if e4m3 else 4
    for n in (4, 12):
        unit = page * Hkv * D * es  # bytes of a page
        need = next(x for x in range(1, 10 ** 6) if (n - 1) * x * unit >= 200000000 + min(x * unit, 2 ** 27) +
                    (e4m3 * max(0, x * unit - 2 ** 27)))
        for pages in (need, need - 1):
            c = ta.Family([(pages, [5] * (n - 1) + [140])], Hq, Hkv, D, page, e4m3, seed=n)
            got = c.run()
            assert mcs.mcs_device_status() == 0
            c.check(*got)
            with pytest.MonkeyPatch.context() as m:
                m.setenv("MCS_TEST_SHARED_WORTH", "0")
                once = c.run()
            if pages == need:
                assert torch.equal(got[0], once[0]) and torch.equal(got[1], once[1])
            else:  # (joined by the same kernel as if something were shared, so not a decode's bits)
                assert not torch.equal(got[1], once[1])


@pytest.mark.parametrize("e4m3,Hq,Hkv,D,page,long", [(False, 8, 2, 128, 16, 0), (True, 4, 4, 64, 32, 0), (False, 16, 16, 128, 64, 1100),
                                                     (True, 9, 1, 128, 16, 300)])
def test_beams_together_with_their_beginnings_read_once(e4m3, Hq, Hkv, D, page, long, monkeypatch):
    monkeypatch.setenv("MCS_TEST_SHARED_WORTH", "0")
    ts.test_beams_of_two_requests_together(e4m3, Hq, Hkv, D, page, long)


# ------------------------------------------------------------------ one key that outweighs all others

def _with_a_sink(c, rows, seed):
    """Scores of log2 weight p in front of all others' 0 for the first key, p from 20 to 34 over the rows; the
    first value is zero in even columns, small in odd ones, the others are about 1."""
    r = np.random.default_rng(seed)
    pid = int(c.table[0, 0])
    value = torch.from_numpy(r.uniform(60, 120, c.v.shape[-1])).to(torch.float8_e4m3fn).view(torch.uint8).cuda()
    hole = c.k == 0x7F
    c.k.masked_fill_(~hole, 0)
    c.v.copy_(torch.where(c.v == 0x7F, c.v, value))
    c.k[pid, :, 0, 0] = 0x7E  # 448
    c.v[pid, :, 0, 0::2] = 0
    c.v[pid, :, 0, 1::2] = 0x58  # 16
    c.q.zero_()
    c.q[..., 0] = torch.linspace(20, 34, rows).to(torch.bfloat16).cuda().view(c.q.shape[0], c.q.shape[1])


SINK_SCALE = float(np.float32(np.log(2) / (448 * tp.KS)))


def _check_sink(out, ls, q, c, oracle):
    """Rounding to bf16; scores and exponentials as in test_gpu_paged_attn; a weight as f16: 2^-11 of it, and where
    it is small 2^-37 of the row's largest: the reference lies 2^12 below the maximum when it is set, f16
    rounds to multiples of 2^-24, and what the maximum grows by makes the sum that divides larger."""
    k, v = (_f64(x) * s for x, s in zip((c.k, c.v), c.scales))
    want, lse, absv, size = oracle(_f64(q), k, v)
    n, D = max(c.lens), c.D
    tol, tol_lse = ta.tolerance(want, lse, absv, size, D, n, True, weight=2.0 ** -11)
    tol = tol + 2.0 ** -37 * n * np.nanmax(np.abs(v))
    assert not np.isnan(want).any()
    off = np.abs(_f64(out) - want)
    assert (off <= tol).all(), (off / tol).max()
    assert (np.abs(_f64(ls) - lse) <= tol_lse).all()
    # the many others are what even columns consist of
    assert (want[..., 0::2] > 2 * tol[..., 0::2]).all()


def _params(c, B, kv=1):
    return mcs.paged(B, c.p.Hq, c.p.Hkv, c.D, c.page, c.p.num_pages, c.p.max_pages, kv=kv, scale=c.p.scale,
                     k_scale=c.p.k_scale, v_scale=c.p.v_scale)


@pytest.mark.parametrize("D,new,tokens,times", [(128, 3, 75600, 1), (64, 40, 75600, 1), (128, 17, 300000, 1),
                                                (128, 2, 75600, 170), (64, 3, 20000, 400)])
def test_many_small_weights_behind_a_large_one(D, new, tokens, times):
    """`times`: the same sequence so many times over, so that a block reads most of it for its rows."""
    c = ta.Step([tokens], [new], 8, 1, D, 128, True, behind=0, scale=SINK_SCALE)
    _with_a_sink(c, new * 8, D)
    q, table = c.q, c.table
    c.q, c.dtable, c.dlens = c.q.repeat(times, 1, 1), _i32(np.repeat(table, times, 0)), _i32([tokens] * times)
    c.p, c.dcu = _params(c, times), _i32(np.arange(times + 1) * new)
    out, ls = (x.view((times, new) + x.shape[1:]) for x in c.attn())
    assert mcs.mcs_device_status() == 0
    assert times == 1 or ls.shape == (times, new, 8)
    _check_sink(out, ls, q, c, lambda q, k, v: po.attn(q, k, v, table, c.lens, c.cu, c.scale))


@pytest.mark.parametrize("Hq,D,tokens,times", [(8, 128, 75648, 1), (20, 64, 75648, 1), (4, 128, 299904, 1),
                                               (8, 128, 75648, 160), (20, 64, 30080, 200)])
def test_many_small_weights_in_a_common_beginning(Hq, D, tokens, times, monkeypatch):
    """`times`: so many groups of two sequences behind the same pages."""
    for worth in ("0", str(1 << 60)):
        monkeypatch.setenv("MCS_TEST_SHARED_WORTH", worth)
        c = ta.Family([(tokens // 128, [1, 40])], Hq, 1, D, 128, True, scale=SINK_SCALE)
        _with_a_sink(c, 2 * Hq, D)
        q, table, lens = c.q, c.table, c.lens
        c.q, c.dtable, c.dlens = q.repeat(times, 1, 1), _i32(np.tile(table, (times, 1))), _i32(lens * times)
        c.p, c.dstarts, c.dshared = _params(c, 2 * times), _i32(np.arange(times + 1) * 2), _i32([tokens // 128] * times)
        c.ws = mcs.empty_workspace(mcs.mcs_paged_decode_shared_workspace(c.p))
        out, ls = (x[:-1].view((times, 2) + x.shape[1:]) for x in c.run())
        assert mcs.mcs_device_status() == 0
        _check_sink(out, ls, q, c, lambda q, k, v: po.decode(q, k, v, table, lens, c.scale))


# ------------------------------------------------------------------ what cannot be

@pytest.mark.parametrize("length", [-1, -2 ** 31, "too long", 2 ** 31 - 1])
def test_attn_reports_lengths_of_sequences_without_new_tokens(length):
    c = ta.Step([300, 90, 70, 40], [10, 0, 9, 0], 4, 2, 64, 16, seed=6)
    for b in (1, 3):
        lens = list(c.lens)
        lens[b] = c.p.max_pages * 16 + 1 if length == "too long" else length
        c.dlens = _i32(lens)
        got = c.attn()
        assert mcs.mcs_device_status() == 6
        c.check_attn(*got)
    c.dlens = _i32([300, 0, 70, c.p.max_pages * 16])
    c.check_attn(*c.attn())
    assert mcs.mcs_device_status() == 0
