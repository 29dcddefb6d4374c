"""Seeded random shapes of the paged cache and of the norm with rotation, against the fp64
oracle with the tolerances that test_gpu_paged.py and test_gpu_norm_rope.py derive."""

import numpy as np
import pytest
import torch

from oracle import paged_oracle as po
from tests import test_gpu_norm_rope as tn
from tests import test_gpu_paged as tp
from token_sparse_attention_gb300 import build as mcs_build
from token_sparse_attention_gb300 import mcs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    mcs_build.build()
    mcs.lib()
    yield
    assert mcs.mcs_device_status() == 0


def _heads(r):
    Hkv = int(r.choice([1, 2, 3, 4, 8]))
    return Hkv * int(r.choice([1, 2, 3, 4, 7, 8, 9, 16, 17, 20])), Hkv


def _lens(r, B, most):
    lens = [int(most ** r.random()) for _ in range(B)]
    for i in range(B):
        if r.random() < 0.15:
            lens[i] = 0
    return lens


@pytest.mark.parametrize("seed", range(24))
def test_decode_and_selection(seed):
    r = np.random.default_rng(1000 + seed)
    (Hq, Hkv), D, page = _heads(r), int(r.choice([64, 128])), int(r.choice([16, 32, 64, 128]))
    B = int(r.integers(1, 12))
    lens = _lens(r, B, int(r.choice([20, 300, 3000])))
    c = tp.Cache(lens, Hq, Hkv, D, page, bool(seed % 2), seed=seed, extra=int(r.integers(0, 40)),
                 scale=float(r.choice([0.0, 0.02, 0.3])),
                 q_stride=int(r.choice([0, Hq * D, (Hq + 2 * Hkv) * D, Hq * D + 8])))
    c.check(*c.run())
    pages = max(1, max(-(-x // page) for x in lens))
    select = int(r.integers(1, pages + 3))
    sink = int(r.integers(0, min(select, 3) + 1))
    recent = int(r.integers(0, min(select - sink, 3) + 1))
    mean = c.means()
    ws = mcs.empty_workspace(mcs.mcs_paged_select_workspace(c.p))
    sel = torch.full((B, Hkv, select), -7, dtype=torch.int32, device="cuda")
    mcs.mcs_paged_select(c.p, c.q, mean, c.dtable, c.dlens, sel, ws, sink=sink, recent=recent)
    want = po.select(tp._f64(c.q), tp._f64(mean), c.table, lens, page, select, sink, recent)
    np.testing.assert_array_equal(sel.cpu().numpy(), want)
    c.check(*c.run(sel), want)
    holes = tp._sel(c, select, seed, True)
    c.check(*c.run(tp._i32(holes)), holes)


@pytest.mark.parametrize("seed", range(16))
def test_plan_and_write(seed):
    r = np.random.default_rng(2000 + seed)
    Hkv, D, page, e4m3 = int(r.choice([1, 2, 5, 8])), int(r.choice([64, 128])), int(r.choice([16, 32, 64, 128])), bool(seed % 2)
    B = int(r.integers(1, 20))
    old, new = np.array(_lens(r, B, 400)), np.array(_lens(r, B, int(r.choice([2, 60, 900]))))
    after = old + new
    c = tp.Cache([int(x) for x in after], Hkv, Hkv, D, page, e4m3, seed=seed)
    have, total = -(-old // page), -(-after // page)
    fresh = np.concatenate([c.table[b, have[b]:total[b]] for b in range(B)])
    skip = int(r.integers(0, 4))  # free pages that earlier steps took
    free = np.concatenate([np.zeros(skip, int), fresh, np.zeros(3, int)])
    table = c.table.copy()
    for b in range(B):
        table[b, have[b]:] = -1
    T = int(new.sum()) + int(r.integers(0, 9))
    want = po.plan(new, old, free, skip, table, page, T, c.p.num_pages)
    got = tp._plan(c.p, new, old, free, skip, table, T, in_place=bool(r.integers(2)))
    for x, y in zip(got, want):
        np.testing.assert_array_equal(x, y)
    if T == 0:
        return
    c.p.kv_stride = int(r.choice([0, Hkv * D, 3 * Hkv * D, Hkv * D + 8]))
    g = torch.Generator(device="cuda").manual_seed(seed)
    k, v = (torch.randn(T, c.p.kv_stride or Hkv * D, generator=g, device="cuda").to(torch.bfloat16)[:, :Hkv * D]
            .view(T, Hkv, D) for _ in range(2))
    mean = c.means()
    before = [x.clone() for x in (c.k, c.v, mean)]
    mcs.mcs_paged_write(c.p, k, v, tp._i32(want[4]), c.k, c.v, mean)
    live = torch.from_numpy(want[4] >= 0).cuda()
    s = tp._i32(want[4])[live].long()
    codes = []
    for x, scale in ((k, tp.KS), (v, tp.VS)):
        x = x.contiguous()
        if e4m3:
            y = torch.empty(x.shape, dtype=torch.uint8, device="cuda")
            mcs.mcs_quantize_e4m3(x, scale, y)
            x = y
        codes.append(x[live])
    for cache, x, old_rows in zip((c.k, c.v), codes, before):
        old_rows[s // page, :, s % page] = x
        assert torch.equal(cache.view(torch.uint8), old_rows.view(torch.uint8))
    held = {}
    for x in want[4][want[4] >= 0]:
        held[x // page] = max(held.get(x // page, 0), x % page + 1)
    got, was = tp._f64(mean), tp._f64(before[2])
    values = tp._f64(c.k) * c.scales[0]
    for pg in range(c.p.num_pages):
        if pg not in held:
            np.testing.assert_array_equal(got[pg], was[pg])
            continue
        rows = values[pg, :, :held[pg]]
        tol = 2.0 ** -8 * np.abs(rows.mean(1)) + (page + 2) * tp.U * np.abs(rows).mean(1)
        assert (np.abs(got[pg] - rows.mean(1)) <= tol).all()


@pytest.mark.parametrize("seed", range(20))
def test_norm_and_gradients(seed):
    r = np.random.default_rng(3000 + seed)
    Hq, Hkv = int(r.integers(1, 41)), int(r.choice([0, 1, 2, 3, 8, 13, 40]))
    D = int(r.choice([64, 128]))
    B, N = int(r.integers(1, 5)), int(1500 ** r.random())
    case = (B, N, Hq, Hkv, D, 16 * int(r.integers(0, D // 16 + 1)), bool(r.integers(2)), int(r.integers(2)),
            bool(r.integers(2)), bool(r.integers(2)), bool(r.integers(2)))
    c = tn.Case(*case, eps=float(r.choice([1e-6, 1e-2])))
    outs, (dx, dw) = c.forward(), c.backward()
    for i in range(2):
        if c.H[i] == 0:
            continue
        x, w, *rest = c.oracle(i)
        want = po.norm_rope(x, w, *rest)
        tol = 2.0 ** -8 * np.abs(want) + (D / 2 + 10) * tn.U * tn._mix(want, c.rot, c.inter) * 2 ** 0.5
        assert (np.abs(c.token_major(outs[i]) - want) <= tol).all()
        dy = c.token_major(c.dy[i])
        want, want_w, _ = po.norm_rope_backward(dy, x, w, *rest)
        rr = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + c.eps)
        g, xh = tn._mix(dy, c.rot, c.inter), np.abs(x * rr)
        tol = 2.0 ** -8 * np.abs(want) + (D + 20) * tn.U * rr * (g * np.abs(w) + xh * (g * np.abs(w) * xh).mean(-1, keepdims=True))
        assert (np.abs(tn._f64(dx[i]) - want) <= tol).all()
        assert (np.abs(tn._f64(dw[i]) - want_w) <= (D / 2 + 410) * tn.U * (g * xh).sum((0, 1, 2))).all()
