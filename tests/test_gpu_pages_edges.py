"""GPU tests of forks, compaction and page copies with requests at the edge of what they may hold."""

import numpy as np
import pytest
import torch

from oracle import mcs_oracle as orc
from oracle import paged_oracle as po
from tests import test_gpu_pages as tg
from tests import test_gpu_paged as tp
from tests import test_gpu_paged_attn as ta
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


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_proposed_tokens_are_taken_back(e4m3):
    """Sequences that propose tokens, keep some of them and give the others back, step by step: lengths are
    lowered, the free list is made anew, and what follows attends to what was kept.  Pages suffice for what is
    held at any time, not for all that was ever asked for."""
    B, Hq, Hkv, D, page, steps = 5, 8, 2, 64, 16, 12
    r = np.random.default_rng(3)
    prompts, most = [40, 16, 1, 77, 32], 40
    num, P = sum(-(-(n + most * 2) // page) + 1 for n in prompts), 12
    g = torch.Generator(device="cuda").manual_seed(3)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)
    ks, vs = (tp.KS, tp.VS) if e4m3 else (1.0, 1.0)
    kc, vc = (torch.full((num, Hkv, page, D), 0x7F if e4m3 else float("nan"), device="cuda").to(torch.uint8 if e4m3 else torch.bfloat16)
              for _ in range(2))
    mean = rand(num, Hkv, D)
    p = mcs.paged(B, Hq, Hkv, D, page, num, P, kv=int(e4m3), k_scale=ks, v_scale=vs)
    free, head, extra = _i32(r.permutation(num)), _i32([0]), _i32([0] * num)
    table, lens = _i32(np.full((B, P), -1)), _i32([0] * B)
    ws, wc = (mcs.empty_workspace(f(p)) for f in (mcs.mcs_paged_attn_workspace, mcs.mcs_paged_compact_workspace))
    kept = [[] for _ in range(B)]  # rows of keys and values
    asked = 0
    for step in range(steps):
        new = prompts if step == 0 else [int(x) for x in r.integers(0, 30, B)]
        T = sum(new)
        asked += sum(-(-n // page) for n in new)
        cu, slots = _i32([0] * (B + 1)), _i32([0] * T)
        mcs.mcs_paged_plan(p, _i32(new), lens, free, head, table, lens, head, cu, slots)
        k, v, q = (rand(T, h, D) for h in (Hkv, Hkv, Hq))
        mcs.mcs_paged_write(p, k, v, slots, kc, vc, mean)
        out, ls = torch.empty_like(q), torch.empty(T, Hq, device="cuda")
        mcs.mcs_paged_attn(p, q, kc, vc, table, lens, cu, out, ws, lse=ls)
        assert mcs.mcs_device_status() == 0
        stored = lambda x, s: (orc.e4m3_decode(orc.e4m3_encode(x.float().cpu().numpy(), s)).astype(np.float64) * s if e4m3
                               else tp._f64(x))
        kx, vx, at = stored(k, ks), stored(v, vs), 0
        for b, n in enumerate(new):
            kept[b] += [(kx[t], vx[t]) for t in range(at, at + n)]
            at += n
        n = [len(x) for x in kept]
        first = np.cumsum([0] + n)
        k1, v1 = (np.stack([row[i] for x in kept for row in x])[:, :, None] for i in (0, 1))
        t1 = np.full((B, max(n)), -1)
        for b in range(B):
            t1[b, :n[b]] = np.arange(first[b], first[b + 1])
        want, lse, absv, size = po.attn(tp._f64(q), k1, v1, t1, n, np.cumsum([0] + list(new)), D ** -0.5)
        tol, tol_lse = ta.tolerance(want, lse, absv, size, D, max(n), e4m3)
        assert (np.abs(tp._f64(out) - want) <= tol).all() and (np.abs(tp._f64(ls) - lse) <= tol_lse).all()
        # some are kept
        back = [0 if step == 0 else int(r.integers(0, x + 1)) for x in new]
        for b in range(B):
            while len(kept[b]) - (n[b] - back[b]) > 0 or len(kept[b]) > most + prompts[b]:
                kept[b].pop()
        lens.copy_(_i32([len(x) for x in kept]))
        mcs.mcs_paged_compact(p, lens, table, extra, table, extra, free, head, _i32(np.zeros((0, 3))), wc)
        held = {int(x) for b, row in enumerate(table.cpu().numpy()) for x in row[:-(-len(kept[b]) // page)]}
        assert len(held) == sum(-(-len(x) // page) for x in kept)
        assert free[int(head):].tolist() == [x for x in range(num) if x not in held]
        assert (extra == 0).all()
    assert asked > num
    assert mcs.mcs_device_status() == 0
