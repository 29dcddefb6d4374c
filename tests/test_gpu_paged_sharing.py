"""Prompts, forks, shared decoding and compaction as a program runs them together, and seeded random
shapes of each against the oracle."""

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

_i32, _f64 = tp._i32, tp._f64


@pytest.fixture(scope="module", autouse=True)
def _lib():
    mcs_build.build()
    mcs.lib()
    yield
    assert mcs.mcs_device_status() == 0


@pytest.mark.parametrize("e4m3,Hq,Hkv,D,page,long", [(False, 8, 2, 128, 16, 0), (True, 4, 4, 64, 32, 0), (False, 16, 16, 128, 64, 1100)])
def test_beams_of_two_requests_together(e4m3, Hq, Hkv, D, page, long):
    """Two prompts in two pieces, each continued by four beams that are reordered every step, over the
    caches of two layers; then the cache is compacted and one more step follows.  What every sequence
    has seen is kept aside, and each attention is checked against it.  `long`: prompts long enough for
    the beams' common beginning to be read once."""
    r, W, B = np.random.default_rng(Hq), 4 if not long else 12, 2
    prompts, steps = [70 + long, 45 + long], 5
    num = 2 * (sum(prompts) // page + 2) + 2 * W * (steps // page + 3)
    P = (max(prompts) + steps) // page + 2
    g = torch.Generator(device="cuda").manual_seed(Hq)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)
    ks, vs = (tp.KS, tp.VS) if e4m3 else (1.0, 1.0)
    kind = torch.uint8 if e4m3 else torch.bfloat16
    caches = [[torch.full((num, Hkv, page, D), 0x7F if e4m3 else float("nan"), device="cuda").to(kind) for _ in range(2)] for _ in range(2)]
    mean = [rand(num, Hkv, D) for _ in range(2)]
    params = lambda n: mcs.paged(n, Hq, Hkv, D, page, num, P, kv=int(e4m3), k_scale=ks, v_scale=vs)
    stored = lambda x, s: (orc.e4m3_decode(orc.e4m3_encode(x.float().cpu().numpy(), s)).astype(np.float64) * s if e4m3 else _f64(x))
    free, head = _i32(r.permutation(num)), _i32([0])
    extra, table, lens = _i32(np.zeros(num)), _i32(np.full((B, P), -1)), _i32([0] * B)
    seen = [[[], []] for _ in range(B)]  # per sequence and layer: (key, value) rows

    def step(new, table, lens, decode=None):
        n, T = len(new), sum(new)
        p = params(n)
        cu, slots = _i32([0] * (n + 1)), _i32([0] * T)
        mcs.mcs_paged_plan(p, _i32(new), lens, free, head, table, lens, head, cu, slots)
        k, v, q = (rand(T, h, D) for h in (Hkv, Hkv, Hq))
        for layer, (kc, vc) in enumerate(caches):
            kl, vl = (k, v) if layer == 0 else (v, k)
            mcs.mcs_paged_write(p, kl, vl, slots, kc, vc, mean[layer])
            kx, vx = stored(kl, ks), stored(vl, vs)
            at = 0
            for b, m in enumerate(new):
                seen[b][layer] += [(kx[t], vx[t]) for t in range(at, at + m)]
                at += m
            out, ls = torch.empty_like(q), torch.empty(T, Hq, device="cuda")
            if decode is None:
                ws = mcs.empty_workspace(mcs.mcs_paged_attn_workspace(p))
                mcs.mcs_paged_attn(p, q, kc, vc, table, lens, cu, out, ws, lse=ls)
            else:
                ws = mcs.empty_workspace(mcs.mcs_paged_decode_shared_workspace(p))
                mcs.mcs_paged_decode_shared(p, q, kc, vc, table, lens, *decode, out, ws, lse=ls)
            assert mcs.mcs_device_status() == 0
            # the same from what was seen, as sequences of pages of one token
            hist = [np.stack([np.stack(x) for x in s[layer]]) for s in seen[:n]]
            k1, v1 = (np.concatenate([h[:, i] for h in hist])[:, :, None] for i in (0, 1))
            first = np.cumsum([0] + [len(h) for h in hist])
            t1 = np.full((n, max(len(h) for h in hist)), -1)
            for b, h in enumerate(hist):
                t1[b, :len(h)] = np.arange(first[b], first[b + 1])
            want, lse, absv, size = po.attn(_f64(q), k1, v1, t1, [len(h) for h in hist], np.cumsum([0] + new), D ** -0.5)
            tol, tol_lse = ta.tolerance(want, lse, absv, size, D, t1.shape[1], e4m3)
            assert (np.abs(_f64(out) - want) <= tol).all() and (np.abs(_f64(ls) - lse) <= tol_lse).all()

    def fork(parents, table, lens):
        n, p = len(parents), params(lens.numel())
        lo, to, moves = _i32([0] * n), _i32(np.zeros((n, P))), _i32(np.zeros((n, 3)))
        ws = mcs.empty_workspace(mcs.mcs_paged_fork_workspace(p))
        mcs.mcs_paged_fork(p, _i32(parents), lens, table, extra, free, head, lo, to, extra, free, head, moves, ws)
        for layer, (kc, vc) in enumerate(caches):
            mcs.mcs_paged_copy(p, moves, kc, vc, mean[layer])
        seen[:] = [[list(x) for x in seen[x]] for x in parents]
        return to, lo

    step([40 + long, 45 + long], table, lens)
    step([30, 0], table, lens)
    table, lens = fork([0] * W + [1] * W, table, lens)
    groups = _i32([0, W, 2 * W])
    for i in range(steps):
        step([1] * 2 * W, table, lens, (groups, _i32([x // page for x in prompts])))
        table, lens = fork([int(r.integers(b // W * W, b // W * W + W)) for b in range(2 * W)], table, lens)
    # holders and the free list are those of the tables
    held = {}
    t, n = table.cpu().numpy(), lens.tolist()
    for b in range(2 * W):
        for j in range(-(-n[b] // page)):
            held[t[b, j]] = held.get(t[b, j], 0) + 1
    assert (extra.cpu().numpy() == [max(held.get(x, 0) - 1, 0) for x in range(num)]).all()
    assert sorted(free[int(head):].tolist()) == [x for x in range(num) if x not in held]
    # some sequences end, the others move to the front
    table, lens = fork([0, 1, W, -1], table, lens)
    seen[3] = [[], []]
    p = params(4)
    moves = _i32(np.zeros((num, 3)))
    mcs.mcs_paged_compact(p, lens, table, extra, table, extra, free, head, moves, mcs.empty_workspace(mcs.mcs_paged_compact_workspace(p)))
    for layer, (kc, vc) in enumerate(caches):
        mcs.mcs_paged_copy(p, moves, kc, vc, mean[layer])
    live = num - (num - int(head))
    assert free[int(head):].tolist() == list(range(live, num))
    seen[3] = [[], []]
    step([3, 1, 2, 5], table, lens)


def _heads(r):
    Hkv = int(r.choice([1, 2, 3, 4, 8]))
    return Hkv * int(r.choice([1, 2, 3, 4, 7, 8, 9, 16, 17, 20])), Hkv


@pytest.mark.parametrize("seed", range(20))
def test_attn_of_random_shapes(seed):
    r = np.random.default_rng(3000 + seed)
    (Hq, Hkv), D, page = _heads(r), int(r.choice([64, 128])), int(r.choice([16, 32, 64, 128]))
    B = int(r.integers(1, 10))
    most = int(r.choice([3, 40, 300, 700]))
    new = [int(most ** r.random()) if r.random() > 0.15 else 0 for _ in range(B)]
    lens = [n + int(int(r.choice([1, 50, 1500])) * r.random()) for n in new]
    c = ta.Step(lens, new, Hq, Hkv, D, page, bool(seed % 2), seed=seed, behind=int(r.integers(0, 9)) + (sum(new) == 0),
                extra=int(r.integers(0, 20)), scale=float(r.choice([0.0, 0.02, 0.3])),
                q_stride=int(r.choice([0, Hq * D, (Hq + 2 * Hkv) * D, Hq * D + 8])))
    c.check_attn(*c.attn())


@pytest.mark.parametrize("seed", range(16))
def test_shared_decode_of_random_shapes(seed):
    r = np.random.default_rng(4000 + seed)
    (Hq, Hkv), D, page = _heads(r), int(r.choice([64, 128])), int(r.choice([16, 32, 64, 128]))
    groups = [(int(int(r.choice([1, 30, 400])) * r.random() * 16 / page), [int(200 ** r.random()) - 1 if r.random() > 0.1 else None
               for _ in range(int(r.integers(1, int(r.choice([2, 9, 40])))))]) for _ in range(int(r.integers(1, 5)))]
    if seed % 4 == 0:  # enough of it to be read once
        groups[0] = (-(-2 ** 27 // (30 * page * Hkv * D * (2 if seed % 2 else 4))) + 1, [int(x) for x in r.integers(0, 90, 32)])
    c = ta.Family(groups, Hq, Hkv, D, page, bool(seed % 2), seed=seed, q_stride=int(r.choice([0, (Hq + 2 * Hkv) * D])))
    c.check(*c.run())


@pytest.mark.parametrize("seed", range(16))
def test_forks_and_compaction_of_random_states(seed):
    r = np.random.default_rng(5000 + seed)
    R, W = int(r.integers(1, 30)), int(r.choice([1, 2, 5, 9]))
    s = tg.State(R, W, int(r.choice([0, 60, 900])), int(r.choice([1, 40, 300])), int(r.choice([16, 32, 64, 128])),
                 int(r.integers(0, 400)), seed=seed, room=int(r.integers(0, 700)), empty=float(r.choice([0, 0.3])))
    parents = [int(x) for x in r.integers(-1, R * W, int(r.integers(1, 2 * R * W + 2)))]
    while po.fork(parents, s.lens, s.table, s.extra, s.free, s.head, s.page, s.num) is None:
        parents = parents[:-1] if len(parents) > 1 else [-1]
    s.check_fork(parents, s.fork(parents, bool(seed % 2)), bool(seed % 2))
    most = int(r.integers(0, s.num + 1))
    s.check_compact(most, s.compact(most, bool(seed % 2)))
