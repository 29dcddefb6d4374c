"""GPU parity of forks, compaction and page copies with the oracle: whole numbers and copied bytes,
equal."""

import numpy as np
import pytest
import torch

from oracle import paged_oracle as po
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


class State:
    """Requests of W sequences that hold their prompt's full pages together, pages in random order, free
    ones among them; table entries past a sequence's end are anything."""

    def __init__(self, R, W, prompt, own, page, spare, seed=0, room=3, empty=0.1):
        r = np.random.default_rng(seed)
        lens, rows, extra, at = [], [], {}, 0
        for _ in range(R):
            p = int(r.integers(0, prompt + 1))
            shared = list(range(at, at + p // page))
            at += len(shared)
            live = []
            for _ in range(W):
                n = 0 if r.random() < empty else p // page * page + int(r.integers(0, own + 1))
                row = shared[:-(-n // page)] if n else []
                if row or n:
                    live.append(n)
                extra_pages = -(-n // page) - len(row)
                row = row + list(range(at, at + extra_pages))
                at += extra_pages
                lens.append(n)
                rows.append(row)
            for x in shared:
                extra[x] = sum(n > 0 for n in lens[-W:]) - 1
        self.page, self.num, P = page, at + spare, max([1] + [len(x) for x in rows]) + room
        order = r.permutation(self.num)
        self.lens, self.table = np.array(lens), r.integers(-5, 2 * self.num, (R * W, P))
        for b, row in enumerate(rows):
            self.table[b, :len(row)] = order[row]
        self.extra = np.zeros(self.num, int)
        for x, n in extra.items():
            self.extra[order[x]] = max(n, 0)
        held = {int(x) for b, row in enumerate(rows) for x in self.table[b, :len(row)]}
        free = [x for x in r.permutation(self.num) if x not in held]
        self.head = self.num - len(free)
        self.free = np.array([-9] * self.head + free)
        self.p = mcs.paged(R * W, 2, 1, 64, page, self.num, P)
        self.r, self.R, self.W = r, R, W

    def fork(self, parents, in_place=False, stream=None):
        n, d = len(parents), {k: _i32(getattr(self, k)) for k in ("lens", "table", "extra", "free")}
        head = _i32([self.head])
        new = lambda x, s: x if in_place else torch.full(s, -77, dtype=torch.int32, device="cuda")
        lens, table, moves = (torch.full(s, -77, dtype=torch.int32, device="cuda") for s in ((n,), (n, self.p.max_pages), (n, 3)))
        extra, free, head_out = new(d["extra"], (self.num,)), new(d["free"], (len(self.free),)), new(head, (1,))
        ws = mcs.empty_workspace(mcs.mcs_paged_fork_workspace(self.p)).fill_(0xA5)
        mcs.mcs_paged_fork(self.p, _i32(parents), d["lens"], d["table"], d["extra"], d["free"], head, lens, table, extra, free,
                           head_out, moves, ws, stream=stream)
        return [x.cpu().numpy() for x in (lens, table, extra, free, head_out, moves)]

    def check_fork(self, parents, got, in_place):
        want = po.fork(parents, self.lens, self.table, self.extra, self.free, self.head, self.page, self.num)
        assert want is not None
        for i in (0, 1, 2, 5):
            np.testing.assert_array_equal(got[i], want[i])
        assert got[4].tolist() == [want[4]]
        np.testing.assert_array_equal(got[3][want[4]:], want[3])
        # in front of the head nothing is touched
        np.testing.assert_array_equal(got[3][:want[4]], self.free[:want[4]] if in_place else -77)

    def compact(self, most, in_place=False, n_free=None):
        d = {k: _i32(getattr(self, k)) for k in ("lens", "table", "extra")}
        new = lambda x: x if in_place else torch.full_like(x, -77)
        table, extra = new(d["table"]), new(d["extra"])
        free = torch.full((self.num if n_free is None else n_free,), -77, dtype=torch.int32, device="cuda")
        head, moves = _i32([-77]), torch.full((most, 3), -77, dtype=torch.int32, device="cuda")
        ws = mcs.empty_workspace(mcs.mcs_paged_compact_workspace(self.p)).fill_(0xA5)
        mcs.mcs_paged_compact(self.p, d["lens"], d["table"], d["extra"], table, extra, free, head, moves, ws)
        return [x.cpu().numpy() for x in (table, extra, free, head, moves)]

    def check_compact(self, most, got, n_free=None):
        want = po.compact(self.lens, self.table, self.extra, self.num if n_free is None else n_free, most, self.page, self.num)
        for i in (0, 1, 4):
            np.testing.assert_array_equal(got[i], want[i])
        assert got[3].tolist() == [want[3]]
        np.testing.assert_array_equal(got[2][want[3]:], want[2])
        assert (got[2][:want[3]] == -77).all()


STATES = [  # R, W, prompt, own, page, spare
    (1, 1, 0, 1, 16, 3), (1, 1, 100, 60, 16, 70), (3, 4, 200, 90, 16, 60), (40, 1, 0, 400, 32, 50), (1, 64, 3000, 40, 64, 200),
    (16, 8, 2000, 200, 16, 300), (700, 2, 60, 40, 16, 5000), (4, 2, 90000, 500, 128, 30), (4096, 1, 0, 40, 16, 9000), (2, 3, 0, 0, 16, 2)]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("R,W,prompt,own,page,spare", STATES)
def test_fork_matches_oracle(R, W, prompt, own, page, spare, in_place):
    s = State(R, W, prompt, own, page, spare, seed=R + W)
    r, B = s.r, R * W
    reorder = [int(r.integers(b // W * W, b // W * W + W)) for b in range(B)]
    ended = [b if r.random() < 0.7 else -1 for b in range(B)]
    more = [int(x) for x in r.integers(-1, B, min(4096, B // 2 + 20))]
    for parents in (list(range(B)), reorder, ended, more, [-1] * 3, [B - 1]):
        if po.fork(parents, s.lens, s.table, s.extra, s.free, s.head, page, s.num) is None:
            parents = parents[:spare]  # as many fresh pages as there are
        s.check_fork(parents, s.fork(parents, in_place), in_place)
    assert mcs.mcs_device_status() == 0


def test_fork_copies_an_open_page_that_others_hold():
    # two sequences hold the same open page, as no call of the library leaves them
    s = State(1, 2, 40, 0, 16, 6, empty=0)
    s.lens[:] = 40
    s.table[:, :3] = s.table[0, :3]
    s.table[0, 2] = s.table[1, 2] = s.free[-1]
    s.extra[:] = 0
    s.extra[s.table[0, :3]] = 1
    s.free, s.head = np.concatenate([[-9], s.free[:-1]]), s.head + 1  # a page less is free
    for parents in ([0, 1], [0, 0, 1], [1], [-1]):
        s.check_fork(parents, s.fork(parents), False)


@pytest.mark.parametrize("what", ["parent", "parent below", "pages", "length", "negative", "page", "page below", "free page", "head",
                                  "holders", "no room"])
def test_fork_refuses_and_takes_nothing(what):
    s = State(3, 2, 100, 90, 16, 9, seed=5, empty=0)
    s.lens[0] += s.lens[0] % 16 == 0
    parents = [0, 0, 2, 3, 4, 5]
    if what.startswith("parent"):
        parents[3] = 6 if what == "parent" else -2
    elif what == "pages":
        s.free, s.head = s.free[:s.head], s.head
    elif what == "length":
        s.lens[1] = s.p.max_pages * 16 + 1
    elif what == "negative":
        s.lens[1] = -1
    elif what.startswith("page"):
        s.table[2, 1] = s.num if what == "page" else -1
    elif what == "free page":
        s.free[s.head] = s.num
    elif what == "head":
        s.head = len(s.free) + 1
    elif what == "holders":
        b = next(b for b in range(6) if s.lens[b] > 32)
        s.extra[s.table[b, 0]], parents = -3, [-1]
    elif what == "no room":
        s.free, s.head, parents = s.free[s.head:], 0, [-1]
    for in_place in (False, True):
        lens, table, extra, free, head, moves = s.fork(parents, in_place)
        assert mcs.mcs_device_status() == 6
        assert (lens == -77).all() and (table == -77).all() and (moves == [-1, -1, 0]).all()
        if in_place:
            assert (extra == s.extra).all() and (free == s.free).all() and head.tolist() == [s.head]
        else:
            assert (extra == -77).all() and (free == -77).all() and (head == -77).all()


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("R,W,prompt,own,page,spare", STATES)
def test_compact_matches_oracle(R, W, prompt, own, page, spare, in_place):
    s = State(R, W, prompt, own, page, spare, seed=R + 3 * W)
    for most in (0, 1, 7, s.num // 2 + 1):
        s.check_compact(most, s.compact(most, in_place))
    holes = s.num - len({int(s.table[b, j]) for b in range(R * W) for j in range(-(-int(s.lens[b]) // page))})
    s.check_compact(5, s.compact(5, in_place, holes + 2), holes + 2)
    s.check_compact(5, s.compact(5, in_place, holes), holes)
    assert mcs.mcs_device_status() == 0
    if holes:
        table, extra, free, head, moves = s.compact(5, in_place, holes - 1)
        assert mcs.mcs_device_status() == 6
        assert (moves == [-1, -1, 0]).all() and (free == -77).all() and (head == -77).all()
        assert (table == (s.table if in_place else -77)).all() and (extra == (s.extra if in_place else -77)).all()


@pytest.mark.parametrize("what", ["length", "negative", "page", "page below"])
def test_compact_refuses_and_changes_nothing(what):
    s = State(3, 2, 100, 90, 16, 9, seed=5, empty=0)
    if what == "length":
        s.lens[1] = s.p.max_pages * 16 + 1
    elif what == "negative":
        s.lens[1] = -1
    else:
        s.table[2, 1] = s.num if what == "page" else -1
    table, extra, free, head, moves = s.compact(4, True)
    assert mcs.mcs_device_status() == 6
    assert (moves == [-1, -1, 0]).all() and (free == -77).all() and (head == -77).all()
    assert (table == s.table).all() and (extra == s.extra).all()


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("Hkv,D,page,num,n", [(1, 64, 16, 9, 2), (8, 128, 64, 60, 20), (3, 128, 128, 20, 10), (5, 64, 32, 900, 400),
                                            (17, 128, 16, 40, 20), (2, 64, 16, 3000, 1500)])
def test_copy_matches_oracle(Hkv, D, page, num, n, e4m3):
    r = np.random.default_rng(num)
    order = r.permutation(num)
    moves = np.stack([order[:n], order[n:2 * n], r.integers(0, page + 1, n)], 1)
    moves[r.random(n) < 0.3] = -1, -1, 0
    moves[0] = order[0], order[n], page
    g = torch.Generator(device="cuda").manual_seed(num)
    k, v = (torch.randint(-2 ** 15, 2 ** 15, (num, Hkv, page, D // (2 if e4m3 else 1)), generator=g, device="cuda").to(torch.int16)
            for _ in range(2))
    mean = torch.randint(-2 ** 15, 2 ** 15, (num, Hkv, D), generator=g, device="cuda").to(torch.int16)
    want = [x.cpu().numpy().copy() for x in (k, v, mean)]
    po.copy(moves, *want)
    p = mcs.paged(1, Hkv, Hkv, D, page, num, 1, kv=int(e4m3))
    kind = torch.uint8 if e4m3 else torch.bfloat16
    keep = mean.clone()
    mcs.mcs_paged_copy(p, _i32(moves), k.view(kind), v.view(kind))
    assert torch.equal(mean, keep)
    mcs.mcs_paged_copy(p, _i32(moves), k.view(kind), v.view(kind), mean.view(torch.bfloat16))
    assert mcs.mcs_device_status() == 0
    for got, x in zip((k, v, mean), want):
        np.testing.assert_array_equal(got.cpu().numpy(), x)


def test_copy_reports_and_skips_what_lies_outside():
    p = mcs.paged(1, 1, 1, 64, 16, 4, 1)
    k, v = (torch.arange(4 * 16 * 64, device="cuda").view(4, 1, 16, 64).to(torch.bfloat16) for _ in range(2))
    before = k.clone()
    for bad in ([4, 1, 3], [0, 4, 3], [0, -1, 3], [0, 1, 17], [0, 1, -1]):
        mcs.mcs_paged_copy(p, _i32([bad, [-1, -1, 0]]), k, v)
        assert mcs.mcs_device_status() == 6
        assert torch.equal(k, before) and torch.equal(v, before)
    mcs.mcs_paged_copy(p, _i32(np.zeros((0, 3))), k, v)
    assert mcs.mcs_device_status() == 0
