"""Pins of the paged and norm-with-rotation oracle (CPU)."""

import math

import numpy as np
import pytest
import torch

from oracle import paged_oracle as po


def _paged(lens, Hkv, page, D, seed):
    """Caches whose used rows hold k, v of each sequence; the others NaN."""
    r = np.random.default_rng(seed)
    n = [-(-x // page) for x in lens]
    order = r.permutation(sum(n) + 2)
    table = np.full((len(lens), max(max(n), 1)), -1)
    k = np.full((sum(n) + 2, Hkv, page, D), np.nan)
    v = k.copy()
    seqs, at = [], 0
    for b, x in enumerate(lens):
        ks, vs = r.standard_normal((2, x, Hkv, D))
        for j in range(n[b]):
            table[b, j] = order[at]
            at += 1
            rows = ks[j * page:(j + 1) * page]
            k[table[b, j], :, :len(rows)] = rows.transpose(1, 0, 2)
            v[table[b, j], :, :len(rows)] = vs[j * page:(j + 1) * page].transpose(1, 0, 2)
        seqs.append((ks, vs))
    return k, v, table, seqs


@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (6, 2)])
def test_decode_is_softmax_attention_over_the_sequence(Hq, Hkv):
    lens, page, D = [5, 0, 1, 33], 16, 8
    k, v, table, seqs = _paged(lens, Hkv, page, D, 1)
    q = np.random.default_rng(2).standard_normal((4, Hq, D))
    out, lse, absv, size = po.decode(q, k, v, table, lens, 0.3)
    for b, (ks, vs) in enumerate(seqs):
        for h in range(Hq):
            if lens[b] == 0:
                assert not out[b, h].any() and lse[b, h] == -math.inf
                continue
            kt, vt = (torch.from_numpy(x[:, h // (Hq // Hkv)]) for x in (ks, vs))
            z = kt @ torch.from_numpy(q[b, h]) * 0.3
            np.testing.assert_allclose(out[b, h], torch.softmax(z, 0) @ vt, rtol=1e-12, atol=1e-13)
            np.testing.assert_allclose(lse[b, h], torch.logsumexp(z, 0), rtol=1e-13)
    # every page selected is the dense result; a part is the attention over that part
    every = np.broadcast_to(np.arange(3), (4, Hkv, 3))
    every = np.where(every < [[[-(-n // page)]] for n in lens], every, -1)
    np.testing.assert_array_equal(po.decode(q, k, v, table, lens, 0.3, every)[0], out)
    part = po.decode(q, k, v, table, lens, 0.3, np.full((4, Hkv, 1), [[[-1]], [[-1]], [[-1]], [[2]]]))
    np.testing.assert_allclose(part[0][3, 0], seqs[3][1][32, 0], rtol=1e-14)


def test_select_orders_scores_and_keeps_ends():
    page, D = 16, 4
    mean = np.zeros((6, 1, D))
    mean[:, 0, 0] = [1, 5, 5, 2, 9, 0]
    table = np.array([[5, 0, 1, 2, 3, 4]])
    q = np.zeros((1, 2, D))
    q[0, :, 0] = 1
    # logical scores: 0 2 10 10 4 18; ties go to the lower page
    assert po.select(q, mean, table, [96], page, 2, 0, 0).tolist() == [[[2, 5]]]
    assert po.select(q, mean, table, [96], page, 3, 0, 0).tolist() == [[[2, 3, 5]]]
    assert po.select(q, mean, table, [96], page, 3, 1, 0).tolist() == [[[0, 2, 5]]]
    assert po.select(q, mean, table, [80], page, 3, 1, 2).tolist() == [[[0, 3, 4]]]
    assert po.select(q, mean, table, [17], page, 3, 0, 0).tolist() == [[[0, 1, -1]]]


def test_plan_and_write_rebuild_the_sequences():
    page, Hkv, D, B, r = 16, 2, 4, 3, np.random.default_rng(3)
    table, lens, head = np.full((B, 5), -1), np.zeros(B, int), 1
    free = r.permutation(20)
    k, v = np.full((2, 20, Hkv, page, D), np.nan)
    mean = np.zeros((20, Hkv, D))
    seqs = [[] for _ in range(B)]
    for new in ([3, 0, 40], [1, 1, 1], [12, 16, 0], [1, 30, 39]):
        T = sum(new) + 2
        lens, head, table, cu, slots, positions = po.plan(new, lens, free, head, table, page, T, 20)
        x = r.standard_normal((T, Hkv, D))
        po.write(x, -x, slots, k, v, mean, lambda y: y)
        for b in range(B):
            seqs[b] += list(x[cu[b]:cu[b + 1]])
            assert positions[cu[b]:cu[b + 1]].tolist() == list(range(lens[b] - new[b], lens[b]))
    for b in range(B):
        got = [k[table[b, t // page], :, t % page] for t in range(lens[b])]
        np.testing.assert_array_equal(got, seqs[b])
        for j in range(-(-lens[b] // page)):
            want = np.mean(seqs[b][j * page:(j + 1) * page], axis=0)
            np.testing.assert_allclose(mean[table[b, j]], want, rtol=1e-12, atol=1e-14)
    # what cannot be met takes nothing
    assert po.plan([1, 0, 1], lens, free, head, table, page, 2, 20) is None  # past the table
    assert po.plan([1, 1, 0], lens, free, head, table, page, 1, 20) is None  # too many tokens
    assert po.plan([0, 9, 0], lens, free[:head], head, table, page, 9, 20) is None  # no free page


@pytest.mark.parametrize("rot,interleaved", [(0, False), (16, True), (32, False), (32, True)])
def test_norm_rope_gradients_match_differences(rot, interleaved):
    r = np.random.default_rng(rot)
    B, N, H, D = 2, 3, 2, 32
    x, dy = r.standard_normal((2, B, N, H, D))
    w = 1 + 0.3 * r.standard_normal(D)
    angle = r.uniform(-3, 3, (7, rot // 2))
    pos = r.integers(0, 7, (B, N))
    f = lambda x, w: (po.norm_rope(x, w, np.cos(angle), np.sin(angle), pos, rot, interleaved,
                                   1e-5) * dy).sum()
    dx, dw, _ = po.norm_rope_backward(dy, x, w, np.cos(angle), np.sin(angle), pos, rot, interleaved,
                                      1e-5)
    # central differences: truncation h^2 f'''/6 ~ 1e-10, rounding 1e-16 |f| / h ~ 1e-9
    h = 1e-5
    for _ in range(12):
        i = tuple(r.integers(0, n) for n in x.shape)
        e = np.zeros_like(x)
        e[i] = h
        assert abs((f(x + e, w) - f(x - e, w)) / (2 * h) - dx[i]) < 1e-7
        e = np.zeros_like(w)
        e[i[-1]] = h
        assert abs((f(x, w + e) - f(x, w - e)) / (2 * h) - dw[i[-1]]) < 1e-7


def test_norm_rope_is_a_rotation_of_the_unit_rows():
    r = np.random.default_rng(0)
    x = r.standard_normal((1, 4, 2, 64)) * 7
    angle = r.uniform(-3, 3, (4, 32))
    y = po.norm_rope(x, np.ones(64), np.cos(angle), np.sin(angle), np.arange(4)[None], 64, True, 0.0)
    np.testing.assert_allclose((y * y).mean(-1), 1, rtol=1e-12)
    z = torch.view_as_complex(torch.from_numpy(x / np.sqrt((x * x).mean(-1, keepdims=True)))
                              .reshape(1, 4, 2, 32, 2).contiguous())
    z = torch.view_as_real(z * torch.polar(torch.ones(4, 32, dtype=torch.float64),
                                           torch.from_numpy(angle))[None, :, None]).reshape(x.shape)
    np.testing.assert_allclose(y, z.numpy(), rtol=1e-12, atol=1e-13)
