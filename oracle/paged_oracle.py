"""Plain fp64 definitions of the paged-cache and norm-with-rotation operators.

Loops over sequences, heads and pages with numpy; used by the tests only.
E4M3 caches are given as codes and decoded with the same functions as the
token-sparse path's oracle.
"""

from __future__ import annotations

import math

import numpy as np


def plan(new, lens, free, head, table, page, T, num_pages):
    """(lens_out, head_out, table, cu_new, slots, positions), or None for a request that
    cannot be met."""
    B, max_pages = table.shape
    table = table.copy()
    cu, slots, positions = [0], np.full(T, -1), np.full(T, -1)
    for b in range(B):
        old, n = int(lens[b]), int(new[b])
        if old < 0 or n < 0 or old + n > max_pages * page or cu[-1] + n > T:
            return None
        if n and old % page and not 0 <= table[b, old // page] < num_pages:
            return None
        for pos in range(old, old + n):
            if pos % page == 0:
                if not 0 <= head < len(free) or not 0 <= free[head] < num_pages:
                    return None
                table[b, pos // page] = free[head]
                head += 1
            t = cu[-1] + pos - old
            slots[t] = table[b, pos // page] * page + pos % page
            positions[t] = pos
        cu.append(cu[-1] + n)
    return np.asarray(lens) + np.asarray(new), head, table, np.array(cu), slots, positions


def write(k, v, slots, k_cache, v_cache, k_mean, values):
    """Stores the rows (already in the caches' type) and takes the means of the touched
    pages; values(x) gives what stored keys stand for, in fp64."""
    page = k_cache.shape[2]
    held = {}
    for t, s in enumerate(slots):
        if s >= 0:
            k_cache[s // page, :, s % page] = k[t]
            v_cache[s // page, :, s % page] = v[t]
            held[s // page] = max(held.get(s // page, 0), s % page + 1)
    if k_mean is not None:
        for p, n in held.items():
            k_mean[p] = values(k_cache[p, :, :n]).mean(1)
    return held


def select(q, k_mean, table, lens, page, keep, sink, recent):
    """sel [B, Hkv, keep] (-1 behind): q [B, Hq, D], k_mean [pages, Hkv, D] in fp64."""
    B, Hkv = len(lens), k_mean.shape[1]
    group = q.shape[1] // Hkv
    sel = np.full((B, Hkv, keep), -1)
    for b in range(B):
        n = -(-int(lens[b]) // page)
        for h in range(Hkv):
            qs = q[b, h * group:(h + 1) * group].sum(0)
            score = [np.float32(qs @ k_mean[table[b, j], h]) for j in range(n)]
            best = sorted(range(n), key=lambda j: (not (j < sink or j >= n - recent), -score[j], j))
            kept = sorted(best[:keep])
            sel[b, h, :len(kept)] = kept
    return sel


def decode(q, k_cache, v_cache, table, lens, scale, sel=None):
    """Attention of one token per sequence, caches in fp64 [pages, Hkv, page, D].

    Returns out [B, Hq, D], lse [B, Hq], and what the error bounds need: the
    mean of |v| under the weights [B, Hq, D] and the largest sum of |q k| scale
    [B, Hq]."""
    B, Hq, D = q.shape
    Hkv, page = k_cache.shape[1:3]
    group = Hq // Hkv
    out, absv = np.zeros((B, Hq, D)), np.zeros((B, Hq, D))
    lse, size = np.full((B, Hq), -math.inf), np.zeros((B, Hq))
    for b in range(B):
        n = int(lens[b])
        for h in range(Hkv):
            pages = range(-(-n // page)) if sel is None else [j for j in sel[b, h] if j >= 0]
            rows = [(table[b, j], r) for j in pages for r in range(page) if j * page + r < n]
            if not rows:
                continue
            at = np.array(rows)
            k, v = k_cache[at[:, 0], h, at[:, 1]], v_cache[at[:, 0], h, at[:, 1]]
            for i in range(h * group, (h + 1) * group):
                z = k @ q[b, i] * scale
                e = np.exp(z - z.max())
                out[b, i] = e @ v / e.sum()
                absv[b, i] = e @ np.abs(v) / e.sum()
                lse[b, i] = z.max() + math.log(e.sum())
                size[b, i] = (np.abs(k) @ np.abs(q[b, i])).max() * scale
    return out, lse, absv, size


def attn(q, k_cache, v_cache, table, lens, cu, scale, num_pages=None):
    """Causal attention of the last cu[b + 1] - cu[b] tokens of each sequence, caches in fp64.

    Returns out [T, Hq, D], lse [T, Hq] (NaN in rows that are no sequence's), the mean of |v| under
    the weights and the largest sum of |q k| scale, as decode() does.  Pages outside
    [0, num_pages) are skipped."""
    T, Hq, D = q.shape
    Hkv, page = k_cache.shape[1:3]
    num_pages = num_pages or k_cache.shape[0]
    group = Hq // Hkv
    out, absv = np.full((T, Hq, D), np.nan), np.zeros((T, Hq, D))
    lse, size = np.full((T, Hq), np.nan), np.zeros((T, Hq))
    for b in range(len(lens)):
        n, new = int(lens[b]), int(cu[b + 1] - cu[b])
        if new <= 0:
            continue
        rows = [(j * page + r, table[b, j], r) for j in range(-(-n // page)) for r in range(page)
                if j * page + r < n and 0 <= table[b, j] < num_pages]
        at = np.array(rows, int).reshape(-1, 3)
        for h in range(Hkv):
            k, v = k_cache[at[:, 1], h, at[:, 2]], v_cache[at[:, 1], h, at[:, 2]]
            for t in range(new):
                sees = at[:, 0] <= n - new + t
                ks, vs, r, hs = k[sees], v[sees], int(cu[b]) + t, slice(h * group, (h + 1) * group)
                if not len(ks):
                    out[r, hs], lse[r, hs] = 0, -math.inf
                    continue
                z = q[r, hs] @ ks.T * scale
                top = z.max(1, keepdims=True)
                e = np.exp(z - top)
                total = e.sum(1, keepdims=True)
                out[r, hs], absv[r, hs] = e @ vs / total, e @ np.abs(vs) / total
                lse[r, hs] = (top + np.log(total))[:, 0]
                size[r, hs] = (np.abs(q[r, hs]) @ np.abs(ks).T).max(1) * scale
    return out, lse, absv, size


def fork(parents, lens, table, extra, free, head, page, num_pages):
    """(lens, table, extra, free list from its head on, head, moves) of the new sequences, or None
    for a request that cannot be met.  Walks over the old sequences' pages with a dictionary of
    holders."""
    B, P = table.shape
    if any(not 0 <= n <= P * page for n in lens) or any(not -1 <= p < B for p in parents) or min(extra) < 0:
        return None
    holders = {}
    for b in range(B):
        for j in range(-(-int(lens[b]) // page)):
            if not 0 <= table[b, j] < num_pages:
                return None
            holders[int(table[b, j])] = int(extra[table[b, j]]) + 1
    before = dict(holders)
    if not 0 <= head <= len(free):
        return None
    n = len(parents)
    lens_out, table_out, moves = np.zeros(n, int), np.full((n, P), -1), np.tile([-1, -1, 0], (n, 1))
    for b in range(B):  # the old sequences let go
        for j in range(-(-int(lens[b]) // page)):
            holders[int(table[b, j])] -= 1
    kept, taken = set(), []
    for i, p in enumerate(parents):
        if p < 0:
            continue
        lens_out[i] = lens[p]
        for j in range(-(-int(lens[p]) // page)):
            pid = int(table[p, j])
            if (j + 1) * page > lens[p] and (p in kept or before[pid] > 1):  # an open page that is not the child's to keep
                at = head + len(taken)
                if at >= len(free) or not 0 <= free[at] < num_pages:
                    return None
                moves[i] = pid, free[at], lens[p] % page
                taken.append(int(free[at]))
                table_out[i, j] = free[at]
            else:
                table_out[i, j] = pid
                holders[pid] += 1
        kept.add(p)
    if any(h < 0 for h in holders.values()):
        return None
    freed = sorted(pid for pid, h in holders.items() if h == 0 and before[pid] > 0)
    head_out = head + len(taken) - len(freed)
    if head_out < 0:
        return None
    extra_out = np.array(extra)
    for pid, h in holders.items():
        extra_out[pid] = max(h - 1, 0)
    return lens_out, table_out, extra_out, freed + [int(x) for x in free[head + len(taken):]], head_out, moves


def compact(lens, table, extra, n_free, most, page, num_pages):
    """(table, extra, free list from its head on, head, moves), or None."""
    B, P = table.shape
    if any(not 0 <= n <= P * page for n in lens):
        return None
    fill = {}
    for b in range(B):
        for j in range(-(-int(lens[b]) // page)):
            if not 0 <= table[b, j] < num_pages:
                return None
            fill[int(table[b, j])] = max(fill.get(int(table[b, j]), 0), min(page, int(lens[b]) - j * page))
    holes = [p for p in range(num_pages) if p not in fill]
    if n_free < len(holes):
        return None
    to = {p: p for p in fill}
    moves = np.tile([-1, -1, 0], (most, 1))
    for i, (src, dst) in enumerate(zip(sorted(fill, reverse=True), holes)):
        if i < most and src > dst:
            to[src], moves[i] = dst, (src, dst, fill[src])
    table_out, extra_out = table.copy(), np.zeros(num_pages, int)
    for b in range(B):
        for j in range(-(-int(lens[b]) // page)):
            table_out[b, j] = to[int(table[b, j])]
    for src, dst in to.items():
        extra_out[dst] = extra[src]
    free = [p for p in range(num_pages) if p not in to.values()]
    return table_out, extra_out, free, n_free - len(free), moves


def copy(moves, k_cache, v_cache, k_mean):
    for src, dst, rows in moves:
        if src >= 0:
            k_cache[dst, :, :rows], v_cache[dst, :, :rows] = k_cache[src, :, :rows].copy(), v_cache[src, :, :rows].copy()
            if k_mean is not None:
                k_mean[dst] = k_mean[src]


def _pairs(D, rot, interleaved):
    one = np.arange(0, rot, 2) if interleaved else np.arange(rot // 2)
    return one, one + (1 if interleaved else rot // 2)


def norm_rope(x, w, cos, sin, positions, rot, interleaved, eps):
    """y [B, N, H, D] from x [B, N, H, D], w [D], tables [rows, rot/2], positions [B, N]."""
    D = x.shape[-1]
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    a, b = _pairs(D, rot, interleaved)
    c, s = cos[positions][:, :, None], sin[positions][:, :, None]
    z = y.copy()
    z[..., a] = y[..., a] * c - y[..., b] * s
    z[..., b] = y[..., b] * c + y[..., a] * s
    return z


def norm_rope_backward(dy, x, w, cos, sin, positions, rot, interleaved, eps):
    """(dx, dw, sum |g xh|): the last is what the error bound of dw needs."""
    D = x.shape[-1]
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    a, b = _pairs(D, rot, interleaved)
    c, s = cos[positions][:, :, None], sin[positions][:, :, None]
    g = dy.copy()
    g[..., a] = dy[..., a] * c + dy[..., b] * s
    g[..., b] = dy[..., b] * c - dy[..., a] * s
    xh = x * r
    wg = w * g
    dx = r * (wg - xh * (wg * xh).mean(-1, keepdims=True))
    return dx, (g * xh).sum((0, 1, 2)), np.abs(g * xh).sum((0, 1, 2))
