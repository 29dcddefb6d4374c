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
