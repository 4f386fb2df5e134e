"""Norms of heads with rotary positions of several axes, attention of several
new tokens per sequence over a paged cache, and the cut of the cache to the
drafted tokens that were kept, in 64 bits and written as loops from the
formulas.  Arrays and caches as in oracle.decode_step."""
from __future__ import annotations

import numpy as np


# ----------------------------------------------------------------------------
# norms and rotations
# ----------------------------------------------------------------------------
def axis_of(pair: int, sections) -> int:
    end = 0
    for a, n in enumerate(sections):
        end += n
        if pair < end:
            return a
    raise IndexError(pair)


def _angles(positions, sections, table, t):
    """(cos, sin) of every pair of token t, or None where it is padding."""
    positions = np.asarray(positions)
    at = [int(positions[a, t]) for a in range(len(sections))]
    if any(not 0 <= p < table.shape[0] for p in at):
        return None
    return np.array([table[at[axis_of(i, sections)], i] for i in range(table.shape[1])])


def _turned(x, cs, layout, sign=1.0):
    """x [H][D] with its pairs turned by cs [pairs][2]."""
    y, half = x.copy(), len(cs)
    for i, (c, s) in enumerate(cs):
        a, b = (i, i + half) if layout == "half" else (2 * i, 2 * i + 1)
        y[:, a], y[:, b] = x[:, a] * c - sign * s * x[:, b], x[:, b] * c + sign * s * x[:, a]
    return y


def rope_axes(x, positions, sections, table, layout="half", transpose=False):
    """x [T][H][D], positions [axes][T]."""
    x, table = np.asarray(x, np.float64), np.asarray(table, np.float64)
    y = np.zeros_like(x)
    for t in range(x.shape[0]):
        cs = _angles(positions, sections, table, t)
        if cs is not None:
            y[t] = _turned(x[t], cs, layout, -1.0 if transpose else 1.0)
    return y


def norm_rope(x, weight, eps, positions, sections, table, layout="half"):
    x = np.asarray(x, np.float64)
    w = np.ones(x.shape[2]) if weight is None else np.asarray(weight, np.float64)
    normed = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    return rope_axes(normed, positions, sections, table, layout)


def norm_rope_grad(x, dy, weight, eps, positions, sections, table, layout="half"):
    """(dx, dweight, and the sum of |terms| of each element of dweight)."""
    x, dy = np.asarray(x, np.float64), np.asarray(dy, np.float64)
    w = np.ones(x.shape[2]) if weight is None else np.asarray(weight, np.float64)
    g = rope_axes(dy, positions, sections, table, layout, True)
    dx, dw, mass = np.zeros_like(x), np.zeros(x.shape[2]), np.zeros(x.shape[2])
    for t in range(x.shape[0]):
        for h in range(x.shape[1]):
            r = 1.0 / np.sqrt((x[t, h] ** 2).mean() + eps)
            u = x[t, h] * r
            dw += g[t, h] * u
            mass += np.abs(g[t, h] * u)
            gw = g[t, h] * w
            dx[t, h] = r * (gw - u * (gw * u).mean())
    padding = [_angles(positions, sections, np.asarray(table, np.float64), t) is None for t in range(x.shape[0])]
    dx[padding] = 0.0
    return dx, dw, mass


# ----------------------------------------------------------------------------
# attention of several new tokens
# ----------------------------------------------------------------------------
def seen_and_distance(n, length, i, first=0, prefix=0, window=0, tree=None):
    """For the i-th of n new tokens of a sequence of `length` slots: which
    slots it sees (bool [length]) and how far they are.  tree: the bits of its
    row, bool [n], or None."""
    ctx, slot = length - n, ctx_slot(length, n, i)
    seen, far = np.zeros(length, bool), np.zeros(length)
    for j in range(length):
        if tree is None:
            seen[j] = j <= slot or j < prefix
            far[j] = abs(slot - j)
        elif j >= ctx:
            seen[j] = tree[j - ctx]
            far[j] = sum(bool(tree[x]) for x in range(j - ctx + 1, n))
        else:
            seen[j] = True
            far[j] = ctx - 1 - j + sum(bool(b) for b in tree)
        if j < first or (window and far[j] >= window):
            seen[j] = False
    return seen, far


def ctx_slot(length, n, i):
    return length - n + i


def attention_tokens(q, k, v, starts, block_table, lengths, scale, softcap=0.0, slopes=None, window=0, first=None,
                     prefix=None, tree=None):
    """q [T][Hq][D], k and v [pages][Hkv][page][D] (fp64), tree bool [T][bits].
    Returns out, lse (NaN for tokens outside all sequences), and the terms that
    error bounds are made of: sum of p |v|, and per row the largest error unit
    of a score's parts: sum |q_d k_d| |scale|, |score| and slope * distance."""
    T, Hq, D = q.shape
    pages, Hkv, page, _ = k.shape
    G = Hq // Hkv
    out, lse = np.full((T, Hq, D), np.nan), np.full((T, Hq), np.nan)
    mass, parts = np.zeros((T, Hq, D)), np.zeros((3, T, Hq))
    for b, length in enumerate(lengths):
        n = starts[b + 1] - starts[b]
        for i in range(n):
            t = starts[b] + i
            bits = None
            if tree is not None:
                bits = np.zeros(n, bool)
                m = min(n, tree.shape[1])
                bits[:m] = tree[t, :m]
            seen, far = seen_and_distance(n, length, i, 0 if first is None else first[t],
                                          0 if prefix is None else prefix[b], window, bits)
            j = np.flatnonzero(seen)
            pg = block_table[b][j // page].astype(np.int64)
            there = (pg >= 0) & (pg < pages)
            j, pg = j[there], pg[there]
            out[t], lse[t] = 0.0, -np.inf
            if not len(j):
                continue
            for h in range(Hq):
                kk, vv = k[pg, h // G, j % page], v[pg, h // G, j % page]
                s = scale * (kk @ q[t, h])
                parts[0, t, h] = (np.abs(kk) @ np.abs(q[t, h])).max() * abs(scale)
                if softcap:
                    s = softcap * np.tanh(s / softcap)
                if slopes is not None:
                    s = s - slopes[h] * far[j]
                    parts[2, t, h] = np.abs(slopes[h] * far[j]).max()
                parts[1, t, h] = np.abs(s).max()
                m = s.max()
                if m == -np.inf:
                    continue
                p = np.exp(s - m)
                total = p.sum()
                out[t, h], lse[t, h] = (p @ vv) / total, m + np.log(total)
                mass[t, h] = (p @ np.abs(vv)) / total
    return out, lse, mass, parts


# ----------------------------------------------------------------------------
# keeping drafted tokens
# ----------------------------------------------------------------------------
def cache_keep(arrays, block_table, lengths, drafted, kept, counts, num_pages, page):
    """New (arrays, lengths): arrays are [pages][kv heads][page]... each."""
    arrays = [None if x is None else x.copy() for x in arrays]
    new = list(lengths)
    for b, length in enumerate(lengths):
        n, count = drafted[b], counts[b]
        if not (0 <= n <= length <= block_table.shape[1] * page and 0 <= count <= min(n, kept.shape[1])):
            continue
        rows = [int(x) for x in kept[b, :count]]
        if any(not 0 <= x < n for x in rows) or any(a >= c for a, c in zip(rows, rows[1:])):
            continue
        slots = [length - n + x for x in rows] + [length - n + i for i in range(count)]
        pg = [int(block_table[b, s // page]) for s in slots]
        if any(not 0 <= p < num_pages for p in pg):
            continue
        new[b] = length - n + count
        for x in arrays:
            if x is None:
                continue
            taken = [x[pg[i], :, slots[i] % page].copy() for i in range(count)]
            for i in range(count):
                x[pg[count + i], :, slots[count + i] % page] = taken[i]
    return arrays, new
