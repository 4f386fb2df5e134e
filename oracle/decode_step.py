"""The decoding step's operators in 64 bits, slot by slot: rotary positions,
the write of k and v into a paged cache, attention of one new token over it
and eviction from it by accumulated attention weight.

Caches are arrays [pages][kv heads][page][head size]; slot s of a cache is
token s % page of page s // page; weights and positions are [pages][kv
heads][page].  Written as loops over sequences and heads from the formulas."""
from __future__ import annotations

import math

import numpy as np


# ----------------------------------------------------------------------------
# rotary positions
# ----------------------------------------------------------------------------
def rope_frequency(i: int, rot: int, base: float, scaling: str = "plain", factor: float = 1.0,
                   original_len: float = 0.0, low: float = 1.0, high: float = 4.0) -> float:
    f = 1.0 / base ** (2 * i / rot)
    if scaling == "linear":
        return f / factor
    if scaling == "bands":
        wave = 2 * math.pi / f
        if wave < original_len / high:
            return f
        if wave > original_len / low:
            return f / factor
        t = (original_len / wave - low) / (high - low)
        return (1 - t) * f / factor + t * f
    if scaling == "yarn":
        def index(turns):
            return rot * math.log(original_len / (turns * 2 * math.pi)) / (2 * math.log(base))
        a, b = max(math.floor(index(high)), 0), min(math.ceil(index(low)), rot - 1)
        t = min(max((i - a) / max(b - a, 0.001), 0.0), 1.0)
        return f * (1 - t) + f / factor * t
    return f


def rope_table(rot, n_pos, base, attention=1.0, **scaling):
    """fp64 [n_pos][rot/2][2]."""
    f = np.array([rope_frequency(i, rot, base, **scaling) for i in range(rot // 2)])
    a = np.arange(n_pos, dtype=np.float64)[:, None] * f
    return np.stack([np.cos(a), np.sin(a)], -1) * attention


def rope(x, positions, table, layout="half", transpose=False):
    """x [T][H][D]; a position outside the table gives zeros."""
    x, table = np.asarray(x, np.float64), np.asarray(table, np.float64)
    half = table.shape[1]
    y = np.zeros_like(x)
    for t, p in enumerate(positions):
        if not 0 <= p < table.shape[0]:
            continue
        y[t] = x[t]
        for i in range(half):
            a, b = (i, i + half) if layout == "half" else (2 * i, 2 * i + 1)
            c, s = table[p, i]
            s = -s if transpose else s
            y[t, :, a] = x[t, :, a] * c - x[t, :, b] * s
            y[t, :, b] = x[t, :, b] * c + x[t, :, a] * s
    return y


# ----------------------------------------------------------------------------
# e4m3 (OCP 8-bit, no infinities): sign, 4 exponent bits of bias 7, 3 mantissa
# bits; all ones are NaN
# ----------------------------------------------------------------------------
def e4m3_values() -> np.ndarray:
    """fp64 [256] by code."""
    out = np.empty(256)
    for code in range(256):
        e, m = (code >> 3) & 15, code & 7
        v = math.nan if (e, m) == (15, 7) else (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        out[code] = -v if code >> 7 else v
    return out


def e4m3_encode(x) -> np.ndarray:
    """Codes of x clamped to +-448 and rounded to nearest, ties to the even
    code."""
    x = np.asarray(x, np.float64)
    grid = e4m3_values()[:127]                      # 0 ... 448, ascending
    a = np.minimum(np.abs(np.where(np.isnan(x), 0.0, x)), 448.0)
    up = np.searchsorted(grid, a)                   # grid[up - 1] < a <= grid[up]
    dn = np.maximum(up - 1, 0)
    du, dd = grid[up] - a, a - grid[dn]
    code = np.where(du < dd, up, np.where(dd < du, dn, np.where(up % 2 == 0, up, dn)))
    code = np.where(grid[up] == a, up, code)
    code = code + 128 * np.signbit(x)
    return np.where(np.isnan(x), 127 + 128 * np.signbit(x), code).astype(np.uint8)


# ----------------------------------------------------------------------------
# attention of one new token
# ----------------------------------------------------------------------------
def paged_attention(q, k, v, block_table, lengths, scale):
    """q [B][Hq][D], k and v [pages][Hkv][page][D] (all fp64).  Returns out
    [B][Hq][D], lse [B][Hq], added weights [pages][Hkv][page], and the terms
    error bounds are made of: per (b, head) the sum of p |v| ([B][Hq][D]) and
    the largest sum of |q_d k_d| over the slots ([B][Hq])."""
    B, Hq, D = q.shape
    pages, Hkv, page, _ = k.shape
    G = Hq // Hkv
    out, lse = np.zeros((B, Hq, D)), np.full((B, Hq), -np.inf)
    mass, dots = np.zeros((B, Hq, D)), np.zeros((B, Hq))
    weights = np.zeros((pages, Hkv, page))
    for b in range(B):
        j = np.arange(max(0, lengths[b]))
        pg = block_table[b][j // page]
        there = (pg >= 0) & (pg < pages)
        pg, off = pg[there], j[there] % page
        if not len(pg):
            continue
        for h in range(Hq):
            kk, vv = k[pg, h // G, off], v[pg, h // G, off]
            s = scale * (kk @ q[b, h])
            m = s.max()
            if m == -np.inf:
                continue
            p = np.exp(s - m)
            total = p.sum()
            out[b, h], lse[b, h] = (p @ vv) / total, m + np.log(total)
            mass[b, h], dots[b, h] = (p @ np.abs(vv)) / total, (np.abs(kk) @ np.abs(q[b, h])).max()
            weights[pg, h // G, off] += p / total
    return out, lse, weights, mass, dots


# ----------------------------------------------------------------------------
# eviction
# ----------------------------------------------------------------------------
def cache_evict(k, v, weights, positions, block_table, lengths, budget, recent):
    """New (k, v, weights, positions, lengths); the inputs stay as they are.
    Slots of a sequence are looked at one by one."""
    k, v, weights, positions = k.copy(), v.copy(), weights.copy(), positions.copy()
    pages, Hkv, page = weights.shape
    new = np.array([max(0, n) for n in lengths], np.int32)
    for b, n in enumerate(new.tolist()):
        pg = block_table[b][: -(-n // page)]
        if n <= budget or ((pg < 0) | (pg >= pages)).any():
            continue
        new[b] = budget
        slot = [(int(pg[j // page]), j % page) for j in range(n)]
        for h in range(Hkv):
            w = [float(weights[p, h, o]) for p, o in slot]
            pos = [int(positions[p, h, o]) for p, o in slot]
            newest = max(pos)

            def order(j):
                if pos[j] > newest - recent:
                    return (0, 0.0, j)
                return (2, 0.0, j) if math.isnan(w[j]) else (1, -w[j], j)

            kept = set(sorted(range(n), key=order)[:budget])
            holes = [j for j in range(budget) if j not in kept]
            fills = [j for j in range(budget, n) if j in kept]
            for d, s in zip(holes, fills):
                (dp, do), (sp, so) = slot[d], slot[s]
                k[dp, h, do], v[dp, h, do] = k[sp, h, so], v[sp, h, so]
                weights[dp, h, do], positions[dp, h, do] = w[s], pos[s]
            for j in range(budget, n):
                weights[slot[j][0], h, slot[j][1]], positions[slot[j][0], h, slot[j][1]] = 0.0, -1
    return k, v, weights, positions, new
