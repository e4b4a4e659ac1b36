"""The paged-cache operators in fp64, written out row by row - TEST
INFRASTRUCTURE (used by the tests only; the product never imports it).

Definitions (include/msa.h, section "Serving: a paged key-value cache").
Caches are float64 arrays [pages, page_size, heads, dim]; token j of row r is
cache[table[r, j // page_size], j % page_size].  All arguments are numpy
arrays (or ints), all results float64.
"""
from __future__ import annotations

import numpy as np

BLOCK, SLOTS = 128, 16


def gather(cache, table_row, lo: int, hi: int) -> np.ndarray:
    """Tokens lo .. hi-1 of a row, [hi - lo, heads, dim]."""
    j = np.arange(lo, hi)
    return cache[np.asarray(table_row)[j // cache.shape[1]], j % cache.shape[1]]


def rotate(x, pos, inv_freq, interleaved: bool) -> np.ndarray:
    """x [n, heads, dim] at positions pos [n]: pair i turns by pos * inv_freq[i]."""
    y = np.array(x, dtype=np.float64)
    half = len(inv_freq)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        angle = np.asarray(pos, dtype=np.float64)[:, None] * float(inv_freq[i])
        c, s = np.cos(angle), np.sin(angle)
        u, v = np.array(x[..., a], np.float64), np.array(x[..., b], np.float64)
        y[..., a], y[..., b] = u * c - v * s, v * c + u * s
    return y


def append(k_cache, v_cache, k, v, table, offs, start, inv_freq=None, interleaved=False, q=None):
    """(k_cache, v_cache, q_rot, k_rot) after the call; rows of q_rot and k_rot
    that no row owns are NaN (not written)."""
    kc, vc = k_cache.copy(), v_cache.copy()
    S = kc.shape[1]
    freq = [] if inv_freq is None else inv_freq
    k_rot = np.full(k.shape, np.nan)
    q_rot = None if q is None else np.full(q.shape, np.nan)
    for r in range(len(start)):
        for t in range(offs[r], offs[r + 1]):
            p = int(start[r]) + t - int(offs[r])
            k_rot[t] = rotate(k[t:t + 1], [p], freq, interleaved)[0]
            if q is not None:
                q_rot[t] = rotate(q[t:t + 1], [p], freq, interleaved)[0]
            kc[table[r, p // S], p % S] = k_rot[t]
            vc[table[r, p // S], p % S] = v[t]
    return kc, vc, q_rot, k_rot


def mean_slot(page: int, last: int, S: int) -> int:
    """Where the mean of the block whose last key is at position ``last`` is kept."""
    return page if S <= BLOCK else page * (S // BLOCK) + last % S // BLOCK


def index(keys, means, ik, table, offs, start):
    """(keys, means) after the call."""
    keys, means = keys.copy(), means.copy()
    S = keys.shape[1]
    for r in range(len(start)):
        p0, p1 = int(start[r]), int(start[r]) + int(offs[r + 1]) - int(offs[r])
        for p in range(p0, p1):
            keys[table[r, p // S], p % S] = ik[offs[r] + p - p0]
        if p1 == p0:
            continue
        for b in range(p0 // BLOCK, (p1 - 1) // BLOCK + 1):
            end = min(b * BLOCK + BLOCK, p1)
            at = mean_slot(table[r, (end - 1) // S], end - 1, S)
            means[at] = gather(keys, table[r], b * BLOCK, end).mean(0)
    return keys, means


def visible(n: int, slots=None) -> np.ndarray:
    """Positions that a row of n keys sees: all, or those in the slots' blocks."""
    j = np.arange(n)
    return j if slots is None else j[np.isin(j // BLOCK, [int(x) for x in slots if x != -1])]


def decode(k_cache, v_cache, q, table, lens, scale, q2k=None):
    """(O [rows, heads, dim], LSE [rows, heads])."""
    rows, heads, dim = q.shape
    kv = k_cache.shape[2]
    share = heads // kv
    O = np.zeros((rows, heads, dim))
    L = np.full((rows, heads), -np.inf)
    for r in range(rows):
        n = int(lens[r])
        if n == 0:
            continue
        K, V = gather(k_cache, table[r], 0, n), gather(v_cache, table[r], 0, n)
        for g in range(kv):
            j = visible(n, None if q2k is None else q2k[g, r])
            if j.size == 0:
                continue
            h = slice(g * share, (g + 1) * share)
            s = scale * (q[r, h] @ K[j, g].T)
            top = s.max(1, keepdims=True)
            p = np.exp(s - top)
            z = p.sum(1, keepdims=True)
            O[r, h] = (p / z) @ V[j, g]
            L[r, h] = (top + np.log(z))[:, 0]
    return O, L


def decode_bounds(k_cache, v_cache, q, table, lens, scale, step: float, tiny: float, q2k=None):
    """Element-wise error bounds (O, LSE) of a kernel that keeps scores and
    states in fp32, gives a weight as the sum of two numbers of a type of
    relative half step ``step`` and smallest half step ``tiny`` (the second is
    what rounding leaves over), and rounds the output to that type.

    u = 2^-24.  A score is a chain of dim fp32 products and sums and one
    scaling (of a constant rounded twice): |ds| <= (dim + 4) u scale sum |q||k|.
    2^x and the differences x - m add 8 u and 2 u |x - m|, |x - m| <= 2 max|s|
    / ln 2 + |ds|; a rescaling of the state (one at most for each 16 keys, and
    one for each join, 400 at most) adds 4 u, a sum over n keys n u.  So
    a weight and the normaliser are each off by e (relative), O by twice that
    times sum p|v|; a weight's two roundings add step^2 * sum p|v| (and tiny for
    each weight whose rest is below the normal range, against a largest weight
    of 2^7 in fp16, whose range is short, and of 1 in bf16), the output's
    step * |O| + tiny.  LSE: e, plus the sum's and logarithm's roundings."""
    u = 2.0 ** -24
    rest = tiny * 2.0 ** -7 if tiny > 2.0 ** -100 else tiny
    O, L = decode(k_cache, v_cache, q, table, lens, scale, q2k)
    BO, BL = np.zeros_like(O), np.zeros_like(L)
    rows, heads, dim = q.shape
    share = heads // k_cache.shape[2]
    for r in range(rows):
        n = int(lens[r])
        if n == 0:
            continue
        K, V = gather(k_cache, table[r], 0, n), gather(v_cache, table[r], 0, n)
        for g in range(k_cache.shape[2]):
            j = visible(n, None if q2k is None else q2k[g, r])
            if j.size == 0:
                continue
            h = slice(g * share, (g + 1) * share)
            s = scale * (q[r, h] @ K[j, g].T)
            ds = (dim + 4) * u * scale * (np.abs(q[r, h]) @ np.abs(K[j, g]).T).max(1)
            biggest = np.abs(s).max(1)
            m = j.size
            e = ds + u * (8 + 4 * biggest) + u * (4 * (m / 16 + 400) + m)
            p = np.exp(s - L[r, h][:, None])
            pv = p @ np.abs(V[j, g])
            BO[r, h] = ((2 * e + step ** 2) * 1.01)[:, None] * pv + step * np.abs(O[r, h]) + tiny \
                + m * rest * np.abs(V[j, g]).max() * np.exp(s.max(1) - L[r, h])[:, None]
            BL[r, h] = 1.01 * e + 4 * u * (np.abs(L[r, h]) + biggest + np.log(m) + 1)
    return O, L, BO, BL


# ------------------------------------------------------------------ rows that show every key
# decode_bounds grows with the number of keys, while O over random values shrinks
# with its root: of a long row it no longer sees a part that is missing.  Here
# page p of the pool holds STRIPE in one channel (p + head) % dim and zeros in
# the others, and all its keys score levels[p], so every stretch of a row is most
# of what one channel holds.
STRIPE = 64.0


def striped_values(pages: int, page_size: int, heads: int, dim: int) -> np.ndarray:
    v = np.zeros((pages, page_size, heads, dim))
    for p in range(pages):
        for g in range(heads):
            v[p, :, g, (p + g) % dim] = STRIPE
    return v


def striped(table_row, n: int, S: int, levels, heads: int, dim: int, times=None):
    """(O [heads, dim], LSE) of a row of n keys over such pages, in closed form;
    times [n]: how often each key counts (once, as it should)."""
    page = np.asarray(table_row)[np.arange(n) // S]
    w = np.bincount(page, weights=times, minlength=len(levels)) * np.exp(levels)
    O = np.zeros((heads, dim))
    for g in range(heads):
        np.add.at(O[g], (np.arange(len(levels)) + g) % dim, STRIPE * w / w.sum())
    return O, float(np.log(w.sum()))


def striped_bounds(O, L: float, n: int, levels, dim: int, step: float, tiny: float):
    """Element-wise bounds (O, LSE) for such a row, q all ones.

    Equal levels of 0: every weight is the same power of two, every sum a whole
    number of them below 2^24, so sums, factors and joins are exact.  What is
    left is 1 / l, the product with it and the output's rounding; for the LSE
    the logarithm, its sum with the maximum (below 32 both) and the product
    with ln 2.  Else as decode_bounds, with sum p|v| = O."""
    u = 2.0 ** -24
    levels = np.asarray(levels)
    if not levels.any():
        return (step + 4 * u) * O + tiny, 8 * u * (L + 7)
    top = float(np.abs(levels).max())
    e = (dim + 4) * u * top + u * (8 + 4 * top) + u * (4 * (n / 16 + 400) + n)
    rest = tiny * 2.0 ** -7 if tiny > 2.0 ** -100 else tiny
    small = n * rest * STRIPE * np.exp(float(levels.max()) - L)
    return (1.01 * (2 * e + step ** 2) + step) * O + tiny + small, \
        1.01 * e + 4 * u * (abs(L) + top + np.log(n) + 1)


# Long rows for them: type ("bf16" or "fp16"), channels, key heads, query heads a
# key head, page size, lengths, range of the levels (0: equal ones).
STRIPED_CASES = {
    "bf16, one row over all thread blocks": ("bf16", 128, 1, 16, 128, [90001], 0.0),
    "fp16, one row over all thread blocks": ("fp16", 64, 2, 5, 256, [70000, 3, 1], 0.0),
    "bf16, short runs": ("bf16", 128, 4, 16, 128, [330001, 5, 70000, 1], 0.0),
    "fp16, short runs": ("fp16", 64, 4, 5, 64, [700003], 0.0),
    "bf16, maxima that differ": ("bf16", 128, 1, 16, 128, [90001, 40000], 16.0),
    "fp16, maxima that differ": ("fp16", 64, 2, 5, 256, [70000, 3], 8.0),
}


def striped_rows(case):
    """(table [rows, width], levels [pages]): a page of the pool for each channel;
    equal levels: in a mixed order; else each page for one stretch of the row,
    levels rising along even rows and falling along odd ones.  A level is a whole
    number of eighths, which a key of equal channels gives exactly."""
    _, dim, _, _, S, lens, span = case
    width = -(-max(lens) // S) + 1
    i = np.arange(width)
    if span == 0:
        return np.stack([(i * 37 + r) % dim for r in range(len(lens))]), np.zeros(dim)
    table = np.stack([np.minimum(i * dim // -(-n // S), dim - 1) for n in lens])
    table[1::2] = dim - 1 - table[1::2]
    return table, np.arange(dim) / dim * span
