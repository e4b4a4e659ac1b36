"""Norm and rotation, and the operators of drafted tokens, in fp64, written out
row by row - TEST INFRASTRUCTURE (used by the tests only; the product never
imports it).

Definitions (include/msa.h: msa_norm_rope and section "Drafted tokens").
All arguments are numpy arrays (or ints), all results float64 or ints.
"""
from __future__ import annotations

import math

import numpy as np

from .paged import BLOCK, gather, rotate

U = 2.0 ** -24


def norm_rope(x, w, pos=None, inv_freq=None, interleaved=False, eps=1e-6):
    """x [T, heads, dim] normed head by head, times w [dim], rotated."""
    n = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    y = x * n * w
    return y if inv_freq is None else rotate(y, pos, inv_freq, interleaved)


def norm_rope_back(dy, x, w, pos=None, inv_freq=None, interleaved=False, eps=1e-6):
    """(dx, dw, sum |g u|): the gradient of norm_rope."""
    n = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    g = dy
    if inv_freq is not None:
        g = rotate(dy, -np.asarray(pos, np.float64), inv_freq, interleaved)
    u = x * n
    gw = g * w
    dx = n * (gw - u * (gw * u).mean(-1, keepdims=True))
    return dx, (g * u).sum((0, 1)), np.abs(g * u).sum((0, 1))


def pair_size(x, rot: int, interleaved: bool):
    """|x| + |its partner in the rotation| (twice |x| where nothing turns)."""
    p = np.abs(x)
    y = 2 * p
    half = rot // 2
    if interleaved:
        both = p[..., 0:rot:2] + p[..., 1:rot:2]
        y[..., 0:rot:2] = y[..., 1:rot:2] = both
    else:
        both = p[..., :half] + p[..., half:rot]
        y[..., :half] = y[..., half:rot] = both
    return y


def norm_bound(x, w, y, rot, inter, eps, step, tiny):
    """Of a kernel in fp32.  Sum of dim squares: 20 roundings in a row at most (16
    of a lane, 3 exchanges, the mean), half of which reach n, its root 2 u, n x w
    2 u, all in all 16 u; angle 2^-22 and the rotation's products and sum, 2^-21
    of both channels; the output's half step."""
    n = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    d = (16 * U + 2.0 ** -21) * pair_size(x * n * w, rot, inter)
    return step * (np.abs(y) + d) + d + tiny


def norm_back_bounds(dy, x, w, dx, sums, pos, freq, rot, inter, eps, step, tiny):
    """(of dx, of dw).  g: 2^-21 of both channels.  The mean: 20 u of its terms'
    sizes, and g's and n's errors (2^-21 + 16 u); n twice, the products: 40 u in
    all, beside g's own; dw: a chain of at most T * heads sums."""
    n = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    size = pair_size(dy, rot, inter) * np.abs(w)
    u = np.abs(x * n)
    d = (2.0 ** -21 + 60 * U) * n * (size + u * (size * u).mean(-1, keepdims=True))
    terms = x.shape[0] * x.shape[1]
    dw = ((terms + 20) * U + 2.0 ** -20) * (pair_size(dy, rot, inter) * u).sum((0, 1))
    return step * (np.abs(dx) + d) + d + tiny, dw


def paths(parents) -> np.ndarray:
    """[n, n]: whether token j has token i on its path, itself included."""
    n = len(parents)
    seen = np.eye(n, dtype=bool)
    for j, p in enumerate(parents):
        if p >= 0:
            seen[j] |= seen[p]
    return seen


def tree(k_cache, v_cache, q, table, offs, lens, parents, scale, q2k=None, step=0.0, tiny=0.0,
         gone=()):
    """(O, LSE, bound of O, bound of LSE), NaN for tokens that no row owns.

    parents None: a chain.  gone: (row, page of the row's table) that are left
    out.  Bounds as oracle.paged.decode_bounds for scores and states, with one
    rounding (step) of each weight; a weight of fp16 is up to 2^7 at least where
    the largest is, so what lies below the type's normal range is off by tiny *
    2^-7 of the largest."""
    T, heads, dim = q.shape
    kv = k_cache.shape[2]
    S = k_cache.shape[1]
    share = heads // kv
    O, BO = np.full((T, heads, dim), np.nan), np.full((T, heads, dim), np.nan)
    L, BL = np.full((T, heads), np.nan), np.full((T, heads), np.nan)
    rest = tiny * 2.0 ** -7 if tiny > 2.0 ** -100 else tiny
    for r in range(len(lens)):
        t0, m, n = int(offs[r]), int(offs[r + 1]) - int(offs[r]), int(lens[r])
        if m <= 0:
            continue
        K, V = gather(k_cache, table[r], 0, n + m), gather(v_cache, table[r], 0, n + m)
        line = paths([j - 1 for j in range(m)] if parents is None else parents[t0:t0 + m])
        there = ~np.isin(np.arange(n + m) // S, [p for row, p in gone if row == r])
        for j in range(m):
            for g in range(kv):
                see = np.concatenate([np.ones(n, bool), line[j]]) & there
                if q2k is not None:
                    see[:n] &= np.isin(np.arange(n) // BLOCK, [int(x) for x in q2k[g, t0 + j]])
                h = slice(g * share, (g + 1) * share)
                i = np.nonzero(see)[0]
                if i.size == 0:
                    O[t0 + j, h], L[t0 + j, h] = 0, -np.inf
                    BO[t0 + j, h], BL[t0 + j, h] = 0, 0
                    continue
                s = scale * (q[t0 + j, h] @ K[i, g].T)
                top = s.max(1, keepdims=True)
                p = np.exp(s - top)
                z = p.sum(1, keepdims=True)
                O[t0 + j, h] = (p / z) @ V[i, g]
                L[t0 + j, h] = (top + np.log(z))[:, 0]
                ds = (dim + 4) * U * scale * (np.abs(q[t0 + j, h]) @ np.abs(K[i, g]).T).max(1)
                big = np.abs(s).max(1)
                e = ds + U * (8 + 4 * big) + U * (4 * (i.size / 16 + 400) + i.size)
                pv = (p / z) @ np.abs(V[i, g])
                BO[t0 + j, h] = ((2 * e + step) * 1.01)[:, None] * pv \
                    + step * np.abs(O[t0 + j, h]) + tiny \
                    + i.size * rest * np.abs(V[i, g]).max() / z
                BL[t0 + j, h] = 1.01 * e + 4 * U * (np.abs(L[t0 + j, h]) + big
                                                    + np.log(i.size) + 1)
    return O, L, BO, BL


def verify(target, tokens, offs, u, u_last, draft=None, parents=None, max_path=64):
    """(path [rows, max_path], count [rows], last [rows]): the definition, r in
    fp32, sums exact."""
    rows, V = len(u_last), target.shape[1]
    path = np.full((rows, max_path), -1)
    count, last = np.zeros(rows, int), np.full(rows, -1)
    f32 = np.float32
    for row in range(rows):
        t0, m = int(offs[row]), int(offs[row + 1]) - int(offs[row])
        if t0 < 0 or m < 1 or m > 64 or offs[row + 1] > len(tokens):
            continue
        up = [j - 1 if parents is None else int(parents[t0 + j]) for j in range(m)]
        cur, kept = 0, [0]
        while True:
            r, S = target[t0 + cur].astype(f32).copy(), 1.0
            at = None
            for j in range(1, m):
                x = int(tokens[t0 + j])
                if len(kept) == max_path or up[j] != cur or up[j] >= j or not 0 <= x < V:
                    continue
                if draft is not None:
                    q = draft[t0 + cur].astype(f32)
                    with np.errstate(over="ignore"):
                        f = f32(1.0 / S) if S > 0 else f32(0)
                    if np.isinf(f):  # so little is left that it is nothing
                        f = f32(0)
                    if float(u[t0 + j]) * float(q[x]) < float(r[x]) * float(f):
                        at = j
                        break
                    r = np.maximum(r * f - q, f32(0))
                    S = math.fsum(r.tolist())
                else:
                    if r[x] > 0 and float(u[t0 + j]) * S < float(r[x]):
                        at = j
                        break
                    S -= float(r[x])
                    r[x] = 0
            if at is None:
                break
            cur = at
            kept.append(at)
        if not r.any():
            r = target[t0 + cur].astype(f32)
        run = np.cumsum(r.astype(np.float64))
        path[row, :len(kept)] = kept
        count[row] = len(kept)
        if run[-1] > 0:
            last[row] = int(np.searchsorted(run, float(u_last[row]) * run[-1], side="right"))
    return path, count, last


def compact(cache, table, lens, path, count):
    """The cache (keys or values) after the call."""
    out = cache.copy()
    S = cache.shape[1]
    for r, n in enumerate(lens):
        for i in range(int(count[r])):
            a, b = int(n) + int(path[r][i]), int(n) + i
            out[table[r][b // S], b % S] = cache[table[r][a // S], a % S]
    return out
