"""The norm and the drafted tokens' operators at the ends of what their calls take,
against their fp64 statement (oracle/drafts.py, where the bounds are derived)."""
import numpy as np
import pytest
import torch

from block_sparse_gqa_msa_gb300 import api
from oracle import drafts
from tests.test_drafts_rules import tiny_rest
from tests.test_gpu_drafts import (BF, DEV, FP, HALF, TINY, _choose, _freq, _gen, _i32, _np, _pages,
                                   _pool, _randn, _within)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ norm and rotation
@pytest.mark.parametrize("dt,dim,hq,hk,rot,T", [
    (BF, 128, 7, 3, 64, 33), (FP, 64, 9, 2, 32, 500), (BF, 64, 24, 4, 0, 5), (FP, 128, 1, 1, 128, 1),
    (BF, 128, 64, 4, 64, 9)])
@pytest.mark.parametrize("inter", [False, True])
def test_norm_without_eps(dt, dim, hq, hk, rot, T, inter):
    """eps = 0 with heads that are not zero; head counts that leave lanes of a warp
    without one."""
    gen = _gen(dim + hq)
    q, k = _randn(gen, (T, hq, dim), dt), _randn(gen, (T, hk, dim), dt)
    wq, wk = (1 + 0.3 * _randn(gen, (dim,)) for _ in range(2))
    gq, gk = _randn(gen, q.shape, dt), _randn(gen, k.shape, dt)
    pos, freq = _i32(range(T)), _freq(rot) if rot else None
    got = api.msa_norm_rope(q, k, wq, wk, pos, freq, eps=0.0, interleaved=inter)
    back = api.msa_norm_rope_backward(gq, gk, q, k, wq, wk, pos, freq, eps=0.0, interleaved=inter)
    p, f = _np(pos), None if freq is None else _np(freq)
    for i, (x, w, g) in enumerate(((q, wq, gq), (k, wk, gk))):
        X, W, G = _np(x), _np(w), _np(g)
        ref = drafts.norm_rope(X, W, p, f, inter, 0.0)
        _within(_np(got[i]), ref, drafts.norm_bound(X, W, ref, rot, inter, 0.0, HALF[dt], TINY[dt]),
                "y")
        dx, dw, sums = drafts.norm_rope_back(G, X, W, p, f, inter, 0.0)
        bx, bw = drafts.norm_back_bounds(G, X, W, dx, sums, p, f, rot, inter, 0.0, HALF[dt], TINY[dt])
        _within(_np(back[i]), dx, bx, "dx")
        _within(_np(back[i + 2]), dw, bw, "dw")


# ------------------------------------------------------------------ attention
@pytest.mark.parametrize("dim,share,S,trees,sparse", [
    (128, 16, 64, [16, 4], False), (64, 3, 16, [5, 64], False), (128, 7, 4, [9, 40], True)])
def test_tree_values_of_the_largest_size(dim, share, S, trees, sparse):
    """Values of 2^60 and scores that grow along the row, so that weights become large
    before the state is scaled."""
    rng, gen, kv = np.random.default_rng(dim), _gen(dim), 2
    lens = [3000, 700]
    offs = np.concatenate([[0], np.cumsum(trees)])
    T = int(offs[-1])
    pool, table = _pages(rng, [n + m for n, m in zip(lens, trees)], S)
    kc = _pool(gen, pool, S, kv, dim, BF)
    vc = _pool(gen, pool, S, kv, dim, BF)
    vc = torch.where(vc >= 0, 2.0 ** 60, -2.0 ** 60).to(BF)
    for r, (n, m) in enumerate(zip(lens, trees)):
        for j in range(n + m):
            kc[int(table[r, j // S]), j % S] *= 3.0 * j / (n + m)
    q = _randn(gen, (T, kv * share, dim), BF)
    q2k = _choose(rng, lens, offs, T, kv) if sparse else None
    ref = drafts.tree(_np(kc), _np(vc), _np(q), table, offs, lens, None, 0.5, q2k, HALF[BF], TINY[BF])
    cache = api.PagedCache(kc, vc)
    o, lse = api.msa_paged_tree(cache, q, _i32(table), _i32(offs), _i32(lens), 0.5,
                                q2k=None if q2k is None else _i32(q2k))
    assert api.msa_paged_read_status(cache) == 0
    _within(_np(o), ref[0], ref[2], "O")
    _within(_np(lse), ref[1], ref[3], "LSE")


# ------------------------------------------------------------------ verification
@pytest.mark.parametrize("rows,V", [(160, 151000), (160, 700001), (160, 1 << 20), (1, 1 << 22)])
def test_verify_sums_keep_their_bits(rows, V):
    """Few likely tokens and many of 2^-35 or so: a drawn token's place needs a sum of
    as many bits.  Probabilities are whole numbers of 2^-59, so the place is exact."""
    rng = np.random.default_rng(V)
    p = np.full(V, 2.0 ** -35, np.float32)
    p[V // 2:] = np.float32(1.9999 * 2.0 ** -35)
    likely = np.concatenate([np.arange(64) + V * b // 16 for b in range(16)])
    p[likely] = 2.0 ** -10
    run = np.cumsum((p.astype(np.float64) * 2.0 ** 59).astype(np.int64))
    total = int(run[-1])
    small = np.setdiff1d(np.arange(V // 2), likely)
    u, want = [], []
    while len(u) < rows:
        x = int(rng.choice(small))
        g = np.float32(run[x] / total)
        goal = int(float(g) * 2 ** 32) * total  # (exact: 24 bits from 2^-8 on)
        if g < 2.0 ** -8:
            continue
        x = int(np.searchsorted(run, goal >> 32, side="right"))
        lo, hi = int(run[x - 1]) << 32, int(run[x]) << 32
        # the sum, the running sum and what is formed of them: 2^-40 of the sum each
        if p[x] == p[small[0]] and min(goal - lo, hi - goal) > total << 32 >> 38:
            u.append(g)
            want.append(x)
    target = torch.as_tensor(p, device=DEV).expand(rows, V).contiguous()
    path, count, last = api.msa_tree_verify(
        target, _i32([0] * rows), _i32(range(rows + 1)), torch.zeros(rows, device=DEV),
        torch.as_tensor(np.array(u), device=DEV), max_path=1)
    assert (count == 1).all() and (path == 0).all()
    assert last.tolist() == want


def test_verify_rest_too_small_for_fp32():
    a = tiny_rest()
    f32 = lambda x: torch.as_tensor(x, device=DEV)
    got = api.msa_tree_verify(f32(a["target"]), _i32(a["tokens"]), _i32(a["offs"]), f32(a["u"]),
                              f32(a["u_last"]), draft=f32(a["draft"]), parents=_i32(a["parents"]),
                              max_path=3)
    for x, want in zip(got, drafts.verify(**a)):
        assert x.tolist() == want.tolist()
