"""The norm and the drafted tokens' operators at the ends of what their calls take,
against their fp64 statement (oracle/drafts.py, where the bounds are derived)."""
import numpy as np
import pytest
import torch

from block_sparse_gqa_msa_gb300 import api
from oracle import drafts
from tests.test_gpu_drafts import BF, DEV, FP, HALF, TINY, _freq, _gen, _i32, _np, _randn, _within

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
