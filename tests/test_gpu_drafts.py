"""Norm with rotation and the operators of drafted tokens on the GPU against
their fp64 statement (oracle/drafts.py, where the bounds are derived)."""
import numpy as np
import pytest
import torch

from block_sparse_gqa_msa_gb300 import api, autograd, inputs
from oracle import drafts, paged

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
BF, FP = torch.bfloat16, torch.float16
HALF = {BF: 2.0 ** -8, FP: 2.0 ** -11}
TINY = {BF: 2.0 ** -134, FP: 2.0 ** -25}  # half the smallest step


def _np(x):
    return x.detach().double().cpu().numpy()


def _i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(gen, shape, dtype=torch.float32):
    return torch.randn(shape, generator=gen, device=DEV).to(dtype)


def _pages(rng, lens, S, spare=3, width=None):
    need = [-(-int(n) // S) for n in lens]
    pool = sum(need) + spare
    order = rng.permutation(pool)
    table = np.full((len(lens), width or max(max(need), 1) + 2), -1, dtype=np.int64)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = order[at:at + n]
        at += n
    return pool, table


def _pool(gen, pool, S, heads, dim, dtype, head_major=False):
    if head_major:
        return _randn(gen, (pool, heads, S, dim), dtype).transpose(1, 2)
    return _randn(gen, (pool, S, heads, dim), dtype)


def _within(got, ref, bound, what):
    assert not np.isnan(got).any(), f"{what}: NaN"
    with np.errstate(invalid="ignore"):
        over = np.where(got == ref, 0.0, np.abs(got - ref) - bound)
    worst = np.unravel_index(np.argmax(over), over.shape)
    assert over[worst] <= 0, (f"{what}: {got[worst]} for {ref[worst]} at {worst}, bound "
                              f"{bound[worst]:.3e}")


def _freq(rot, theta=10000.0):
    return torch.tensor(theta ** (-np.arange(0, rot, 2) / rot), dtype=torch.float32, device=DEV)


# ------------------------------------------------------------------ norm and rotation
NORM_CASES = [
    # type, dim, q heads, k heads, rot, interleaved, tokens, fp32 weights, one projection
    (BF, 128, 64, 4, 64, False, 37, True, True),
    (BF, 128, 7, 3, 128, True, 1, False, False),
    (BF, 64, 24, 8, 48, False, 9, True, True),
    (FP, 64, 1, 1, 16, True, 333, False, False),
    (FP, 128, 5, 5, 128, False, 2, True, True),
    (FP, 64, 9, 2, 0, False, 6, True, False),
    (BF, 128, 3, 1, 112, True, 5000, False, True),
    (FP, 64, 65, 33, 32, False, 700, True, True),
]


def _norm_case(case, seed=3):
    dt, dim, hq, hk, rot, inter, T, wide, fused = case
    gen = _gen(seed)
    if fused:
        x = _randn(gen, (T, hq + 2 * hk, dim), dt)
        q, k = x[:, :hq], x[:, hq:hq + hk]
    else:
        q, k = _randn(gen, (T, hq, dim), dt), _randn(gen, (T, hk, dim), dt)
    q[T // 2] *= 0.01
    wd = torch.float32 if wide else dt
    wq, wk = (1 + 0.3 * _randn(gen, (dim,))).to(wd), (1 + 0.3 * _randn(gen, (dim,))).to(wd)
    pos = torch.randint(0, 1 << 20, (T,), generator=gen, device=DEV).to(torch.int32)
    freq = _freq(rot) if rot else None
    return q, k, wq, wk, pos, freq, gen


@pytest.mark.parametrize("case", NORM_CASES, ids=str)
def test_norm_and_gradient_match_fp64(case):
    dt, dim, hq, hk, rot, inter, T, _, _ = case
    q, k, wq, wk, pos, freq, gen = _norm_case(case)
    eps = 1e-5
    gq, gk = _randn(gen, q.shape, dt), _randn(gen, k.shape, dt)
    got = api.msa_norm_rope(q, k, wq, wk, pos, freq, eps=eps, interleaved=inter)
    back = api.msa_norm_rope_backward(gq, gk, q, k, wq, wk, pos, freq, eps=eps, interleaved=inter)
    again = api.msa_norm_rope_backward(gq, gk, q, k, wq, wk, pos, freq, eps=eps, interleaved=inter)
    leaves = [x.detach().requires_grad_() for x in (q, k, wq, wk)]
    outs = autograd.msa_norm_rope(*leaves, pos, freq, eps=eps, interleaved=inter)
    grads = torch.autograd.grad(outs, leaves, (gq, gk))
    torch.cuda.synchronize()
    p, f = _np(pos), None if freq is None else _np(freq)
    e = float(np.float32(eps))
    for i, (x, w, g) in enumerate(((q, wq, gq), (k, wk, gk))):
        X, W, G = _np(x), _np(w), _np(g)
        ref = drafts.norm_rope(X, W, p, f, inter, e)
        _within(_np(got[i]), ref, drafts.norm_bound(X, W, ref, rot, inter, e, HALF[dt], TINY[dt]),
                "y")
        dx, dw, sums = drafts.norm_rope_back(G, X, W, p, f, inter, e)
        bx, bw = drafts.norm_back_bounds(G, X, W, dx, sums, p, f, rot, inter, e, HALF[dt], TINY[dt])
        _within(_np(back[i]), dx, bx, "dx")
        _within(_np(back[i + 2]), dw, bw, "dw")
        assert torch.equal(outs[i], got[i]) and torch.equal(grads[i], back[i])
        assert torch.equal(grads[i + 2], back[i + 2].to(w.dtype))
        assert torch.equal(again[i], back[i]) and torch.equal(again[i + 2], back[i + 2])


def test_norm_in_place_and_of_zeros():
    q, k, wq, wk, pos, freq, _ = _norm_case(NORM_CASES[1])
    want = api.msa_norm_rope(q, k, wq, wk, pos, freq, interleaved=True)
    got = api.msa_norm_rope(q, k, wq, wk, pos, freq, interleaved=True, q_out=q, k_out=k)
    assert got[0] is q and torch.equal(q, want[0]) and torch.equal(k, want[1])
    z = torch.zeros(3, 4, 64, dtype=BF, device=DEV)
    w = torch.ones(64, device=DEV)
    y = api.msa_norm_rope(z, z, w, w)
    g = api.msa_norm_rope_backward(torch.ones_like(z), torch.ones_like(z), z, z, w, w)
    assert all((x == 0).all() for x in (*y, *g[2:]))
    # dx = n (g w - 0) = 1000, rounded to bf16
    assert (g[0] == 1000).all()


def test_norm_strides_and_gradients_that_are_broadcast():
    gen = _gen(17)
    wide = _randn(gen, (50, 40, 64), BF)
    w = (1 + 0.2 * _randn(gen, (64,))).requires_grad_()
    q = wide[::7, 3:14].detach().requires_grad_()
    k = wide[10:18, 37:].detach().requires_grad_()
    pos, freq = _i32([0, -5, 2 ** 29 - 1, 7, 1, 2, -2 ** 29, 3]), _freq(32)
    with pytest.raises(api.MSAError):  # tokens that overlap are refused
        api.msa_norm_rope(q, k[:1].expand(8, 3, 64), w, w, pos, freq)
    outs = autograd.msa_norm_rope(q, k, w, w, pos, freq)
    gq, gk = _randn(gen, (1, 11, 64), BF).expand(8, 11, 64), _randn(gen, (8, 1, 64), BF).expand(8, 3, 64)
    got = torch.autograd.grad(outs, (q, k, w), (gq, gk))
    c = [x.detach().contiguous() for x in (q, k, gq, gk)]
    assert all(torch.equal(x, y) for x, y in zip(outs, api.msa_norm_rope(*c[:2], w.detach(), w.detach(), pos, freq)))
    dq, dk, wq, wk = api.msa_norm_rope_backward(c[2], c[3], c[0], c[1], w.detach(), w.detach(), pos, freq)
    assert torch.equal(got[0], dq) and torch.equal(got[1], dk) and torch.equal(got[2], wq + wk)
    ref = drafts.norm_rope(_np(q), _np(w), _np(pos), _np(freq), False, float(np.float32(1e-6)))
    _within(_np(outs[0]), ref, drafts.norm_bound(_np(q), _np(w), ref, 32, False, 1e-6, HALF[BF], TINY[BF]), "y")


def test_calls_at_once_and_in_graphs():
    """Norm, its gradient, verification and compaction on two streams at a time and in a
    graph whose inputs change between replays."""
    gen, rng = _gen(18), np.random.default_rng(18)
    q, k = _randn(gen, (900, 24, 128), BF), _randn(gen, (900, 8, 128), BF)
    w, pos, freq = 1 + 0.1 * _randn(gen, (128,)), _i32(range(900)), _freq(64)
    p = torch.softmax(30 * _randn(gen, (30, 9000)), 1)  # most of it in one token
    tok, offs = _i32(rng.integers(0, 9000, 30)), _i32(range(0, 31, 6))
    for t in range(30):  # likely drafts
        tok[t] = p[max(t - 1, 0)].argmax()
    u, ul = torch.rand(30, generator=gen, device=DEV), torch.rand(5, generator=gen, device=DEV)
    kc, vc = (_randn(gen, (20, 16, 2, 64), FP) for _ in range(2))
    tab, lens = _i32(rng.permutation(20).reshape(5, 4)), _i32([3, 40, 0, 17, 31])

    def calls(stream=None):
        out = list(api.msa_norm_rope(q, k, w, w, pos, freq, stream=stream))
        out += api.msa_norm_rope_backward(*out, q, k, w, w, pos, freq, stream=stream)
        path, count, last = api.msa_tree_verify(p, tok, offs, u, ul, max_path=6, stream=stream)
        with torch.cuda.stream(stream):
            c = api.PagedCache(kc.clone(), vc.clone())
        new = api.msa_paged_compact(c, tab, lens, path, count, stream=stream)
        return out + [path, count, last, new, c.k, c.v]

    here = torch.cuda.current_stream()
    want = calls(here)
    assert int(want[7].max()) > 1
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for got in [calls(x) for x in sides]:
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = calls(torch.cuda.current_stream())
    for x in (q, u, kc):  # the step after
        x.copy_(x.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    now = calls(here)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, now)) and not torch.equal(got[0], want[0])


def test_norm_through_training_attention():
    """A step as trained: projection, norm with rotation, attention; the gradient of
    the projection's output is that of the two calls one after the other."""
    w = inputs.custom([300, 77], 5)
    gen = _gen(6)
    T = 377
    x = _randn(gen, (T, 72, 128), BF).requires_grad_()
    wq, wk = ((1 + 0.2 * _randn(gen, (128,))).requires_grad_() for _ in range(2))
    pos = _i32(list(range(300)) + list(range(77)))
    freq = _freq(64)
    q, k = autograd.msa_norm_rope(x[:, :64], x[:, 64:68], wq, wk, pos, freq)
    o = autograd.msa_attention(q, k, x[:, 68:].contiguous(), w.q2k.to(DEV), w.doc_offsets.to(DEV))
    do = w.do.to(DEV)
    dx, dwq, dwk = torch.autograd.grad(o, (x, wq, wk), do)
    plan = api.msa_build_plan(w.q2k.to(DEV), w.doc_offsets.to(DEV))
    v = x[:, 68:].detach().contiguous()
    O, lse = api.msa_forward(plan, q.detach(), k.detach(), v, 128 ** -0.5)
    dq, dk, dv = api.msa_backward(plan, q.detach(), k.detach(), v, O, lse, do, 128 ** -0.5)
    e = 1e-6
    gq, gk, rq, rk = api.msa_norm_rope_backward(dq, dk, x[:, :64].detach(), x[:, 64:68].detach(),
                                                wq.detach(), wk.detach(), pos, freq, eps=e)
    # the attention's gradients are summed by atomics: two runs differ by their last bits
    for a, b in ((dx[:, :64], gq), (dx[:, 64:68], gk), (dx[:, 68:], dv), (dwq, rq), (dwk, rk)):
        a, b = a.float(), b.float()
        assert (a - b).norm() <= 1e-2 * b.norm()


# ------------------------------------------------------------------ attention
def _random_parents(rng, n, chain=False):
    return [-1] + [j - 1 if chain else int(rng.integers(-1 if j % 5 == 0 else 0, j))
                   for j in range(1, n)]


def _choose(rng, lens, offs, T, kv, most=16):
    """Slots of each token: distinct blocks of the cached tokens in any order, some twice, some
    unused; now and then none."""
    q2k = np.full((kv, T, 16), -1)
    for r, n in enumerate(lens):
        blocks = -(-n // 128)
        for t in range(offs[r], offs[r + 1]):
            for g in range(kv):
                c = rng.integers(0, min(most, blocks) + 1)
                v = rng.choice(blocks, c, replace=False) if blocks else np.zeros(0, int)
                at = rng.permutation(16)[:c]
                q2k[g, t, at] = v
                if 0 < c < 16 and rng.random() < 0.3:
                    q2k[g, t, np.setdiff1d(np.arange(16), at)[0]] = v[0]
    return q2k


def _tree_case(dt, dim, kv, share, S, lens, trees, sparse, chain=False, seed=1, pad=0,
               head_major=False, scale=None, growing=False, stream=None):
    rng, gen = np.random.default_rng(seed), _gen(seed)
    offs = np.concatenate([[0], np.cumsum(trees)])
    T = int(offs[-1]) + pad
    pool, table = _pages(rng, [n + m for n, m in zip(lens, trees)], S)
    kc, vc = (_pool(gen, pool, S, kv, dim, dt, head_major) for _ in range(2))
    parents = [p for m in trees for p in (_random_parents(rng, m, chain) if m else [])] + [99] * pad
    q = _randn(gen, (T, kv * share, dim), dt)
    if growing:  # scores that rise along the row, to about 40
        for r, (n, m) in enumerate(zip(lens, trees)):
            for j in range(n + m):
                kc[int(table[r, j // S]), j % S] *= 3.0 * j / (n + m)
    scale = scale or dim ** -0.5
    q2k = _choose(rng, lens, offs, T, kv) if sparse else None
    # what lies past a row's tokens, and in pages of nobody, must not matter
    ref = drafts.tree(_np(kc), _np(vc), _np(q), table, offs, lens, None if chain else parents,
                      float(np.float32(scale)), q2k, HALF[dt], TINY[dt])
    for r, (n, m) in enumerate(zip(lens, trees)):
        for j in range(n + m, -(-(n + m) // S) * S):
            kc[int(table[r, j // S]), j % S] = float("nan")
            vc[int(table[r, j // S]), j % S] = float("inf")
    cache = api.PagedCache(kc, vc)
    o = torch.full((T, kv * share, dim), 7.0, dtype=dt, device=DEV)
    lse = torch.full((T, kv * share), 7.0, device=DEV)
    args = (cache, q, _i32(table), _i32(offs), _i32(lens), scale)
    kw = dict(parents=None if chain else _i32(parents), q2k=None if q2k is None else _i32(q2k))
    api.msa_paged_tree(*args, o=o, lse=lse, **kw)
    torch.cuda.synchronize()
    assert api.msa_paged_read_status(cache) == 0
    n = int(offs[-1])
    assert (o[n:] == 7).all() and (lse[n:] == 7).all()
    _within(_np(o)[:n], ref[0][:n], ref[2][:n], "O")
    _within(_np(lse)[:n], ref[1][:n], ref[3][:n], "LSE")
    return args, kw, o, lse


@pytest.mark.parametrize("sparse", [False, True])
@pytest.mark.parametrize("dt,dim,kv,share,S", [
    (BF, 128, 4, 16, 64), (FP, 64, 2, 3, 16), (BF, 64, 1, 1, 1), (FP, 128, 3, 7, 256),
    (BF, 128, 2, 8, 2), (FP, 64, 1, 16, 1024)])
def test_tree_matches_fp64(dt, dim, kv, share, S, sparse):
    lens = [300, 0, 1, 127, 128, 129, 1000, 65]
    trees = [5, 3, 1, 64, 17, 0, 9, 33]
    _tree_case(dt, dim, kv, share, S, lens, trees, sparse, pad=3, seed=S + sparse,
               head_major=S == 256)


@pytest.mark.parametrize("chain", [False, True])
@pytest.mark.parametrize("n,m", [(0, 1), (1, 1), (5, 8), (128, 64), (2900, 8), (3000, 16), (100, 64)])
def test_tree_one_row(n, m, chain):
    _tree_case(BF, 128, 4, 16, 64, [n], [m], False, chain=chain, seed=n + m)


def test_tree_many_rows_with_many_segments_a_run():
    rng = np.random.default_rng(4)
    trees = [int(x) for x in rng.integers(0, 7, 700)]
    lens = [int(x) for x in rng.integers(0, 200, 700)]
    _tree_case(FP, 64, 2, 5, 16, lens, trees, False, pad=1, seed=4)
    _tree_case(BF, 128, 1, 7, 32, lens[:300], trees[:300], True, seed=5)


def test_tree_rows_of_two_tokens_in_two_items():
    # 7 heads a key head: token 36 has heads on both sides of matrix row 256
    _tree_case(BF, 128, 1, 7, 64, [500, 260], [64, 40], False, seed=8)
    _tree_case(FP, 64, 2, 7, 32, [3000, 260], [64, 40], True, seed=9)
    _tree_case(BF, 64, 1, 13, 16, [400], [63], True, seed=10)


@pytest.mark.parametrize("seed", range(4))
def test_tree_rows_of_all_kinds_together(seed):
    """Rows whose items take both slots next to rows that share a tile, empty ones between
    them, in tables of any width (few tiles or many by it) and strides."""
    rng = np.random.default_rng(50 + seed)
    rows = int(rng.integers(2, 60))
    trees = [int(rng.choice([0, 1, 2, 8, 9, 16, 17, 33, 64])) for _ in range(rows)]
    lens = [int(rng.choice([0, 1, 100, 127, 128, 129, 255, 256, 400, 1500])) for _ in range(rows)]
    _tree_case([BF, FP][seed % 2], [128, 64][seed // 2], int(rng.integers(1, 4)),
               int(rng.integers(1, 17)), int(rng.choice([4, 8, 16, 64])), lens, trees, seed == 3,
               pad=seed, seed=60 + seed)


@pytest.mark.parametrize("dt", [BF, FP])
def test_tree_scores_that_grow_along_the_row(dt):
    _tree_case(dt, 128, 1, 16, 64, [3000, 700], [16, 4], False, seed=6, growing=True, scale=0.5)
    _tree_case(dt, 64, 2, 4, 16, [2000, 900], [20, 64], True, seed=7, growing=True, scale=0.5)


@pytest.mark.parametrize("dt,dim,kv,share,S,n,m", [
    (BF, 128, 1, 16, 128, 60001, 8), (BF, 128, 1, 16, 64, 60001, 64), (FP, 64, 2, 5, 256, 50000, 3),
    (BF, 128, 4, 16, 16, 20011, 16)])
def test_tree_counts_every_key_of_a_long_row_once(dt, dim, kv, share, S, n, m):
    """Equal scores; block b of the row has its values in channel b % dim: what a
    channel holds is the share of its blocks' keys, whole numbers and one division."""
    rng = np.random.default_rng(n)
    pool, table = _pages(rng, [n + m, 300], S)
    kc = torch.zeros(pool, S, kv, dim, dtype=dt, device=DEV)
    vc = torch.zeros_like(kc)
    pos = torch.arange(n + m, device=DEV)
    at = _i32(table[0]).long()[pos // S]
    vc[at, pos % S, :, (pos // 128) % dim] = 64.0
    q = torch.ones(m + 1, kv * share, dim, dtype=dt, device=DEV)
    cache = api.PagedCache(kc, vc)
    o, lse = api.msa_paged_tree(cache, q, _i32(table), _i32([0, m, m + 1]), _i32([n, 299]), 1.0)
    assert api.msa_paged_read_status(cache) == 0
    for j in range(m):
        keys = n + j + 1
        want = np.bincount((np.arange(keys) // 128) % dim, minlength=dim) * 64.0 / keys
        want = np.broadcast_to(want, (kv * share, dim))
        _within(_np(o[j]), want, (HALF[dt] + 4 * U) * want + TINY[dt], "O")
        _within(_np(lse[j]), np.full(kv * share, np.log(keys)), np.full(kv * share, 8 * U * 20), "LSE")


def test_tree_bad_input_is_left_out():
    gen = _gen(11)
    S, dim = 16, 64
    kc, vc = (_randn(gen, (40, S, 2, dim), BF) for _ in range(2))
    cache = api.PagedCache(kc, vc)
    table = np.arange(32).reshape(2, 16)
    q = _randn(gen, (70, 6, dim), BF)

    def call(table, offs, lens, code, parents=None, q2k=None, gone=(), ref_lens=None,
             ref_parents=None, ref_q2k=None):
        o, lse = (torch.full(s, 7.0, dtype=d, device=DEV) for s, d in (
            ((70, 6, dim), BF), ((70, 6), torch.float32)))
        api.msa_paged_tree(cache, q, _i32(table), _i32(offs), _i32(lens), 0.125,
                           parents=None if parents is None else _i32(parents),
                           q2k=None if q2k is None else _i32(q2k), o=o, lse=lse)
        assert api.msa_paged_read_status(cache, clear=True) == code
        if ref_lens is None:
            return o, lse
        safe = np.clip(np.asarray(table), 0, 39)
        up = ref_parents if ref_parents is not None else parents
        ref = drafts.tree(_np(kc), _np(vc), _np(q), safe, offs, ref_lens, up,
                          0.125, ref_q2k, HALF[BF], TINY[BF], gone)
        n = offs[-1]
        _within(_np(o)[:n], ref[0][:n], ref[2][:n], "O")
        _within(_np(lse)[:n], ref[1][:n], ref[3][:n], "LSE")
        return o, lse

    # pages outside the pool: their keys are left out
    bad = table.copy()
    bad[0, 3], bad[1, 0], bad[1, 7] = -1, 40, 1 << 30
    call(bad, [0, 5, 9], [100, 110], 11, gone=[(0, 3), (1, 0), (1, 7)], ref_lens=[100, 110])
    # all of a row's keys in bad pages
    none = table.copy()
    none[0, 0] = -5
    o, lse = call(none, [0, 5, 9], [3, 110], 11, gone=[(0, 0)], ref_lens=[3, 110])
    assert (o[:5] == 0).all() and (lse[:5] == -np.inf).all()
    # a length outside the table, below 0
    for n in (252, -1, 2 ** 31 - 1):
        o, lse = call(table, [0, 5, 9], [n, 110], 11)
        assert (o[:5] == 0).all() and (lse[:5] == -np.inf).all()
        assert torch.isfinite(lse[5:9]).all() and (o[9:] == 7).all() and (lse[9:] == 7).all()
    # too many tokens
    o, lse = call(table, [0, 65, 69], [10, 110], 12)
    assert (o[:65] == 0).all() and (lse[:65] == -np.inf).all() and torch.isfinite(lse[65:69]).all()
    # parents that do not come before their tokens stand for the cached ones
    call(table, [0, 4, 7], [50, 60], 12, parents=[-1, 1, 7, -2, -1, 0, 1] + [0] * 63,
         ref_lens=[50, 60], ref_parents=[-1, -1, -1, -1, -1, 0, 1])
    # blocks that the cached tokens do not have
    q2k = np.full((2, 70, 16), -1)
    q2k[:, :9, 0] = 0
    good = q2k.copy()
    q2k[0, 1, 3], q2k[1, 6, 5], q2k[1, 2, 2] = 1, -2, 1 << 30
    call(table, [0, 5, 9], [100, 110], 6, q2k=q2k, ref_lens=[100, 110], ref_q2k=good)
    # offsets
    o, lse = call(table, [0, 5, 71], [100, 110], 7)
    assert torch.isfinite(lse[:5]).all() and (lse[5:] == 7).all()
    o, lse = call(table, [-2, 5, 9], [100, 110], 7)
    assert (lse[:5] == 7).all() and torch.isfinite(lse[5:9]).all() and (lse[9:] == 7).all()


@pytest.mark.parametrize("dt,dim,share,S,n,m,sparse", [
    (BF, 128, 16, 64, 100, 40, False), (FP, 64, 3, 16, 3000, 9, False), (BF, 128, 7, 4, 250, 64, True),
    (FP, 128, 16, 32, 0, 64, False), (BF, 64, 5, 8, 1000, 21, True), (FP, 128, 2, 256, 9000, 64, True)])
def test_tree_values_that_are_not_finite_reach_those_who_see_them(dt, dim, share, S, n, m, sparse):
    rng, gen, kv = np.random.default_rng(m), _gen(m + n), 2
    lens, trees, offs = [n, 70], [m, 3], [0, m, m + 3]
    T = m + 3
    pool, table = _pages(rng, [a + b for a, b in zip(lens, trees)], S)
    kc, vc = (_pool(gen, pool, S, kv, dim, dt) for _ in range(2))
    q = _randn(gen, (T, kv * share, dim), dt)
    parents = _random_parents(rng, m) + [-1, 0, 0]
    q2k = _choose(rng, lens, offs, T, kv) if sparse else None
    odd = {}  # token of row 0, key head, channel -> value
    for i, j in enumerate(rng.choice(m, min(m, 6), replace=False)):
        for c in rng.choice(dim, 2, replace=False):
            odd[int(j), i % kv, int(c)] = [float("inf"), -float("inf"), float("nan")][i % 3]
    place = lambda j: (int(table[0, (n + j) // S]), (n + j) % S)
    for (j, g, c) in odd:
        vc[place(j)][g, c] = 0.0
    scale = dim ** -0.5
    ref = drafts.tree(_np(kc), _np(vc), _np(q), table, offs, lens, parents,
                      float(np.float32(scale)), q2k, HALF[dt], TINY[dt])
    want, bound = ref[0].copy(), ref[2].copy()
    # also a token that none of the others continues: its keys are not to be seen
    leaf = [j for j in range(m) if j not in parents[:m]][-1]
    for (j, g, c), x in odd.items():
        vc[place(j)][g, c] = x
        for t in range(m):
            up = t
            while up > j:
                up = parents[up]
            if up == j:
                with np.errstate(invalid="ignore"):  # inf - inf
                    want[t, g * share:(g + 1) * share, c] += x
    kc[place(leaf)] = float("inf")
    cache = api.PagedCache(kc, vc)
    o, lse = api.msa_paged_tree(cache, q, _i32(table), _i32(offs), _i32(lens), scale,
                                parents=_i32(parents), q2k=None if q2k is None else _i32(q2k))
    assert api.msa_paged_read_status(cache) == 0
    rest = [t for t in range(T) if t != leaf]
    got, want, bound = _np(o)[rest], want[rest], bound[rest]
    finite = np.isfinite(want)
    assert not finite.all()
    assert np.array_equal(got[~finite], want[~finite], equal_nan=True)
    _within(np.where(finite, got, 0.0), np.where(finite, want, 0.0), np.where(finite, bound, 0.0), "O")
    _within(_np(lse)[rest], ref[1][rest], ref[3][rest], "LSE")


def test_tree_repeats_its_bits_on_streams_and_in_a_graph():
    args, kw, o, lse = _tree_case(BF, 128, 2, 16, 64, [3000, 5, 700], [16, 3, 40], True, seed=12)
    cache, q, table, offs, lens, scale = args
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o1, lse1 = api.msa_paged_tree(*args, **kw, stream=side)
    o2, lse2 = api.msa_paged_tree(*args, **kw)  # at the same time
    side.synchronize()
    torch.cuda.synchronize()
    for a, b in ((o1, lse1), (o2, lse2)):
        assert torch.equal(a, o) and torch.equal(b, lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        og, lg = api.msa_paged_tree(*args, **kw)
    lens -= 1  # the step after: other lengths, the same graph
    graph.replay()
    want = api.msa_paged_tree(*args, **kw)
    assert torch.equal(og, want[0]) and torch.equal(lg, want[1]) and not torch.equal(og, o)
    lens += 1
    graph.replay()
    assert torch.equal(og, o) and torch.equal(lg, lse)


def test_tree_in_a_cache_of_more_than_2_to_the_31_elements():
    S, kv, dim, n, m = 128, 4, 128, 777, 5
    pool = 2 ** 31 // (S * kv * dim) + 600
    kc = torch.empty(pool, S, kv, dim, dtype=BF, device=DEV)
    vc = torch.empty(pool, S, kv, dim, dtype=BF, device=DEV)
    gen = _gen(13)
    table = np.array([[pool - 1 - i for i in range(7)]])
    small_k, small_v = (_randn(gen, (7, S, kv, dim), BF) for _ in range(2))
    kc[_i32(table[0]).long()], vc[_i32(table[0]).long()] = small_k, small_v
    q = _randn(gen, (m, 64, dim), BF)
    tail = (_i32([0, m]), _i32([n]), 0.1)
    a = api.msa_paged_tree(api.PagedCache(kc, vc), q, _i32(table), *tail)
    b = api.msa_paged_tree(api.PagedCache(small_k, small_v), q, _i32([range(7)]), *tail)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    # and the moves of such pages
    path, count = _i32([[0, 2, 4]]), _i32([3])
    big, tiny = api.PagedCache(kc, vc), api.PagedCache(small_k, small_v)
    for c, t in ((big, table), (tiny, [range(7)])):
        assert api.msa_paged_compact(c, _i32(t), _i32([n]), path, count).tolist() == [n + 3]
    assert torch.equal(kc[_i32(table[0]).long()], small_k)
    assert torch.equal(vc[_i32(table[0]).long()], small_v)


# ------------------------------------------------------------------ verification
def _verify_case(rows, trees, V, drawn, chain, seed, sharp=1.0, skew=0, max_path=64):
    rng, gen = np.random.default_rng(seed), _gen(seed)
    offs = np.concatenate([[0], np.cumsum(trees)])
    T = int(offs[-1])
    wide = torch.randn(T, V + skew, generator=gen, device=DEV) * sharp
    near = wide + 0.8 * torch.randn(T, V + skew, generator=gen, device=DEV)
    target = torch.zeros(T, V + skew, device=DEV)
    target[:, skew // 2:skew // 2 + V] = torch.softmax(wide[:, :V], 1)
    target = target[:, skew // 2:skew // 2 + V]  # rows begin at any address
    draft = torch.softmax(near[:, :V], 1)
    parents = [p for m in trees for p in (_random_parents(rng, m, chain) if m else [])]
    base = np.repeat(offs[:-1], trees)
    at = torch.as_tensor(base + np.maximum(parents, 0), device=DEV)
    tokens = torch.multinomial(draft[at], 1, generator=gen)[:, 0].to(torch.int32)
    u, ul = torch.rand(T, generator=gen, device=DEV), torch.rand(rows, generator=gen, device=DEV)
    got = api.msa_tree_verify(target, tokens, _i32(offs), u, ul, draft=draft if drawn else None,
                              parents=None if chain else _i32(parents), max_path=max_path)
    f32 = lambda x: x.cpu().numpy()
    ref = drafts.verify(f32(target), f32(tokens), offs, f32(u), f32(ul),
                        f32(draft) if drawn else None, None if chain else parents, max_path)
    for a, b, what in zip(got, ref, ("path", "count", "last")):
        assert np.array_equal(a.cpu().numpy(), b), what
    return ref


@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("rows,trees,V,chain,sharp,skew", [
    (1, [6], 32000, True, 3.0, 0),
    (5, [1, 64, 7, 0, 30], 1009, False, 1.0, 3),
    (3, [9, 9, 9], 151, False, 0.3, 1),
    (2, [64, 12], 70001, False, 2.0, 2),
    (40, [5] * 40, 5000, False, 2.0, 0),
    (600, [3] * 600, 1, True, 1.0, 0),
    (200, [4] * 200, 7, False, 1.0, 1),
    (160, [1, 3, 5, 4] * 40, 49161, False, 2.0, 1),  # more CTAs than the chip holds
])
def test_verify_matches_the_definition(rows, trees, V, chain, sharp, skew, drawn):
    _verify_case(rows, trees, V, drawn, chain, rows + V, sharp, skew)


def test_verify_stops_at_max_path():
    _verify_case(30, [12] * 30, 50, True, True, 5, 0.1, max_path=3)
    _verify_case(30, [12] * 30, 50, False, True, 6, 3.0, max_path=1)


@pytest.mark.parametrize("parents", [[-1, 0, 0, 0], [-1, 0, 1, 1]])
def test_verify_keeps_the_targets_distribution(parents):
    gen, V, m, rows = _gen(21), 6, 4, 20000
    p = torch.softmax(1.5 * torch.randn(m, V, generator=gen, device=DEV), 1).repeat(rows, 1)
    q = torch.softmax(1.5 * torch.randn(m, V, generator=gen, device=DEV), 1).repeat(rows, 1)
    at = torch.arange(rows, device=DEV)[:, None] * m + _i32(parents).long().clamp(min=0)
    tokens = torch.multinomial(q[at.flatten()], 1, generator=gen)[:, 0].to(torch.int32)
    path, count, last = api.msa_tree_verify(
        p, tokens, _i32(range(0, rows * m + 1, m)), torch.rand(rows * m, generator=gen, device=DEV),
        torch.rand(rows, generator=gen, device=DEV), draft=q, parents=_i32(parents * rows), max_path=4)
    first = torch.where(count > 1, tokens.view(rows, m).gather(1, path[:, 1:2].long().clamp(min=0))[:, 0],
                        last)
    seen = np.bincount(first.cpu().numpy(), minlength=V)
    want = _np(p[0]) * rows
    # binomial counts: five standard deviations
    assert (np.abs(seen - want) <= 5 * np.sqrt(want)).all()


def test_verify_edges():
    V = 3000
    p = torch.zeros(4, V, device=DEV)
    p[0, 2999], p[1, 0], p[2, 1500] = 1, 1, 1
    tok, one = _i32([5, 2999, 0, 7]), torch.full((1,), 0.999999, device=DEV)
    zero = torch.zeros(1, device=DEV)
    run = lambda **kw: [x.tolist() for x in api.msa_tree_verify(
        p, tok, _i32([0, 3]) if "offs" not in kw else _i32(kw.pop("offs")),
        torch.full((4,), 0.5, device=DEV), kw.pop("ul", zero), max_path=4, **kw)]
    # one-hot targets keep the drafts that agree, with equal drafts or none of theirs
    for draft in (None, p):
        for ul in (zero, one):
            assert run(draft=draft, ul=ul) == [[[0, 1, 2, -1]], [3], [1500]]
    # a rejected draft that had all there was: the distribution itself is drawn from
    same = p.clone()
    same[0, 2999] = 0.25
    got = api.msa_tree_verify(same, tok, _i32([0, 2]), torch.full((4,), 0.5, device=DEV), zero,
                              draft=same * 4, max_path=2)
    assert [x.tolist() for x in got] == [[[0, -1]], [1], [2999]]
    # nothing to draw from, not a number, an infinity
    for bad in (0.0, float("nan"), float("inf")):
        x = torch.full((4, V), bad, device=DEV)
        got = api.msa_tree_verify(x, tok, _i32([0, 1]), zero.expand(4).contiguous(), zero, max_path=1)
        assert [v.tolist() for v in got] == [[[0]], [1], [-1]]
    # rows without tokens or with bad offsets
    for offs in ([0, 0], [0, 5], [-1, 2], [3, 2]):
        assert run(offs=offs) == [[[-1] * 4], [0], [-1]]
    many = torch.full((70, 4), 0.25, device=DEV)
    got = api.msa_tree_verify(many, _i32([0] * 70), _i32([0, 65, 70]), torch.zeros(70, device=DEV),
                              torch.zeros(2, device=DEV), max_path=5)
    assert got[1].tolist() == [0, 5] and got[2].tolist() == [-1, 0]
    # tokens outside the vocabulary and bad parents are not tried
    t = _i32([0, V, -1, 2999])
    got = api.msa_tree_verify(p, t, _i32([0, 4]), torch.zeros(4, device=DEV), zero,
                              parents=_i32([0, 0, 0, 3]), max_path=4)
    assert [x.tolist() for x in got] == [[[0, -1, -1, -1]], [1], [2999]]
    # u_last of 1 or more takes the last token with anything in it
    flat = torch.full((1, 5), 0.2, device=DEV)
    flat[0, 4] = 0
    got = api.msa_tree_verify(flat, _i32([0]), _i32([0, 1]), zero, torch.full((1,), 1.5, device=DEV))
    assert got[2].tolist() == [3]


# ------------------------------------------------------------------ compaction
@pytest.mark.parametrize("dt,dim,kv,S,head_major", [(BF, 128, 4, 64, False), (FP, 64, 9, 1, False),
                                                    (BF, 64, 64, 16, True), (FP, 128, 1, 1024, False)])
def test_compact_matches_the_definition(dt, dim, kv, S, head_major):
    rng, gen = np.random.default_rng(S), _gen(S)
    trees = [1, 64, 64, 5, 9, 2, 33]
    lens = [0, 100, 63, 1000, 7, 128, 0]
    pool, table = _pages(rng, [n + m for n, m in zip(lens, trees)], S)
    kc, vc = (_pool(gen, pool, S, kv, dim, dt, head_major) for _ in range(2))
    count = [1, 64, 40, 0, 4, 1, 11]
    path = np.full((7, 64), -1)
    for r, (c, m) in enumerate(zip(count, trees)):
        path[r, :c] = np.sort(rng.choice(m, c, replace=False))
    want = [drafts.compact(_np(x), table, lens, path, count) for x in (kc, vc)]
    cache = api.PagedCache(kc, vc)
    got = api.msa_paged_compact(cache, _i32(table), _i32(lens), _i32(path), _i32(count))
    assert got.tolist() == [n + c for n, c in zip(lens, count)]
    assert api.msa_paged_read_status(cache) == 0
    assert np.array_equal(_np(kc), want[0]) and np.array_equal(_np(vc), want[1])


def test_compact_leaves_bad_rows_alone():
    gen, S = _gen(31), 4
    kc, vc = (_randn(gen, (12, S, 2, 64), BF) for _ in range(2))
    before = kc.clone(), vc.clone()
    cache = api.PagedCache(kc, vc)
    table = np.arange(12).reshape(2, 6)
    for path, count, lens, code in (
            ([[0, 2, 2]], [3], [5], 12), ([[3, 2, 4]], [3], [5], 12), ([[-1, 2, 4]], [3], [5], 12),
            ([[0, 2, 4]], [4], [5], 12), ([[0, 2, 4]], [-1], [5], 12),
            ([[0, 2, 4]], [3], [20], 11), ([[0, 2, 4]], [3], [-1], 11),
            ([[0, 2, 1 << 30]], [3], [5], 11), ([[0, 2, 2 ** 31 - 1]], [3], [2 ** 31 - 1], 11)):
        # the row beside it is moved all the same
        got = api.msa_paged_compact(cache, _i32(table), _i32(lens + [3]), _i32(path + [[1, 2, 3]]),
                                    _i32(count + [3]))
        assert got.tolist() == [lens[0], 6]
        assert api.msa_paged_read_status(cache, clear=True) == code
        assert torch.equal(kc[:6], before[0][:6]) and torch.equal(vc[:6], before[1][:6])
    bad = table.copy()
    bad[0, 2] = 12
    got = api.msa_paged_compact(cache, _i32(bad), _i32([5, 3]), _i32([[0, 2, 4]] * 2), _i32([3, 0]))
    assert got.tolist() == [5, 3] and api.msa_paged_read_status(cache, clear=True) == 11
    assert torch.equal(kc[:6], before[0][:6])


# ------------------------------------------------------------------ a step of all of them
@pytest.mark.parametrize("sparse", [False, True])
def test_a_step_with_drafts_as_served(sparse):
    """Norm and rotation by depth, append, selection, attention, verification,
    compaction, index: afterwards the cache is what it would be had the kept tokens
    been appended one by one, and the next token's attention is the same."""
    rng, gen = np.random.default_rng(41), _gen(41)
    kv, heads, dim, S, V = 4, 64, 128, 64, 500
    lens, trees = [2500, 130, 3000], [9, 6, 12]
    rows, T = 3, sum(trees)
    offs = np.concatenate([[0], np.cumsum(trees)])
    pool, table = _pages(rng, [n + m + 2 for n, m in zip(lens, trees)], S)
    kc, vc = (_randn(gen, (pool, S, kv, dim), BF) for _ in range(2))
    keys = torch.zeros(pool, S, 4, 64, dtype=BF, device=DEV)
    cache = api.PagedCache(kc, vc)
    index = api.PagedIndex(keys, torch.zeros(api.paged_means_shape(pool, S, 4, 64), device=DEV))
    past = _randn(gen, (sum(lens), 4, 64), BF)
    tab = _i32(table)
    api.msa_paged_index(index, past, tab, _i32(np.concatenate([[0], np.cumsum(lens)])), _i32([0] * rows))
    old = kc.clone(), vc.clone()

    parents = [p for m in trees for p in _random_parents(rng, m)]
    row = np.repeat(np.arange(rows), trees)
    depth = np.zeros(T, int)
    for t in range(T):
        p = parents[t]
        depth[t] = depth[offs[row[t]] + p] + 1 if p >= 0 else 0
    qkv = _randn(gen, (T, heads + 2 * kv, dim), BF)
    iq, ik = _randn(gen, (T, 4, 64), BF), _randn(gen, (T, 4, 64), BF)
    w, freq = torch.ones(dim, device=DEV), _freq(64)
    pos = _i32(np.asarray(lens)[row] + depth)
    L = _i32(lens)
    q, k = api.msa_norm_rope(qkv[:, :heads], qkv[:, heads:heads + kv], w, w, pos, freq)
    v = qkv[:, heads + kv:]
    api.msa_paged_append(cache, k, v, tab, _i32(offs), L)
    q2k = None
    if sparse:
        q2k = api.msa_paged_select(index, iq, tab[torch.as_tensor(row, device=DEV)].contiguous(),
                                   L[torch.as_tensor(row, device=DEV)].contiguous())
    o, lse = api.msa_paged_tree(cache, q, tab, _i32(offs), L, dim ** -0.5, parents=_i32(parents),
                                q2k=q2k)
    ref = drafts.tree(_np(kc), _np(vc), _np(q), table, offs, lens, parents, float(np.float32(dim ** -0.5)),
                      None if q2k is None else q2k.cpu().numpy(), HALF[BF], TINY[BF])
    _within(_np(o), ref[0], ref[2], "O")
    _within(_np(lse), ref[1], ref[3], "LSE")
    # a stand-in for the model's head
    probs = torch.softmax(o.float().flatten(1)[:, :V] * 30, 1)
    tokens = torch.randint(0, V, (T,), generator=gen, device=DEV).to(torch.int32)
    for t in range(T):  # likely drafts, so that some stay
        if parents[t] >= 0:
            tokens[t] = probs[offs[row[t]] + parents[t]].argmax()
    path, count, last = api.msa_tree_verify(probs, tokens, _i32(offs), torch.rand(T, generator=gen, device=DEV),
                                            torch.rand(rows, generator=gen, device=DEV),
                                            parents=_i32(parents), max_path=12)
    new_len = api.msa_paged_compact(cache, tab, L, path, count)
    torch.cuda.synchronize()
    c, at = count.tolist(), path.cpu().numpy()
    assert max(c) > 2 and new_len.tolist() == [n + x for n, x in zip(lens, c)]
    kept = [offs[r] + at[r, i] for r in range(rows) for i in range(c[r])]
    kept_t = torch.as_tensor(kept, device=DEV)
    o2 = _i32(np.concatenate([[0], np.cumsum(c)]))
    api.msa_paged_index(index, ik[kept_t].contiguous(), tab, o2, L)
    # one by one: positions follow one another, so the cache's own rotation gives the keys
    want = api.PagedCache(*(x.clone() for x in old))
    plain, _ = api.msa_norm_rope(qkv[:, heads:heads + kv], qkv[:, heads:heads + kv], w, w)
    api.msa_paged_append(want, plain[kept_t].contiguous(), v[kept_t].contiguous(), tab, o2, L,
                         inv_freq=freq)
    for r in range(rows):
        n = lens[r] + c[r]
        j = torch.arange(n, device=DEV)
        place = tab[r].long()[j // S], j % S
        assert torch.equal(cache.v[place], want.v[place])
        # normed, rounded, then rotated and rounded again: two half steps more
        a, b = cache.k[place].float(), want.k[place].float()
        assert torch.equal(a[:lens[r]], b[:lens[r]])
        size = torch.as_tensor(drafts.pair_size(_np(b), 64, False), device=DEV)
        assert ((a - b).abs() <= 3 * HALF[BF] * size).all()
    # the next token: decode and a tree of one see the same
    q1 = _randn(gen, (rows, heads, dim), BF)
    k1, v1 = _randn(gen, (rows, kv, dim), BF), _randn(gen, (rows, kv, dim), BF)
    one = _i32(range(rows + 1))
    api.msa_paged_append(cache, k1, v1, tab, one, new_len)
    d, dl = api.msa_paged_decode(cache, q1, tab, new_len + 1, dim ** -0.5)
    t, tl = api.msa_paged_tree(cache, q1, tab, one, new_len, dim ** -0.5)
    ref = drafts.tree(_np(kc), _np(vc), _np(q1), table, list(range(rows + 1)), new_len.tolist(), None,
                      float(np.float32(dim ** -0.5)), None, HALF[BF], TINY[BF])
    for a, b in ((d, dl), (t, tl)):
        _within(_np(a), ref[0], ref[2], "O")
        _within(_np(b), ref[1], ref[3], "LSE")
    for x in (cache, index):
        assert api.msa_paged_read_status(x) == 0


def test_binding_refuses_mismatches():
    z = lambda *s, dt=BF: torch.zeros(*s, dtype=dt, device=DEV)
    w = torch.ones(64, device=DEV)
    q = z(4, 8, 64)
    cache = api.PagedCache(z(4, 16, 2, 64), z(4, 16, 2, 64))
    tab, offs, lens = _i32([[0, 1]]), _i32([0, 4]), _i32([3])
    for call, err in [
        (lambda: api.msa_norm_rope(q, z(3, 2, 64), w, w), ValueError),
        (lambda: api.msa_norm_rope(q, z(4, 2, 64, dt=FP), w, w), TypeError),
        (lambda: api.msa_norm_rope(q.float(), q, w, w), TypeError),
        (lambda: api.msa_norm_rope(q, q, w.half(), w.half()), TypeError),
        (lambda: api.msa_norm_rope(q, q, w, w.bfloat16()), TypeError),
        (lambda: api.msa_norm_rope(q, q, w, w, None, _freq(16)), ValueError),
        (lambda: api.msa_norm_rope(q, q, w, w, eps=-1.0), api.MSAError),
        (lambda: api.msa_norm_rope(z(4, 8, 32), z(4, 8, 32), w[:32], w[:32]), api.MSAError),
        (lambda: api.msa_norm_rope(q.transpose(0, 1), q, w, w), ValueError),
        (lambda: api.msa_norm_rope_backward(q, q[:3], q, q, w, w), ValueError),
        (lambda: api.msa_paged_tree(cache, z(4, 3, 64), tab, offs, lens, 0.1), api.MSAError),
        (lambda: api.msa_paged_tree(cache, z(4, 34, 64), tab, offs, lens, 0.1), api.MSAError),
        (lambda: api.msa_paged_tree(cache, q.half(), tab, offs, lens, 0.1), TypeError),
        (lambda: api.msa_paged_tree(cache, q, tab, offs, lens, 0.0), api.MSAError),
        (lambda: api.msa_paged_tree(cache, q, tab, offs, lens, 0.1, parents=_i32([0])), ValueError),
        (lambda: api.msa_paged_tree(cache, q, tab, offs, lens, 0.1, workspace=z(16, dt=torch.uint8)),
         api.MSAError),
        (lambda: api.msa_tree_verify(q[0].float(), _i32([0] * 8), offs, w[:8], w[:1], max_path=65),
         ValueError),
        (lambda: api.msa_tree_verify(q[0], _i32([0] * 8), offs, w[:8], w[:1]), TypeError),
        (lambda: api.msa_tree_verify(q[0].float(), _i32([0] * 7), offs, w[:8], w[:1]), ValueError),
        (lambda: api.msa_tree_verify(q[0].float().t(), _i32([0] * 64), offs, w, w[:1]), ValueError),
        (lambda: api.msa_paged_compact(cache, tab, lens, _i32([[0] * 65]), _i32([1])), api.MSAError),
        (lambda: api.msa_paged_compact(cache, tab, lens, _i32([[0]]), _i32([1]), new_len=lens),
         api.MSAError),
    ]:
        with pytest.raises(err):
            call()
