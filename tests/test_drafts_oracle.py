"""The fp64 statements of the norm and of the drafted tokens' operators
(oracle/drafts.py) against other statements of the same: differences, torch's
autograd, a mask built from the definition, and the distribution that
verification is to keep."""
import itertools

import numpy as np
import pytest
import torch

from oracle import drafts, paged


@pytest.mark.parametrize("inter", [False, True])
def test_norm_gradient_against_differences_and_autograd(inter):
    rng = np.random.default_rng(1)
    x, dy, w = rng.normal(size=(3, 2, 16)), rng.normal(size=(3, 2, 16)), rng.normal(size=16)
    pos, freq = np.array([0, 5, 70000]), 10.0 ** -np.arange(4.0)
    dx, dw, _ = drafts.norm_rope_back(dy, x, w, pos, freq, inter, 0.1)
    h = 1e-6
    for at in itertools.product(range(3), range(2), (0, 3, 6, 15)):
        e = np.zeros_like(x)
        e[at] = h
        lo, hi = (drafts.norm_rope(x + s * e, w, pos, freq, inter, 0.1) for s in (-1, 1))
        # central differences of values of order 1: h^2 times a third derivative below
        # 100, and roundings 2^-52 / h of the sum of 96 terms
        assert abs(((hi - lo) * dy).sum() / (2 * h) - dx[at]) < 1e-7
    for c in (0, 9):
        e = np.zeros_like(w)
        e[c] = h
        lo, hi = (drafts.norm_rope(x, w + s * e, pos, freq, inter, 0.1) for s in (-1, 1))
        assert abs(((hi - lo) * dy).sum() / (2 * h) - dw[c]) < 1e-7
    # against torch's autograd, the turn as a complex product
    X = torch.tensor(x, requires_grad=True)
    W = torch.tensor(w, requires_grad=True)
    y = X / torch.sqrt((X ** 2).mean(-1, keepdim=True) + 0.1) * W
    i = torch.arange(4)
    lo, hi = (2 * i, 2 * i + 1) if inter else (i, i + 4)
    z = torch.complex(y[..., lo], y[..., hi]) * torch.exp(
        1j * torch.tensor(pos)[:, None, None] * torch.tensor(freq))
    out = y.clone()
    out[..., lo], out[..., hi] = z.real, z.imag
    assert np.allclose(out.detach().numpy(), drafts.norm_rope(x, w, pos, freq, inter, 0.1), atol=1e-12)
    out.backward(torch.tensor(dy))
    assert np.allclose(X.grad.numpy(), dx, atol=1e-12) and np.allclose(W.grad.numpy(), dw, atol=1e-12)


def test_tree_attention_against_a_masked_softmax_and_decode():
    rng = np.random.default_rng(2)
    S, kv, share, dim, n = 4, 2, 3, 8, 300
    parents = [-1, 0, 0, 1, 2, -1]
    m = len(parents)
    pages = -(-(n + m) // S)
    K, V = rng.normal(size=(2, pages + 2, S, kv, dim))
    table = rng.permutation(pages + 2)[None, :pages]
    q = rng.normal(size=(m, kv * share, dim))
    q2k = np.full((kv, m, 16), -1)
    q2k[:, :, 0] = rng.integers(0, 3, (kv, m))
    q2k[:, :, 1] = 0
    on = {0: [0], 1: [0, 1], 2: [0, 2], 3: [0, 1, 3], 4: [0, 2, 4], 5: [5]}
    for slots in (None, q2k):
        O, L, _, _ = drafts.tree(K, V, q, table, [0, m], [n], parents, 0.3, slots)
        k, v = paged.gather(K, table[0], 0, n + m), paged.gather(V, table[0], 0, n + m)
        for j, h in itertools.product(range(m), range(kv * share)):
            g = h // share
            mask = np.full(n + m, -np.inf)
            mask[:n] = 0 if slots is None else np.where(
                np.isin(np.arange(n) // 128, slots[g, j][:2]), 0, -np.inf)
            mask[[n + i for i in on[j]]] = 0
            s = torch.tensor(0.3 * (k[:, g] @ q[j, h]) + mask)
            assert np.allclose(torch.softmax(s, 0).numpy() @ v[:, g], O[j, h], atol=1e-12)
            assert abs(float(torch.logsumexp(s, 0)) - L[j, h]) < 1e-12
    # a chain is one decode row for each token
    O, L, _, _ = drafts.tree(K, V, q, table, [0, m], [n], None, 0.3)
    for j in range(m):
        o, l = paged.decode(K, V, q[j:j + 1], table, [n + j + 1], 0.3)
        assert np.allclose(o[0], O[j], atol=1e-12) and np.allclose(l[0], L[j], atol=1e-12)


@pytest.mark.parametrize("drawn", [True, False])
@pytest.mark.parametrize("parents", [[-1, 0, 0, 0], [-1, 0, 1, 2], [-1, 0, 0, 1]])
def test_verification_keeps_the_targets_distribution(parents, drawn):
    """The first token behind token 0 - a draft that stays, or the drawn one - has
    the target's distribution, whatever the drafting model's."""
    rng = np.random.default_rng(len(parents) + sum(parents) + drawn)
    V, m, runs = 4, len(parents), 4000
    p, q = (rng.dirichlet(np.ones(V), size=m).astype(np.float32) for _ in range(2))
    seen = np.zeros(V)
    for _ in range(runs):
        # drafts drawn from q behind their parent, or the two best of another model
        tokens = [0] + [int(rng.choice(V, p=q[a] / q[a].sum(dtype=np.float64))) if drawn
                        else int(np.argsort(-q[a])[parents[1:j + 1].count(a)])
                        for j, a in enumerate(parents[1:])]
        path, count, last = drafts.verify(p, tokens, [0, m], rng.random(m, np.float32),
                                          rng.random(1, np.float32), q if drawn else None, parents)
        seen[tokens[path[0][1]] if count[0] > 1 else last[0]] += 1
    # binomial counts: five standard deviations
    assert (np.abs(seen - runs * p[0]) <= 5 * np.sqrt(runs * p[0] * (1 - p[0])) + 1).all()


def test_verification_by_hand():
    p = np.array([[.5, .25, .25, 0], [0, 0, 1, 0], [.25, .25, .25, .25]], np.float32)
    q = np.array([[.25, .5, .25, 0], [.5, .5, 0, 0], [0, 0, 0, 1]], np.float32)
    tok = [9, 1, 0]
    # a chain of two: token 1 stays if u < .5, token 0 behind it never (p = 0)
    run = lambda u, last, **kw: [x.tolist() for x in drafts.verify(p, tok, [0, 3], u, [last], **kw)]
    assert run([0, .49, 0], .5, draft=q, max_path=3) == [[[0, 1, -1]], [2], [2]]
    # not kept: what is left is (.25, 0, 0, 0)
    assert run([0, .5, 0], .99, draft=q, max_path=2) == [[[0, -1]], [1], [0]]
    # a tree: 1 fails, then 0 is kept (left: all of it on 0, q(0) = .25, any u)
    assert run([0, .5, .99], .7, draft=q, parents=[-1, 0, 0], max_path=3) == [[[0, 2, -1]], [2], [2]]
    # not drawn: 1 fails (u >= .25), 0 is kept if u * .75 < .5
    assert run([0, .25, .66], .7, parents=[-1, 0, 0], max_path=3) == [[[0, 2, -1]], [2], [2]]
    assert run([0, .25, .67], .7, parents=[-1, 0, 0], max_path=3) == [[[0, -1, -1]], [1], [2]]
    # the walk ends at max_path
    assert run([0, 0, 0], .3, draft=q, max_path=1) == [[[0]], [1], [0]]


def test_compact_by_hand():
    c = np.arange(12.0).reshape(3, 4, 1, 1)
    got = drafts.compact(c, [[2, 0, 1]], [2], [[0, 2, 3, 5]], [4])
    # row: 8 9 10 11 | 0 1 2 3 | 4 5 6 7; slots 2, 4, 5, 7 go to 2, 3, 4, 5
    assert got[[2, 0, 1]].ravel().tolist() == [8, 9, 10, 0, 1, 3, 2, 3, 4, 5, 6, 7]
