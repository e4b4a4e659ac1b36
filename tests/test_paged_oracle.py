"""The paged-cache oracle pinned: closed forms, and agreement with the
training oracle where both compute the same thing (no GPU)."""
import math

import numpy as np
import pytest
import torch

import oracle
from oracle import paged

RNG = np.random.default_rng


def _cache(rng, lens, S, heads, dim, extra=2):
    """Shuffled pages, a table with -1 behind each row's pages."""
    need = [-(-n // S) for n in lens]
    pool = sum(need) + extra
    order = rng.permutation(pool)
    table = np.full((len(lens), max(need) + 1), -1, dtype=np.int64)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = order[at:at + n]
        at += n
    return rng.standard_normal((pool, S, heads, dim)), table


def test_rotation_by_known_angles():
    x = np.arange(1.0, 9.0).reshape(1, 1, 8)
    quarter = [math.pi / 2, math.pi]  # per position
    y = paged.rotate(x, [1], quarter, False)   # pairs (0, 2), (1, 3); channels 4 .. stay
    assert np.allclose(y[0, 0], [-3, -2, 1, -4, 5, 6, 7, 8])
    y = paged.rotate(x, [1], quarter, True)    # pairs (0, 1), (2, 3)
    assert np.allclose(y[0, 0], [-2, 1, -3, -4, 5, 6, 7, 8])
    assert np.allclose(paged.rotate(x, [4], quarter, True), x)


def test_rotation_keeps_products_of_equal_distance():
    rng = RNG(1)
    q, k = rng.standard_normal((1, 1, 16)), rng.standard_normal((1, 1, 16))
    f = 10000.0 ** (-np.arange(8) / 8)
    for inter in (False, True):
        dots = [float((paged.rotate(q, [p + 7], f, inter) * paged.rotate(k, [p], f, inter)).sum())
                for p in (0, 5, 1000)]
        assert np.allclose(dots, dots[0])


def test_append_places_tokens_and_nothing_else():
    rng = RNG(2)
    lens = [5, 9]
    kc, table = _cache(rng, lens, 4, 2, 8)
    vc = rng.standard_normal(kc.shape)
    k, v = rng.standard_normal((4, 2, 8)), rng.standard_normal((4, 2, 8))
    k2, v2, _, k_rot = paged.append(kc, vc, k, v, table, [0, 1, 3], [4, 7])
    assert np.array_equal(k2[table[0, 1], 0], k[0]) and np.array_equal(v2[table[1, 1], 3], v[1])
    assert np.array_equal(k2[table[1, 2], 0], k[2])
    assert (k2 != kc).any((2, 3)).sum() == 3 and np.isnan(k_rot[3]).all()


def test_means_of_blocks_match_the_scores_of_the_training_oracle():
    rng = RNG(3)
    n, S = 128 * 18 + 40, 32
    ik = rng.integers(-8, 9, (n, 4, 16)) / 4.0
    iq = rng.integers(-8, 9, (n, 4, 16)) / 4.0
    keys, table = _cache(rng, [n], S, 4, 16)
    means = np.full((keys.shape[0], 4, 16), np.nan)
    # in three calls, cut inside blocks
    for a, b in ((0, 200), (200, 1000), (1000, n)):
        keys, means = paged.index(keys, means, ik[a:b], table, [0, b - a], [a])
    t = n - 1
    ref = oracle.block_scores(torch.from_numpy(iq).bfloat16(), torch.from_numpy(ik).bfloat16(),
                              np.array([0, n]), [[g, t] for g in range(4)])  # exact in bf16
    for g in range(4):
        for v in range(19):
            last = min(v * 128 + 127, t)
            at = paged.mean_slot(table[0, last // S], last, S)
            assert np.isclose(means[at, g] @ iq[t, g], ref[g, v])


def test_decode_matches_the_training_oracle_on_a_document():
    rng = RNG(4)
    n = 300
    q, k, v = (rng.standard_normal((n, h, 128)) for h in (64, 4, 4))
    q2k = np.full((4, n, 16), -1, dtype=np.int32)
    for g in range(4):
        q2k[g, :, 3] = 0
        q2k[g, 256:, 5] = 2 - (g % 2)
    P = oracle.Problem(q, k, v, q2k, np.array([0, n], np.int32), 0.07)
    O, L = P.forward(np.array([n - 1]))
    kc, table = _cache(rng, [n], 16, 4, 128)
    vc = np.zeros_like(kc)
    kc, vc, _, _ = paged.append(kc, vc, k, v, table, [0, n], [0])
    o, lse = paged.decode(kc, vc, q[n - 1:], table, [n], 0.07, q2k[:, n - 1:])
    assert np.allclose(o[0], O[0]) and np.allclose(lse[0], L[0])


def test_decode_equal_scores_average_the_values():
    kc = np.zeros((3, 2, 1, 4))
    vc = np.arange(24.0).reshape(3, 2, 1, 4)
    table = np.array([[2, 0, -1]])
    o, lse = paged.decode(kc, vc, np.ones((1, 2, 4)), table, [3], 1.0)
    assert np.allclose(o[0, 0], (vc[2, 0, 0] + vc[2, 1, 0] + vc[0, 0, 0]) / 3)
    assert np.allclose(lse, math.log(3))
    o, lse = paged.decode(kc, vc, np.ones((1, 2, 4)), table, [0], 1.0)
    assert (o == 0).all() and (lse == -np.inf).all()


def test_striped_rows_are_what_the_oracle_gives():
    for levels in (np.zeros(8), np.arange(8) / 4):
        table = np.array([[3, 0, 7, 7, 1, 5, 2]])
        k = np.ones((8, 4, 2, 8)) * levels[:, None, None, None] / 8
        v = paged.striped_values(8, 4, 2, 8)
        for n in (1, 4, 23, 28):
            o, lse = paged.decode(k, v, np.ones((1, 6, 8)), table, [n], 1.0)
            O, L = paged.striped(table[0], n, 4, levels, 2, 8)
            assert np.allclose(o[0], np.repeat(O, 3, axis=0)) and np.allclose(lse, L)


@pytest.mark.parametrize("name", paged.STRIPED_CASES)
@pytest.mark.parametrize("times", [0, 2])
def test_a_part_of_a_striped_row_lost_or_counted_twice_is_out_of_bounds(name, times):
    """Mistakes of the split over 304 thread blocks, planted here: with equal
    levels one tile of a warp in O and in LSE, else a run in O."""
    case = paged.STRIPED_CASES[name]
    dt, dim, _, _, S, lens, span = case
    step, tiny = (2.0 ** -8, 2.0 ** -134) if dt == "bf16" else (2.0 ** -11, 2.0 ** -25)
    table, levels = paged.striped_rows(case)
    for r, n in enumerate(lens):
        if n < 10000:
            continue
        O, L = paged.striped(table[r], n, S, levels, 1, dim)
        BO, BL = paged.striped_bounds(O, L, n, levels, dim, step, tiny)
        part = n // 304 if span else 2048 // dim
        for at in range(0, n - part, max(n // 150 // part, 1) * part):
            count = np.ones(n)
            count[at:at + part] = times
            o, lse = paged.striped(table[r], n, S, levels, 1, dim, count)
            assert (np.abs(o - O) > BO).any(), at
            assert span or abs(lse - L) > BL, at
