"""The paged-cache operators on the GPU against their fp64 statement
(oracle/paged.py), and against the training path where both compute the same.

Error bounds are element-wise and derived (u = 2^-24, h = half a step of the
cache's type relative to the value: bf16 2^-8, fp16 2^-11):
  rotation  an angle's turns are rounded once to fp32 (2 f <= 1: pi 2^-25) and
            sine and cosine are good to 2 u: 2^-22 absolute; with the products'
            and the sum's roundings d = 2^-21 (|x| + |y|), then h (|result| + d)
  means     n - 1 sums and a division: (n + 1) u mean|x|
  attention oracle.paged.decode_bounds
"""
import numpy as np
import pytest
import torch

import oracle
from block_sparse_gqa_msa_gb300 import api, inputs
from oracle import paged
from tests.helpers import check_lse, check_o

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


def _pages(rng, lens, S, spare=3, width=None):
    """(pool size, table [rows, width] with -1 where a row has no page)."""
    need = [-(-n // S) for n in lens]
    pool = sum(need) + spare
    order = rng.permutation(pool)
    table = np.full((len(lens), width or max(max(need), 1) + 2), -1, dtype=np.int64)
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = order[at:at + n]
        at += n
    return pool, table


def _randn(gen, shape, dtype=torch.float32):
    return torch.randn(shape, generator=gen, device=DEV).to(dtype)


def _pool(gen, pool, S, heads, dim, dtype, head_major=False):
    if head_major:
        return _randn(gen, (pool, heads, S, dim), dtype).transpose(1, 2)
    return _randn(gen, (pool, S, heads, dim), dtype)


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _within(got, ref, bound, what):
    over = np.abs(got - ref) - bound
    assert not np.isnan(got).any(), f"{what}: NaN"
    worst = np.unravel_index(np.argmax(over), over.shape)
    assert over[worst] <= 0, (f"{what}: {got[worst]} for {ref[worst]} at {worst}, bound "
                              f"{bound[worst]:.3e}")


def _rot_bound(x, ref, rot, inter, dt):
    """Bound of a rotated tensor; channels past rot are copied exactly."""
    part = np.array(x)
    half = rot // 2
    if inter:
        part[..., 0:rot:2], part[..., 1:rot:2] = x[..., 1:rot:2], x[..., 0:rot:2]
    else:
        part[..., :half], part[..., half:rot] = x[..., half:rot], x[..., :half]
    d = 2.0 ** -21 * (np.abs(x) + np.abs(part))
    b = HALF[dt] * (np.abs(ref) + d) + d + TINY[dt]
    b[..., rot:] = 0
    return b


# ------------------------------------------------------------------ append
def _append_case(dt, dim, kv, heads, S, rot, inter, fresh, start, pad, seed, head_major=False,
                 fused=False, theta=10000.0):
    rng, gen = np.random.default_rng(seed), _gen(seed)
    pool, table = _pages(rng, [f + s for f, s in zip(fresh, start)], S)
    offs = np.concatenate([[0], np.cumsum(fresh)])
    T = int(offs[-1]) + pad
    kc, vc = (_pool(gen, pool, S, kv, dim, dt, head_major) for _ in range(2))
    if fused:  # one projection's output, sliced
        qkv = _randn(gen, (T, heads + 2 * kv, dim), dt)
        q, k, v = qkv[:, :heads], qkv[:, heads:heads + kv], qkv[:, heads + kv:]
    else:
        q, k, v = (_randn(gen, (T, h, dim), dt) for h in (heads, kv, kv))
    freq = torch.tensor(theta ** (-np.arange(0, rot, 2) / max(rot, 1)), dtype=torch.float32,
                        device=DEV) if rot else None
    ref = paged.append(_np(kc), _np(vc), _np(k), _np(v), table, offs, start,
                       None if freq is None else _np(freq), inter, _np(q))
    cache = api.PagedCache(kc, vc)
    k_out = torch.full((T, kv, dim), 7.0, dtype=dt, device=DEV)
    q_out = torch.full((T, heads, dim), 7.0, dtype=dt, device=DEV)
    before = _np(kc)
    api.msa_paged_append(cache, k, v, _i32(table), _i32(offs), _i32(start), inv_freq=freq,
                         interleaved=inter, q=q, q_out=q_out, k_out=k_out)
    torch.cuda.synchronize()
    assert api.msa_paged_read_status(cache) == 0
    kc2, vc2, q_ref, k_ref = ref
    n = int(offs[-1])
    assert (_np(q_out)[n:] == 7).all() and (_np(k_out)[n:] == 7).all()
    _within(_np(q_out)[:n], q_ref[:n], _rot_bound(_np(q)[:n], q_ref[:n], rot, inter, dt), "q")
    _within(_np(k_out)[:n], k_ref[:n], _rot_bound(_np(k)[:n], k_ref[:n], rot, inter, dt), "k")
    assert np.array_equal(_np(vc), vc2)
    # the cache holds exactly the rotated keys handed back, and is unchanged elsewhere
    want = before
    for r in range(len(start)):
        for t in range(offs[r], offs[r + 1]):
            p = start[r] + t - offs[r]
            want[table[r, p // S], p % S] = _np(k_out)[t]
    assert np.array_equal(_np(kc), want)


@pytest.mark.parametrize("dt,dim,kv,heads,S,rot,inter,fused,head_major", [
    (BF, 128, 4, 64, 128, 64, False, False, False),
    (BF, 128, 4, 64, 16, 128, True, True, False),
    (FP, 64, 8, 24, 32, 64, False, False, True),
    (FP, 128, 1, 7, 1, 32, True, True, True),
    (BF, 64, 3, 3, 1024, 16, False, True, False),
    (BF, 128, 2, 2, 64, 0, False, False, False),
])
def test_append_matches_fp64(dt, dim, kv, heads, S, rot, inter, fused, head_major):
    _append_case(dt, dim, kv, heads, S, rot, inter, [1, 0, 130, 3, 17], [5, 9, 0, 1000, 127], 4,
                 seed=S + rot, fused=fused, head_major=head_major)


def test_append_one_token_per_row_many_rows():
    rng = np.random.default_rng(5)
    start = rng.integers(0, 40, 1500).tolist()
    fresh = (rng.random(1500) < 0.9).astype(int).tolist()
    _append_case(BF, 64, 1, 2, 8, 32, False, fresh, start, 1, seed=6)


def test_append_one_token():
    _append_case(BF, 128, 4, 64, 64, 64, False, [1], [0], 0, seed=7)
    _append_case(FP, 128, 4, 64, 64, 64, True, [1], [777], 0, seed=8)


@pytest.mark.parametrize("dt,dim,kv,heads,S,rot,inter,fused", [
    (BF, 64, 1, 1, 64, 64, False, False), (FP, 64, 3, 3, 16, 16, True, True),
    (BF, 128, 2, 8, 128, 64, False, True), (FP, 128, 1, 6, 8, 128, True, False)])
def test_append_many_tokens_of_few_heads(dt, dim, kv, heads, S, rot, inter, fused):
    # rows that begin and end anywhere in a group of tokens, empty rows, padding behind the last
    _append_case(dt, dim, kv, heads, S, rot, inter, [1, 0, 2003, 1, 3, 0, 2501, 2], [5, 9, 0, 77, 1,
                 3, 127, 64], 13, seed=21 + dim, fused=fused, head_major=False)


def test_append_bad_places_among_many_tokens():
    gen = _gen(22)
    S, T = 16, 1600
    kc, vc = (_pool(gen, 101, S, 1, 64, BF) for _ in range(2))
    k, v = (_randn(gen, (T, 1, 64), BF) for _ in range(2))
    k0, v0 = kc.clone(), vc.clone()
    table = torch.randperm(101, generator=gen, device=DEV)[:100].to(torch.int32)[None]
    bad = [3, 4, 50, 99]
    table[0, bad] = _i32([-1, 101, 2**31 - 1, -2**31])
    cache = api.PagedCache(kc, vc)
    k_out = torch.full((T, 1, 64), 9.0, dtype=BF, device=DEV)
    api.msa_paged_append(cache, k, v, table, _i32([0, T - 1]), _i32([1]), k_out=k_out)
    assert api.msa_paged_read_status(cache) == 11
    for t in range(T - 1):
        pg, slot = divmod(t + 1, S)
        if pg in bad:
            assert bool((k_out[t] == 9).all())
        else:
            k0[table[0, pg].item(), slot], v0[table[0, pg].item(), slot] = k[t], v[t]
    assert torch.equal(kc, k0) and torch.equal(vc, v0) and bool((k_out[T - 1] == 9).all())
    fine = [t for t in range(T - 1) if (t + 1) // S not in bad]
    assert torch.equal(k_out[fine], k[fine])


@pytest.mark.parametrize("pad", [3, 1500])
def test_append_padding_may_hold_anything(pad):
    # beside few tokens and beside many (several to a thread block)
    gen = _gen(63)
    kc, vc = (torch.zeros(4, 16, 1, 64, dtype=FP, device=DEV) for _ in range(2))
    q, k, v = (_randn(gen, (5 + pad, h, 64), FP) for h in (2, 1, 1))
    for x, bad in ((q, float("nan")), (k, float("inf")), (v, float("nan"))):
        x[5:] = bad
    cache = api.PagedCache(kc, vc)
    outs = [torch.full_like(x, 7.0) for x in (q, k)]
    api.msa_paged_append(cache, k, v, _i32([[3, 1], [0, 2]]), _i32([0, 2, 5]), _i32([15, 14]),
                         inv_freq=torch.rand(16, generator=gen, device=DEV), q=q, q_out=outs[0],
                         k_out=outs[1])
    assert api.msa_paged_read_status(cache) == 0
    for x in (kc, vc, *outs):
        assert bool(x.isfinite().all())
    assert all(bool((x[5:] == 7).all()) for x in outs)
    for c, new in ((kc, outs[1]), (vc, v)):
        want = torch.zeros_like(c)
        for t, (pg, slot) in enumerate(((3, 15), (1, 0), (0, 14), (0, 15), (2, 0))):
            want[pg, slot] = new[t]
        assert torch.equal(c, want)


def test_append_wide_tokens_take_several_rounds():
    _append_case(BF, 128, 64, 256, 16, 128, False, [3], [2], 0, seed=9)


def test_append_far_positions():
    # every entry of the table names the same few pages: only the last position is written
    S, pos = 1024, [1_000_003, 99_999_999]
    gen = _gen(11)
    kc, vc = (_pool(gen, 4, S, 2, 128, BF) for _ in range(2))
    q, k, v = (_randn(gen, (2, h, 128), BF) for h in (4, 2, 2))
    width = max(pos) // S + 1
    table = torch.zeros(2, width, dtype=torch.int32, device=DEV)
    table[1] = 3
    freq = torch.tensor(5e6 ** (-np.arange(0, 128, 2) / 128), dtype=torch.float32, device=DEV)
    cache = api.PagedCache(kc, vc)
    q_out, _ = api.msa_paged_append(cache, k, v, table, _i32([0, 1, 2]), _i32(pos), inv_freq=freq,
                                    q=q)
    torch.cuda.synchronize()
    assert api.msa_paged_read_status(cache) == 0
    ref = paged.rotate(_np(q), pos, _np(freq), False)
    _within(_np(q_out), ref, _rot_bound(_np(q), ref, 128, False, BF), "q")
    ref = paged.rotate(_np(k), pos, _np(freq), False)
    for r, pg in ((0, 0), (1, 3)):
        _within(_np(kc[pg, pos[r] % S]), ref[r], _rot_bound(_np(k[r]), ref[r], 128, False, BF), "k")
        assert torch.equal(vc[pg, pos[r] % S], v[r])


def test_append_in_place_and_without_queries():
    gen = _gen(12)
    kc, vc = (_pool(gen, 6, 16, 2, 64, BF) for _ in range(2))
    q, k, v = (_randn(gen, (5, h, 64), BF) for h in (6, 2, 2))
    freq = torch.rand(16, generator=gen, device=DEV)
    args = (_i32([[1, 2], [4, 0]]), _i32([0, 3, 5]), _i32([0, 14]))
    cache = api.PagedCache(kc, vc)
    want, _ = api.msa_paged_append(cache, k, v, *args, inv_freq=freq, q=q)
    k1 = kc.clone()
    kc.zero_()
    none, _ = api.msa_paged_append(cache, k, v, *args, inv_freq=freq)
    got, _ = api.msa_paged_append(cache, k, v, *args, inv_freq=freq, q=q, q_out=q)
    torch.cuda.synchronize()
    assert none is None and got is q and torch.equal(q, want)
    touched = kc.abs().sum((2, 3)) > 0
    assert torch.equal(kc[touched], k1[touched]) and int(touched.sum()) == 5


def test_append_bad_places_are_skipped():
    gen = _gen(13)
    kc, vc = (_pool(gen, 4, 16, 2, 64, FP) for _ in range(2))
    k, v = (_randn(gen, (6, 2, 64), FP) for _ in range(2))
    cache = api.PagedCache(kc, vc)
    before = kc.clone()
    table = _i32([[0, -1], [4, 1], [2, 3]])
    # row 0: positions 15 (page 0), 16 (no page); row 1: 0 (page 4 of 4), 16 is fine;
    # row 2: 31 (page 3), 32 (past the table)
    k_out = torch.full((6, 2, 64), 9.0, dtype=FP, device=DEV)
    api.msa_paged_append(cache, k, v, table, _i32([0, 2, 4, 6]), _i32([15, 15, 31]), k_out=k_out)
    assert api.msa_paged_read_status(cache, clear=True) == 11
    assert api.msa_paged_read_status(cache) == 0
    ok = [0, 3, 4]
    for t, (pg, slot) in zip(ok, ((0, 15), (1, 0), (3, 15))):
        assert torch.equal(kc[pg, slot], k[t]) and torch.equal(vc[pg, slot], v[t])
        before[pg, slot] = k[t]
        assert torch.equal(k_out[t], k[t])
    assert torch.equal(kc, before)
    assert (k_out[[1, 2, 5]] == 9).all()
    # a negative position, and offsets that decrease or pass T
    api.msa_paged_append(cache, k[:1], v[:1], table[:1], _i32([0, 1]), _i32([-1]))
    assert api.msa_paged_read_status(cache, clear=True) == 11 and torch.equal(kc, before)
    for offs in ([0, 2, 1, 6], [0, 2, 4, 7], [1, 2, 4, 6]):
        api.msa_paged_append(cache, k, v, _i32([[0], [1], [2]]), _i32(offs), _i32([0, 0, 0]))
        assert api.msa_paged_read_status(cache, clear=True) == 7


# ------------------------------------------------------------------ index
@pytest.mark.parametrize("S,heads,dim,head_major", [(128, 4, 64, False), (16, 4, 128, False),
                                                    (1, 3, 8, False), (512, 4, 32, True),
                                                    (64, 5, 120, True)])
def test_index_matches_fp64(S, heads, dim, head_major):
    rng, gen = np.random.default_rng(S), _gen(S)
    steps = [([0, 5, 130, 300, 1], [0, 0, 0, 0, 0]), ([1, 0, 1, 1, 1], [0, 5, 130, 300, 1]),
             ([400, 1, 126, 90, 0], [1, 5, 131, 301, 2])]
    final = [401, 6, 257, 391, 2]
    pool, table = _pages(rng, final, S)
    keys = _pool(gen, pool, S, heads, dim, BF, head_major)
    means = torch.full(api.paged_means_shape(pool, S, heads, dim), 3.0, device=DEV)
    index = api.PagedIndex(keys, means)
    for fresh, start in steps:
        offs = np.concatenate([[0], np.cumsum(fresh)])
        ik = _randn(gen, (int(offs[-1]) + 2, heads + 1, dim), BF)[:, :heads]
        k0, m0 = _np(keys), _np(means)
        k_ref, m_ref = paged.index(k0, m0, _np(ik), table, offs, start)
        api.msa_paged_index(index, ik, _i32(table), _i32(offs), _i32(start))
        torch.cuda.synchronize()
        assert np.array_equal(_np(keys), k_ref)
        m_abs = paged.index(np.abs(k0), np.abs(m0), np.abs(_np(ik)), table, offs, start)[1]
        bound = 129 * U * m_abs
        bound[m_ref == m0] = 0  # not touched
        _within(_np(means), m_ref, bound, "means")
    assert api.msa_paged_read_status(index) == 0


def test_index_long_prompts():
    rng, gen = np.random.default_rng(1), _gen(1)
    fresh, start, S = [5000, 1, 3333], [77, 128, 0], 64
    pool, table = _pages(rng, [f + s for f, s in zip(fresh, start)], S)
    offs = np.concatenate([[0], np.cumsum(fresh)])
    ik = _randn(gen, (int(offs[-1]), 4, 64), BF)
    keys = _pool(gen, pool, S, 4, 64, BF)
    index = api.PagedIndex(keys, torch.zeros(api.paged_means_shape(pool, S, 4, 64), device=DEV))
    k0, m0 = _np(keys), _np(index.means)
    k_ref, m_ref = paged.index(k0, m0, _np(ik), table, offs, start)
    m_abs = paged.index(np.abs(k0), m0, np.abs(_np(ik)), table, offs, start)[1]
    api.msa_paged_index(index, ik, _i32(table), _i32(offs), _i32(start))
    torch.cuda.synchronize()
    assert np.array_equal(_np(keys), k_ref)
    _within(_np(index.means), m_ref, 129 * U * m_abs, "means")
    assert api.msa_paged_read_status(index) == 0


def test_index_bad_pages_leave_the_block_out():
    gen = _gen(2)
    keys = _pool(gen, 4, 64, 4, 8, BF)
    before = keys.clone()
    index = api.PagedIndex(keys, torch.zeros(4, 4, 8, device=DEV))
    ik = _randn(gen, (130, 4, 8), BF)
    # block 0 (pages 0, 9 of 4) is left out, block 1 (page 2) is not
    api.msa_paged_index(index, ik, _i32([[0, 9, 2]]), _i32([0, 130]), _i32([0]))
    assert api.msa_paged_read_status(index, clear=True) == 11
    before[2, :2] = ik[128:]
    assert torch.equal(keys, before)
    assert torch.equal(index.means[2], ik[128:].float().sum(0) / 2)
    assert (index.means[[0, 1, 3]] == 0).all()
    api.msa_paged_index(index, ik[:1], _i32([[0, 1]]), _i32([0, 1]), _i32([128]))
    assert api.msa_paged_read_status(index, clear=True) == 11
    api.msa_paged_index(index, ik[:1], _i32([[0, 1]]), _i32([0, 1]), _i32([-3]))
    assert api.msa_paged_read_status(index, clear=True) == 11 and torch.equal(keys, before)


@pytest.mark.parametrize("narrow", [False, True])
@pytest.mark.parametrize("offs", [[0, 2, 4, 7],     # the last row ends past T
                                  [0, 2, 9, 11],    # one before it does
                                  [1, 2, 4, 6],     # token 0 is nobody's
                                  [-3, 2, 4, 6]])   # nor are a row's that begins below 0
def test_bad_offsets_leave_the_same_tokens_out_of_both_caches(offs, narrow):
    gen, S, T = _gen(62), 16, 6
    more = 2000 if narrow else 0  # tokens behind, so that append takes several to a thread block
    kc, vc = (torch.zeros(8, S, 1, 64, dtype=BF, device=DEV) for _ in range(2))
    keys = torch.zeros(8, S, 1, 64, dtype=BF, device=DEV)
    k = _randn(gen, (T + more, 1, 64), BF)
    first, table = [15, 3, 14], [[0, 1], [2, 3], [4, 5]]
    owned = [(r, a, min(b, T + more)) for r, (a, b) in enumerate(zip(offs, offs[1:]))
             if 0 <= a < T + more]
    cache, index = api.PagedCache(kc, vc), api.PagedIndex(keys, torch.zeros(8, 1, 64, device=DEV))
    args = (_i32(table), _i32(offs), _i32(first))
    api.msa_paged_append(cache, k, k, *args)
    api.msa_paged_index(index, k, *args)
    code = 7 if offs[0] != 0 or offs[-1] > T + more else 0
    assert api.msa_paged_read_status(cache) == code and api.msa_paged_read_status(index) == code
    want, means = torch.zeros_like(kc), torch.zeros_like(index.means)
    for r, a, b in owned:
        for t in range(a, b):
            p = first[r] + t - a
            want[table[r][p // S], p % S] = k[t]
        end = first[r] + b - a
        seen = torch.cat([want[pg] for pg in table[r]])[:end]  # the keys before are zeros
        means[table[r][(end - 1) // S]] = seen.double().sum(0).div(end).float()
    for got in (kc, vc, keys):
        assert torch.equal(got, want)
    # 7 sums at most and a division, of values up to 6
    assert (index.means - means).abs().max() <= 9 * U * 6


# ------------------------------------------------------------------ select
def _filled_index(lens, S, dim, seed, heads=4):
    rng, gen = np.random.default_rng(seed), _gen(seed)
    pool, table = _pages(rng, lens, S)
    offs = np.concatenate([[0], np.cumsum(lens)])
    ik = _randn(gen, (int(offs[-1]), heads, dim), BF)
    keys = torch.zeros(pool, S, heads, dim, dtype=BF, device=DEV)
    index = api.PagedIndex(keys, torch.full(api.paged_means_shape(pool, S, heads, dim),
                                            float("nan"), device=DEV))
    api.msa_paged_index(index, ik, _i32(table), _i32(offs), _i32([0] * len(lens)))
    return index, table, offs, ik, _randn(gen, ik.shape, BF)


@pytest.mark.parametrize("lens,S,dim,force", [
    ([2500, 300, 3100, 129, 1], 64, 64, True),
    ([2500, 300, 3100, 129, 1], 16, 64, False),
    ([2049, 2048, 2176, 2177], 128, 128, False),
    ([40000, 5000], 512, 32, False),
    ([150000], 128, 64, True),
    ([600000], 1024, 8, False),
])
def test_select_equals_the_training_selection(lens, S, dim, force):
    """Bit for bit: the same sums and products in the same order."""
    index, table, offs, ik, iq = _filled_index(lens, S, dim, sum(lens) + S)
    ref = api.msa_select_blocks(iq, ik, _i32(offs), force_local=force)
    last = torch.as_tensor(offs[1:] - 1, device=DEV)
    got = api.msa_paged_select(index, iq[last].contiguous(), _i32(table), _i32(lens),
                               force_local=force)
    torch.cuda.synchronize()
    assert torch.equal(got, ref[:, last])
    assert api.msa_paged_read_status(index) == 0
    if force:  # the own block is kept without a score: any shorter length as well
        rng = np.random.default_rng(3)
        cut = np.array([rng.integers(1, n + 1) for n in lens])
        at = torch.as_tensor(offs[:-1] + cut - 1, device=DEV)
        got = api.msa_paged_select(index, iq[at].contiguous(), _i32(table), _i32(cut))
        assert torch.equal(got, ref[:, at])


@pytest.mark.parametrize("heads,dim", [(1, 8), (3, 40), (64, 24), (5, 120), (7, 104), (2, 72)])
@pytest.mark.parametrize("force", [False, True])
def test_select_of_any_heads_and_channels(heads, dim, force):
    """Against the plain statement, on means and queries whose products and sums
    are exact in 32 bits (whole numbers of 2^-11 below 2^6), so that the choice
    does not depend on the order of a sum."""
    lens, S = [128 * 40 + 5, 1, 2049, 128 * 300, 0, 128 * 17], 32
    rng, gen = np.random.default_rng(heads * dim), _gen(heads * dim)
    pool, table = _pages(rng, lens, S)
    grid = torch.randint(-64, 65, (pool, heads, dim), generator=gen, device=DEV).float() / 512
    iq = (torch.randint(-16, 17, (len(lens), heads, dim), generator=gen, device=DEV) / 4.0).to(BF)
    index = api.PagedIndex(torch.zeros(pool, S, heads, dim, dtype=BF, device=DEV), grid)
    got = api.msa_paged_select(index, iq, _i32(table), _i32(lens), force_local=force)
    assert api.msa_paged_read_status(index) == 0
    want = np.full((heads, len(lens), 16), -1)
    for r, n in enumerate(lens):
        nb = -(-n // 128)
        if nb == 0:
            continue
        last = np.minimum(np.arange(nb) * 128 + 127, n - 1)
        score = np.einsum("vhd,hd->hv", _np(grid)[table[r, last // S]], _np(iq[r]))
        if force:
            score[:, [0, nb - 1]] = np.inf
        for h in range(heads):
            best = np.sort(np.argsort(-score[h], kind="stable")[:16])
            want[h, r, :len(best)] = best
    assert np.array_equal(got.cpu().numpy(), want)


def test_select_ties_go_to_the_lowest_block():
    n = 128 * 40
    gen = _gen(4)
    pool, table = _pages(np.random.default_rng(4), [n], 128)
    index = api.PagedIndex(torch.zeros(pool, 128, 4, 8, dtype=BF, device=DEV),
                           torch.zeros(pool, 4, 8, device=DEV))
    iq = _randn(gen, (1, 4, 8), BF)
    got = api.msa_paged_select(index, iq, _i32(table), _i32([n]), force_local=False)
    assert got.cpu().tolist() == [[list(range(16))]] * 4
    index.means[torch.as_tensor(table[0, 1::2].copy(), device=DEV).clamp(min=0)] = -0.0
    got = api.msa_paged_select(index, -iq.abs(), _i32(table), _i32([n]), force_local=False)
    assert got.cpu().tolist() == [[list(range(16))]] * 4
    got = api.msa_paged_select(index, iq, _i32(table), _i32([n]), force_local=True)
    assert got.cpu().tolist() == [[list(range(15)) + [39]]] * 4


def test_select_unused_rows_bad_lengths_and_pages():
    lens = [2600, 2600, 2600, 2600]
    index, table, offs, ik, iq = _filled_index(lens, 128, 16, 5)
    last = torch.as_tensor(offs[1:] - 1, device=DEV)
    q = iq[last].contiguous()
    good = api.msa_paged_select(index, q, _i32(table), _i32(lens)).cpu().numpy()
    assert api.msa_paged_read_status(index) == 0
    table = table.copy()
    table[2, 4:] = -1       # only blocks 0 .. 3 have a page
    got = api.msa_paged_select(index, q, _i32(table), _i32([0, 2600, 2600, 128 * 99])).cpu().numpy()
    assert api.msa_paged_read_status(index, clear=True) == 11
    assert (got[:, 0] == -1).all() and np.array_equal(got[:, 1], good[:, 1])
    assert (got[:, 3] == -1).all()
    for h in range(4):  # the blocks with a page, and the two that are always kept
        assert got[h, 2].tolist() == [0, 1, 2, 3, 20] + [-1] * 11


# ------------------------------------------------------------------ decode
def _decode_case(dt, dim, kv, share, S, lens, sparse, seed, head_major=False, poison=True,
                 scale=None, spread=1.0):
    rng, gen = np.random.default_rng(seed), _gen(seed)
    pool, table = _pages(rng, lens, S)
    kc, vc = (_pool(gen, pool, S, kv, dim, dt, head_major) for _ in range(2))
    q = (_randn(gen, (len(lens), kv * share, dim)) * spread).to(dt)
    q2k = None
    if sparse:
        q2k = np.full((kv, len(lens), 16), -1, dtype=np.int64)
        for g in range(kv):
            for r, n in enumerate(lens):
                nb = -(-n // 128)
                if nb == 0 or rng.random() < 0.1:
                    continue  # no slot used
                pick = rng.permutation(nb)[:rng.integers(1, 17)]
                if rng.random() < 0.7:
                    pick = np.unique(np.append(pick, nb - 1))[-16:]
                slots = rng.permutation(16)[:len(pick)]
                q2k[g, r, slots] = pick
                free = [i for i in range(16) if i not in slots]
                if free and rng.random() < 0.5:
                    q2k[g, r, free[0]] = pick[0]  # the same block twice counts once
    scale = scale or dim ** -0.5
    ref = paged.decode_bounds(_np(kc), _np(vc), _np(q), table, lens, scale, HALF[dt], TINY[dt], q2k)
    if poison:  # whatever lies where no row has a key must not matter
        used = np.zeros((pool, S), dtype=bool)
        for r, n in enumerate(lens):
            j = np.arange(n)
            used[table[r, j // S], j % S] = True
        free = torch.as_tensor(~used, device=DEV)
        for c, bad in ((kc, float("nan")), (vc, float("inf"))):
            c[free] = bad
    cache = api.PagedCache(kc, vc)
    o, lse = api.msa_paged_decode(cache, q, _i32(table), _i32(lens), scale,
                                  q2k=None if q2k is None else _i32(q2k))
    torch.cuda.synchronize()
    assert api.msa_paged_read_status(cache) == 0
    O, L, BO, BL = ref
    fin = np.isfinite(L)
    got = _np(lse)
    assert np.array_equal(got == -np.inf, ~fin)
    _within(np.where(fin, got, 0), np.where(fin, L, 0), BL, "LSE")
    _within(_np(o), O, BO, "O")
    assert (_np(o)[~fin] == 0).all()
    o2, lse2 = api.msa_paged_decode(cache, q, _i32(table), _i32(lens), scale,
                                    q2k=None if q2k is None else _i32(q2k))
    assert torch.equal(o, o2) and torch.equal(lse, lse2), "not the same twice"


EDGES = [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 191, 300, 1000]


@pytest.mark.parametrize("dt,dim,kv,share,S,head_major", [
    (BF, 128, 4, 16, 128, False),
    (BF, 128, 4, 16, 16, True),
    (FP, 64, 8, 3, 32, False),
    (FP, 128, 2, 7, 64, True),
    (BF, 64, 1, 1, 1, False),
    (BF, 64, 3, 8, 8, False),
    (FP, 128, 1, 9, 1024, False),
    (BF, 128, 2, 16, 4, True),
])
@pytest.mark.parametrize("sparse", [False, True])
def test_decode_matches_fp64(dt, dim, kv, share, S, head_major, sparse):
    _decode_case(dt, dim, kv, share, S, EDGES, sparse, seed=S + dim + share,
                 head_major=head_major)


@pytest.mark.parametrize("n", [1, 64, 65, 128, 1000, 2500])
@pytest.mark.parametrize("sparse", [False, True])
def test_decode_one_row(n, sparse):
    _decode_case(BF, 128, 4, 16, 64, [n], sparse, seed=n)


@pytest.mark.parametrize("dt,dim,kv,share,S,head_major", [
    (BF, 128, 4, 16, 128, False), (FP, 64, 2, 3, 32, True), (FP, 128, 1, 9, 16, False),
    (BF, 64, 3, 16, 8, False),
])
@pytest.mark.parametrize("sparse", [False, True])
def test_decode_few_short_rows(dt, dim, kv, share, S, head_major, sparse):
    # one cluster of CTAs a unit; parts without a tile among them
    for lens in ([0, 1, 129, 1000, 16], [64, 65, 513, 2100], [0], [2048]):
        _decode_case(dt, dim, kv, share, S, lens, sparse, seed=S + dim + len(lens),
                     head_major=head_major)


def test_decode_row_without_keys_alone():
    _decode_case(BF, 128, 4, 16, 64, [0], False, seed=1)
    _decode_case(FP, 64, 1, 2, 64, [0, 0], True, seed=2)


def test_decode_many_rows():
    rng = np.random.default_rng(8)
    _decode_case(BF, 64, 2, 4, 16, rng.integers(0, 200, 700).tolist(), False, seed=8)
    _decode_case(BF, 128, 4, 16, 32, rng.integers(0, 700, 90).tolist(), True, seed=9)
    # 64 channels: two heads at once, and each alone (an odd number, pages by head, blocks)
    # (the kernel reads a head's 64 channels alone in each of them: heads beside one another
    # in a token, an odd number of them, pages by head, selected blocks)
    lens = rng.integers(0, 300, 200).tolist()
    _decode_case(FP, 64, 4, 16, 32, lens, False, seed=40)
    _decode_case(FP, 64, 3, 5, 32, lens, False, seed=41)
    _decode_case(BF, 64, 2, 9, 64, lens, False, seed=42, head_major=True)
    _decode_case(BF, 64, 4, 3, 16, lens, True, seed=43)


def test_decode_one_long_row_split_over_all_ctas():
    _decode_case(BF, 128, 1, 16, 128, [90001], False, seed=10)
    _decode_case(FP, 64, 2, 5, 256, [70000, 3], False, seed=11)


def test_decode_sparse_in_long_rows():
    _decode_case(BF, 128, 4, 16, 128, [40000, 17, 9000], True, seed=12)


def test_decode_peaked_and_growing_scores():
    # large scores: the running maximum moves often, most weights vanish
    _decode_case(BF, 128, 2, 16, 64, [700, 129], False, seed=13, spread=30.0)
    _decode_case(FP, 64, 2, 4, 64, [700, 129], False, seed=14, spread=12.0)


@pytest.mark.parametrize("dt,dim", [(FP, 64), (FP, 128), (BF, 128)])
@pytest.mark.parametrize("nats", [16.0, 17.0, 18.0])
def test_decode_keeps_the_tail_behind_a_dominant_key(dt, dim, nats):
    """One key `nats` above all others, with a value of 0: O is what the tail
    leaves.  Two units an SM, a run each: all of a unit's keys meet the dominant
    one's warp or the three beside it."""
    gen, S, n = _gen(61), 128, 16384
    rows = 2 * torch.cuda.get_device_properties(0).multi_processor_count
    kc, vc = (_pool(gen, 9, S, 1, dim, dt) for _ in range(2))
    kc.mul_(0.02)
    vc.add_(2.0)
    q = torch.ones(rows, 4, dim, dtype=dt, device=DEV)
    q[:, 1::2] *= 0.9375
    scale = dim ** -0.5
    kc[8, 0] = nats / (dim * scale)
    vc[8, 0] = 0
    table = torch.randint(8, (1, n // S), generator=gen, device=DEV, dtype=torch.int32)
    table[0, 0] = 8
    cache = api.PagedCache(kc, vc)
    o, lse = api.msa_paged_decode(cache, q, table.expand(rows, -1).contiguous(), _i32([n] * rows),
                                  scale)
    torch.cuda.synchronize()
    assert api.msa_paged_read_status(cache) == 0
    O, L, BO, BL = paged.decode_bounds(_np(kc), _np(vc), _np(q[:1]), _np(table).astype(int), [n],
                                       scale, HALF[dt], TINY[dt])
    assert (BO < 0.1 * np.abs(O)).all()  # a quarter of the tail is missed if one warp's is
    one = np.ones((rows, 1, 1))
    _within(_np(lse), L * one[..., 0], BL * one[..., 0], "LSE")
    _within(_np(o), O * one, BO * one, "O")


@pytest.mark.parametrize("sparse", [False, True])
def test_decode_lengths_that_the_stream_has_just_written(sparse):
    # steps in a row, each with lengths from the kernel before it, eager and captured
    gen = _gen(31)
    rows, kv, S, steps = 61, 4, 64, 8
    pool, width = 300, 72  # 4608 tokens; the longest row comes to 4376
    kc, vc = (_pool(gen, pool, S, kv, 128, BF) for _ in range(2))
    cache = api.PagedCache(kc, vc)
    q = _randn(gen, (rows, kv * 16, 128), BF)
    table = torch.randint(pool, (rows, width), generator=gen, device=DEV, dtype=torch.int32)
    first = torch.randint(0, 2000, (rows,), generator=gen, device=DEV, dtype=torch.int32)
    q2k = None
    if sparse:
        q2k = torch.arange(16, dtype=torch.int32, device=DEV).repeat(kv, rows, 1)
        q2k[:, :, 7:] = -1
        first += 900  # all the blocks named are there
    ws = torch.empty(api.paged_decode_workspace_bytes(cache, rows, kv * 16), dtype=torch.uint8,
                     device=DEV)
    want = []
    for i in range(steps):  # one at a time
        lens = first + 211 * i
        torch.cuda.synchronize()
        want.append(api.msa_paged_decode(cache, q, table, lens, 0.09, q2k, workspace=ws))
        torch.cuda.synchronize()
    lens = first.clone()
    outs = [[torch.empty_like(x) for x in w] for w in want]

    def run():
        lens.copy_(first)
        for o, lse in outs:
            api.msa_paged_decode(cache, q, table, lens, 0.09, q2k, o=o, lse=lse, workspace=ws)
            lens.add_(211)

    run()
    runs = [[[x.clone() for x in p] for p in outs]]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        run()
    for _ in range(5):
        graph.replay()
        runs.append([[x.clone() for x in p] for p in outs])
    torch.cuda.synchronize()
    assert api.msa_paged_read_status(cache) == 0
    for got in runs:
        for (o, lse), (wo, wl) in zip(got, want):
            assert torch.equal(o, wo) and torch.equal(lse, wl)


def _decode_shared_pages(dt, dim, kv, share, S, lens, sparse, seed):
    """Long rows over few pages: the table names each many times, so the fp64
    result is a sum over the pool's keys with their counts."""
    rng, gen = np.random.default_rng(seed), _gen(seed)
    pool = 24
    width = -(-max(lens) // S) + 1
    table = rng.integers(0, pool, (len(lens), width))
    kc, vc = (_pool(gen, pool, S, kv, dim, dt) for _ in range(2))
    q = _randn(gen, (len(lens), kv * share, dim), dt)
    q2k = None
    if sparse:
        q2k = np.stack([[np.sort(rng.permutation(-(-n // 128))[:16]) for n in lens]
                        for _ in range(kv)])
    scale = dim ** -0.5
    cache = api.PagedCache(kc, vc)
    args = (cache, q, _i32(table), _i32(lens), scale, None if q2k is None else _i32(q2k))
    o, lse = api.msa_paged_decode(*args)
    again = [api.msa_paged_decode(*args) for _ in range(5)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        replayed = api.msa_paged_decode(*args)
    for _ in range(3):
        for x in replayed:
            x.zero_()
        graph.replay()
        again.append([x.clone() for x in replayed])
    torch.cuda.synchronize()
    assert api.msa_paged_read_status(cache) == 0
    for x, y in again:
        assert torch.equal(x, o) and torch.equal(y, lse), "not the same twice"
    K, V, Q = _np(kc).reshape(pool * S, kv, dim), _np(vc).reshape(pool * S, kv, dim), _np(q)
    O, L, BO, BL = (np.zeros((len(lens), kv * share) + x) for x in ((dim,), (), (dim,), ()))
    for r, n in enumerate(lens):
        for g in range(kv):
            j = paged.visible(n, None if q2k is None else q2k[g, r])
            at, count = np.unique(table[r, j // S] * S + j % S, return_counts=True)
            h = slice(g * share, (g + 1) * share)
            s = scale * (Q[r, h] @ K[at, g].T)
            top = s.max(1, keepdims=True)
            w = count * np.exp(s - top)
            z = w.sum(1, keepdims=True)
            O[r, h], L[r, h] = (w / z) @ V[at, g], (top + np.log(z))[:, 0]
            # as oracle.paged.decode_bounds
            ds = (dim + 4) * U * scale * (np.abs(Q[r, h]) @ np.abs(K[at, g]).T).max(1)
            big = np.abs(s).max(1)
            e = ds + U * (8 + 4 * big) + U * (4 * (j.size / 16 + 400) + j.size)
            pv = (w / z) @ np.abs(V[at, g])
            BO[r, h] = (1.01 * (2 * e + HALF[dt] ** 2))[:, None] * pv + HALF[dt] * np.abs(O[r, h]) \
                + TINY[dt] + j.size * TINY[dt] * np.abs(V[at, g]).max() / z
            BL[r, h] = 1.01 * e + 4 * U * (np.abs(L[r, h]) + big + np.log(j.size) + 1)
    _within(_np(lse), L, BL, "LSE")
    _within(_np(o), O, BO, "O")


@pytest.mark.parametrize("name", paged.STRIPED_CASES)
def test_decode_counts_every_key_of_a_long_row_once(name):
    """Rows that show a part left out or counted twice, where random ones do not:
    tests/test_paged_oracle.py plants both."""
    case = paged.STRIPED_CASES[name]
    dt, dim, kv, share, S, lens, span = case
    dt = BF if dt == "bf16" else FP
    table, levels = paged.striped_rows(case)
    scale = 0.125
    gen = _gen(64)
    vc = torch.as_tensor(paged.striped_values(dim, S, kv, dim), device=DEV).to(dt)
    q = torch.ones(len(lens), kv * share, dim, dtype=dt, device=DEV)
    if span:
        kc = torch.as_tensor(levels / (dim * scale), device=DEV).to(dt)
        assert np.array_equal(_np(kc) * dim * scale, levels)
        kc = kc[:, None, None, None].expand(dim, S, kv, dim).contiguous()
    else:
        kc, q = _pool(gen, dim, S, kv, dim, dt), torch.zeros_like(q)
    cache = api.PagedCache(kc, vc)
    o, lse = api.msa_paged_decode(cache, q, _i32(table), _i32(lens), scale)
    torch.cuda.synchronize()
    assert api.msa_paged_read_status(cache) == 0
    for r, n in enumerate(lens):
        O, L = paged.striped(table[r], n, S, levels, kv, dim)
        BO, BL = paged.striped_bounds(O, L, n, levels, dim, HALF[dt], TINY[dt])
        O, BO = (np.repeat(x, share, axis=0) for x in (O, BO))
        _within(_np(o[r]), O, BO, f"O of row {r}")
        _within(_np(lse[r]), np.full(kv * share, L), np.full(kv * share, BL), f"LSE of row {r}")


def test_decode_enough_tiles_for_the_short_runs():
    _decode_shared_pages(BF, 128, 4, 16, 128, [330001, 5, 70000], False, seed=31)
    _decode_shared_pages(FP, 64, 4, 5, 64, [700003], False, seed=32)
    _decode_shared_pages(BF, 128, 4, 16, 64, [2100 + 7 * i for i in range(190)], True, seed=33)


def test_caches_of_more_than_2_to_the_31_elements():
    """Pages whose first element lies past 2^31 (and past 2^32 bytes)."""
    gen, S, pool = _gen(34), 128, 33000
    kc, vc = (torch.empty(pool, S, 4, 128, dtype=BF, device=DEV) for _ in range(2))
    keys = torch.empty(2 * pool, S, 4, 128, dtype=BF, device=DEV)
    used = [pool - 1, 3, pool - 2, 0]
    n = 400
    table = np.array([used])
    cache = api.PagedCache(kc, vc)
    q, k, v = (_randn(gen, (n, h, 128), BF) for h in (64, 4, 4))
    ik, t = _randn(gen, (n, 4, 128), BF), _i32(table)
    offs, start = _i32([0, n]), _i32([0])
    k_out = torch.empty_like(k)
    api.msa_paged_append(cache, k, v, t, offs, start, inv_freq=torch.rand(64, device=DEV), q=q,
                         k_out=k_out)
    index = api.PagedIndex(keys, torch.zeros(2 * pool, 4, 128, device=DEV))
    api.msa_paged_index(index, ik, _i32([[2 * pool - 1, 3, 2 * pool - 2, 0]]), offs, start)
    o, lse = api.msa_paged_decode(cache, q[:1], t, _i32([n]), 0.09)
    torch.cuda.synchronize()
    for i, pg in enumerate(used):
        here = slice(128 * i, min(n, 128 * i + 128))
        m = here.stop - here.start
        assert torch.equal(kc[pg, :m], k_out[here]) and torch.equal(vc[pg, :m], v[here])
    assert torch.equal(keys[2 * pool - 1], ik[:128])
    small = np.array([[0, 1, 2, 3]])
    K = np.stack([_np(kc[p]) for p in used])
    V = np.stack([_np(vc[p]) for p in used])
    O, L, BO, BL = paged.decode_bounds(K, V, _np(q[:1]), small, [n], 0.09, HALF[BF], TINY[BF])
    _within(_np(lse), L, BL, "LSE")
    _within(_np(o), O, BO, "O")


def test_decode_bad_slots_pages_and_lengths():
    rng, gen = np.random.default_rng(15), _gen(15)
    lens = [300, 300, 300, 300, 300]
    pool, table = _pages(rng, lens, 16)
    kc, vc = (_pool(gen, pool, 16, 2, 64, BF) for _ in range(2))
    q = _randn(gen, (5, 8, 64), BF)
    cache = api.PagedCache(kc, vc)
    q2k = np.full((2, 5, 16), -1)
    q2k[:, :, 2], q2k[:, :, 9] = 0, 2
    bad = q2k.copy()
    bad[0, 1, 0], bad[1, 1, 5], bad[:, 2, 15] = 3, -2, 2 ** 31 - 1
    good = api.msa_paged_decode(cache, q, _i32(table), _i32(lens), 0.125, q2k=_i32(q2k))
    assert api.msa_paged_read_status(cache) == 0
    got = api.msa_paged_decode(cache, q, _i32(table), _i32(lens), 0.125, q2k=_i32(bad))
    assert api.msa_paged_read_status(cache, clear=True) == 6
    assert torch.equal(got[0], good[0]) and torch.equal(got[1], good[1])
    # row 3's second page is bad: as if its keys were not there; rows 0 and 4: bad lengths
    broken = table.copy()
    broken[3, 1] = pool
    wrong = [-1, 300, 300, 300, 16 * table.shape[1] + 1]
    for slots in (None, q2k):
        got = api.msa_paged_decode(cache, q, _i32(broken), _i32(wrong), 0.125,
                                   q2k=None if slots is None else _i32(slots))
        assert api.msa_paged_read_status(cache, clear=True) == 11
        for r in (0, 4):
            assert (got[0][r] == 0).all() and (got[1][r] == -float("inf")).all()
        # positions 16 .. 31 moved out of the row
        j = [x for x in range(300) if not 16 <= x < 32]
        for g in range(2):
            see = [x for x in j if slots is None or x // 128 in (0, 2)]
            K = np.stack([_np(kc[table[3, x // 16], x % 16, g]) for x in see])
            s = 0.125 * _np(q[3, 4 * g:4 * g + 4]) @ K.T
            L = np.log(np.exp(s).sum(1))
            assert np.abs(_np(got[1][3, 4 * g:4 * g + 4]) - L).max() < 1e-4
        ok = [1, 2]
        full = api.msa_paged_decode(cache, q, _i32(table), _i32(lens), 0.125,
                                    q2k=None if slots is None else _i32(slots))
        # the split of the keys over CTAs differs with the lengths: equal up to rounding
        assert (full[1][ok] - got[1][ok]).abs().max() < 1e-5


def test_decode_on_another_stream_and_into_given_tensors():
    gen = _gen(16)
    pool, table = _pages(np.random.default_rng(16), [500, 90], 32)
    kc, vc = (_pool(gen, pool, 32, 4, 128, BF) for _ in range(2))
    q = _randn(gen, (2, 64, 128), BF)
    cache = api.PagedCache(kc, vc)
    t, n = _i32(table), _i32([500, 90])
    want = api.msa_paged_decode(cache, q, t, n, 0.1)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = api.msa_paged_decode(cache, q, t, n, 0.1, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    o, lse = torch.full_like(want[0], 5.0), torch.full_like(want[1], 5.0)
    ws = torch.full((api.paged_decode_workspace_bytes(cache, 2, 64),), 255, dtype=torch.uint8,
                    device=DEV)
    got = api.msa_paged_decode(cache, q, t, n, 0.1, o=o, lse=lse, workspace=ws)
    assert got[0] is o and torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_calls_at_the_same_time_on_two_streams():
    """Two batches, each on its own stream with its own workspace, over and over
    (long enough for the short runs, so that both take CTAs at once)."""
    rng = np.random.default_rng(18)
    jobs = []
    for i, (rows, n) in enumerate(((40, 9000), (3, 120000))):
        gen = _gen(180 + i)
        kc, vc = (_pool(gen, 64, 128, 4, 128, BF) for _ in range(2))
        cache = api.PagedCache(kc, vc)
        lens = rng.integers(n // 2, n, rows)
        args = (cache, _randn(gen, (rows, 64, 128), BF),
                _i32(rng.integers(0, 64, (rows, -(-n // 128)))), _i32(lens), 0.09)
        want = api.msa_paged_decode(*args)
        ws = torch.empty(api.paged_decode_workspace_bytes(cache, rows, 64), dtype=torch.uint8,
                         device=DEV)
        jobs.append((cache, args, want, ws, torch.cuda.Stream(), []))
    torch.cuda.synchronize()
    for _ in range(12):
        for cache, args, want, ws, stream, got in jobs:
            with torch.cuda.stream(stream):
                got.append(api.msa_paged_decode(*args, workspace=ws))
    torch.cuda.synchronize()
    for cache, args, want, ws, stream, got in jobs:
        assert api.msa_paged_read_status(cache) == 0
        for o, lse in got:
            assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_one_pool_for_keys_and_values_and_a_slice_of_a_table():
    """k and v as halves of one tensor's pages, heads out of a wider pool, the
    table a slice of a larger one: same results as with tensors of their own."""
    rng, gen = np.random.default_rng(19), _gen(19)
    lens, S = [333, 1, 90], 16
    pool, table = _pages(rng, lens, S)
    both = _randn(gen, (pool, 2, S, 6, 128), BF)
    kc, vc = both[:, 0, :, 1:5], both[:, 1, :, 2:6]
    big = torch.full((5, table.shape[1] + 9), -7, dtype=torch.int32, device=DEV)
    t = big[1:4, 4:4 + table.shape[1]]
    t.copy_(_i32(table))
    n = _i32(lens)
    q, k, v = (_randn(gen, (3, h, 128), BF) for h in (64, 4, 4))
    freq = torch.rand(64, generator=gen, device=DEV)
    own = api.PagedCache(kc.contiguous(), vc.contiguous())
    views = api.PagedCache(kc, vc)
    outside = both.clone()
    for cache, tab in ((own, _i32(table)), (views, t)):
        api.msa_paged_append(cache, k, v, tab, _i32([0, 1, 2, 3]), n - 1, inv_freq=freq)
    torch.cuda.synchronize()
    assert torch.equal(kc, own.k) and torch.equal(vc, own.v)
    outside[:, 0, :, 1:5], outside[:, 1, :, 2:6] = kc, vc
    assert torch.equal(both, outside)
    for x, y in zip(api.msa_paged_decode(own, q, _i32(table), n, 0.1),
                    api.msa_paged_decode(views, q, t, n, 0.1)):
        assert torch.equal(x, y)
    assert api.msa_paged_read_status(views) == 0


def test_binding_refuses_mismatches():
    gen = _gen(17)
    kc, vc = (_pool(gen, 4, 16, 2, 64, BF) for _ in range(2))
    cache = api.PagedCache(kc, vc)
    t, n, q = _i32([[0, 1]]), _i32([20]), _randn(gen, (1, 8, 64), BF)
    for kw in (dict(q=q.half()), dict(q=q[:, :, :32]), dict(q=q[0]), dict(n=_i32([20, 3])),
               dict(n=n.long()), dict(n=n.cpu()), dict(t=t.cpu()), dict(q2k=_i32([[0] * 16])),
               dict(o=torch.empty(1, 8, 64, device=DEV)), dict(lse=q[:, :, 0].double()),
               dict(workspace=torch.empty(8, dtype=torch.uint8, device=DEV)),
               dict(scale=0.0), dict(q=_randn(gen, (1, 7, 64), BF)),
               dict(q=_randn(gen, (1, 34, 64), BF))):
        a = {**dict(q=q, t=t, n=n, scale=0.1), **kw}
        with pytest.raises((TypeError, ValueError, api.MSAError)):
            api.msa_paged_decode(cache, a["q"], a["t"], a["n"], a["scale"], q2k=a.get("q2k"),
                                 o=a.get("o"), lse=a.get("lse"), workspace=a.get("workspace"))
    with pytest.raises(ValueError):
        api.PagedCache(kc, vc[:3])
    with pytest.raises(TypeError):
        api.PagedCache(kc, vc.half())
    with pytest.raises(ValueError):
        api.PagedCache(kc[:1].expand(4, 16, 2, 64), vc)
    with pytest.raises(api.MSAError):
        api.PagedCache(kc[:, :12], vc[:, :12])
    with pytest.raises(api.MSAError):
        api.PagedCache(kc[..., :32], vc[..., :32])
    assert api.msa_paged_read_status(cache) == 0


# ------------------------------------------------------------------ together
def test_prompt_then_steps_as_served():
    """A prompt through append, index and the training path's forward, then
    token by token: every step's output must be what the training path and
    the fp64 oracle give for that token of the whole document."""
    rng, gen = np.random.default_rng(21), _gen(21)
    lens, steps, S, dim = [2300, 129, 700], 4, 64, 64
    full = [n + steps for n in lens]
    pool, table = _pages(rng, full, S)
    t = _i32(table)
    offs_full = np.concatenate([[0], np.cumsum(full)])
    T = int(offs_full[-1])
    q, k, v = (_randn(gen, (T, h, 128), BF) for h in (64, 4, 4))
    iq, ik = (_randn(gen, (T, 4, dim), BF) for _ in range(2))
    freq = torch.tensor(10000.0 ** (-np.arange(0, 64, 2) / 64), dtype=torch.float32, device=DEV)
    scale = 128 ** -0.5

    cache = api.PagedCache(*(torch.zeros(pool, S, 4, 128, dtype=BF, device=DEV) for _ in range(2)))
    index = api.PagedIndex(torch.zeros(pool, S, 4, dim, dtype=BF, device=DEV),
                           torch.zeros(api.paged_means_shape(pool, S, 4, dim), device=DEV))
    q_rot, k_rot = torch.empty_like(q), torch.empty_like(k)

    def tokens(begin, end):  # each row's tokens begin[r] .. end[r]-1
        return torch.as_tensor(np.concatenate([np.arange(offs_full[r] + begin[r],
                                                         offs_full[r] + end[r])
                                               for r in range(3)]), device=DEV)

    def feed(begin, end):
        at = tokens(begin, end)
        offs = _i32(np.concatenate([[0], np.cumsum(np.array(end) - np.array(begin))]))
        k_out = torch.empty(len(at), 4, 128, dtype=BF, device=DEV)
        qr, kr = api.msa_paged_append(cache, k[at], v[at], t, offs, _i32(begin), inv_freq=freq,
                                      q=q[at], k_out=k_out)
        api.msa_paged_index(index, ik[at], t, offs, _i32(begin))
        q_rot[at], k_rot[at] = qr, kr
        return qr

    # the prompt: handed-back queries and keys through the training path
    qr = feed([0, 0, 0], lens)
    at = tokens([0, 0, 0], lens)
    offs = _i32(np.concatenate([[0], np.cumsum(lens)]))
    q2k = api.msa_select_blocks(iq[at], ik[at], offs)
    plan = api.msa_build_plan(q2k, offs)
    o, lse = api.msa_forward(plan, qr, k_rot[at], v[at], scale)
    last = (offs[1:] - 1).long()
    got = api.msa_paged_decode(cache, qr[last].contiguous(), t, _i32(lens), scale,
                               q2k=q2k[:, last].contiguous())
    torch.cuda.synchronize()
    check_o(_np(got[0]), _np(o[last]))
    check_lse(_np(got[1]), _np(lse[last]))

    # then step by step
    served = []
    for i in range(steps):
        n = [x + i for x in lens]
        qr = feed(n, [x + 1 for x in n])
        at = tokens(n, [x + 1 for x in n])
        chosen = api.msa_paged_select(index, iq[at], t, _i32([x + 1 for x in n]))
        served.append((at, chosen, api.msa_paged_decode(cache, qr, t, _i32([x + 1 for x in n]),
                                                        scale, q2k=chosen)))
    torch.cuda.synchronize()
    assert api.msa_paged_read_status(cache) == 0 and api.msa_paged_read_status(index) == 0

    offs = _i32(offs_full)
    q2k = api.msa_select_blocks(iq, ik, offs)
    plan = api.msa_build_plan(q2k, offs)
    o, lse = api.msa_forward(plan, q_rot, k_rot, v, scale)
    P = oracle.Problem(q_rot.cpu(), k_rot.cpu(), v.cpu(), q2k.cpu().numpy(),
                       offs_full.astype(np.int32), scale)
    for at, chosen, (so, sl) in served:
        assert torch.equal(chosen, q2k[:, at])
        check_o(_np(so), _np(o[at]))
        check_lse(_np(sl), _np(lse[at]))
        O, L = P.forward(at.cpu().numpy())
        check_o(_np(so), O)
        check_lse(_np(sl), L)


@pytest.mark.parametrize("S", [16, 64, 256])
def test_tokens_behind_a_cached_prefix_one_row_each(S):
    """Several new tokens of a row as rows of their own over the same pages, as the
    header describes it: selection with force_local equals the training path's
    for the whole document, attention its forward's, whatever the page size."""
    gen, rng = _gen(65), np.random.default_rng(65)
    n, cached, dim = 2900, 2437, 32  # the prefix ends inside a block; new tokens over four blocks
    pool, table = _pages(rng, [n], S)
    q, k, v = (_randn(gen, (n, h, 128), BF) for h in (64, 4, 4))
    iq, ik = (_randn(gen, (n, 4, dim), BF) for _ in range(2))
    cache = api.PagedCache(*(torch.zeros(pool, S, 4, 128, dtype=BF, device=DEV) for _ in range(2)))
    index = api.PagedIndex(torch.zeros(pool, S, 4, dim, dtype=BF, device=DEV),
                           torch.full(api.paged_means_shape(pool, S, 4, dim), float("nan"),
                                      device=DEV))
    t = _i32(table)
    for a, b in ((0, cached), (cached, n)):
        offs, start = _i32([0, b - a]), _i32([a])
        api.msa_paged_append(cache, k[a:b], v[a:b], t, offs, start)
        api.msa_paged_index(index, ik[a:b], t, offs, start)
    new = torch.arange(cached, n, device=DEV)
    rows, lens = t.expand(len(new), -1).contiguous(), (new + 1).int()
    chosen = api.msa_paged_select(index, iq[new], rows, lens)
    o, lse = api.msa_paged_decode(cache, q[new], rows, lens, 128 ** -0.5, q2k=chosen)
    doc = _i32([0, n])
    q2k = api.msa_select_blocks(iq, ik, doc)
    want, want_lse = api.msa_forward(api.msa_build_plan(q2k, doc), q, k, v, 128 ** -0.5)
    torch.cuda.synchronize()
    assert api.msa_paged_read_status(cache) == 0 and api.msa_paged_read_status(index) == 0
    assert torch.equal(chosen, q2k[:, new])
    check_o(_np(o), _np(want[new]))
    check_lse(_np(lse), _np(want_lse[new]))


def test_a_step_captured_and_replayed():
    """One step in a CUDA graph, replayed with other lengths, tables and
    inputs, some rows not in use; a second graph of another batch size beside
    it; every replay equals the eager calls."""
    rng, gen = np.random.default_rng(22), _gen(22)
    S, dim, most = 32, 32, 4000
    pool = 900
    cache = api.PagedCache(*(_pool(gen, pool, S, 4, 128, BF) for _ in range(2)))
    index = api.PagedIndex(_pool(gen, pool, S, 4, dim, BF),
                           _randn(gen, api.paged_means_shape(pool, S, 4, dim)))
    freq = torch.rand(32, generator=gen, device=DEV)

    def state(rows):
        return dict(q=torch.zeros(rows, 64, 128, dtype=BF, device=DEV),
                    k=torch.zeros(rows, 4, 128, dtype=BF, device=DEV),
                    v=torch.zeros(rows, 4, 128, dtype=BF, device=DEV),
                    iq=torch.zeros(rows, 4, dim, dtype=BF, device=DEV),
                    ik=torch.zeros(rows, 4, dim, dtype=BF, device=DEV),
                    t=torch.zeros(rows, -(-most // S), dtype=torch.int32, device=DEV),
                    offs=torch.zeros(rows + 1, dtype=torch.int32, device=DEV),
                    start=torch.zeros(rows, dtype=torch.int32, device=DEV),
                    n=torch.zeros(rows, dtype=torch.int32, device=DEV))

    def step(s):
        qr, _ = api.msa_paged_append(cache, s["k"], s["v"], s["t"], s["offs"], s["start"],
                                     inv_freq=freq, q=s["q"], q_out=s.get("qr"))
        api.msa_paged_index(index, s["ik"], s["t"], s["offs"], s["start"])
        chosen = api.msa_paged_select(index, s["iq"], s["t"], s["n"])
        return (chosen, *api.msa_paged_decode(cache, qr, s["t"], s["n"], 0.09, q2k=chosen))

    graphs = []
    for rows in (5, 3):
        s = state(rows)
        s["qr"] = torch.zeros(rows, 64, 128, dtype=BF, device=DEV)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step(s)
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step(s)
        graphs.append((rows, s, g, out))
    for turn in range(4):
        for rows, s, g, out in graphs:
            order, at = rng.permutation(pool), 0
            used = int(rng.integers(1, rows + 1))
            new = state(rows)
            start = np.zeros(rows, int)
            start[:used] = rng.integers(0, most - 1, used)
            new["start"].copy_(_i32(start))
            new["n"][:used] = _i32(start[:used] + 1)
            new["offs"].copy_(_i32(np.minimum(np.arange(rows + 1), used)))
            new["t"].fill_(-1)
            for r in range(used):
                np_ = start[r] // S + 1
                new["t"][r, :np_] = _i32(order[at:at + np_])
                at += np_
            for x in ("q", "k", "v", "iq", "ik"):
                new[x].copy_(_randn(gen, new[x].shape, BF))
            for x in new:
                s[x].copy_(new[x])
            saved = [x.clone() for x in (cache.k, cache.v, index.keys, index.means)]
            g.replay()
            torch.cuda.synchronize()
            for x, y in zip((cache.k, cache.v, index.keys, index.means), saved):
                x.copy_(y)
            eager = step(s)
            for x, y in zip(out, eager):
                assert torch.equal(x, y)
            assert (out[0][:, used:] == -1).all() and (out[1][used:] == 0).all()
            assert (out[2][used:] == -float("inf")).all()
    assert api.msa_paged_read_status(cache) == 0 and api.msa_paged_read_status(index) == 0
