"""What the norm and the drafted tokens' calls refuse on the host, without a GPU."""
import ctypes

import pytest

from block_sparse_gqa_msa_gb300 import api
from block_sparse_gqa_msa_gb300 import build as msa_build
from tests.test_paged_host import BAD_POOLS, BAD_TABLES, _cache, _table

INVALID, ALIGN, WORKSPACE = 1, 3, 4
G = 0x10000  # an aligned address that no refused call reads


@pytest.fixture(scope="module")
def lib():
    msa_build.build()
    return api.lib()


def _norm(lib, back=False, outs=(G, G), ws=1 << 30, **kw):
    d = dict(q=G, k=G, q_stride=8192, k_stride=512, q_weight=G, k_weight=G, positions=G, inv_freq=G,
             T=3, q_heads=64, k_heads=4, head_dim=128, rotary_dim=64, interleaved=0, dtype=0,
             weight_dtype=2, eps=1e-6)
    d.update(kw)
    a = ctypes.byref(api.MsaNormRopeStruct(**d))
    if back:
        return lib.msa_norm_rope_backward(a, *outs, G, G, G, G, G, ws, None)
    return lib.msa_norm_rope(a, *outs, None)


@pytest.mark.parametrize("bad,code", [
    (dict(q=None), 1), (dict(k=None), 1), (dict(q_weight=None), 1), (dict(T=0), 1),
    (dict(T=(1 << 20) + 1), 1), (dict(head_dim=96), 1), (dict(q_heads=0), 1), (dict(k_heads=1025), 1),
    (dict(dtype=2), 1), (dict(weight_dtype=3), 1), (dict(q_stride=8184), 1), (dict(k_stride=516), 1),
    (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(positions=None), 1), (dict(rotary_dim=8), 1),
    (dict(rotary_dim=144), 1), (dict(q=G + 8), 3), (dict(q_weight=G + 2), 3), (dict(positions=G + 2), 3),
    (dict(outs=(None, G)), 1), (dict(outs=(G, G + 4)), 3)])
def test_norm_refusals(lib, bad, code):
    assert _norm(lib, **bad) == code
    assert _norm(lib, back=True, **bad) == code


def test_norm_in_place_needs_contiguous_rows_and_workspace(lib):
    assert _norm(lib, outs=(G, 2 * G), q_stride=9000) == INVALID
    n = ctypes.c_size_t(0)
    assert lib.msa_norm_rope_workspace_bytes(128, ctypes.byref(n)) == 0
    assert _norm(lib, back=True, ws=n.value - 1) == WORKSPACE
    assert lib.msa_norm_rope_workspace_bytes(96, ctypes.byref(n)) == INVALID


def _tree(lib, cache=None, table=None, **kw):
    d = dict(offs=G, lens=G, parents=G, T=9, q=G, heads=64, scale=0.1, q2k=None, o=G, lse=G, ws=G,
             n=1 << 30)
    d.update(kw)
    return lib.msa_paged_tree(cache or _cache(), table or _table(), d["offs"], d["lens"], d["parents"],
                              d["T"], d["q"], d["heads"], d["scale"], d["q2k"], d["o"], d["lse"],
                              d["ws"], d["n"], None)


def test_tree_refusals(lib):
    for bad in BAD_POOLS:
        assert _tree(lib, cache=_cache(**bad)) == INVALID
    for bad in BAD_TABLES:
        assert _tree(lib, table=_table(**bad)) == INVALID
    for bad in (dict(offs=None), dict(lens=None), dict(q=None), dict(o=None), dict(lse=None),
                dict(ws=None), dict(T=0), dict(T=(1 << 20) + 1), dict(heads=0), dict(heads=66),
                dict(heads=68), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan"))):
        assert _tree(lib, **bad) == INVALID
    for bad in (dict(q=G + 2), dict(o=G + 8), dict(ws=G + 4), dict(lens=G + 1), dict(parents=G + 2),
                dict(q2k=G + 2), dict(lse=G + 2)):
        assert _tree(lib, **bad) == ALIGN
    # tiles past 32 bits: 4 groups of rows, 2^14 rows, 2^20 tokens
    assert _tree(lib, table=_table(rows=1 << 14, width=1 << 13, stride=1 << 13), T=1000) == INVALID
    n = ctypes.c_size_t(0)
    ref = ctypes.byref(_cache())
    assert lib.msa_paged_tree_workspace_bytes(ref, 3, 9, 64, ctypes.byref(n)) == 0
    assert _tree(lib, n=n.value - 1) == WORKSPACE
    for rows, T, heads in ((0, 9, 64), (65537, 9, 64), (3, 0, 64), (3, 9, 63), (3, 9, 68)):
        assert lib.msa_paged_tree_workspace_bytes(ref, rows, T, heads, ctypes.byref(n)) == INVALID


def test_verify_refusals(lib):
    def call(**kw):
        d = dict(p=G, ps=100, q=G, qs=100, tok=G, up=G, offs=G, rows=2, T=9, V=100, u=G, ul=G, width=8,
                 path=G, count=G, last=G)
        d.update(kw)
        return lib.msa_tree_verify(*d.values(), None)
    for bad in (dict(p=None), dict(tok=None), dict(offs=None), dict(u=None), dict(ul=None),
                dict(path=None), dict(count=None), dict(last=None), dict(rows=0), dict(rows=65537),
                dict(T=0), dict(V=0), dict(V=(1 << 24) + 1), dict(ps=99), dict(qs=99), dict(width=0),
                dict(width=65)):
        assert call(**bad) == INVALID
    for name in ("p", "q", "tok", "up", "offs", "u", "ul", "path", "count", "last"):
        assert call(**{name: G + 2}) == ALIGN


def test_compact_refusals(lib):
    def call(cache=None, table=None, **kw):
        d = dict(lens=G, path=G, width=8, count=G, new=2 * G)
        d.update(kw)
        return lib.msa_paged_compact(cache or _cache(), table or _table(), *d.values(), None)
    for bad in BAD_POOLS:
        assert call(cache=_cache(**bad)) == INVALID
    for bad in BAD_TABLES:
        assert call(table=_table(**bad)) == INVALID
    for bad in (dict(lens=None), dict(path=None), dict(count=None), dict(new=None), dict(new=G),
                dict(width=0), dict(width=65)):
        assert call(**bad) == INVALID
    for name in ("lens", "path", "count", "new"):
        assert call(**{name: G + 2}) == ALIGN
