"""The paged-cache calls without a GPU: struct layouts, and every refusal that
is decided on the host, in the C ABI and in the Python binding."""
import ctypes
import importlib.util
import os
import shutil
import subprocess
import tempfile

import pytest
import torch

from block_sparse_gqa_msa_gb300 import api
from block_sparse_gqa_msa_gb300 import build as msa_build

OK, INVALID, ALIGN, WORKSPACE = 0, 1, 3, 4
CPU = torch.device("cpu")
G = 0x10000  # an aligned address that no refused call reads


@pytest.fixture(scope="module")
def lib():
    msa_build.build()
    return api.lib()


def _cache(**kw):
    d = dict(k=G, v=G, k_stride=(65536, 512, 128), v_stride=(65536, 512, 128), num_pages=10,
             page_size=128, kv_heads=4, head_dim=128, dtype=0, status=G)
    d.update(kw)
    for n in ("k_stride", "v_stride"):
        d[n] = (ctypes.c_int64 * 3)(*d[n])
    return api.MsaPagedCacheStruct(**d)


def _index(**kw):
    d = dict(keys=G, key_stride=(32768, 256, 64), means=G, num_pages=10, page_size=128, heads=4,
             dim=64, reserved=0, status=G)
    d.update(kw)
    d["key_stride"] = (ctypes.c_int64 * 3)(*d["key_stride"])
    return api.MsaPagedIndexStruct(**d)


def _table(**kw):
    return api.MsaPageTableStruct(**{**dict(pages=G, stride=8, rows=3, width=8), **kw})


BAD_TABLES = [dict(pages=None), dict(rows=0), dict(rows=65537), dict(width=0), dict(stride=7),
              dict(width=1 << 24, stride=1 << 24)]
BAD_POOLS = [dict(num_pages=0), dict(num_pages=1 << 31), dict(page_size=0), dict(page_size=48),
             dict(page_size=2048), dict(status=None)]


def _append(lib, cache=None, table=None, **kw):
    d = dict(offs=G, start=G, T=3, k=G, ks=512, v=G, vs=512, q=G, qs=8192, heads=64, freq=G,
             rot=64, inter=0, q_out=G, k_out=None)
    d.update(kw)
    return lib.msa_paged_append(cache or _cache(), table or _table(), d["offs"], d["start"],
                                d["T"], d["k"], d["ks"], d["v"], d["vs"], d["q"], d["qs"],
                                d["heads"], d["freq"], d["rot"], d["inter"], d["q_out"],
                                d["k_out"], None)


@pytest.mark.parametrize("kw", [
    dict(offs=None), dict(start=None), dict(T=0), dict(T=(1 << 20) + 1), dict(k=None),
    dict(v=None), dict(ks=511), dict(ks=516), dict(vs=504), dict(q_out=None), dict(heads=0),
    dict(heads=1025), dict(qs=8188), dict(qs=8190), dict(q_out=G, q=G, qs=8200), dict(q=None),
    dict(rot=8), dict(rot=24), dict(rot=144), dict(rot=0)])
def test_append_refuses(lib, kw):
    assert _append(lib, **kw) == INVALID


def test_append_refuses_caches_tables_and_alignment(lib):
    for kw in BAD_POOLS + [dict(k=None), dict(v=None), dict(kv_heads=0), dict(kv_heads=65),
                           dict(head_dim=96), dict(dtype=2), dict(k_stride=(65536, 512, 4)),
                           dict(v_stride=(65536, 0, 128)), dict(k_stride=(-8, 512, 128))]:
        assert _append(lib, cache=_cache(**kw)) == INVALID, kw
    for kw in BAD_TABLES:
        assert _append(lib, table=_table(**kw)) == INVALID, kw
    for kw in (dict(k=G + 8), dict(v=G + 2), dict(q=G + 8), dict(q_out=G + 4), dict(k_out=G + 8),
               dict(offs=G + 2), dict(start=G + 1), dict(freq=G + 2)):
        assert _append(lib, **kw) == ALIGN, kw
    assert _append(lib, cache=_cache(k=G + 8)) == ALIGN
    assert _append(lib, cache=_cache(status=G + 4)) == ALIGN
    assert _append(lib, table=_table(pages=G + 2)) == ALIGN


def test_index_and_select_refuse(lib):
    def index(cache=None, table=None, offs=G, start=G, T=3, ik=G, s=256):
        return lib.msa_paged_index(cache or _index(), table or _table(), offs, start, T, ik, s, None)

    def select(cache=None, table=None, lens=G, iq=G, q2k=G):
        return lib.msa_paged_select(cache or _index(), table or _table(), lens, iq, 1, q2k, None)
    for kw in (dict(offs=None), dict(start=None), dict(T=0), dict(T=(1 << 20) + 1), dict(ik=None),
               dict(s=248), dict(s=260)):
        assert index(**kw) == INVALID, kw
    for kw in (dict(lens=None), dict(iq=None), dict(q2k=None)):
        assert select(**kw) == INVALID, kw
    for kw in (dict(ik=G + 8), dict(offs=G + 2)):
        assert index(**kw) == ALIGN, kw
    for kw in (dict(iq=G + 8), dict(q2k=G + 8), dict(lens=G + 2)):
        assert select(**kw) == ALIGN, kw
    for call in (index, select):
        for kw in BAD_POOLS + [dict(keys=None), dict(means=None), dict(heads=0), dict(heads=65),
                               dict(dim=4), dict(dim=12), dict(dim=136),
                               dict(key_stride=(32768, 256, 0))]:
            assert call(cache=_index(**kw)) == INVALID, kw
        for kw in BAD_TABLES:
            assert call(table=_table(**kw)) == INVALID, kw
        assert call(cache=_index(keys=G + 8)) == ALIGN and call(cache=_index(means=G + 4)) == ALIGN


def test_decode_refuses(lib):
    n = ctypes.c_size_t(0)
    c = _cache()
    assert lib.msa_paged_decode_workspace_bytes(c, 3, 64, ctypes.byref(n)) == OK and n.value > 0
    for rows, heads in ((0, 64), (65537, 64), (3, 0), (3, 6), (3, 68)):
        assert lib.msa_paged_decode_workspace_bytes(c, rows, heads, ctypes.byref(n)) == INVALID
    assert lib.msa_paged_decode_workspace_bytes(c, 3, 64, None) == INVALID
    assert lib.msa_paged_decode_workspace_bytes(None, 3, 64, ctypes.byref(n)) == INVALID
    need = n.value

    def decode(cache=None, table=None, lens=G, q=G, heads=64, scale=0.1, q2k=G, o=G, lse=G, ws=G,
               nbytes=need):
        return lib.msa_paged_decode(cache or _cache(), table or _table(), lens, q, heads, scale,
                                    q2k, o, lse, ws, nbytes, None)
    for kw in (dict(lens=None), dict(q=None), dict(o=None), dict(lse=None), dict(ws=None),
               dict(heads=0), dict(heads=63), dict(heads=68), dict(scale=0.0), dict(scale=-1.0),
               dict(scale=float("nan")), dict(scale=float("inf"))):
        assert decode(**kw) == INVALID, kw
    for kw in BAD_TABLES:
        assert decode(table=_table(**kw)) == INVALID, kw
    for kw in (dict(q=G + 8), dict(o=G + 8), dict(ws=G + 8), dict(lens=G + 2), dict(lse=G + 2),
               dict(q2k=G + 1)):
        assert decode(**kw) == ALIGN, kw
    assert decode(nbytes=need - 1) == WORKSPACE
    assert lib.msa_paged_read_status(None, None) == INVALID
    assert lib.msa_paged_read_status(G + 4, None) == ALIGN


def test_binding_refuses_cpu_and_overlapping_tensors():
    x = torch.zeros(4, 16, 4, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        api.PagedCache(x, x.clone())
    with pytest.raises(ValueError):
        api.PagedIndex(x, torch.zeros(4, 4, 128))
    with pytest.raises(TypeError):
        api.PagedCache(None, x)
    assert api.paged_means_shape(7, 16, 4, 64) == (7, 4, 64)
    assert api.paged_means_shape(7, 512, 4, 64) == (28, 4, 64)


def test_binding_checks_layouts():
    with pytest.raises(TypeError):
        api._table(torch.zeros(2, 3, dtype=torch.int64), CPU)
    with pytest.raises(ValueError):
        api._table(torch.zeros(3, dtype=torch.int32), CPU)
    with pytest.raises(ValueError):
        api._table(torch.zeros(3, 2, dtype=torch.int32).t(), CPU)
    with pytest.raises(ValueError):
        api._table(torch.zeros(1, 5, dtype=torch.int32).expand(4, 5), CPU)
    with pytest.raises(ValueError):
        api._table(torch.zeros(3, 2, dtype=torch.int32), torch.device("cuda:0"))
    t = api._table(torch.zeros(4, 9, dtype=torch.int32)[1:3, 2:7], CPU)
    assert (t.rows, t.width, t.stride) == (2, 5, 9)
    one = api._table(torch.zeros(4, 9, dtype=torch.int32)[:1, :5], CPU)
    assert one.stride >= one.width
    qkv = torch.zeros(5, 72, 128, dtype=torch.float16)
    assert api._tokens(qkv[:, 64:68], "k", torch.float16, 5, 4, 128, CPU) == 72 * 128
    for x, dt, h, d in ((qkv, torch.bfloat16, 72, 128), (qkv, torch.float16, 4, 128),
                        (qkv, torch.float16, 72, 64), (qkv[0], torch.float16, 72, 128),
                        (qkv[:, ::2], torch.float16, 36, 128),
                        (qkv.transpose(1, 2), torch.float16, 128, 72)):
        with pytest.raises((TypeError, ValueError)):
            api._tokens(x, "x", dt, None, h, d, CPU)
    with pytest.raises(ValueError):
        api._tokens(qkv, "x", torch.float16, 6, 72, 128, CPU)


def test_status_of_a_cache_on_another_device_is_refused(monkeypatch):
    # it would wait for the current device's stream, not for the one that the calls ran on
    class Cache:
        device = torch.device("cuda", 1)
        status = torch.zeros(1, dtype=torch.int64)

    monkeypatch.setattr(api, "_current_device", lambda: 0)
    monkeypatch.setattr(api, "_raw_stream", lambda device: 0)
    monkeypatch.setattr(api, "lib", lambda: pytest.fail("the library was called"))
    for clear in (False, True):
        with pytest.raises(ValueError, match="cuda:1"):
            api.msa_paged_read_status(Cache, clear=clear)


def test_binding_imports_without_a_cuda_build_of_torch(monkeypatch):
    """Without torch's own bindings the module still loads and asks the public calls."""
    for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
        monkeypatch.delattr(torch._C, name, raising=False)
    spec = importlib.util.spec_from_file_location("api_without_cuda", api.__file__)
    fresh = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(fresh)
    asked = []

    class Stream:
        cuda_stream = 77

    monkeypatch.setattr(torch.cuda, "current_stream", lambda device: asked.append(device) or Stream)
    monkeypatch.setattr(fresh, "_current_device", lambda: 3)
    assert fresh._stream(None) == 77 and asked == [3]
    assert fresh._stream(Stream) == 77


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs a C++ compiler")
def test_a_question_to_the_device_is_asked_once_also_if_it_fails(tmp_path):
    """What decides the way of a call never changes within a process."""
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text("""
#include <cstdio>
#include "asked_once.cuh"
static msa::AskedOnce<4, 8> known;
int main() {
  int asked = 0;
  auto says = [&](int x) { return [&asked, x] { ++asked; return x; }; };
  const int got[] = {known.get(0, 1, says(-1)), known.get(0, 1, says(9)),  // failed: 0, and stays
                     known.get(0, 2, says(0)), known.get(0, 2, says(9)),
                     known.get(3, 1, says(38)), known.get(3, 1, says(-1)),
                     known.get(4, 0, says(9)), known.get(-1, 0, says(9))};
  for (int x : got) std::printf("%d ", x);
  std::printf("%d", asked);
}
""")
    csrc = os.path.join(os.path.dirname(api.__file__), "csrc")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", csrc, str(src), "-o", str(exe)],
                   check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout
    assert out.split() == "0 0 0 0 38 38 0 0 3".split()


@pytest.mark.skipif(shutil.which("gcc") is None, reason="needs a C compiler")
def test_paged_struct_layouts_match_header():
    mirrors = {"msa_paged_cache": api.MsaPagedCacheStruct,
               "msa_paged_index_cache": api.MsaPagedIndexStruct,
               "msa_page_table": api.MsaPageTableStruct}
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "msa.h"', "int main(void) {"]
    for cname, py in mirrors.items():
        lines.append(f'  printf("{cname} size %zu\\n", sizeof({cname}));')
        for field, _ in py._fields_:
            lines.append(f'  printf("{cname} {field} %zu\\n", offsetof({cname}, {field}));')
    lines.append('  printf("x MSA_BF16 %d\\nx MSA_F16 %d\\nx bad_page %d\\n", MSA_BF16, MSA_F16, '
                 'MSA_ERR_BAD_PAGE);\n  return 0; }')
    with tempfile.TemporaryDirectory() as d:
        src, exe = os.path.join(d, "p.c"), os.path.join(d, "p")
        with open(src, "w") as f:
            f.write("\n".join(lines))
        subprocess.run(["gcc", "-I", os.path.dirname(api.HEADER_PATH), src, "-o", exe], check=True)
        out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout
    got = {tuple(x.split()[:2]): int(x.split()[2]) for x in out.splitlines()}
    for cname, py in mirrors.items():
        assert got[(cname, "size")] == ctypes.sizeof(py)
        for field, _ in py._fields_:
            assert got[(cname, field)] == getattr(py, field).offset, (cname, field)
    assert got[("x", "MSA_BF16")] == api.PAGED_DTYPES[torch.bfloat16]
    assert got[("x", "MSA_F16")] == api.PAGED_DTYPES[torch.float16]
    assert api.STATUS[got[("x", "bad_page")]] == "MSA_ERR_BAD_PAGE"
