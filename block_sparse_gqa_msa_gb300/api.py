"""Python binding of libmsa (include/msa.h): argument marshalling only.

Every step of MSA runs in the library's CUDA kernels; this module checks
shapes / dtypes / devices of torch tensors, allocates outputs and workspaces
with torch's caching allocator, and passes raw pointers plus the current CUDA
stream through the C ABI.  There is no fallback: if libmsa.so is missing or
cannot run, calls raise MSAError.

Names follow the C ABI: msa_build_plan, msa_forward, msa_backward.
"""
from __future__ import annotations

import ctypes
import os
import threading

import numpy as np
import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmsa.so")
HEADER_PATH = os.path.join(os.path.dirname(HERE), "include", "msa.h")

NUM_Q_HEADS, NUM_KV_HEADS, HEAD_DIM, TOPK = 64, 4, 128, 16

STATUS = {
    0: "MSA_OK", 1: "MSA_ERR_INVALID_ARG", 2: "MSA_ERR_UNSUPPORTED", 3: "MSA_ERR_ALIGNMENT",
    4: "MSA_ERR_WORKSPACE", 5: "MSA_ERR_CUDA", 6: "MSA_ERR_BAD_Q2K", 7: "MSA_ERR_BAD_OFFSETS",
    8: "MSA_ERR_TIMEOUT", 9: "MSA_ERR_CAPACITY", 10: "MSA_ERR_RANGE",
    11: "MSA_ERR_BAD_PAGE",
}
MSA_OK = 0


class MSAError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {STATUS.get(code, code)}")


class MsaPlanStruct(ctypes.Structure):
    _fields_ = [
        ("T", ctypes.c_int64), ("num_docs", ctypes.c_int32), ("super_block", ctypes.c_int32),
        ("dq_accum", ctypes.c_int32), ("o_accum", ctypes.c_int32),
        ("dense_blocks", ctypes.c_int32), ("nb_cap", ctypes.c_int64), ("tri_cap", ctypes.c_int64), ("nnz_cap", ctypes.c_int64),
        ("task_cap", ctypes.c_int64),
        ("q2k", ctypes.c_void_p), ("doc_offsets", ctypes.c_void_p), ("header", ctypes.c_void_p),
        ("doc_info", ctypes.c_void_p), ("doc_tri", ctypes.c_void_p), ("cnt", ctypes.c_void_p),
        ("off", ctypes.c_void_p), ("col", ctypes.c_void_p), ("tcnt", ctypes.c_void_p),
        ("toff", ctypes.c_void_p), ("tasks", ctypes.c_void_p), ("scan_tmp", ctypes.c_void_p),
        ("scan_tmp_len", ctypes.c_int64),
        ("item_cap", ctypes.c_int64), ("grouped", ctypes.c_void_p), ("items", ctypes.c_void_p),
        ("fflag", ctypes.c_void_p), ("fpos", ctypes.c_void_p), ("ftasks", ctypes.c_void_p),
        ("rows", ctypes.c_void_p),
    ]


class MsaPlanOptions(ctypes.Structure):
    _fields_ = [("super_block", ctypes.c_int32), ("dq_accum", ctypes.c_int32),
                ("o_accum", ctypes.c_int32), ("dense_blocks", ctypes.c_int32),
                ("reserved", ctypes.c_int32 * 4)]


class MsaPagedCacheStruct(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_stride", ctypes.c_int64 * 3),
                ("v_stride", ctypes.c_int64 * 3), ("num_pages", ctypes.c_int64),
                ("page_size", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("status", ctypes.c_void_p)]


class MsaPagedIndexStruct(ctypes.Structure):
    _fields_ = [("keys", ctypes.c_void_p), ("key_stride", ctypes.c_int64 * 3),
                ("means", ctypes.c_void_p), ("num_pages", ctypes.c_int64),
                ("page_size", ctypes.c_int32), ("heads", ctypes.c_int32), ("dim", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("status", ctypes.c_void_p)]


class MsaPageTableStruct(ctypes.Structure):
    _fields_ = [("pages", ctypes.c_void_p), ("stride", ctypes.c_int64), ("rows", ctypes.c_int32),
                ("width", ctypes.c_int32)]


DQ_ACCUM = {"f16": 0, "bf16": 1, "f32": 2}
O_ACCUM = {"f32": 0, "bf16": 1}


_lock = threading.Lock()
_lib = None

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I32 = ctypes.c_int32
_SZ = ctypes.c_size_t
_F = ctypes.c_float
_PLAN = ctypes.POINTER(MsaPlanStruct)
_CACHE = ctypes.POINTER(MsaPagedCacheStruct)
_INDEX = ctypes.POINTER(MsaPagedIndexStruct)
_TABLE = ctypes.POINTER(MsaPageTableStruct)

SIGNATURES = {
    "msa_status_string": ([_I32], ctypes.c_char_p),
    "msa_plan_workspace_bytes": ([_I64, _I32, ctypes.POINTER(_SZ)], _I32),
    "msa_build_plan": ([_P, _P, _I64, _I32, ctypes.POINTER(MsaPlanOptions), _P, _SZ, _P, _PLAN],
                       _I32),
    "msa_build_plan_static": ([_P, _P, _I64, _I32, ctypes.POINTER(MsaPlanOptions), _P, _PLAN],
                              _I32),
    "msa_forward_workspace_bytes": ([_PLAN, ctypes.POINTER(_SZ)], _I32),
    "msa_forward": ([_PLAN, _P, _P, _P, _F, _P, _P, _P, _SZ, _P], _I32),
    "msa_backward_workspace_bytes": ([_PLAN, ctypes.POINTER(_SZ)], _I32),
    "msa_backward": ([_PLAN, _P, _P, _P, _P, _P, _P, _F, _P, _P, _P, _P, _SZ, _P], _I32),
    "msa_read_status": ([_PLAN, _P], _I32),
    "msa_plan_counts": ([_PLAN, _P, ctypes.POINTER(_I64)], _I32),
    "msa_plan_export": ([_PLAN, _P, _P, _I64, _P, _I64], _I32),
    "msa_plan_export_groups": ([_PLAN, _P, _P, _I64, _P, _I64, _P, _I64], _I32),
    "msa_profile_enable": ([_I32], _I32),
    "msa_profile_reset": ([], _I32),
    "msa_profile_read": ([ctypes.c_char_p, ctypes.POINTER(_I64), ctypes.POINTER(ctypes.c_double)],
                         _I32),
    "msa_launch_count": ([], _I64),
    "msa_pack_thd": ([_P, _I32, _I32, _I32, _P, _P, _P, _P], _I32),
    "msa_unpack_bshd": ([_P, _I32, _I32, _I32, _P, _P, _P, _P], _I32),
    "msa_select_workspace_bytes": ([_I64, _I32, _I32, ctypes.POINTER(_SZ)], _I32),
    "msa_select_blocks": ([_P, _P, _I64, _I32, _P, _I32, _I32, _P, _P, _SZ, _P], _I32),
    "msa_paged_read_status": ([_P, _P], _I32),
    "msa_paged_append": ([_CACHE, _TABLE, _P, _P, _I64, _P, _I64, _P, _I64, _P, _I64, _I32, _P,
                          _I32, _I32, _P, _P, _P], _I32),
    "msa_paged_index": ([_INDEX, _TABLE, _P, _P, _I64, _P, _I64, _P], _I32),
    "msa_paged_select": ([_INDEX, _TABLE, _P, _P, _I32, _P, _P], _I32),
    "msa_paged_decode_workspace_bytes": ([_CACHE, _I32, _I32, ctypes.POINTER(_SZ)], _I32),
    "msa_paged_decode": ([_CACHE, _TABLE, _P, _P, _I32, _F, _P, _P, _P, _P, _SZ, _P], _I32),
}


def lib():
    """The loaded libmsa (built in-tree by build.py); raises MSAError if absent."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise MSAError(1, f"{LIB_PATH} is not built (run __graft_entry__.build())")
            L = ctypes.CDLL(LIB_PATH)
            for name, (args, res) in SIGNATURES.items():
                fn = getattr(L, name)
                fn.argtypes = args
                fn.restype = res
            _lib = L
    return _lib


def _check(code: int, what: str):
    if code != MSA_OK:
        raise MSAError(code, what)


def _public_raw_stream(device: int) -> int:
    return torch.cuda.current_stream(device).cuda_stream


# The current device, and its current stream's handle without a Stream object (4
# us of a call), where this build of torch offers them; else the public calls.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _public_raw_stream)


def _stream(stream) -> int:
    if stream is None:
        return _raw_stream(_current_device())
    return stream.cuda_stream


def _ptr(t: torch.Tensor) -> ctypes.c_void_p:
    return ctypes.c_void_p(t.data_ptr())


def _need(t: torch.Tensor, name: str, dtype, shape):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


class Plan:
    """A built plan: the C struct plus the tensors it points into."""

    def __init__(self, struct: MsaPlanStruct, workspace: torch.Tensor, q2k: torch.Tensor,
                 doc_offsets: torch.Tensor):
        self.struct = struct
        self.workspace = workspace
        self.q2k = q2k
        self.doc_offsets = doc_offsets

    @property
    def T(self) -> int:
        return int(self.struct.T)

    @property
    def num_docs(self) -> int:
        return int(self.struct.num_docs)

    def ref(self):
        return ctypes.byref(self.struct)


def plan_workspace_bytes(T: int, num_docs: int) -> int:
    n = _SZ(0)
    _check(lib().msa_plan_workspace_bytes(T, num_docs, ctypes.byref(n)), "msa_plan_workspace_bytes")
    return int(n.value)


def msa_build_plan(q2k: torch.Tensor, doc_offsets: torch.Tensor, super_block: int = 64,
                   workspace: torch.Tensor | None = None, stream=None,
                   dq_accum: str = "f16", o_accum: str = "f32", dense_blocks: int = 0) -> Plan:
    """Device-side plan from q2k int32 [4,T,16] and doc_offsets int32 [D+1].
    dq_accum: precision of the backward's dQ pool ("f16", "bf16" or "f32");
    o_accum: precision of the forward's O pool (only "f32" is accepted; the
    library rejects "bf16", whose O error exceeds the forward's bar);
    dense_blocks: bound on the query block (b + 1 <= dense_blocks) of the
    forward's dense octets (0: the default, 32; -1: none)."""
    if q2k.dim() != 3:
        raise ValueError("q2k must be [4, T, 16]")
    T = int(q2k.shape[1])
    D = int(doc_offsets.numel()) - 1
    _need(q2k, "q2k", torch.int32, (NUM_KV_HEADS, T, TOPK))
    _need(doc_offsets, "doc_offsets", torch.int32, (D + 1,))
    nbytes = plan_workspace_bytes(T, D)
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=q2k.device)
    opts = MsaPlanOptions(super_block=super_block, dq_accum=DQ_ACCUM[dq_accum],
                          o_accum=O_ACCUM[o_accum], dense_blocks=dense_blocks)
    st = MsaPlanStruct()
    _check(lib().msa_build_plan(_ptr(q2k), _ptr(doc_offsets), T, D, ctypes.byref(opts),
                                _ptr(workspace), workspace.numel(), _stream(stream),
                                ctypes.byref(st)), "msa_build_plan")
    return Plan(st, workspace, q2k, doc_offsets)


def msa_build_plan_static(q2k: torch.Tensor, doc_offsets: torch.Tensor, super_block: int = 64,
                          stream=None, dq_accum: str = "f16", o_accum: str = "f32",
                          dense_blocks: int = 0) -> Plan:
    """Like msa_build_plan, but the plan tables live in the library's own
    static device array, so nothing is allocated.  For callers that cannot
    allocate device memory; the plan is valid until the next call."""
    if q2k.dim() != 3:
        raise ValueError("q2k must be [4, T, 16]")
    T = int(q2k.shape[1])
    D = int(doc_offsets.numel()) - 1
    _need(q2k, "q2k", torch.int32, (NUM_KV_HEADS, T, TOPK))
    _need(doc_offsets, "doc_offsets", torch.int32, (D + 1,))
    opts = MsaPlanOptions(super_block=super_block, dq_accum=DQ_ACCUM[dq_accum],
                          o_accum=O_ACCUM[o_accum], dense_blocks=dense_blocks)
    st = MsaPlanStruct()
    _check(lib().msa_build_plan_static(_ptr(q2k), _ptr(doc_offsets), T, D, ctypes.byref(opts),
                                       _stream(stream), ctypes.byref(st)), "msa_build_plan_static")
    return Plan(st, None, q2k, doc_offsets)


def forward_workspace_bytes(plan: Plan) -> int:
    n = _SZ(0)
    _check(lib().msa_forward_workspace_bytes(plan.ref(), ctypes.byref(n)), "msa_forward_workspace_bytes")
    return int(n.value)


def backward_workspace_bytes(plan: Plan) -> int:
    n = _SZ(0)
    _check(lib().msa_backward_workspace_bytes(plan.ref(), ctypes.byref(n)),
           "msa_backward_workspace_bytes")
    return int(n.value)


def msa_forward(plan: Plan, q, k, v, softmax_scale: float, o=None, lse=None, workspace=None,
                stream=None):
    """(O bf16 [T,64,128], LSE fp32 [T,64])."""
    T = plan.T
    _need(q, "q", torch.bfloat16, (T, NUM_Q_HEADS, HEAD_DIM))
    _need(k, "k", torch.bfloat16, (T, NUM_KV_HEADS, HEAD_DIM))
    _need(v, "v", torch.bfloat16, (T, NUM_KV_HEADS, HEAD_DIM))
    o = torch.empty_like(q) if o is None else o
    lse = torch.empty((T, NUM_Q_HEADS), dtype=torch.float32, device=q.device) if lse is None else lse
    _need(o, "o", torch.bfloat16, (T, NUM_Q_HEADS, HEAD_DIM))
    _need(lse, "lse", torch.float32, (T, NUM_Q_HEADS))
    if workspace is None:
        workspace = torch.empty(forward_workspace_bytes(plan), dtype=torch.uint8, device=q.device)
    _check(lib().msa_forward(plan.ref(), _ptr(q), _ptr(k), _ptr(v), float(softmax_scale), _ptr(o),
                             _ptr(lse), _ptr(workspace), workspace.numel(), _stream(stream)),
           "msa_forward")
    return o, lse


def msa_backward(plan: Plan, q, k, v, o, lse, dout, softmax_scale: float, dq=None, dk=None,
                 dv=None, workspace=None, stream=None):
    """(dQ bf16 [T,64,128], dK bf16 [T,4,128], dV bf16 [T,4,128])."""
    T = plan.T
    _need(q, "q", torch.bfloat16, (T, NUM_Q_HEADS, HEAD_DIM))
    _need(k, "k", torch.bfloat16, (T, NUM_KV_HEADS, HEAD_DIM))
    _need(v, "v", torch.bfloat16, (T, NUM_KV_HEADS, HEAD_DIM))
    _need(o, "o", torch.bfloat16, (T, NUM_Q_HEADS, HEAD_DIM))
    _need(lse, "lse", torch.float32, (T, NUM_Q_HEADS))
    _need(dout, "dout", torch.bfloat16, (T, NUM_Q_HEADS, HEAD_DIM))
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    if workspace is None:
        workspace = torch.empty(backward_workspace_bytes(plan), dtype=torch.uint8, device=q.device)
    _check(lib().msa_backward(plan.ref(), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse),
                              _ptr(dout), float(softmax_scale), _ptr(dq), _ptr(dk), _ptr(dv),
                              _ptr(workspace), workspace.numel(), _stream(stream)),
           "msa_backward")
    return dq, dk, dv


def msa_read_status(plan: Plan, stream=None) -> int:
    """Synchronising read of the plan's device status word (0 = OK)."""
    return int(lib().msa_read_status(plan.ref(), _stream(stream)))


def msa_plan_counts(plan: Plan, stream=None) -> dict:
    c = (_I64 * 7)()
    _check(lib().msa_plan_counts(plan.ref(), _stream(stream), c), "msa_plan_counts")
    return {"NB": c[0], "nnz": c[1], "ntasks": c[2], "pairs": c[3], "entries": c[4],
            "items": c[5], "ftasks": c[6]}


def msa_plan_export(plan: Plan, stream=None):
    """(col int32 [nnz], tasks int32 [ntasks, 4]) copied to host."""
    cnt = msa_plan_counts(plan, stream)
    col = np.zeros(max(cnt["nnz"], 1), dtype=np.int32)
    tasks = np.zeros((max(cnt["ntasks"], 1), 4), dtype=np.int32)
    _check(lib().msa_plan_export(plan.ref(), _stream(stream), col.ctypes.data_as(_P), col.size,
                                 tasks.ctypes.data_as(_P), tasks.shape[0]), "msa_plan_export")
    return col[:cnt["nnz"]], tasks[:cnt["ntasks"]]


def msa_plan_export_groups(plan: Plan, stream=None):
    """(grouped uint8 [4, T], items int32 [n_items, 36], ftasks int32
    [n_ftasks, 4]) - the forward's octet groups - copied to host."""
    cnt = msa_plan_counts(plan, stream)
    T = plan.struct.T
    grouped = np.zeros((4, T), dtype=np.uint8)
    items = np.zeros((max(cnt["items"], 1), 36), dtype=np.int32)
    ftasks = np.zeros((max(cnt["ftasks"], 1), 4), dtype=np.int32)
    _check(lib().msa_plan_export_groups(plan.ref(), _stream(stream), grouped.ctypes.data_as(_P),
                                        T, items.ctypes.data_as(_P), items.shape[0],
                                        ftasks.ctypes.data_as(_P), ftasks.shape[0]),
           "msa_plan_export_groups")
    return grouped, items[:cnt["items"]], ftasks[:cnt["ftasks"]]


def profile_enable(on: bool = True):
    _check(lib().msa_profile_enable(1 if on else 0), "msa_profile_enable")


def profile_reset():
    _check(lib().msa_profile_reset(), "msa_profile_reset")


def profile_read(name: str):
    n = _I64(0)
    ms = ctypes.c_double(0.0)
    _check(lib().msa_profile_read(name.encode(), ctypes.byref(n), ctypes.byref(ms)),
           "msa_profile_read")
    return int(n.value), float(ms.value)


def launch_count() -> int:
    return int(lib().msa_launch_count())


# ---------------------------------------------------------------- THD packing
def _row_bytes(x: torch.Tensor, lead: int) -> int:
    return int(x[(0,) * lead].numel() * x.element_size()) if x.numel() else 0


def pack_thd(x: torch.Tensor, row_len: torch.Tensor, total: int | None = None, stream=None):
    """Padded packed rows -> compact THD.

    x: CUDA tensor [B, S, ...] (each token row a multiple of 16 bytes);
    row_len: int32 [B] on the same device, tokens 0..row_len[b]-1 of row b are
    real.  Returns (y [T, ...], row_offsets int32 [B+1]).  ``total`` = T if
    known; otherwise it is read from row_len (one device-to-host copy).
    """
    if not (x.is_cuda and row_len.is_cuda):
        raise ValueError("pack_thd needs CUDA tensors")
    if x.dim() < 2 or not x.is_contiguous():
        raise ValueError("x must be a contiguous [B, S, ...] tensor")
    B, S = int(x.shape[0]), int(x.shape[1])
    _need(row_len, "row_len", torch.int32, (B,))
    if total is None:
        total = int(row_len.clamp(0, S).sum().item())
    y = torch.empty((total,) + tuple(x.shape[2:]), dtype=x.dtype, device=x.device)
    offs = torch.empty(B + 1, dtype=torch.int32, device=x.device)
    _check(lib().msa_pack_thd(_ptr(x), B, S, _row_bytes(x, 2), _ptr(row_len), _ptr(y),
                              _ptr(offs), _stream(stream)), "msa_pack_thd")
    return y, offs


def unpack_bshd(y: torch.Tensor, row_len: torch.Tensor, row_offsets: torch.Tensor, S: int,
                out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Compact THD -> padded packed rows [B, S, ...] (padding rows zero)."""
    if not (y.is_cuda and row_len.is_cuda and row_offsets.is_cuda):
        raise ValueError("unpack_bshd needs CUDA tensors")
    if y.dim() < 1 or not y.is_contiguous():
        raise ValueError("y must be a contiguous [T, ...] tensor")
    B = int(row_len.shape[0])
    _need(row_len, "row_len", torch.int32, (B,))
    _need(row_offsets, "row_offsets", torch.int32, (B + 1,))
    if out is None:
        out = torch.empty((B, S) + tuple(y.shape[1:]), dtype=y.dtype, device=y.device)
    row_bytes = int(out[0, 0].numel() * out.element_size())
    _check(lib().msa_unpack_bshd(_ptr(y), B, S, row_bytes, _ptr(row_len), _ptr(row_offsets),
                                 _ptr(out), _stream(stream)), "msa_unpack_bshd")
    return out


# ---------------------------------------------------------------- block selection
def select_workspace_bytes(T: int, num_docs: int, dim: int) -> int:
    n = _SZ(0)
    _check(lib().msa_select_workspace_bytes(T, num_docs, dim, ctypes.byref(n)),
           "msa_select_workspace_bytes")
    return int(n.value)


def msa_select_blocks(iq: torch.Tensor, ik: torch.Tensor, doc_offsets: torch.Tensor,
                      force_local: bool = True, q2k: torch.Tensor | None = None,
                      workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """q2k int32 [4, T, 16] from index queries / keys bf16 [T, 4, dim] (see
    msa_select_blocks in include/msa.h for the scoring and tie rules)."""
    if iq.dim() != 3:
        raise ValueError("iq must be [T, 4, dim]")
    T, dim = int(iq.shape[0]), int(iq.shape[2])
    _need(iq, "iq", torch.bfloat16, (T, NUM_KV_HEADS, dim))
    _need(ik, "ik", torch.bfloat16, (T, NUM_KV_HEADS, dim))
    D = int(doc_offsets.numel()) - 1
    _need(doc_offsets, "doc_offsets", torch.int32, (D + 1,))
    if q2k is None:
        q2k = torch.empty((NUM_KV_HEADS, T, TOPK), dtype=torch.int32, device=iq.device)
    _need(q2k, "q2k", torch.int32, (NUM_KV_HEADS, T, TOPK))
    if workspace is None:
        workspace = torch.empty(select_workspace_bytes(T, D, dim), dtype=torch.uint8,
                                device=iq.device)
    _check(lib().msa_select_blocks(_ptr(iq), _ptr(ik), T, dim, _ptr(doc_offsets), D,
                                   1 if force_local else 0, _ptr(q2k), _ptr(workspace),
                                   workspace.numel(), _stream(stream)), "msa_select_blocks")
    return q2k


# ---------------------------------------------------------------- paged cache (serving)
BLOCK = 128
PAGED_DTYPES = {torch.bfloat16: 0, torch.float16: 1}


def _pool(x, name: str, dtypes):
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if x.dtype not in dtypes:
        raise TypeError(f"{name} must be one of {tuple(dtypes)}, got {x.dtype}")
    if x.dim() != 4 or x.numel() == 0:
        raise ValueError(f"{name} must be [num_pages, page_size, heads, dim]")
    if x.stride(3) != 1:
        raise ValueError(f"{name}: a head's channels must be contiguous")
    # outermost first, every dimension must step over all that the inner ones cover
    covered = x.shape[3]
    for stride, n in sorted((x.stride(i), x.shape[i]) for i in range(3)):
        if n > 1 and stride < covered:
            raise ValueError(f"{name}: elements overlap (strides {x.stride()})")
        covered = max(covered, stride * n)


def _pool_strides(x):
    # the stride of a dimension of one element means nothing; any valid one will do
    return (_I64 * 3)(*(x.stride(i) if x.shape[i] > 1 else x.shape[3] for i in range(3)))


class PagedCache:
    """Keys and values in pages: two tensors [num_pages, page_size, kv_heads,
    head_dim], bf16 or fp16, any strides with contiguous channels (so pages
    may also lie head-major).  page_size is a power of two up to 1024,
    head_dim 64 or 128.  Holds the tensors and a device status word."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor):
        _pool(k, "k", PAGED_DTYPES)
        _pool(v, "v", (k.dtype,))
        if k.shape != v.shape:
            raise ValueError(f"k {tuple(k.shape)} and v {tuple(v.shape)} must have one shape")
        if k.device != v.device:
            raise ValueError("k and v must be on one device")
        self.k, self.v = k, v
        self.device, self.dtype = k.device, k.dtype
        self.num_pages, self.page_size, self.kv_heads, self.head_dim = map(int, k.shape)
        self.status = torch.zeros(1, dtype=torch.int64, device=k.device)
        self.struct = MsaPagedCacheStruct(
            k=k.data_ptr(), v=v.data_ptr(), k_stride=_pool_strides(k), v_stride=_pool_strides(v),
            num_pages=self.num_pages, page_size=self.page_size, kv_heads=self.kv_heads,
            head_dim=self.head_dim, dtype=PAGED_DTYPES[k.dtype], status=self.status.data_ptr())
        self._ref = ctypes.byref(self.struct)
        # the library's own check of the cache, before the first call
        paged_decode_workspace_bytes(self, 1, self.kv_heads)

    def ref(self):
        return self._ref


def paged_means_shape(num_pages: int, page_size: int, heads: int, dim: int):
    """Shape of the block means that belong to index keys in pages."""
    return num_pages * max(1, page_size // BLOCK), heads, dim


class PagedIndex:
    """Index keys in pages, bf16 [num_pages, page_size, heads, dim] (strides
    as for PagedCache), and the fp32 means of their 128-key blocks
    (``paged_means_shape``, contiguous).  Holds both and a status word."""

    def __init__(self, keys: torch.Tensor, means: torch.Tensor):
        _pool(keys, "keys", (torch.bfloat16,))
        shape = paged_means_shape(*map(int, keys.shape))
        _need(means, "means", torch.float32, shape)
        if keys.device != means.device:
            raise ValueError("keys and means must be on one device")
        self.keys, self.means, self.device = keys, means, keys.device
        self.num_pages, self.page_size, self.heads, self.dim = map(int, keys.shape)
        self.status = torch.zeros(1, dtype=torch.int64, device=keys.device)
        self.struct = MsaPagedIndexStruct(
            keys=keys.data_ptr(), key_stride=_pool_strides(keys), means=means.data_ptr(),
            num_pages=self.num_pages, page_size=self.page_size, heads=self.heads, dim=self.dim,
            reserved=0, status=self.status.data_ptr())
        self._ref = ctypes.byref(self.struct)

    def ref(self):
        return self._ref


def _current(device):
    if device.index != _current_device():
        raise ValueError(f"the cache is on {device}, the current device is "
                         f"cuda:{_current_device()}")


def _arg(t, name: str, dtype, shape, device) -> int:
    """Address of a contiguous tensor of this type and shape on the cache's device."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
            and t.device == device and t.is_contiguous()):
        return t.data_ptr()
    _need(t, name, dtype, shape)
    raise ValueError(f"{name} must be on {device}, got {t.device}")


def _table(page_table: torch.Tensor, device) -> MsaPageTableStruct:
    if not isinstance(page_table, torch.Tensor):
        raise TypeError("page_table must be a torch.Tensor")
    if page_table.dtype is not torch.int32:
        raise TypeError(f"page_table must be torch.int32, got {page_table.dtype}")
    if page_table.device != device:
        raise ValueError(f"page_table must be on {device}, got {page_table.device}")
    if page_table.dim() != 2 or page_table.numel() == 0:
        raise ValueError("page_table must be [rows, pages of a row]")
    rows, width = page_table.shape
    stride, step = page_table.stride()
    if rows == 1:
        stride = width
    if (width > 1 and step != 1) or stride < width:
        raise ValueError("page_table: a row's entries must be contiguous, rows must not overlap")
    return MsaPageTableStruct(page_table.data_ptr(), stride, rows, width)


def _tokens(x, name: str, dtype, tokens: int | None, heads: int | None, dim: int, device) -> int:
    """Token stride of [T, heads, dim] with contiguous tokens."""
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if x.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {x.dtype}")
    if x.device != device:
        raise ValueError(f"{name} must be on {device}, got {x.device}")
    shape = x.shape
    if (len(shape) != 3 or shape[2] != dim or (heads is not None and shape[1] != heads)
            or (tokens is not None and shape[0] != tokens)):
        raise ValueError(f"{name} must be [{'T' if tokens is None else tokens}, "
                         f"{'heads' if heads is None else heads}, {dim}], got {tuple(shape)}")
    st, sh, sd = x.stride()
    h = shape[1]
    if sd != 1 or (h > 1 and sh != dim):
        raise ValueError(f"{name}: a token's heads must be contiguous")
    return st if shape[0] > 1 else h * dim


def _empty(shape, dtype, device, stream):
    """What a call allocates belongs to the stream that it runs on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def paged_decode_workspace_bytes(cache: PagedCache, rows: int, q_heads: int) -> int:
    n = _SZ(0)
    _check(lib().msa_paged_decode_workspace_bytes(cache.ref(), rows, q_heads, ctypes.byref(n)),
           "msa_paged_decode_workspace_bytes")
    return int(n.value)


def msa_paged_read_status(cache, stream=None, clear: bool = False) -> int:
    """Synchronising read of the status word of a PagedCache or PagedIndex (0 =
    OK; the lowest-numbered status otherwise).  ``clear`` resets the word.  The
    cache's device must be the current one, as for the calls that set it."""
    _current(cache.device)
    code = int(lib().msa_paged_read_status(_ptr(cache.status), _stream(stream)))
    if clear:
        with torch.cuda.stream(stream):  # the current one if None
            cache.status.zero_()
    return code


def msa_paged_append(cache: PagedCache, k: torch.Tensor, v: torch.Tensor,
                     page_table: torch.Tensor, row_offsets: torch.Tensor,
                     start_pos: torch.Tensor, inv_freq: torch.Tensor | None = None,
                     interleaved: bool = False, q: torch.Tensor | None = None,
                     q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None,
                     stream=None):
    """New tokens into the cache, keys (and queries) rotated by position.

    k, v: [T, kv_heads, head_dim] and q: [T, q_heads, head_dim] of the cache's
    type, each token contiguous, any token stride (slices of one projection
    will do).  Row r owns tokens row_offsets[r] .. row_offsets[r+1]-1 (int32
    [rows + 1]), at positions from start_pos[r] (int32 [rows]) on; tokens at
    row_offsets[rows] and behind are padding and left alone.  page_table:
    int32 [rows, width].  inv_freq: fp32 [rotary_dim / 2], or None for no
    rotation; pairs are channels (i, i + rotary_dim / 2), or (2 i, 2 i + 1)
    when ``interleaved``.  Returns (q_out, k_out): the rotated queries (None
    without q; q itself may be given as q_out) and, where a k_out [T,
    kv_heads, head_dim] is given, the rotated keys.  Padding rows of both are
    left as they were.  Not differentiable."""
    device, dt, dim, kv = cache.device, cache.dtype, cache.head_dim, cache.kv_heads
    _current(device)
    table = _table(page_table, device)
    rows = table.rows
    ks = _tokens(k, "k", dt, None, kv, dim, device)
    T = k.shape[0]
    vs = _tokens(v, "v", dt, T, kv, dim, device)
    offs = _arg(row_offsets, "row_offsets", torch.int32, (rows + 1,), device)
    start = _arg(start_pos, "start_pos", torch.int32, (rows,), device)
    qs = heads = rot = 0
    qp = qo = ko = freq = None
    if q is not None:
        qs = _tokens(q, "q", dt, T, None, dim, device)
        qp, heads = q.data_ptr(), q.shape[1]
        if q_out is None:
            q_out = _empty((T, heads, dim), dt, device, stream)
            qo = q_out.data_ptr()
        else:
            qo = _arg(q_out, "q_out", dt, (T, heads, dim), device)
    elif q_out is not None:
        raise ValueError("q_out needs q")
    if inv_freq is not None:
        rot = 2 * inv_freq.numel()
        freq = _arg(inv_freq, "inv_freq", torch.float32, (rot // 2,), device)
    if k_out is not None:
        ko = _arg(k_out, "k_out", dt, (T, kv, dim), device)
    _check(lib().msa_paged_append(
        cache._ref, ctypes.byref(table), offs, start, T, k.data_ptr(), ks, v.data_ptr(), vs, qp,
        qs, heads, freq, rot, 1 if interleaved else 0, qo, ko, _stream(stream)),
        "msa_paged_append")
    return q_out, k_out


def msa_paged_index(index: PagedIndex, ik: torch.Tensor, page_table: torch.Tensor,
                    row_offsets: torch.Tensor, start_pos: torch.Tensor, stream=None) -> None:
    """New tokens' index keys (bf16 [T, heads, dim], each token contiguous)
    into their pages, and the means of the blocks they fall in.  Rows,
    positions and padding as for ``msa_paged_append``."""
    device = index.device
    _current(device)
    table = _table(page_table, device)
    s = _tokens(ik, "ik", torch.bfloat16, None, index.heads, index.dim, device)
    offs = _arg(row_offsets, "row_offsets", torch.int32, (table.rows + 1,), device)
    start = _arg(start_pos, "start_pos", torch.int32, (table.rows,), device)
    _check(lib().msa_paged_index(index._ref, ctypes.byref(table), offs, start, ik.shape[0],
                                 ik.data_ptr(), s, _stream(stream)), "msa_paged_index")


def msa_paged_select(index: PagedIndex, iq: torch.Tensor, page_table: torch.Tensor,
                     kv_len: torch.Tensor, force_local: bool = True,
                     q2k: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """q2k int32 [heads, rows, 16] for the newest token of each row from its
    index query (bf16 [rows, heads, dim]) and the cached block means; the
    rules of ``msa_select_blocks``.  kv_len: int32 [rows], the new token
    included, 0 for a row that is not in use."""
    device, heads = index.device, index.heads
    _current(device)
    table = _table(page_table, device)
    rows = table.rows
    qp = _arg(iq, "iq", torch.bfloat16, (rows, heads, index.dim), device)
    lens = _arg(kv_len, "kv_len", torch.int32, (rows,), device)
    if q2k is None:
        q2k = _empty((heads, rows, TOPK), torch.int32, device, stream)
        out = q2k.data_ptr()
    else:
        out = _arg(q2k, "q2k", torch.int32, (heads, rows, TOPK), device)
    _check(lib().msa_paged_select(index._ref, ctypes.byref(table), lens, qp,
                                  1 if force_local else 0, out, _stream(stream)),
           "msa_paged_select")
    return q2k


def msa_paged_decode(cache: PagedCache, q: torch.Tensor, page_table: torch.Tensor,
                     kv_len: torch.Tensor, softmax_scale: float,
                     q2k: torch.Tensor | None = None, o: torch.Tensor | None = None,
                     lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                     stream=None):
    """Attention of one token of each row over the cache: (O [rows, q_heads,
    head_dim], LSE fp32 [rows, q_heads]).

    q: [rows, q_heads, head_dim] of the cache's type, up to 16 query heads a
    key head; kv_len: int32 [rows], keys that each row attends (0: none, O = 0
    and LSE = -inf); q2k: int32 [kv_heads, rows, 16], or None for every key.
    A workspace serves one call at a time.  Not differentiable."""
    device = cache.device
    _current(device)
    table = _table(page_table, device)
    rows = table.rows
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise ValueError("q must be a [rows, q_heads, head_dim] tensor")
    heads = q.shape[1]
    shape = (rows, heads, cache.head_dim)
    qp = _arg(q, "q", cache.dtype, shape, device)
    lens = _arg(kv_len, "kv_len", torch.int32, (rows,), device)
    slots = None
    if q2k is not None:
        slots = _arg(q2k, "q2k", torch.int32, (cache.kv_heads, rows, TOPK), device)
    if o is None:
        o = _empty(shape, cache.dtype, device, stream)
        op = o.data_ptr()
    else:
        op = _arg(o, "o", cache.dtype, shape, device)
    if lse is None:
        lse = _empty((rows, heads), torch.float32, device, stream)
        lp = lse.data_ptr()
    else:
        lp = _arg(lse, "lse", torch.float32, (rows, heads), device)
    if workspace is None:
        workspace = _empty(paged_decode_workspace_bytes(cache, rows, heads), torch.uint8, device,
                           stream)
    nbytes = workspace.numel()
    _check(lib().msa_paged_decode(
        cache._ref, ctypes.byref(table), lens, qp, heads, float(softmax_scale), slots, op, lp,
        _arg(workspace, "workspace", torch.uint8, (nbytes,), device), nbytes, _stream(stream)),
        "msa_paged_decode")
    return o, lse
