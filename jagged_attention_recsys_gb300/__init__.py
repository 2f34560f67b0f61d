"""Python binding of libjfa (Jagged Flash Attention for GB300): argument marshalling only.

Every function here has the name of the C entry point it calls (see
``include/jfa.h``) and forwards torch CUDA tensors as raw device pointers on
the current CUDA stream.  No attention arithmetic happens in Python and there
is no fallback: if the compiled library is missing or no CUDA device is
present, the calls raise.

Build the library with ``python -m jagged_attention_recsys_gb300.build``.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os

import numpy as np
import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_build", "libjfa.so")

JFA_OK = 0
JFA_ERR_INVALID_ARG = 1
JFA_ERR_UNSUPPORTED = 2
JFA_ERR_WORKSPACE = 3
JFA_ERR_BAD_OFFSETS = 4
JFA_ERR_TIMEOUT = 5
JFA_ERR_CUDA = 6
JFA_ERR_BAD_PAGES = 7

JFA_F32 = 0
JFA_BF16 = 1
JFA_MXFP8 = 2

JFA_PLANNED = 1

KERNEL_KINDS = {"schedule": 0, "fwd": 1, "bwd_d": 2, "bwd_dkdv": 3, "bwd_dq": 4, "aux": 5,
                "norm_rope": 6, "cache": 7, "paged": 8}

ROPE_LAYOUTS = {"halves": 0, "pairs": 1}
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}

# Every symbol include/jfa.h declares.
EXPORTS = ("jfa_workspace_size", "jfa_fwd", "jfa_bwd", "jfa_cross_fwd", "jfa_cross_bwd",
           "jfa_gdpa_fwd", "jfa_gdpa_bwd", "jfa_status_check", "jfa_status_string",
           "jfa_profile_enable", "jfa_profile_reset", "jfa_profile_read", "jfa_path_for",
           "jfa_fwd_noalloc", "jfa_bbs_plan", "jfa_pooled_workspace_size", "jfa_pooled_fwd",
           "jfa_pooled_bwd", "jfa_block_workspace_size", "jfa_block_fwd", "jfa_block_bwd",
           "jfa_test_hold", "jfa_block_rope_fwd", "jfa_block_rope_bwd", "jfa_plan",
           "jfa_block_plan", "jfa_norm_rope_workspace_size", "jfa_norm_rope_fwd",
           "jfa_norm_rope_bwd", "jfa_paged_workspace_size", "jfa_cache_write", "jfa_cache_read",
           "jfa_paged_plan", "jfa_paged_fwd")


class JfaError(RuntimeError):
    def __init__(self, code, where):
        self.code = code
        super().__init__("%s: %s (status %d)" % (where, status_string(code), code))


class jfa_params(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("total_q", ctypes.c_int64),
                ("total_k", ctypes.c_int64), ("heads", ctypes.c_int32),
                ("dim_qk", ctypes.c_int32), ("dim_v", ctypes.c_int32),
                ("scale", ctypes.c_float), ("causal", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("flags", ctypes.c_int32)]


class _rope(ctypes.Structure):
    _fields_ = [("dim", ctypes.c_int32), ("layout", ctypes.c_int32), ("scaling", ctypes.c_int32),
                ("amp", ctypes.c_float), ("base", ctypes.c_double), ("factor", ctypes.c_double),
                ("orig_len", ctypes.c_double), ("turns_fast", ctypes.c_double),
                ("turns_slow", ctypes.c_double)]


class jfa_norm_rope_params(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("stride_q", ctypes.c_int64),
                ("stride_k", ctypes.c_int64), ("stride_yq", ctypes.c_int64),
                ("stride_yk", ctypes.c_int64), ("stride_dq", ctypes.c_int64),
                ("stride_dk", ctypes.c_int64), ("heads_q", ctypes.c_int32),
                ("heads_k", ctypes.c_int32), ("dim", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("norm", ctypes.c_int32), ("eps", ctypes.c_float), ("rope", _rope)]


class jfa_paged_params(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("total_q", ctypes.c_int64), ("pages", ctypes.c_int64),
                ("stride_q", ctypes.c_int64), ("stride_k", ctypes.c_int64),
                ("stride_v", ctypes.c_int64), ("heads_q", ctypes.c_int32),
                ("heads_k", ctypes.c_int32), ("dim_qk", ctypes.c_int32), ("dim_v", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("scale", ctypes.c_float), ("causal", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("cache_dtype", ctypes.c_int32), ("flags", ctypes.c_int32)]


_lib = None


def lib():
    """The loaded libjfa (ctypes.CDLL); raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libjfa is not built (%s missing); run "
                               "`python -m jagged_attention_recsys_gb300.build`" % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        vp, i64p, fp = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p
        P = ctypes.POINTER(jfa_params)
        sz = ctypes.c_size_t
        L.jfa_workspace_size.argtypes = [P]
        L.jfa_workspace_size.restype = sz
        L.jfa_path_for.argtypes = [P]
        L.jfa_path_for.restype = ctypes.c_int
        L.jfa_fwd.argtypes = [P, vp, vp, vp, i64p, vp, fp, vp, sz, vp]
        L.jfa_bwd.argtypes = [P, vp, vp, vp, vp, fp, vp, i64p, vp, vp, vp, vp, sz, vp]
        L.jfa_cross_fwd.argtypes = [P, vp, vp, vp, i64p, i64p, vp, fp, vp, sz, vp]
        L.jfa_cross_bwd.argtypes = [P, vp, vp, vp, vp, fp, vp, i64p, i64p, vp, vp, vp, vp, sz, vp]
        L.jfa_gdpa_fwd.argtypes = [P, vp, vp, vp, i64p, i64p, vp, vp, sz, vp]
        L.jfa_gdpa_bwd.argtypes = [P, vp, vp, vp, vp, i64p, i64p, vp, vp, vp, vp, sz, vp]
        for f in ("jfa_fwd", "jfa_bwd", "jfa_cross_fwd", "jfa_cross_bwd", "jfa_gdpa_fwd",
                  "jfa_gdpa_bwd"):
            getattr(L, f).restype = ctypes.c_int
        L.jfa_fwd_noalloc.argtypes = [P, vp, vp, vp, i64p, vp, fp, vp]
        L.jfa_fwd_noalloc.restype = ctypes.c_int
        L.jfa_status_check.argtypes = [vp, vp]
        L.jfa_status_check.restype = ctypes.c_int
        L.jfa_status_string.argtypes = [ctypes.c_int]
        L.jfa_status_string.restype = ctypes.c_char_p
        L.jfa_test_hold.argtypes = [ctypes.c_int]
        L.jfa_test_hold.restype = ctypes.c_int
        L.jfa_profile_enable.argtypes = [ctypes.c_int]
        L.jfa_profile_enable.restype = ctypes.c_int
        L.jfa_profile_reset.argtypes = []
        L.jfa_profile_reset.restype = ctypes.c_int
        L.jfa_profile_read.argtypes = [ctypes.c_int, ctypes.POINTER(ctypes.c_int64),
                                       ctypes.POINTER(ctypes.c_double)]
        L.jfa_profile_read.restype = ctypes.c_int
        L.jfa_bbs_plan.argtypes = [vp, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, vp, vp, vp]
        L.jfa_bbs_plan.restype = ctypes.c_int
        i32 = ctypes.c_int32
        L.jfa_pooled_workspace_size.argtypes = [P, i32]
        L.jfa_pooled_workspace_size.restype = sz
        L.jfa_pooled_fwd.argtypes = [P, i32, vp, vp, vp, i64p, vp, fp, vp, sz, vp]
        L.jfa_pooled_fwd.restype = ctypes.c_int
        L.jfa_pooled_bwd.argtypes = [P, i32, vp, vp, vp, vp, fp, vp, i64p, vp, vp, vp, vp, sz, vp]
        L.jfa_pooled_bwd.restype = ctypes.c_int
        L.jfa_block_workspace_size.argtypes = [P]
        L.jfa_block_workspace_size.restype = sz
        L.jfa_block_fwd.argtypes = [P, vp, vp, vp, i64p, vp, fp, vp, sz, vp]
        L.jfa_block_fwd.restype = ctypes.c_int
        L.jfa_block_bwd.argtypes = [P, vp, vp, vp, vp, fp, vp, i64p, vp, vp, vp, vp, sz, vp]
        L.jfa_block_bwd.restype = ctypes.c_int
        L.jfa_block_rope_fwd.argtypes = [P, vp, vp, vp, i64p, vp, fp, vp, sz, vp]
        L.jfa_block_rope_fwd.restype = ctypes.c_int
        L.jfa_block_rope_bwd.argtypes = [P, vp, vp, vp, vp, fp, vp, i64p, vp, vp, vp, vp, sz, vp]
        L.jfa_block_rope_bwd.restype = ctypes.c_int
        L.jfa_plan.argtypes = [P, i64p, i64p, vp, sz, vp]
        L.jfa_plan.restype = ctypes.c_int
        L.jfa_block_plan.argtypes = [P, i64p, vp, sz, vp]
        L.jfa_block_plan.restype = ctypes.c_int
        N = ctypes.POINTER(jfa_norm_rope_params)
        G = ctypes.POINTER(jfa_paged_params)
        L.jfa_norm_rope_workspace_size.argtypes = [N]
        L.jfa_norm_rope_workspace_size.restype = sz
        L.jfa_norm_rope_fwd.argtypes = [N] + [vp] * 8
        L.jfa_norm_rope_bwd.argtypes = [N] + [vp] * 12 + [sz, vp]
        L.jfa_paged_workspace_size.argtypes = [G]
        L.jfa_paged_workspace_size.restype = sz
        L.jfa_cache_write.argtypes = [G] + [vp] * 10 + [sz, vp]
        L.jfa_cache_read.argtypes = [G] + [vp] * 10 + [sz, vp]
        L.jfa_paged_plan.argtypes = [G, vp, vp, vp, sz, vp]
        L.jfa_paged_fwd.argtypes = [G] + [vp] * 11 + [sz, vp]
        for f in ("jfa_norm_rope_fwd", "jfa_norm_rope_bwd", "jfa_cache_write", "jfa_cache_read",
                  "jfa_paged_plan", "jfa_paged_fwd"):
            getattr(L, f).restype = ctypes.c_int
        _lib = L
    return _lib


def status_string(code: int) -> str:
    return lib().jfa_status_string(int(code)).decode()


def _check(code, where):
    if code != JFA_OK:
        raise JfaError(code, where)


def _dtype_code(t: torch.dtype) -> int:
    if t == torch.float32:
        return JFA_F32
    if t == torch.bfloat16:
        return JFA_BF16
    raise TypeError("libjfa takes fp32 or bf16 tensors, got %s" % t)


def make_params(batch, total_q, total_k, heads, dim_qk, dim_v, dtype, scale=None, causal=False):
    if scale is None:
        scale = 1.0 / math.sqrt(dim_qk)
    return jfa_params(int(batch), int(total_q), int(total_k), int(heads), int(dim_qk),
                      int(dim_v), float(scale), int(bool(causal)), _dtype_code(dtype))


def params_for(q, k, v, offs_q, scale=None, causal=False):
    return make_params(offs_q.numel() - 1, q.shape[0], k.shape[0], q.shape[1], q.shape[2],
                       v.shape[2], q.dtype, scale, causal)


def jfa_workspace_size(p: jfa_params) -> int:
    return int(lib().jfa_workspace_size(ctypes.byref(p)))


def jfa_path_for(p: jfa_params) -> int:
    return int(lib().jfa_path_for(ctypes.byref(p)))


def jfa_bbs_plan(cost, sub=128, ranks=1):
    """Base Batch Shuffling plan (host only): returns (sub_rank, sub_slot, rank_cost) numpy
    arrays for per-sample costs `cost`, `sub` samples per sub-batch and `ranks` ranks."""
    c = np.ascontiguousarray(np.asarray(cost, dtype=np.int64))
    n_sub = -(-c.size // int(sub)) if int(sub) > 0 else 0
    sub_rank = np.zeros(max(n_sub, 1), np.int32)
    sub_slot = np.zeros(max(n_sub, 1), np.int32)
    rank_cost = np.zeros(max(int(ranks), 1), np.int64)
    _check(lib().jfa_bbs_plan(c.ctypes.data if c.size else None, c.size, int(sub), int(ranks),
                              sub_rank.ctypes.data, sub_slot.ctypes.data, rank_cost.ctypes.data),
           "jfa_bbs_plan")
    return sub_rank[:n_sub], sub_slot[:n_sub], rank_cost[:int(ranks)]


def workspace(p: jfa_params, device="cuda") -> torch.Tensor:
    """A device workspace large enough for every call with these params."""
    return torch.empty(max(jfa_workspace_size(p), 256), dtype=torch.uint8, device=device)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _check_tensors(q, k, v, offs_q, offs_k=None):
    for t in (q, k, v):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("q, k, v must be contiguous CUDA tensors")
    for o in (offs_q, offs_k):
        if o is not None and (o.dtype != torch.int64 or not o.is_cuda):
            raise ValueError("offsets must be int64 CUDA tensors")


def _prep(q, k, v, offs_q, offs_k, ws, scale, causal, planned=False):
    _check_tensors(q, k, v, offs_q, offs_k)
    p = params_for(q, k, v, offs_q, scale, causal)
    if planned:
        if ws is None:
            raise ValueError("a planned call needs the workspace its plan was built in")
        p.flags = JFA_PLANNED
    if ws is None:
        ws = workspace(p, q.device)
    return p, ws


def jfa_plan(q, k, v, offs_q, offs_k=None, *, scale=None, causal=False, ws=None, stream=None):
    """Builds the work lists of the forward and backward calls on these inputs' shapes and
    offsets into ``ws`` (allocated if None) and returns ``ws``; later calls given
    ``planned=True``, the same offsets and this workspace skip their own scheduling.
    offs_k=None means self-attention."""
    offs_k = offs_q if offs_k is None else offs_k
    p, ws = _prep(q, k, v, offs_q, offs_k, ws, scale, causal)
    _check(lib().jfa_plan(ctypes.byref(p), _ptr(offs_q), _ptr(offs_k), _ptr(ws), ws.numel(),
                          _stream(stream)), "jfa_plan")
    return ws


def jfa_fwd(q, k, v, offs, *, scale=None, causal=False, o=None, lse=None, ws=None, stream=None,
            planned=False):
    """Softmax self-attention forward; returns (o, lse)."""
    p, ws = _prep(q, k, v, offs, None, ws, scale, causal, planned)
    if o is None:
        o = torch.empty(q.shape[0], q.shape[1], v.shape[2], dtype=q.dtype, device=q.device)
    if lse is None:
        lse = torch.empty(q.shape[0], q.shape[1], dtype=torch.float32, device=q.device)
    _check(lib().jfa_fwd(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(offs), _ptr(o),
                         _ptr(lse), _ptr(ws), ws.numel(), _stream(stream)), "jfa_fwd")
    return o, lse


def jfa_fwd_noalloc(q, k, v, offs, *, scale=None, causal=False, o=None, lse=None, stream=None):
    """jfa_fwd without a workspace (scratch in a static device array); returns (o, lse).

    For callers that cannot allocate device memory; pass preallocated ``o`` and ``lse``
    to keep the call itself free of allocations.
    """
    p = params_for(q, k, v, offs, scale, causal)
    if o is None:
        o = torch.empty(q.shape[0], q.shape[1], v.shape[2], dtype=q.dtype, device=q.device)
    if lse is None:
        lse = torch.empty(q.shape[0], q.shape[1], dtype=torch.float32, device=q.device)
    _check(lib().jfa_fwd_noalloc(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(offs),
                                 _ptr(o), _ptr(lse), _stream(stream)), "jfa_fwd_noalloc")
    return o, lse


def jfa_bwd(q, k, v, o, lse, dout, offs, *, scale=None, causal=False, dq=None, dk=None,
            dv=None, ws=None, stream=None, planned=False):
    """Softmax self-attention backward; returns (dq, dk, dv)."""
    p, ws = _prep(q, k, v, offs, None, ws, scale, causal, planned)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    _check(lib().jfa_bwd(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse),
                         _ptr(dout), _ptr(offs), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(ws),
                         ws.numel(), _stream(stream)), "jfa_bwd")
    return dq, dk, dv


def jfa_cross_fwd(q, k, v, offs_q, offs_k, *, scale=None, o=None, lse=None, ws=None,
                  stream=None, planned=False):
    """Softmax cross-attention forward (independent key offsets); returns (o, lse)."""
    p, ws = _prep(q, k, v, offs_q, offs_k, ws, scale, False, planned)
    if o is None:
        o = torch.empty(q.shape[0], q.shape[1], v.shape[2], dtype=q.dtype, device=q.device)
    if lse is None:
        lse = torch.empty(q.shape[0], q.shape[1], dtype=torch.float32, device=q.device)
    _check(lib().jfa_cross_fwd(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(offs_q),
                               _ptr(offs_k), _ptr(o), _ptr(lse), _ptr(ws), ws.numel(),
                               _stream(stream)), "jfa_cross_fwd")
    return o, lse


def jfa_cross_bwd(q, k, v, o, lse, dout, offs_q, offs_k, *, scale=None, dq=None, dk=None,
                  dv=None, ws=None, stream=None, planned=False):
    """Backward of jfa_cross_fwd; returns (dq, dk, dv)."""
    p, ws = _prep(q, k, v, offs_q, offs_k, ws, scale, False, planned)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    _check(lib().jfa_cross_bwd(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse),
                               _ptr(dout), _ptr(offs_q), _ptr(offs_k), _ptr(dq), _ptr(dk),
                               _ptr(dv), _ptr(ws), ws.numel(), _stream(stream)), "jfa_cross_bwd")
    return dq, dk, dv


def jfa_gdpa_fwd(q, k, v, offs_q, offs_k=None, *, scale=None, causal=False, o=None, ws=None,
                 stream=None, planned=False):
    """SiLU(s)/L attention forward; returns o.  offs_k=None means self-attention."""
    offs_k = offs_q if offs_k is None else offs_k
    p, ws = _prep(q, k, v, offs_q, offs_k, ws, scale, causal, planned)
    if o is None:
        o = torch.empty(q.shape[0], q.shape[1], v.shape[2], dtype=q.dtype, device=q.device)
    _check(lib().jfa_gdpa_fwd(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(offs_q),
                              _ptr(offs_k), _ptr(o), _ptr(ws), ws.numel(), _stream(stream)),
           "jfa_gdpa_fwd")
    return o


def jfa_gdpa_bwd(q, k, v, dout, offs_q, offs_k=None, *, scale=None, causal=False, dq=None,
                 dk=None, dv=None, ws=None, stream=None, planned=False):
    """Backward of jfa_gdpa_fwd; returns (dq, dk, dv)."""
    offs_k = offs_q if offs_k is None else offs_k
    p, ws = _prep(q, k, v, offs_q, offs_k, ws, scale, causal, planned)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    _check(lib().jfa_gdpa_bwd(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(dout),
                              _ptr(offs_q), _ptr(offs_k), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(ws),
                              ws.numel(), _stream(stream)), "jfa_gdpa_bwd")
    return dq, dk, dv


def jfa_status_check(ws, stream=None) -> int:
    """Synchronises the stream and returns the device status word of the last call on ``ws``."""
    return int(lib().jfa_status_check(_ptr(ws), _stream(stream)))


def jfa_test_hold(on: bool):
    """Test hook of the kernels' bounded waits (see jfa_test_hold in include/jfa.h)."""
    _check(lib().jfa_test_hold(int(bool(on))), "jfa_test_hold")


def jfa_profile_enable(on: bool = True):
    _check(lib().jfa_profile_enable(int(bool(on))), "jfa_profile_enable")


def jfa_profile_reset():
    _check(lib().jfa_profile_reset(), "jfa_profile_reset")


def jfa_profile_read(kind: str):
    """(launches, total_ms) of one kernel kind since the last reset."""
    n = ctypes.c_int64(0)
    ms = ctypes.c_double(0.0)
    _check(lib().jfa_profile_read(KERNEL_KINDS[kind], ctypes.byref(n), ctypes.byref(ms)),
           "jfa_profile_read")
    return int(n.value), float(ms.value)


# ----------------------------------------------------------------------------- pooled attention
def pooled_params(q, k, v, offs_k, scale=None):
    """Params of a pooled call: q [m,H,Dqk] shared rows; B = len(offs_k)-1; o has B*m rows."""
    B, m = offs_k.numel() - 1, q.shape[0]
    return make_params(B, B * m, k.shape[0], q.shape[1], q.shape[2], v.shape[2], q.dtype, scale,
                       False), m


def pooled_workspace(p: jfa_params, m: int, device="cuda") -> torch.Tensor:
    n = int(lib().jfa_pooled_workspace_size(ctypes.byref(p), int(m)))
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def _pooled_prep(q, k, v, offs_k, ws, scale):
    _check_tensors(q, k, v, offs_k)
    p, m = pooled_params(q, k, v, offs_k, scale)
    if ws is None:
        ws = pooled_workspace(p, m, q.device)
    return p, m, ws


def jfa_pooled_fwd(q, k, v, offs_k, *, scale=None, o=None, lse=None, ws=None, stream=None):
    """Pooled multi-head attention forward: the m rows of q attend every sequence;
    returns (o [B*m,H,Dv], lse [B*m,H])."""
    p, m, ws = _pooled_prep(q, k, v, offs_k, ws, scale)
    if o is None:
        o = torch.empty(p.total_q, q.shape[1], v.shape[2], dtype=q.dtype, device=q.device)
    if lse is None:
        lse = torch.empty(p.total_q, q.shape[1], dtype=torch.float32, device=q.device)
    _check(lib().jfa_pooled_fwd(ctypes.byref(p), m, _ptr(q), _ptr(k), _ptr(v), _ptr(offs_k),
                                _ptr(o), _ptr(lse), _ptr(ws), ws.numel(), _stream(stream)),
           "jfa_pooled_fwd")
    return o, lse


def jfa_pooled_bwd(q, k, v, o, lse, dout, offs_k, *, scale=None, dq=None, dk=None, dv=None,
                   ws=None, stream=None):
    """Backward of jfa_pooled_fwd; returns (dq [m,H,Dqk] summed over sequences, dk, dv)."""
    p, m, ws = _pooled_prep(q, k, v, offs_k, ws, scale)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    _check(lib().jfa_pooled_bwd(ctypes.byref(p), m, _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse),
                                _ptr(dout), _ptr(offs_k), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(ws),
                                ws.numel(), _stream(stream)), "jfa_pooled_bwd")
    return dq, dk, dv


# ----------------------------------------------------------------------------- BlockAttention
def block_workspace(p: jfa_params, device="cuda") -> torch.Tensor:
    n = int(lib().jfa_block_workspace_size(ctypes.byref(p)))
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


def _block_prep(q, k, v, offs, ws, scale, causal, planned=False):
    _check_tensors(q, k, v, offs)
    p = params_for(q, k, v, offs, scale, causal)
    if planned:
        if ws is None:
            raise ValueError("a planned call needs the workspace its plan was built in")
        p.flags = JFA_PLANNED
    return p, block_workspace(p, q.device) if ws is None else ws


def jfa_block_plan(q, k, v, offs, *, scale=None, causal=False, ws=None, stream=None):
    """The block offsets, rotary table and work lists of the BlockAttention calls on these
    inputs, built into ``ws`` (allocated if None); returns ``ws``."""
    p, ws = _block_prep(q, k, v, offs, ws, scale, causal)
    _check(lib().jfa_block_plan(ctypes.byref(p), _ptr(offs), _ptr(ws), ws.numel(),
                                _stream(stream)), "jfa_block_plan")
    return ws


def jfa_block_fwd(q, k, v, offs, *, scale=None, causal=False, o=None, lse=None, ws=None,
                  stream=None, rope=False, planned=False):
    """BlockAttention forward (softmax within fixed 64-row blocks); returns (o, lse).
    With ``rope``, the fused rotary position embedding (jfa_block_rope_fwd)."""
    p, ws = _block_prep(q, k, v, offs, ws, scale, causal, planned)
    if o is None:
        o = torch.empty(q.shape[0], q.shape[1], v.shape[2], dtype=q.dtype, device=q.device)
    if lse is None:
        lse = torch.empty(q.shape[0], q.shape[1], dtype=torch.float32, device=q.device)
    name = "jfa_block_rope_fwd" if rope else "jfa_block_fwd"
    _check(getattr(lib(), name)(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(offs), _ptr(o),
                                _ptr(lse), _ptr(ws), ws.numel(), _stream(stream)), name)
    return o, lse


def jfa_block_bwd(q, k, v, o, lse, dout, offs, *, scale=None, causal=False, dq=None, dk=None,
                  dv=None, ws=None, stream=None, rope=False, planned=False):
    """Backward of jfa_block_fwd; returns (dq, dk, dv).  With ``rope``, the backward of the
    fused rotary position embedding as well (jfa_block_rope_bwd)."""
    p, ws = _block_prep(q, k, v, offs, ws, scale, causal, planned)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    name = "jfa_block_rope_bwd" if rope else "jfa_block_bwd"
    _check(getattr(lib(), name)(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse),
                                _ptr(dout), _ptr(offs), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(ws),
                                ws.numel(), _stream(stream)), name)
    return dq, dk, dv


# ----------------------------------------------------------------------------- shared checks
# The handle alone: building a torch Stream around it costs 2.5 us a call.
_current_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _on(device):
    """The raw current stream of ``device``, which must be the current one."""
    if device.index != _current_device():
        raise ValueError("tensors are on %s, which is not the current device" % device)
    return _current_raw_stream(device.index)


def _in_stream(fn):
    """Calls with a ``stream`` run with it current: what they allocate belongs to it."""
    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        if stream is None:
            return fn(*args, **kw)
        with torch.cuda.stream(stream):
            return fn(*args, **kw)
    return call


def _rows(name, t, dtype, device, heads=None, dim=None, tokens=None):
    """Checks [T, heads, dim] rows with contiguous heads; returns the stride between tokens."""
    if t is None or t.dim() != 3 or t.dtype is not dtype or t.device != device:
        raise ValueError("%s must be a [tokens, heads, dim] %s tensor on %s" % (name, dtype, device))
    T, H, D = t.shape
    if heads not in (None, H) or dim not in (None, D) or tokens not in (None, T):
        raise ValueError("%s has shape %s, which does not fit the other arguments" % (name, tuple(t.shape)))
    st, sh, sd = t.stride()
    if (D > 1 and sd != 1) or (H > 1 and sh != D):
        if T * H * D:
            raise ValueError("%s: the heads of a token must be contiguous" % name)
    return st if T > 1 else H * D


def _plain(name, t, dtype, shape, device):
    if t is None or t.dtype is not dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s tensor of shape %s on %s"
                         % (name, dtype, tuple(shape), device))


def _addr(t):
    return None if t is None else t.data_ptr()


# ----------------------------------------------------------------------------- norms, rotary positions
def jfa_rope(dim, *, layout="halves", base=10000.0, scaling="none", factor=1.0, orig_len=0.0,
             turns_fast=32.0, turns_slow=1.0, amp=1.0):
    """The rotation of jfa_norm_rope_*: the first ``dim`` columns of every head, in ``layout``
    "halves" or "pairs", frequencies changed by ``scaling`` ("none", "linear", "ntk", "yarn")."""
    return _rope(int(dim), ROPE_LAYOUTS[layout], ROPE_SCALINGS[scaling], amp, base, factor, orig_len,
                 turns_fast, turns_slow)


def _norm_rope_params(q, k, pos, wq, wk, eps, rope, norm):
    x = q if q is not None else k
    if x is None:
        raise ValueError("q and k are both None")
    if x.dim() != 3 or not x.is_cuda:
        raise ValueError("q and k must be [tokens, heads, dim] CUDA tensors")
    if not norm and (wq is not None or wk is not None):
        raise ValueError("norm=False takes no weights")
    (T, _, D), dtype, dev = x.shape, x.dtype, x.device
    sq = hq = sk = hk = 0
    if rope is not None and rope.dim:
        _plain("pos", pos, torch.int64, (T,), dev)
    if q is not None:
        sq, hq = _rows("q", q, dtype, dev, None, D, T), q.shape[1]
    if k is not None:
        sk, hk = _rows("k", k, dtype, dev, None, D, T), k.shape[1]
    if wq is not None:
        _plain("wq", wq, torch.float32, (D,), dev)
    if wk is not None:
        _plain("wk", wk, torch.float32, (D,), dev)
    p = jfa_norm_rope_params(T, sq, sk, 0, 0, 0, 0, hq, hk, D, _dtype_code(dtype), 1 if norm else 0, eps)
    if rope is not None:
        p.rope = rope
    return p, x


def _rows_like(t):
    """An empty contiguous tensor of the rows of ``t`` (the copied options cost less than given ones)."""
    return torch.empty_like(t) if t.is_contiguous() else torch.empty(t.shape, dtype=t.dtype, device=t.device)


def _out(name, t, like, make=True):
    """A tensor of the rows of ``like`` and its stride between tokens; made if None."""
    T, H, D = like.shape
    if t is None and make:
        return _rows_like(like), H * D
    return t, _rows(name, t, like.dtype, like.device, H, D, T)


@_in_stream
def jfa_norm_rope_fwd(q, k, pos, wq=None, wk=None, *, rope=None, eps=1e-6, norm=True, yq=None,
                      yk=None, stream=None):
    """RMS norm of every head of q [T, Hq, D] and k [T, Hk, D] (either may be None) with the
    rotary position embedding ``rope`` (jfa_rope) at positions ``pos`` [T]; returns (yq, yk)."""
    p, x = _norm_rope_params(q, k, pos, wq, wk, eps, rope, norm)
    if q is not None:
        yq, p.stride_yq = _out("yq", yq, q)
    if k is not None:
        yk, p.stride_yk = _out("yk", yk, k)
    _check(lib().jfa_norm_rope_fwd(ctypes.byref(p), _addr(q), _addr(k), _addr(pos), _addr(wq), _addr(wk),
                                   _addr(yq), _addr(yk), _on(x.device)), "jfa_norm_rope_fwd")
    return yq, yk


@_in_stream
def jfa_norm_rope_bwd(q, k, pos, dyq, dyk, wq=None, wk=None, *, rope=None, eps=1e-6, norm=True,
                      dq=None, dk=None, dwq=None, dwk=None, ws=None, stream=None):
    """Backward of jfa_norm_rope_fwd; returns (dq, dk, dwq, dwk).  The weights' gradients are
    summed over tokens and heads in fp32 (None where the norm has no such weight)."""
    p, x = _norm_rope_params(q, k, pos, wq, wk, eps, rope, norm)
    f32 = dict(dtype=torch.float32, device=x.device)
    if q is not None:
        p.stride_yq = _out("dyq", dyq, q, False)[1]
        dq, p.stride_dq = _out("dq", dq, q)
        if wq is not None and dwq is None:
            dwq = torch.empty(p.dim, **f32)
    if k is not None:
        p.stride_yk = _out("dyk", dyk, k, False)[1]
        dk, p.stride_dk = _out("dk", dk, k)
        if wk is not None and dwk is None:
            dwk = torch.empty(p.dim, **f32)
    for name, w in (("dwq", dwq), ("dwk", dwk)):
        if w is not None:
            _plain(name, w, torch.float32, (p.dim,), x.device)
    if ws is None:
        n = int(lib().jfa_norm_rope_workspace_size(ctypes.byref(p)))
        ws = torch.empty(max(n, 256), dtype=torch.uint8, device=x.device)
    _check(lib().jfa_norm_rope_bwd(ctypes.byref(p), _addr(q), _addr(k), _addr(pos), _addr(wq), _addr(wk),
                                   _addr(dyq), _addr(dyk), _addr(dq), _addr(dk), _addr(dwq), _addr(dwk),
                                   _addr(ws), ws.numel(), _on(x.device)), "jfa_norm_rope_bwd")
    return dq, dk, dwq, dwk


# ----------------------------------------------------------------------------- paged cache
class PagedCache:
    """The arrays of a paged cache: k [pages, heads, page_size, dim], v likewise; with
    k_scale and v_scale (uint8 [pages, heads, page_size, dim / 32]) k and v are uint8 MXFP8
    codes, without them values."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        if k.dim() != 4 or v.dim() != 4 or k.shape[:3] != v.shape[:3]:
            raise ValueError("k and v must be [pages, heads, page_size, dim] with the same pages")
        if (k_scale is None) != (v_scale is None):
            raise ValueError("k_scale and v_scale belong together")
        if not k.is_cuda or v.device != k.device or not k.is_contiguous() or not v.is_contiguous():
            raise ValueError("the cache's arrays must be contiguous CUDA tensors on one device")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.mxfp8 = k_scale is not None
        self.pages, self.heads, self.page_size, self.dim_qk = k.shape
        self.dim_v = v.shape[3]
        if self.mxfp8:
            if k.dtype is not torch.uint8 or v.dtype is not torch.uint8 or (self.dim_qk | self.dim_v) % 32:
                raise ValueError("MXFP8 codes must be uint8, columns a multiple of 32")
            _plain("k_scale", k_scale, torch.uint8, k.shape[:3] + (self.dim_qk // 32,), k.device)
            _plain("v_scale", v_scale, torch.uint8, k.shape[:3] + (self.dim_v // 32,), k.device)
            self.dtype_code = JFA_MXFP8
        else:
            if v.dtype is not k.dtype:
                raise ValueError("k and v must be of one type")
            self.dtype_code = _dtype_code(k.dtype)

    @property
    def device(self):
        return self.k.device


def paged_cache(pages, heads, dim_qk, dim_v=None, *, page_size=64, dtype=torch.bfloat16, mxfp8=False,
                device="cuda"):
    """An empty PagedCache of values of ``dtype``, or of MXFP8 codes."""
    dim_v = dim_qk if dim_v is None else dim_v
    new = lambda d, t: torch.zeros(pages, heads, page_size, d, dtype=t, device=device)
    if not mxfp8:
        return PagedCache(new(dim_qk, dtype), new(dim_v, dtype))
    u = torch.uint8
    return PagedCache(new(dim_qk, u), new(dim_v, u), new(dim_qk // 32, u), new(dim_v // 32, u))


def paged_params(cache, table, offs, lens, total, dtype, *, heads_q=None, scale=None, causal=True):
    """Params of the calls on a paged cache (strides of contiguous rows)."""
    hk, d, dv = cache.heads, cache.dim_qk, cache.dim_v
    hq = hk if heads_q is None else heads_q
    return jfa_paged_params(offs.numel() - 1, total, cache.pages, hq * d, hk * d, hk * dv, hq, hk, d, dv,
                            cache.page_size, table.shape[1],
                            1.0 / math.sqrt(d) if scale is None else scale, 1 if causal else 0,
                            _dtype_code(dtype), cache.dtype_code, 0)


def paged_workspace(p: jfa_paged_params, device="cuda") -> torch.Tensor:
    """A workspace for every call on a paged cache with these params."""
    return torch.empty(max(int(lib().jfa_paged_workspace_size(ctypes.byref(p))), 256), dtype=torch.uint8,
                       device=device)


def _paged_prep(cache, table, offs, lens, total, dtype, heads_q, scale, causal, ws, planned):
    dev = cache.device
    if offs.dim() != 1 or table.dim() != 2 or offs.numel() < 1:
        raise ValueError("offs must be [B + 1], table [B, max_pages]")
    B = offs.numel() - 1
    _plain("offs", offs, torch.int64, (B + 1,), dev)
    _plain("lens", lens, torch.int64, (B,), dev)
    _plain("table", table, torch.int32, (B, table.shape[1]), dev)
    p = paged_params(cache, table, offs, lens, total, dtype, heads_q=heads_q, scale=scale, causal=causal)
    if planned:
        if ws is None:
            raise ValueError("a planned call needs the workspace its plan was built in")
        p.flags = JFA_PLANNED
    if ws is None:
        ws = paged_workspace(p, dev)
    elif ws.device != dev or ws.dtype is not torch.uint8 or not ws.is_contiguous():
        raise ValueError("ws must be a contiguous uint8 tensor on %s" % dev)
    return p, ws


@_in_stream
def jfa_cache_write(k, v, cache, table, offs, lens, *, ws=None, stream=None, planned=False):
    """Writes the new tokens' k [T, Hk, Dqk] and v [T, Hk, Dv] into their pages of ``cache``:
    token i of sequence b at position lens[b] - L_b + i.  Returns the workspace, whose status
    word jfa_status_check reads."""
    stride_k = _rows("k", k, k.dtype, cache.device, cache.heads, cache.dim_qk)
    stride_v = _rows("v", v, k.dtype, cache.device, cache.heads, cache.dim_v, k.shape[0])
    p, ws = _paged_prep(cache, table, offs, lens, k.shape[0], k.dtype, None, None, True, ws, planned)
    p.stride_k, p.stride_v = stride_k, stride_v
    _check(lib().jfa_cache_write(ctypes.byref(p), _addr(k), _addr(v), _addr(offs), _addr(lens), _addr(table),
                                 _addr(cache.k), _addr(cache.v), _addr(cache.k_scale), _addr(cache.v_scale),
                                 _addr(ws), ws.numel(), _on(cache.device)), "jfa_cache_write")
    return ws


@_in_stream
def jfa_cache_read(cache, table, offs, lens, total, *, dtype=torch.bfloat16, k=None, v=None, ws=None,
                   stream=None, planned=False):
    """The last L_b cached rows of every sequence, ``total`` = offs[B] of them, gathered into
    (k [total, Hk, Dqk], v [total, Hk, Dv]) of ``dtype``."""
    p, ws = _paged_prep(cache, table, offs, lens, total, dtype, None, None, True, ws, planned)
    dev = cache.device
    kshape, vshape = (total, cache.heads, cache.dim_qk), (total, cache.heads, cache.dim_v)
    if k is None:
        k = torch.empty(kshape, dtype=dtype, device=dev)
    else:
        _plain("k", k, dtype, kshape, dev)
    if v is None:
        v = torch.empty(vshape, dtype=dtype, device=dev)
    else:
        _plain("v", v, dtype, vshape, dev)
    _check(lib().jfa_cache_read(ctypes.byref(p), _addr(cache.k), _addr(cache.v), _addr(cache.k_scale),
                                _addr(cache.v_scale), _addr(offs), _addr(lens), _addr(table), _addr(k),
                                _addr(v), _addr(ws), ws.numel(), _on(dev)), "jfa_cache_read")
    return k, v


@_in_stream
def jfa_paged_plan(q, cache, table, offs, lens, *, causal=True, ws=None, stream=None):
    """The shares of work of a step's calls on ``cache`` (same offs and lens), built into
    ``ws`` (allocated if None); returns ``ws`` for calls with ``planned=True``."""
    stride_q = _rows("q", q, q.dtype, cache.device, None, cache.dim_qk)
    p, ws = _paged_prep(cache, table, offs, lens, q.shape[0], q.dtype, q.shape[1], None, causal, ws, False)
    p.stride_q = stride_q
    _check(lib().jfa_paged_plan(ctypes.byref(p), _addr(offs), _addr(lens), _addr(ws), ws.numel(),
                                _on(cache.device)), "jfa_paged_plan")
    return ws


@_in_stream
def jfa_paged_fwd(q, cache, table, offs, lens, *, scale=None, causal=True, o=None, lse=None, ws=None,
                  stream=None, planned=False):
    """Attention of the new tokens' queries q [T, Hq, Dqk] over their sequences' cached keys
    and values (the new tokens' own among them), Hq a multiple of the cache's heads; returns
    (o [T, Hq, Dv], lse [T, Hq])."""
    dev = cache.device
    stride_q = _rows("q", q, q.dtype, dev, None, cache.dim_qk)
    p, ws = _paged_prep(cache, table, offs, lens, q.shape[0], q.dtype, q.shape[1], scale, causal, ws, planned)
    p.stride_q = stride_q
    T, H = q.shape[0], q.shape[1]
    if o is None:
        o = _rows_like(q) if cache.dim_v == cache.dim_qk else torch.empty((T, H, cache.dim_v), dtype=q.dtype, device=dev)
    else:
        _plain("o", o, q.dtype, (T, H, cache.dim_v), dev)
    if lse is None:
        lse = torch.empty((T, H), dtype=torch.float32, device=dev)
    else:
        _plain("lse", lse, torch.float32, (T, H), dev)
    _check(lib().jfa_paged_fwd(ctypes.byref(p), _addr(q), _addr(cache.k), _addr(cache.v), _addr(cache.k_scale),
                               _addr(cache.v_scale), _addr(offs), _addr(lens), _addr(table), _addr(o),
                               _addr(lse), _addr(ws), ws.numel(), _on(dev)), "jfa_paged_fwd")
    return o, lse
