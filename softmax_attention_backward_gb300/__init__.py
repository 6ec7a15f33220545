"""GB300 softmax-attention training kernels: thin Python binding of libattn.so.

Every function here only marshals torch tensors (device memory and the current
stream) into the C ABI declared in include/attn.h; all arithmetic runs in the
library's CUDA kernels.  There is no CPU or eager fallback: if the library is
missing or a call fails, an exception is raised.

Entry points (same names as the C ABI):
  attn_fwd, attn_bwd_workspace_size, attn_bwd_preprocess, attn_bwd, attn_bwd_postprocess,
  sparse_attn_fwd, sparse_attn_bwd_workspace_size, sparse_attn_bwd,
  sparse_attn_bwd_deterministic_workspace_size, sparse_attn_bwd_deterministic,
  attn_bwd_fixed_scratch, attn_status_string, attn_version   (include/attn.h)
  dsa_indexer_fwd, dsa_topk, dsa_indexer_bwd_workspace_size, dsa_indexer_bwd, dsa_sparse_kl,
  csa_compressor_fwd, csa_compressor_bwd_workspace_size, csa_compressor_bwd  (include/dsa.h)
  attn_cache_append, attn_cache_fwd_workspace_size, attn_cache_fwd  (include/cache.h)
  attn_rotary_table, attn_rotary_fwd, attn_rotary_bwd  (include/rotary.h)
  linear_attn_fwd_workspace_size, linear_attn_fwd, linear_attn_bwd_workspace_size, linear_attn_bwd,
  linear_attn_step  (include/linear.h)
"""
from __future__ import annotations

import ctypes
import math
import os
import warnings

import torch

__all__ = [
    "ATTN_DQ_ATOMIC", "ATTN_DQ_SPLIT", "AttnError", "lib", "attn_fwd", "attn_bwd_workspace_size",
    "attn_bwd_preprocess", "attn_bwd", "attn_bwd_postprocess", "sparse_attn_fwd", "sparse_attn_bwd_workspace_size",
    "sparse_attn_bwd", "sparse_attn_bwd_deterministic_workspace_size", "sparse_attn_bwd_deterministic",
    "attn_status_string", "attn_version", "dense_backward",
    "SPARSE_DIM_QK", "SPARSE_DIM_V", "EXPORTED_SYMBOLS", "attn_bwd_fixed_scratch",
    "FIXED_SCRATCH_BYTES", "csa_compressor_fwd", "csa_compressor_bwd_workspace_size",
    "csa_compressor_bwd", "dsa_indexer_fwd", "dsa_topk", "dsa_indexer_bwd_workspace_size",
    "dsa_indexer_bwd", "dsa_sparse_kl", "INDEXER_HEAD_DIM", "attn_wait_selftest",
    "attn_cache_append", "attn_cache_fwd_workspace_size", "attn_cache_fwd", "attn_cache_empty",
    "attn_rotary_table", "attn_rotary_fwd", "attn_rotary_bwd",
    "linear_attn_fwd_workspace_size", "linear_attn_fwd", "linear_attn_bwd_workspace_size",
    "linear_attn_bwd", "linear_attn_step",
]

ATTN_DQ_ATOMIC = 0
ATTN_DQ_SPLIT = 1
SPARSE_DIM_QK = 576
SPARSE_DIM_V = 512
LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libattn.so")

EXPORTED_SYMBOLS = (
    "attn_fwd", "attn_bwd_workspace_size", "attn_bwd_preprocess", "attn_bwd", "attn_bwd_postprocess",
    "sparse_attn_fwd", "sparse_attn_bwd_workspace_size", "sparse_attn_bwd",
    "sparse_attn_bwd_deterministic_workspace_size", "sparse_attn_bwd_deterministic",
    "attn_status_string", "attn_version", "attn_bwd_fixed_scratch",
    "csa_compressor_fwd", "csa_compressor_bwd_workspace_size", "csa_compressor_bwd",
    "dsa_indexer_fwd", "dsa_topk", "dsa_indexer_bwd_workspace_size", "dsa_indexer_bwd",
    "dsa_sparse_kl", "attn_wait_selftest",
    "attn_cache_append", "attn_cache_fwd_workspace_size", "attn_cache_fwd",
    "attn_rotary_table", "attn_rotary_fwd", "attn_rotary_bwd",
    "linear_attn_fwd_workspace_size", "linear_attn_fwd", "linear_attn_bwd_workspace_size",
    "linear_attn_bwd", "linear_attn_step",
)
INDEXER_HEAD_DIM = 128
FIXED_SCRATCH_BYTES = 16 << 20


class AttnError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn}: {attn_status_string(code)} (status {code})")
        self.code = code


class _Problem(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int), ("seqlen", ctypes.c_int), ("heads_q", ctypes.c_int),
        ("heads_kv", ctypes.c_int), ("head_dim", ctypes.c_int), ("causal", ctypes.c_int),
        ("scale", ctypes.c_float), ("cu_seqlens", ctypes.c_void_p), ("num_seqs", ctypes.c_int),
        ("capacity", ctypes.c_int), ("max_seqlen", ctypes.c_int), ("error_word", ctypes.c_void_p),
    ]


class _SparseProblem(ctypes.Structure):
    _fields_ = [
        ("tokens", ctypes.c_int), ("heads", ctypes.c_int), ("dim_qk", ctypes.c_int),
        ("dim_v", ctypes.c_int), ("topk", ctypes.c_int), ("scale", ctypes.c_float),
        ("error_word", ctypes.c_void_p),
    ]


class _CsaProblem(ctypes.Structure):
    _fields_ = [
        ("tokens", ctypes.c_int), ("comp_capacity", ctypes.c_int), ("num_seqs", ctypes.c_int),
        ("head_dim", ctypes.c_int), ("ratio", ctypes.c_int), ("coff", ctypes.c_int),
        ("cu_seqlens", ctypes.c_void_p), ("cu_seqlens_comp", ctypes.c_void_p),
        ("error_word", ctypes.c_void_p),
    ]


class _IndexerProblem(ctypes.Structure):
    _fields_ = [
        ("tokens", ctypes.c_int), ("heads", ctypes.c_int), ("head_dim", ctypes.c_int),
        ("topk", ctypes.c_int), ("use_relu", ctypes.c_int), ("logits_ld", ctypes.c_int),
        ("cu_seqlens", ctypes.c_void_p), ("num_seqs", ctypes.c_int),
        ("error_word", ctypes.c_void_p),
    ]


class _CacheProblem(ctypes.Structure):
    _fields_ = [
        ("num_seqs", ctypes.c_int), ("tokens", ctypes.c_int), ("heads_q", ctypes.c_int),
        ("heads_kv", ctypes.c_int), ("head_dim", ctypes.c_int), ("cache_type", ctypes.c_int),
        ("page_size", ctypes.c_int), ("num_pages", ctypes.c_int), ("max_pages", ctypes.c_int),
        ("max_new", ctypes.c_int), ("causal", ctypes.c_int), ("scale", ctypes.c_float),
        ("rot_dim", ctypes.c_int), ("rot_interleaved", ctypes.c_int),
        ("max_position", ctypes.c_int), ("q_stride", ctypes.c_int64),
        ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64),
        ("cu_seqlens", ctypes.c_void_p), ("seqlens_kv", ctypes.c_void_p),
        ("page_table", ctypes.c_void_p), ("error_word", ctypes.c_void_p),
    ]


class _RotaryTable(ctypes.Structure):
    _fields_ = [
        ("max_position", ctypes.c_int), ("rot_dim", ctypes.c_int), ("base", ctypes.c_double),
        ("scaling", ctypes.c_int), ("factor", ctypes.c_double), ("original", ctypes.c_int),
        ("fast", ctypes.c_double), ("slow", ctypes.c_double), ("magnitude", ctypes.c_double),
    ]


class _RotaryProblem(ctypes.Structure):
    _fields_ = [
        ("tokens", ctypes.c_int), ("heads_q", ctypes.c_int), ("heads_k", ctypes.c_int),
        ("head_dim", ctypes.c_int), ("rot_dim", ctypes.c_int), ("rot_offset", ctypes.c_int),
        ("interleaved", ctypes.c_int), ("max_position", ctypes.c_int), ("seqlen", ctypes.c_int),
        ("num_seqs", ctypes.c_int), ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
        ("cu_seqlens", ctypes.c_void_p), ("positions", ctypes.c_void_p),
        ("error_word", ctypes.c_void_p),
    ]


class _LinearProblem(ctypes.Structure):
    _fields_ = [
        ("num_seqs", ctypes.c_int), ("seqlen", ctypes.c_int), ("tokens", ctypes.c_int),
        ("heads_q", ctypes.c_int), ("heads_kv", ctypes.c_int), ("head_dim", ctypes.c_int),
        ("scale", ctypes.c_float), ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
        ("v_stride", ctypes.c_int64), ("dout_stride", ctypes.c_int64),
        ("cu_seqlens", ctypes.c_void_p), ("log_decay", ctypes.c_void_p),
        ("error_word", ctypes.c_void_p),
    ]


class _LinearStep(ctypes.Structure):
    _fields_ = [
        ("num_seqs", ctypes.c_int), ("num_slots", ctypes.c_int), ("heads_q", ctypes.c_int),
        ("heads_kv", ctypes.c_int), ("head_dim", ctypes.c_int), ("scale", ctypes.c_float),
        ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64), ("v_stride", ctypes.c_int64),
        ("slots", ctypes.c_void_p), ("log_decay", ctypes.c_void_p),
        ("error_word", ctypes.c_void_p),
    ]


_LIB = None


def lib() -> ctypes.CDLL:
    """Loads libattn.so (built by __graft_entry__.build() or build.py)."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m softmax_attention_backward_gb300.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, sz, i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
        P = ctypes.POINTER(_Problem)
        SP = ctypes.POINTER(_SparseProblem)
        L.attn_fwd.argtypes = [P, vp, vp, vp, vp, vp, vp]
        L.attn_bwd_workspace_size.argtypes = [P, i32]
        L.attn_bwd_workspace_size.restype = sz
        L.attn_bwd_preprocess.argtypes = [P, i32, vp, vp, vp, vp, sz, vp]
        L.attn_bwd.argtypes = [P, i32, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.attn_bwd_postprocess.argtypes = [P, i32, vp, sz, vp, vp, vp, vp]
        L.sparse_attn_fwd.argtypes = [SP, vp, vp, vp, vp, vp, vp]
        L.sparse_attn_bwd_workspace_size.argtypes = [SP]
        L.sparse_attn_bwd_workspace_size.restype = sz
        L.sparse_attn_bwd.argtypes = [SP, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.sparse_attn_bwd_deterministic_workspace_size.argtypes = [SP]
        L.sparse_attn_bwd_deterministic_workspace_size.restype = sz
        L.sparse_attn_bwd_deterministic.argtypes = [SP, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.attn_bwd_fixed_scratch.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
        CP = ctypes.POINTER(_CsaProblem)
        L.csa_compressor_fwd.argtypes = [CP, vp, vp, vp, vp, vp]
        L.csa_compressor_bwd_workspace_size.argtypes = [CP]
        L.csa_compressor_bwd_workspace_size.restype = sz
        L.csa_compressor_bwd.argtypes = [CP, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        IP = ctypes.POINTER(_IndexerProblem)
        L.dsa_indexer_fwd.argtypes = [IP, vp, vp, vp, vp, vp]
        L.dsa_topk.argtypes = [IP, vp, vp, vp, vp, vp]
        L.dsa_indexer_bwd_workspace_size.argtypes = [IP]
        L.dsa_indexer_bwd_workspace_size.restype = sz
        L.dsa_indexer_bwd.argtypes = [IP, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.dsa_sparse_kl.argtypes = [SP, vp, vp, vp, vp, vp, vp, vp, vp, vp]
        KP = ctypes.POINTER(_CacheProblem)
        L.attn_cache_append.argtypes = [KP, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp]
        L.attn_cache_fwd_workspace_size.argtypes = [KP]
        L.attn_cache_fwd_workspace_size.restype = sz
        L.attn_cache_fwd.argtypes = [KP, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        RP = ctypes.POINTER(_RotaryProblem)
        L.attn_rotary_table.argtypes = [ctypes.POINTER(_RotaryTable), vp, vp]
        L.attn_rotary_fwd.argtypes = [RP, vp, vp, vp, vp, vp, vp]
        L.attn_rotary_bwd.argtypes = [RP, vp, vp, vp, vp, vp, vp]
        LP = ctypes.POINTER(_LinearProblem)
        L.linear_attn_fwd_workspace_size.argtypes = [LP]
        L.linear_attn_fwd_workspace_size.restype = sz
        L.linear_attn_fwd.argtypes = [LP, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.linear_attn_bwd_workspace_size.argtypes = [LP]
        L.linear_attn_bwd_workspace_size.restype = sz
        L.linear_attn_bwd.argtypes = [LP, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
        L.linear_attn_step.argtypes = [ctypes.POINTER(_LinearStep), vp, vp, vp, vp, vp, vp]
        L.attn_wait_selftest.argtypes = [vp, ctypes.c_uint, vp, vp]
        L.attn_wait_selftest.restype = i32
        L.attn_status_string.argtypes = [i32]
        L.attn_status_string.restype = ctypes.c_char_p
        L.attn_version.argtypes = []
        for name in ("attn_fwd", "attn_bwd_preprocess", "attn_bwd", "attn_bwd_postprocess",
                     "sparse_attn_fwd", "sparse_attn_bwd", "attn_bwd_fixed_scratch",
                     "csa_compressor_fwd", "csa_compressor_bwd", "dsa_indexer_fwd", "dsa_topk",
                     "dsa_indexer_bwd", "dsa_sparse_kl", "attn_cache_append", "attn_cache_fwd",
                     "attn_rotary_table", "attn_rotary_fwd", "attn_rotary_bwd", "linear_attn_fwd",
                     "linear_attn_bwd", "linear_attn_step"):
            getattr(L, name).restype = i32
        _LIB = L
    return _LIB


def attn_status_string(code: int) -> str:
    return lib().attn_status_string(int(code)).decode()


def attn_version() -> int:
    return int(lib().attn_version())


def attn_wait_selftest(limit_us=1000, *, device=None, stream=None):
    """Runs the bounded-wait self-test; returns (result bits, error word)
    after synchronizing (7 and ATTN_DEVERR_TIMEOUT when the mechanism works)."""
    dev = device if device is not None else torch.device("cuda", torch.cuda.current_device())
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    res = torch.full((1,), -1, dtype=torch.int32, device=dev)
    _check("attn_wait_selftest", lib().attn_wait_selftest(_ptr(err), int(limit_us), _ptr(res),
                                                          _stream(stream)))
    torch.cuda.synchronize(dev)
    return int(res.item()), int(err.item())


# ----------------------------------------------------------------------------
# marshalling helpers
# ----------------------------------------------------------------------------
def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _check(fn, code):
    if code != 0:
        raise AttnError(fn, code)


def _need(t, name, dtype, device=None):
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    return t


def _nondeterministic(what: str, instead: str):
    if torch.are_deterministic_algorithms_enabled():
        msg = f"{what} accumulates with fp32 atomics and is not bitwise reproducible"
        if torch.is_deterministic_algorithms_warn_only_enabled():
            warnings.warn(msg, RuntimeWarning, stacklevel=3)
        else:
            raise RuntimeError(f"{msg}; use {instead}")


def _problem(q, k, causal, scale, cu_seqlens, max_seqlen, error_word):
    p = _Problem()
    if cu_seqlens is None:
        if q.dim() != 4:
            raise ValueError("dense q must be [batch, seqlen, heads, head_dim]")
        p.batch, p.seqlen, p.heads_q, p.head_dim = q.shape
        p.heads_kv = k.shape[2]
        p.cu_seqlens = None
        p.num_seqs = 0
        p.capacity = 0
        p.max_seqlen = q.shape[1]
    else:
        if q.dim() != 3:
            raise ValueError("THD q must be [capacity, heads, head_dim]")
        _need(cu_seqlens, "cu_seqlens", torch.int32, q.device)
        p.batch, p.seqlen = 1, 0
        p.capacity, p.heads_q, p.head_dim = q.shape
        p.heads_kv = k.shape[1]
        p.cu_seqlens = cu_seqlens.data_ptr()
        p.num_seqs = cu_seqlens.numel() - 1
        if max_seqlen is None:
            # Deriving it from cu_seqlens would read device memory on the host: a
            # hidden synchronisation, and a stale value under graph capture.
            raise ValueError("THD calls need max_seqlen, an upper bound on every "
                             "sequence length (the host never reads cu_seqlens)")
        p.max_seqlen = int(max_seqlen)
    p.causal = 1 if causal else 0
    p.scale = float(scale if scale is not None else 1.0 / math.sqrt(p.head_dim))
    p.error_word = None if error_word is None else error_word.data_ptr()
    return p


def _lse_shape(q, cu_seqlens):
    if cu_seqlens is None:
        return (q.shape[0], q.shape[2], q.shape[1])
    return (q.shape[1], q.shape[0])


# ----------------------------------------------------------------------------
# dense / THD
# ----------------------------------------------------------------------------
def attn_fwd(q, k, v, *, causal=False, scale=None, cu_seqlens=None, max_seqlen=None, out=None,
             lse=None, error_word=None, stream=None):
    """Returns (o, lse).  Dense: q [B,S,Hq,D], k/v [B,S,Hkv,D], lse [B,Hq,S].
    THD: q [cap,Hq,D], k/v [cap,Hkv,D], cu_seqlens int32 [n+1], lse [Hq,cap]."""
    dev = q.device
    for n, t in (("q", q), ("k", k), ("v", v)):
        _need(t, n, torch.bfloat16, dev)
    o = out if out is not None else torch.empty_like(q)
    lse = lse if lse is not None else torch.empty(_lse_shape(q, cu_seqlens), dtype=torch.float32,
                                                  device=dev)
    _need(o, "out", torch.bfloat16, dev)
    _need(lse, "lse", torch.float32, dev)
    p = _problem(q, k, causal, scale, cu_seqlens, max_seqlen, error_word)
    _check("attn_fwd", lib().attn_fwd(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(o),
                                      _ptr(lse), _stream(stream)))
    return o, lse


def attn_bwd_workspace_size(q, k, *, mode=ATTN_DQ_ATOMIC, causal=False, cu_seqlens=None,
                            max_seqlen=None, scale=None) -> int:
    p = _problem(q, k, causal, scale, cu_seqlens, max_seqlen, None)
    return int(lib().attn_bwd_workspace_size(ctypes.byref(p), int(mode)))


def attn_bwd_preprocess(q, k, o, dout, *, mode=ATTN_DQ_ATOMIC, workspace=None, causal=False,
                        scale=None, cu_seqlens=None, max_seqlen=None, delta=None,
                        error_word=None, stream=None):
    """Returns delta = rowsum(dO * O) (fp32, layout of lse); clears the atomic
    dQ accumulator inside `workspace` (a uint8 CUDA tensor)."""
    dev = q.device
    _need(o, "o", torch.bfloat16, dev)
    _need(dout, "dout", torch.bfloat16, dev)
    delta = delta if delta is not None else torch.empty(_lse_shape(q, cu_seqlens),
                                                        dtype=torch.float32, device=dev)
    p = _problem(q, k, causal, scale, cu_seqlens, max_seqlen, error_word)
    ws_ptr, ws_bytes = (None, 0) if workspace is None else (_ptr(workspace), workspace.numel())
    _check("attn_bwd_preprocess",
           lib().attn_bwd_preprocess(ctypes.byref(p), int(mode), _ptr(o), _ptr(dout), _ptr(delta),
                                     ws_ptr, ws_bytes, _stream(stream)))
    return delta


def attn_bwd(q, k, v, dout, lse, delta, *, mode=ATTN_DQ_ATOMIC, workspace, causal=False,
             scale=None, cu_seqlens=None, max_seqlen=None, dk=None, dv=None, error_word=None,
             stream=None):
    """Main backward pass: returns (dk, dv) bf16 and leaves dQ (fp32) in the
    workspace.  Call attn_bwd_preprocess before and attn_bwd_postprocess after,
    with the same workspace and mode."""
    if int(mode) == ATTN_DQ_ATOMIC:
        _nondeterministic("attn_bwd(dq_mode=ATTN_DQ_ATOMIC)", "dq_mode=ATTN_DQ_SPLIT")
    dev = q.device
    for n, t in (("q", q), ("k", k), ("v", v), ("dout", dout)):
        _need(t, n, torch.bfloat16, dev)
    _need(lse, "lse", torch.float32, dev)
    _need(delta, "delta", torch.float32, dev)
    dk = dk if dk is not None else torch.empty_like(k)
    dv = dv if dv is not None else torch.empty_like(v)
    p = _problem(q, k, causal, scale, cu_seqlens, max_seqlen, error_word)
    _check("attn_bwd",
           lib().attn_bwd(ctypes.byref(p), int(mode), _ptr(q), _ptr(k), _ptr(v), _ptr(dout),
                          _ptr(lse), _ptr(delta), _ptr(dk), _ptr(dv), _ptr(workspace),
                          workspace.numel(), _stream(stream)))
    return dk, dv


def attn_bwd_postprocess(q, k, dk, dv, *, mode=ATTN_DQ_ATOMIC, workspace, causal=False, scale=None,
                         cu_seqlens=None, max_seqlen=None, dq=None, error_word=None, stream=None):
    """Writes dq (bf16) from the workspace of attn_bwd; returns dq."""
    dq = dq if dq is not None else torch.empty_like(q)
    _need(dq, "dq", torch.bfloat16, q.device)
    p = _problem(q, k, causal, scale, cu_seqlens, max_seqlen, error_word)
    _check("attn_bwd_postprocess",
           lib().attn_bwd_postprocess(ctypes.byref(p), int(mode), _ptr(workspace),
                                      workspace.numel(), _ptr(dq), _ptr(dk), _ptr(dv),
                                      _stream(stream)))
    return dq


def dense_backward(q, k, v, o, lse, dout, *, mode=ATTN_DQ_ATOMIC, causal=False, scale=None,
                   cu_seqlens=None, max_seqlen=None, workspace=None, error_word=None,
                   stream=None):
    """Preprocess + backward with a workspace allocated here when not given."""
    if workspace is None:
        n = attn_bwd_workspace_size(q, k, mode=mode, causal=causal, cu_seqlens=cu_seqlens,
                                    max_seqlen=max_seqlen)
        workspace = torch.empty(max(n, 16), dtype=torch.uint8, device=q.device)
    kw = dict(mode=mode, causal=causal, scale=scale, cu_seqlens=cu_seqlens, max_seqlen=max_seqlen,
              error_word=error_word, stream=stream)
    delta = attn_bwd_preprocess(q, k, o, dout, workspace=workspace, **kw)
    dk, dv = attn_bwd(q, k, v, dout, lse, delta, workspace=workspace, **kw)
    dq = attn_bwd_postprocess(q, k, dk, dv, workspace=workspace, **kw)
    return dq, dk, dv


def attn_bwd_fixed_scratch(q, k, v, o, dout, lse, *, causal=False, scale=None, cu_seqlens=None,
                           max_seqlen=None, dq=None, dk=None, dv=None, error_word=None,
                           stream=None):
    """Backward for callers that cannot allocate device memory: no workspace
    argument; Delta and the fp32 dQ accumulator live in a 16 MiB array the
    library owns on each GPU.  Returns (dq, dk, dv).  Problems whose scratch
    need exceeds the array raise ValueError; calls that overlap on the GPU race
    on the shared array."""
    _nondeterministic("attn_bwd_fixed_scratch", "attn_bwd with dq_mode=ATTN_DQ_SPLIT")
    dev = q.device
    for n, t in (("q", q), ("k", k), ("v", v), ("o", o), ("dout", dout)):
        _need(t, n, torch.bfloat16, dev)
    _need(lse, "lse", torch.float32, dev)
    rows = q.shape[0] if cu_seqlens is not None else q.shape[0] * q.shape[1]
    hq, d = q.shape[-2], q.shape[-1]
    need = (rows * hq * d * 4 + 255) // 256 * 256 + rows * hq * 4
    if need > FIXED_SCRATCH_BYTES:
        raise ValueError(f"attn_bwd_fixed_scratch: problem needs {need} bytes of scratch, "
                         f"more than the fixed {FIXED_SCRATCH_BYTES}")
    dq = dq if dq is not None else torch.empty_like(q)
    dk = dk if dk is not None else torch.empty_like(k)
    dv = dv if dv is not None else torch.empty_like(v)
    p = _problem(q, k, causal, scale, cu_seqlens, max_seqlen, error_word)
    _check("attn_bwd_fixed_scratch",
           lib().attn_bwd_fixed_scratch(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(o),
                                        _ptr(dout), _ptr(lse), _ptr(dq), _ptr(dk), _ptr(dv),
                                        _stream(stream)))
    return dq, dk, dv


# ----------------------------------------------------------------------------
# top-k sparse
# ----------------------------------------------------------------------------
def _sparse_problem(q, idx, scale, error_word):
    p = _SparseProblem()
    p.tokens, p.heads, p.dim_qk = q.shape
    p.dim_v = SPARSE_DIM_V
    p.topk = idx.shape[1]
    p.scale = float(scale if scale is not None else 1.0 / math.sqrt(p.dim_qk))
    p.error_word = None if error_word is None else error_word.data_ptr()
    return p


def sparse_attn_fwd(q, kv, idx, *, scale=None, out=None, lse=None, error_word=None, stream=None):
    """q [T,H,576], kv [T,576], idx int32 [T,K] -> (o [T,H,512], lse [T,H])."""
    dev = q.device
    _need(q, "q", torch.bfloat16, dev)
    _need(kv, "kv", torch.bfloat16, dev)
    _need(idx, "idx", torch.int32, dev)
    T, H, _ = q.shape
    o = out if out is not None else torch.empty(T, H, SPARSE_DIM_V, dtype=torch.bfloat16, device=dev)
    lse = lse if lse is not None else torch.empty(T, H, dtype=torch.float32, device=dev)
    p = _sparse_problem(q, idx, scale, error_word)
    _check("sparse_attn_fwd",
           lib().sparse_attn_fwd(ctypes.byref(p), _ptr(q), _ptr(kv), _ptr(idx), _ptr(o), _ptr(lse),
                                 _stream(stream)))
    return o, lse


def sparse_attn_bwd_workspace_size(q, idx, *, scale=None) -> int:
    p = _sparse_problem(q, idx, scale, None)
    return int(lib().sparse_attn_bwd_workspace_size(ctypes.byref(p)))


def sparse_attn_bwd(q, kv, idx, o, dout, lse, *, scale=None, workspace=None, dq=None, dkv=None,
                    error_word=None, stream=None):
    """Returns (dq [T,H,576], dkv [T,576]) bf16."""
    _nondeterministic("sparse_attn_bwd (dKV)", "sparse_attn_bwd_deterministic")
    dev = q.device
    for n, t in (("q", q), ("kv", kv), ("o", o), ("dout", dout)):
        _need(t, n, torch.bfloat16, dev)
    _need(idx, "idx", torch.int32, dev)
    _need(lse, "lse", torch.float32, dev)
    if workspace is None:
        n = sparse_attn_bwd_workspace_size(q, idx, scale=scale)
        workspace = torch.empty(max(n, 16), dtype=torch.uint8, device=dev)
    dq = dq if dq is not None else torch.empty_like(q)
    dkv = dkv if dkv is not None else torch.empty_like(kv)
    p = _sparse_problem(q, idx, scale, error_word)
    _check("sparse_attn_bwd",
           lib().sparse_attn_bwd(ctypes.byref(p), _ptr(q), _ptr(kv), _ptr(idx), _ptr(o),
                                 _ptr(dout), _ptr(lse), _ptr(dq), _ptr(dkv), _ptr(workspace),
                                 workspace.numel(), _stream(stream)))
    return dq, dkv


def sparse_attn_bwd_deterministic_workspace_size(q, idx, *, scale=None) -> int:
    p = _sparse_problem(q, idx, scale, None)
    return int(lib().sparse_attn_bwd_deterministic_workspace_size(ctypes.byref(p)))


def sparse_attn_bwd_deterministic(q, kv, idx, o, dout, lse, *, scale=None, workspace=None, dq=None,
                                  dkv=None, error_word=None, stream=None):
    """Returns (dq [T,H,576], dkv [T,576]) bf16 with dkv bitwise reproducible
    (fixed per-key-row summation order; see include/attn.h for the workspace)."""
    dev = q.device
    for n, t in (("q", q), ("kv", kv), ("o", o), ("dout", dout)):
        _need(t, n, torch.bfloat16, dev)
    _need(idx, "idx", torch.int32, dev)
    _need(lse, "lse", torch.float32, dev)
    if workspace is None:
        n = sparse_attn_bwd_deterministic_workspace_size(q, idx, scale=scale)
        workspace = torch.empty(max(n, 16), dtype=torch.uint8, device=dev)
    dq = dq if dq is not None else torch.empty_like(q)
    dkv = dkv if dkv is not None else torch.empty_like(kv)
    p = _sparse_problem(q, idx, scale, error_word)
    _check("sparse_attn_bwd_deterministic",
           lib().sparse_attn_bwd_deterministic(ctypes.byref(p), _ptr(q), _ptr(kv), _ptr(idx),
                                               _ptr(o), _ptr(dout), _ptr(lse), _ptr(dq), _ptr(dkv),
                                               _ptr(workspace), workspace.numel(), _stream(stream)))
    return dq, dkv


# ----------------------------------------------------------------------------
# CSA compressor gated pooling (include/dsa.h)
# ----------------------------------------------------------------------------
def _csa_problem(kv, cu_seqlens, cu_seqlens_comp, ratio, coff, comp_capacity, error_word):
    p = _CsaProblem()
    if kv.dim() != 2 or kv.shape[1] % coff:
        raise ValueError("kv must be [tokens, coff * head_dim]")
    _need(cu_seqlens, "cu_seqlens", torch.int32, kv.device)
    _need(cu_seqlens_comp, "cu_seqlens_comp", torch.int32, kv.device)
    if cu_seqlens.numel() != cu_seqlens_comp.numel():
        raise ValueError("cu_seqlens and cu_seqlens_comp must have the same length")
    p.tokens = kv.shape[0]
    p.comp_capacity = int(comp_capacity)
    p.num_seqs = cu_seqlens.numel() - 1
    p.head_dim = kv.shape[1] // coff
    p.ratio, p.coff = int(ratio), int(coff)
    p.cu_seqlens = cu_seqlens.data_ptr()
    p.cu_seqlens_comp = cu_seqlens_comp.data_ptr()
    p.error_word = None if error_word is None else error_word.data_ptr()
    return p


def csa_compressor_fwd(kv, score, ape, cu_seqlens, cu_seqlens_comp, *, ratio=4, coff=2,
                       comp_capacity, out=None, error_word=None, stream=None):
    """kv/score bf16 [T, coff*D], ape fp32 [ratio, coff*D] -> out bf16 [comp_capacity, D]."""
    dev = kv.device
    _need(kv, "kv", torch.bfloat16, dev)
    _need(score, "score", torch.bfloat16, dev)
    _need(ape, "ape", torch.float32, dev)
    p = _csa_problem(kv, cu_seqlens, cu_seqlens_comp, ratio, coff, comp_capacity, error_word)
    out = out if out is not None else torch.empty(p.comp_capacity, p.head_dim,
                                                  dtype=torch.bfloat16, device=dev)
    _need(out, "out", torch.bfloat16, dev)
    _check("csa_compressor_fwd",
           lib().csa_compressor_fwd(ctypes.byref(p), _ptr(kv), _ptr(score), _ptr(ape), _ptr(out),
                                    _stream(stream)))
    return out


def csa_compressor_bwd_workspace_size(kv, cu_seqlens, cu_seqlens_comp, *, ratio=4, coff=2,
                                      comp_capacity) -> int:
    p = _csa_problem(kv, cu_seqlens, cu_seqlens_comp, ratio, coff, comp_capacity, None)
    return int(lib().csa_compressor_bwd_workspace_size(ctypes.byref(p)))


def csa_compressor_bwd(kv, score, ape, dout, cu_seqlens, cu_seqlens_comp, *, ratio=4, coff=2,
                       workspace=None, dkv=None, dscore=None, dape=None, error_word=None,
                       stream=None):
    """Returns (dkv, dscore) bf16 [T, coff*D] and dape fp32 [ratio, coff*D], all
    bitwise reproducible."""
    dev = kv.device
    for n, t in (("kv", kv), ("score", score), ("dout", dout)):
        _need(t, n, torch.bfloat16, dev)
    _need(ape, "ape", torch.float32, dev)
    p = _csa_problem(kv, cu_seqlens, cu_seqlens_comp, ratio, coff, dout.shape[0], error_word)
    if workspace is None:
        n = int(lib().csa_compressor_bwd_workspace_size(ctypes.byref(p)))
        workspace = torch.empty(max(n, 16), dtype=torch.uint8, device=dev)
    dkv = dkv if dkv is not None else torch.empty_like(kv)
    dscore = dscore if dscore is not None else torch.empty_like(score)
    dape = dape if dape is not None else torch.empty_like(ape)
    _check("csa_compressor_bwd",
           lib().csa_compressor_bwd(ctypes.byref(p), _ptr(kv), _ptr(score), _ptr(ape), _ptr(dout),
                                    _ptr(dkv), _ptr(dscore), _ptr(dape), _ptr(workspace),
                                    workspace.numel(), _stream(stream)))
    return dkv, dscore, dape


# ----------------------------------------------------------------------------
# DSA lightning indexer, top-k and sparse KL (include/dsa.h)
# ----------------------------------------------------------------------------
def logits_ld(tokens: int) -> int:
    """Row stride of the logits buffer: tokens rounded up to a multiple of 4."""
    return (int(tokens) + 3) // 4 * 4


def _indexer_problem(q, topk, use_relu, cu_seqlens, error_word, ld=None):
    p = _IndexerProblem()
    if q.dim() != 3:
        raise ValueError("indexer q must be [tokens, heads, head_dim]")
    p.tokens, p.heads, p.head_dim = q.shape
    p.topk = int(topk)
    p.use_relu = 1 if use_relu else 0
    p.logits_ld = logits_ld(p.tokens) if ld is None else int(ld)
    if cu_seqlens is not None:
        _need(cu_seqlens, "cu_seqlens", torch.int32, q.device)
        p.cu_seqlens = cu_seqlens.data_ptr()
        p.num_seqs = cu_seqlens.numel() - 1
    else:
        p.cu_seqlens, p.num_seqs = None, 0
    p.error_word = None if error_word is None else error_word.data_ptr()
    return p


def dsa_indexer_fwd(q, k, w, *, use_relu=True, cu_seqlens=None, logits=None, error_word=None,
                    stream=None):
    """q bf16 [T,H,128], k bf16 [T,128], w fp32 [T,H] -> logits fp32 [T, logits_ld(T)]
    (columns past T unwritten; use logits[:, :T])."""
    dev = q.device
    _need(q, "q", torch.bfloat16, dev)
    _need(k, "k", torch.bfloat16, dev)
    _need(w, "w", torch.float32, dev)
    p = _indexer_problem(q, 1, use_relu, cu_seqlens, error_word)
    if logits is None:
        logits = torch.empty(p.tokens, p.logits_ld, dtype=torch.float32, device=dev)
    _need(logits, "logits", torch.float32, dev)
    p.logits_ld = logits.shape[1]
    _check("dsa_indexer_fwd", lib().dsa_indexer_fwd(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(w),
                                                    _ptr(logits), _stream(stream)))
    return logits


def dsa_topk(logits, topk, *, heads=1, cu_seqlens=None, idx=None, length=None, scores=None,
             error_word=None, stream=None):
    """logits fp32 [T, ld] -> (idx int32 [T,topk], length int32 [T], scores fp32 [T,topk])."""
    dev = logits.device
    _need(logits, "logits", torch.float32, dev)
    T = logits.shape[0]
    p = _IndexerProblem()
    p.tokens, p.heads, p.head_dim, p.topk = T, int(heads), INDEXER_HEAD_DIM, int(topk)
    p.use_relu, p.logits_ld = 1, logits.shape[1]
    if cu_seqlens is not None:
        _need(cu_seqlens, "cu_seqlens", torch.int32, dev)
        p.cu_seqlens, p.num_seqs = cu_seqlens.data_ptr(), cu_seqlens.numel() - 1
    else:
        p.cu_seqlens, p.num_seqs = None, 0
    p.error_word = None if error_word is None else error_word.data_ptr()
    idx = idx if idx is not None else torch.empty(T, topk, dtype=torch.int32, device=dev)
    length = length if length is not None else torch.empty(T, dtype=torch.int32, device=dev)
    scores = scores if scores is not None else torch.empty(T, topk, dtype=torch.float32, device=dev)
    _check("dsa_topk", lib().dsa_topk(ctypes.byref(p), _ptr(logits), _ptr(idx), _ptr(length),
                                      _ptr(scores), _stream(stream)))
    return idx, length, scores


def dsa_indexer_bwd(q, k, w, idx, grad, *, use_relu=True, workspace=None, dq=None, dk=None,
                    dw=None, error_word=None, stream=None):
    """Gradients (dq bf16 [T,H,128], dk bf16 [T,128], dw fp32 [T,H]) of
    sum_j grad[t, j] * logits[t, idx[t, j]]."""
    _nondeterministic("dsa_indexer_bwd (dk)", "a reproducible reduction of dk")
    dev = q.device
    _need(q, "q", torch.bfloat16, dev)
    _need(k, "k", torch.bfloat16, dev)
    _need(w, "w", torch.float32, dev)
    _need(idx, "idx", torch.int32, dev)
    _need(grad, "grad", torch.float32, dev)
    p = _indexer_problem(q, idx.shape[1], use_relu, None, error_word)
    if workspace is None:
        n = int(lib().dsa_indexer_bwd_workspace_size(ctypes.byref(p)))
        workspace = torch.empty(max(n, 16), dtype=torch.uint8, device=dev)
    dq = dq if dq is not None else torch.empty_like(q)
    dk = dk if dk is not None else torch.empty_like(k)
    dw = dw if dw is not None else torch.empty_like(w)
    _check("dsa_indexer_bwd",
           lib().dsa_indexer_bwd(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(w), _ptr(idx), _ptr(grad),
                                 _ptr(dq), _ptr(dk), _ptr(dw), _ptr(workspace), workspace.numel(),
                                 _stream(stream)))
    return dq, dk, dw


def dsa_sparse_kl(q, kv, lse, idx, scores, *, scale=None, loss=None, grad=None, target=None,
                  want_target=False, error_word=None, stream=None):
    """Sparse KL of the attention target from softmax(scores) per token:
    returns (loss fp32 [T], grad fp32 [T,K], target fp32 [T,K] or None)."""
    dev = q.device
    _need(q, "q", torch.bfloat16, dev)
    _need(kv, "kv", torch.bfloat16, dev)
    _need(lse, "lse", torch.float32, dev)
    _need(idx, "idx", torch.int32, dev)
    _need(scores, "scores", torch.float32, dev)
    T = q.shape[0]
    p = _sparse_problem(q, idx, scale, error_word)
    loss = loss if loss is not None else torch.empty(T, dtype=torch.float32, device=dev)
    grad = grad if grad is not None else torch.empty_like(scores)
    if want_target and target is None:
        target = torch.empty_like(scores)
    _check("dsa_sparse_kl",
           lib().dsa_sparse_kl(ctypes.byref(p), _ptr(q), _ptr(kv), _ptr(lse), _ptr(idx),
                               _ptr(scores), _ptr(loss), _ptr(grad), _ptr(target), _stream(stream)))
    return loss, grad, target


# ----------------------------------------------------------------------------
# paged key/value cache (include/cache.h)
# ----------------------------------------------------------------------------
_CACHE_TYPES = {torch.bfloat16: 0, torch.float8_e4m3fn: 1}


def attn_cache_empty(num_pages, heads_kv, page_size, head_dim, *, dtype=torch.bfloat16, device=None):
    """An empty cache: (k_cache, v_cache, k_scale, v_scale), the pools
    [num_pages, heads_kv, page_size, head_dim] of `dtype` (bfloat16 or
    float8_e4m3fn) uninitialized, the scales fp32 [num_pages, heads_kv] (None for
    bfloat16)."""
    if dtype not in _CACHE_TYPES:
        raise TypeError(f"a cache is bfloat16 or float8_e4m3fn, not {dtype}")
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    k, v = (torch.empty(num_pages, heads_kv, page_size, head_dim, dtype=dtype, device=dev)
            for _ in range(2))
    if dtype == torch.bfloat16:
        return k, v, None, None
    ks, vs = (torch.ones(num_pages, heads_kv, dtype=torch.float32, device=dev) for _ in range(2))
    return k, v, ks, vs


def _need_rows(t, name, heads, dim, device):
    """bf16 [tokens, heads, dim] whose tokens may lie apart (a slice of a fused
    projection); returns the elements between two tokens, 0 for dense ones."""
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dim() != 3 or t.shape[1] != heads or t.shape[2] != dim:
        raise ValueError(f"{name} must be [tokens, {heads}, {dim}], got {tuple(t.shape)}")
    if t.is_contiguous():
        return 0
    st = t.stride()
    if st[2] != 1 or (heads > 1 and st[1] != dim):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    if t.shape[0] <= 1:
        return 0
    if st[0] < heads * dim:   # (0 would mean dense to the library)
        raise ValueError(f"{name}: the tokens must not overlap (a broadcast tensor: call contiguous())")
    return st[0]


# A step of one token takes the GPU a few microseconds, so the checks below look
# at each tensor once, in one expression, and leave the wording to _need.
def _cache_problem(k_cache, v_cache, k_scale, v_scale, page_table, seqlens_kv, cu_seqlens,
                   max_new, error_word, tokens, heads_q, causal=1, scale=1.0):
    dtype, shape, gpu = k_cache.dtype, k_cache.shape, k_cache.get_device()
    kind = _CACHE_TYPES.get(dtype)
    if kind is None:
        raise TypeError(f"k_cache must be bfloat16 or float8_e4m3fn, got {dtype}")
    if len(shape) != 4:
        raise ValueError("k_cache must be [num_pages, heads_kv, page_size, head_dim]")
    if (gpu < 0 or not k_cache.is_contiguous() or v_cache.dtype is not dtype
            or v_cache.get_device() != gpu or not v_cache.is_contiguous()):
        _need(k_cache, "k_cache", dtype)
        _need(v_cache, "v_cache", dtype, k_cache.device)
    if v_cache.shape != shape:
        raise ValueError("k_cache and v_cache must have the same shape")
    if kind:
        for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            if _need(t, name, torch.float32, k_cache.device).shape != shape[:2]:
                raise ValueError(f"{name} must be [num_pages, heads_kv]")
    elif k_scale is not None or v_scale is not None:
        raise ValueError("k_scale, v_scale: a bfloat16 cache has no scales")
    i32 = torch.int32
    if (page_table.dtype is not i32 or seqlens_kv.dtype is not i32 or cu_seqlens.dtype is not i32
            or page_table.get_device() != gpu or seqlens_kv.get_device() != gpu
            or cu_seqlens.get_device() != gpu or not page_table.is_contiguous()
            or not seqlens_kv.is_contiguous() or not cu_seqlens.is_contiguous()):
        for t, name in ((page_table, "page_table"), (seqlens_kv, "seqlens_kv"),
                        (cu_seqlens, "cu_seqlens")):
            _need(t, name, i32, k_cache.device)
    if error_word is not None:
        error_word = _need(error_word, "error_word", i32, k_cache.device).data_ptr()
    n, table = seqlens_kv.numel(), page_table.shape
    if len(table) != 2 or table[0] != n or cu_seqlens.numel() != n + 1:
        raise ValueError("seqlens_kv [n], cu_seqlens [n + 1] and page_table [n, max_pages] disagree")
    if max_new > 0x7fffffff or table[1] > 0x7fffffff:
        raise ValueError("max_new and page_table's columns must be below 2^31")
    return _CacheProblem(n, tokens, heads_q, shape[1], shape[3], kind, shape[2], shape[0], table[1],
                         max_new, causal, scale, 0, 0, 0, 0, 0, 0, cu_seqlens.data_ptr(),
                         seqlens_kv.data_ptr(), page_table.data_ptr(), error_word)


def _rows_stride(t, name, tokens, heads, dim, gpu, device):
    if (t.dtype is torch.bfloat16 and t.get_device() == gpu and t.shape == (tokens, heads, dim)
            and t.is_contiguous()):
        return 0
    stride = _need_rows(t, name, heads, dim, device)
    if t.shape[0] != tokens:
        raise ValueError("q, k and v must have the same tokens")
    return stride


def _on(device, stream):
    """The context in which a call on `device` runs and allocates (so that what it
    allocates belongs to the stream that writes it), None for the present one, and
    that stream's handle."""
    if stream is not None:
        if stream.device != device:
            raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
        return torch.cuda.stream(stream), stream.cuda_stream
    handle = torch._C._cuda_getCurrentRawStream(device.index)
    if device.index == torch._C._cuda_getDevice():
        return None, handle
    return torch.cuda.device(device), handle


def _at(t):
    return None if t is None else t.data_ptr()


def attn_cache_append(q, k, v, k_cache, v_cache, *, page_table, seqlens_kv, cu_seqlens, max_new,
                      k_scale=None, v_scale=None, cos_sin=None, interleaved=False, q_out=None,
                      error_word=None, stream=None):
    """Writes the new tokens' keys and values (k, v bf16 [T, Hkv, D]) into the
    paged cache and returns the rotated queries (q bf16 [T, Hq, D], or None for
    both).  k_cache, v_cache [pages, Hkv, page_size, D] bfloat16, or
    float8_e4m3fn with k_scale, v_scale fp32 [pages, Hkv]; page_table int32
    [n, max_pages]; seqlens_kv int32 [n], the lengths including the new tokens;
    cu_seqlens int32 [n + 1]; max_new bounds the new tokens of a sequence.
    cos_sin fp32 [positions, rot_dim] (cosines, then sines) rotates q and k, None
    leaves them; `interleaved` pairs neighbouring dims.  The tokens of q, k and v
    may lie apart, as in a fused projection, but not over each other (expand).  A
    step without a token (T = 0) does nothing."""
    dev = k_cache.device
    if q is None:
        if q_out is not None:
            raise ValueError("q_out is given without q")
        heads_q = k_cache.shape[1]
    else:
        if q.dim() != 3:
            raise ValueError("q must be [tokens, heads, head_dim]")
        heads_q = q.shape[1]
    T = k.shape[0]
    p = _cache_problem(k_cache, v_cache, k_scale, v_scale, page_table, seqlens_kv, cu_seqlens,
                       int(max_new), error_word, T, heads_q)
    _, heads, _, dim = k_cache.shape
    p.k_stride = _rows_stride(k, "k", T, heads, dim, dev.index, dev)
    p.v_stride = _rows_stride(v, "v", T, heads, dim, dev.index, dev)
    if cos_sin is not None:
        if _need(cos_sin, "cos_sin", torch.float32, dev).dim() != 2:
            raise ValueError("cos_sin must be [positions, rot_dim]")
        p.max_position, p.rot_dim = cos_sin.shape
        p.rot_interleaved = 1 if interleaved else 0
    if q is not None:
        p.q_stride = _rows_stride(q, "q", T, heads_q, dim, dev.index, dev)
        if q_out is not None and _need(q_out, "q_out", torch.bfloat16, dev).shape != q.shape:
            raise ValueError("q_out must have the shape of q")
    ctx, s = _on(dev, stream)
    if ctx is None:
        return _append_here(p, q, k, v, cos_sin, q_out, k_cache, v_cache, k_scale, v_scale, s)
    with ctx:
        return _append_here(p, q, k, v, cos_sin, q_out, k_cache, v_cache, k_scale, v_scale, s)


def _append_here(p, q, k, v, cos_sin, q_out, k_cache, v_cache, k_scale, v_scale, s):
    if q is not None and q_out is None:
        q_out = torch.empty_like(q) if p.q_stride == 0 else q.new_empty(q.shape)
    code = (_LIB or lib()).attn_cache_append(ctypes.byref(p), _at(q), k.data_ptr(), v.data_ptr(),
                                             _at(cos_sin), _at(q_out), k_cache.data_ptr(),
                                             v_cache.data_ptr(), _at(k_scale), _at(v_scale), s)
    if code:
        raise AttnError("attn_cache_append", code)
    return q_out


def _cache_fwd_problem(q, k_cache, v_cache, k_scale, v_scale, page_table, seqlens_kv, cu_seqlens,
                       max_new, causal, scale, error_word):
    if q.dim() != 3:
        raise ValueError("q must be [tokens, heads, head_dim]")
    p = _cache_problem(k_cache, v_cache, k_scale, v_scale, page_table, seqlens_kv, cu_seqlens,
                       int(max_new), error_word, q.shape[0], q.shape[1], 1 if causal else 0,
                       float(scale) if scale is not None else 1.0 / math.sqrt(q.shape[2]))
    dev = k_cache.device
    p.q_stride = _rows_stride(q, "q", q.shape[0], q.shape[1], k_cache.shape[3], dev.index, dev)
    return p


def attn_cache_fwd_workspace_size(q, k_cache, v_cache, *, page_table, seqlens_kv, cu_seqlens,
                                  max_new, k_scale=None, v_scale=None) -> int:
    p = _cache_fwd_problem(q, k_cache, v_cache, k_scale, v_scale, page_table, seqlens_kv,
                           cu_seqlens, max_new, True, None, None)
    return int(lib().attn_cache_fwd_workspace_size(ctypes.byref(p)))


def attn_cache_fwd(q, k_cache, v_cache, *, page_table, seqlens_kv, cu_seqlens, max_new,
                   k_scale=None, v_scale=None, causal=True, scale=None, out=None, lse=None,
                   workspace=None, error_word=None, stream=None):
    """Attention of the new tokens' queries (q bf16 [T, Hq, D], rotated) over the
    paged cache, which holds their own keys already; arguments as for
    attn_cache_append.  Returns (o bf16 [T, Hq, D], lse fp32 [Hq, T]).  A
    workspace is allocated here when none is given."""
    dev = k_cache.device
    p = _cache_fwd_problem(q, k_cache, v_cache, k_scale, v_scale, page_table, seqlens_kv,
                           cu_seqlens, max_new, causal, scale, error_word)
    if out is not None and _need(out, "out", torch.bfloat16, dev).shape != q.shape:
        raise ValueError("out must have the shape of q")
    if lse is not None and _need(lse, "lse", torch.float32, dev).shape != (p.heads_q, p.tokens):
        raise ValueError("lse must be [heads, tokens]")
    if workspace is not None:
        _need(workspace, "workspace", torch.uint8, dev)
    ctx, s = _on(dev, stream)
    if ctx is None:
        return _fwd_here(p, q, k_cache, v_cache, k_scale, v_scale, out, lse, workspace, s)
    with ctx:
        return _fwd_here(p, q, k_cache, v_cache, k_scale, v_scale, out, lse, workspace, s)


def _fwd_here(p, q, k_cache, v_cache, k_scale, v_scale, out, lse, workspace, s):
    L, ref = _LIB or lib(), ctypes.byref(p)
    if out is None:
        out = torch.empty_like(q) if p.q_stride == 0 else q.new_empty(q.shape)
    if lse is None:
        lse = q.new_empty((p.heads_q, p.tokens), dtype=torch.float32)
    if workspace is None:
        n = L.attn_cache_fwd_workspace_size(ref) or 16
        workspace = q.new_empty(n, dtype=torch.uint8)
    else:
        n = workspace.numel()
    code = L.attn_cache_fwd(ref, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), _at(k_scale),
                            _at(v_scale), out.data_ptr(), lse.data_ptr(), workspace.data_ptr(), n, s)
    if code:
        raise AttnError("attn_cache_fwd", code)
    return out, lse


# ----------------------------------------------------------------------------
# rotation by position (include/rotary.h)
# ----------------------------------------------------------------------------
_ROTARY_SCALINGS = {"none": 0, "linear": 1, "base": 2, "parts": 3}


def attn_rotary_table(max_position, rot_dim, *, base=10000.0, scaling="none", factor=1.0,
                      original=0, fast=32.0, slow=1.0, magnitude=1.0, out=None, device=None,
                      stream=None):
    """The table of cosines and sines of attn_rotary_fwd and attn_cache_append: fp32
    [max_position, rot_dim], magnitude times the cosines of position * frequency,
    then the sines.  scaling "none", "linear" (frequencies divided by factor),
    "base" (the base grown so that the lowest is) or "parts" (those divided that
    turn less than `slow` times over `original` positions, those kept that turn
    more than `fast` times, a ramp between)."""
    if scaling not in _ROTARY_SCALINGS:
        raise ValueError(f"scaling must be one of {', '.join(_ROTARY_SCALINGS)}, got {scaling!r}")
    max_position, rot_dim = _size(int(max_position), "positions"), _size(int(rot_dim), "rotated dims")
    if out is None:
        dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        if dev.type != "cuda":
            raise ValueError(f"device must be a CUDA device, got {dev}")
        if dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
    else:
        dev = _need(out, "out", torch.float32).device
        if out.shape != (max_position, rot_dim):
            raise ValueError("out must be [max_position, rot_dim]")
        if device is not None and torch.device(device) not in (dev, torch.device("cuda")):
            raise ValueError(f"out is on {dev}, device is {device}")
    p = _RotaryTable(max_position, rot_dim, float(base), _ROTARY_SCALINGS[scaling],
                     float(factor), _size(int(original), "original positions"), float(fast), float(slow), float(magnitude))
    ctx, s = _on(dev, stream)
    if ctx is None:
        return _table_here(p, out, dev, s)
    with ctx:
        return _table_here(p, out, dev, s)


def _size(n, what):
    """A size that the library takes in 32 bits (ctypes would cut off what is above)."""
    if not -1 << 31 <= n < 1 << 31:
        raise ValueError(f"{n} {what}: at most {(1 << 31) - 1} are supported")
    return n


def _table_here(p, out, dev, s):
    if out is None:
        out = torch.empty((max(0, p.max_position), max(0, p.rot_dim)), dtype=torch.float32, device=dev)
    code = (_LIB or lib()).attn_rotary_table(ctypes.byref(p), out.data_ptr(), s)
    if code:
        raise AttnError("attn_rotary_table", code)
    return out


def _token_rows(t, name, lead, heads, dim, device):
    """bf16 [*lead, heads, dim] (lead one or two dims) whose tokens may lie apart,
    equally far (a slice of a fused projection); returns the elements between two
    tokens, 0 for dense ones."""
    if t.shape != (*lead, heads, dim):
        raise ValueError(f"{name} must be {[*lead, heads, dim]}, got {list(t.shape)}")
    if len(lead) == 1:
        return _need_rows(t, name, heads, dim, device)
    if lead[0] > 1 and lead[1] > 1 and t.stride(0) != lead[1] * t.stride(1) and t.numel():
        raise ValueError(f"{name}: the sequences must follow each other as the tokens of one do")
    row = t.stride(1) if lead[1] > 1 else t.stride(0)
    if t.numel() == 0:
        row = heads * dim
    return _need_rows(t.as_strided((lead[0] * lead[1], heads, dim), (row, t.stride(2), t.stride(3)),
                                   t.storage_offset()), name, heads, dim, device)


# As for the cache, a call on few tokens takes the GPU a few microseconds: the
# checks below look at each tensor once and leave the wording to the functions
# above.
def _ok(t, dtype, gpu):
    return t.dtype is dtype and t.get_device() == gpu and t.is_contiguous()


def _gpu_of(t, name):
    """The device of a tensor that decides a call's, and its index."""
    gpu = t.get_device()
    if gpu < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return gpu, t.device


def _lead(shape, cu_seqlens, gpu, device):
    """The leading dims of a dense [batch, seqlen, heads, dim] or packed [tokens,
    heads, dim] tensor: tokens, sequences, their length and cu_seqlens' address."""
    if cu_seqlens is None:
        if len(shape) != 4:
            raise ValueError("dense q must be [batch, seqlen, heads, head_dim]")
        n, length = shape[0], shape[1]
        return _size(n * length, "tokens"), _size(n, "sequences"), _size(length, "tokens of a sequence"), None
    if len(shape) != 3:
        raise ValueError("THD q must be [tokens, heads, head_dim]")
    if not _ok(cu_seqlens, torch.int32, gpu):
        _need(cu_seqlens, "cu_seqlens", torch.int32, device)
    n = cu_seqlens.numel() - 1
    if cu_seqlens.dim() != 1 or n < 1:
        raise ValueError("cu_seqlens must be [num_seqs + 1]")
    return _size(shape[0], "tokens"), _size(n, "sequences"), 0, cu_seqlens.data_ptr()


def _word(error_word, gpu, device):
    if error_word is None:
        return None
    if not _ok(error_word, torch.int32, gpu):
        _need(error_word, "error_word", torch.int32, device)
    return error_word.data_ptr()


def _out_like(t, name, like, gpu, device):
    """A given bf16 output, dense with the shape of `like`."""
    if not _ok(t, torch.bfloat16, gpu):
        _need(t, name, torch.bfloat16, device)
    if t.shape != like.shape:
        raise ValueError(f"{name} must be {list(like.shape)}, got {list(t.shape)}")


def _rotary(name, q, k, cos_sin, positions, cu_seqlens, interleaved, rot_offset, q_out, k_out,
            error_word, stream):
    bf16 = torch.bfloat16
    gpu, dev = _gpu_of(q, "q")
    shape = q.shape
    lead = shape[:-2]
    if positions is None:
        tokens, n, length, cu = _lead(shape, cu_seqlens, gpu, dev)
        at = None
    else:
        if cu_seqlens is not None:
            raise ValueError("positions and cu_seqlens exclude each other")
        if len(shape) not in (3, 4):
            raise ValueError("q must be [tokens, heads, head_dim] or [batch, seqlen, heads, head_dim]")
        if not _ok(positions, torch.int32, gpu):
            _need(positions, "positions", torch.int32, dev)
        if positions.shape != lead:
            raise ValueError(f"positions must be {list(lead)}, got {list(positions.shape)}")
        tokens, n, length, cu, at = _size(positions.numel(), "tokens"), 0, 0, None, positions.data_ptr()
    heads, dim = shape[-2], shape[-1]
    q_stride = 0 if _ok(q, bf16, gpu) else _token_rows(q, "q", lead, heads, dim, dev)
    heads_k = k_stride = 0
    if k is not None:
        kshape = k.shape
        if len(kshape) != len(shape):
            raise ValueError("q and k must have the same leading dims")
        heads_k = kshape[-2]
        if kshape[:-2] != lead or kshape[-1] != dim or not _ok(k, bf16, gpu):
            k_stride = _token_rows(k, "k", lead, heads_k, dim, dev)
    elif k_out is not None:
        raise ValueError("k_out is given without k")
    if not _ok(cos_sin, torch.float32, gpu):
        _need(cos_sin, "cos_sin", torch.float32, dev)
    if cos_sin.dim() != 2:
        raise ValueError("cos_sin must be [positions, rot_dim]")
    if q_out is not None:
        _out_like(q_out, "q_out", q, gpu, dev)
    if k_out is not None:
        _out_like(k_out, "k_out", k, gpu, dev)
    rows, rot = cos_sin.shape
    p = _RotaryProblem(tokens, _size(heads, "heads"), _size(heads_k, "heads"), dim, rot,
                       _size(int(rot_offset), "dims before the rotated ones"), 1 if interleaved else 0,
                       _size(rows, "positions"), length, n, q_stride, k_stride, cu, at, _word(error_word, gpu, dev))
    ctx, s = _on(dev, stream)
    if ctx is None:
        return _rotary_here(name, p, q, k, cos_sin, q_out, k_out, s)
    with ctx:
        return _rotary_here(name, p, q, k, cos_sin, q_out, k_out, s)


def _new_like(t, stride):
    """A dense tensor like t, whose tokens may lie apart."""
    return torch.empty_like(t) if stride == 0 else t.new_empty(t.shape)


def _rotary_here(name, p, q, k, cos_sin, q_out, k_out, s):
    if q_out is None:
        q_out = _new_like(q, p.q_stride)
    if k is not None and k_out is None:
        k_out = _new_like(k, p.k_stride)
    code = getattr(_LIB or lib(), name)(ctypes.byref(p), q.data_ptr(), _at(k), cos_sin.data_ptr(),
                                        q_out.data_ptr(), _at(k_out), s)
    if code:
        raise AttnError(name, code)
    return q_out, k_out


def attn_rotary_fwd(q, k, cos_sin, *, positions=None, cu_seqlens=None, interleaved=False,
                    rot_offset=0, q_out=None, k_out=None, error_word=None, stream=None):
    """Rotates q (bf16 [B, S, H, D], or packed [T, H, D]) and k (likewise, or None) by
    position: dims rot_offset .. rot_offset + rot_dim by the rows of cos_sin (fp32
    [positions, rot_dim], cosines then sines), the other dims copied.  Positions
    are a token's place in its sequence, or `positions` (int32 [*leading dims],
    -1 for padding).  q_out, k_out may be q, k.  Returns (q_out, k_out)."""
    return _rotary("attn_rotary_fwd", q, k, cos_sin, positions, cu_seqlens, interleaved,
                   rot_offset, q_out, k_out, error_word, stream)


def attn_rotary_bwd(dq, dk, cos_sin, *, positions=None, cu_seqlens=None, interleaved=False,
                    rot_offset=0, dq_out=None, dk_out=None, error_word=None, stream=None):
    """Backward of attn_rotary_fwd: the gradients of the rotated rows in, those of
    the rows out (the transposed rotation).  Returns (dq_out, dk_out)."""
    return _rotary("attn_rotary_bwd", dq, dk, cos_sin, positions, cu_seqlens, interleaved,
                   rot_offset, dq_out, dk_out, error_word, stream)


# ----------------------------------------------------------------------------
# linear attention with a decay for each head (include/linear.h)
# ----------------------------------------------------------------------------
def _linear_heads(q, k, v, log_decay, gpu, dev):
    """Shape and stride checks of a call's rows: heads_kv and the strides."""
    bf16 = torch.bfloat16
    shape, kshape = q.shape, k.shape
    lead, dim = shape[:-2], shape[-1]
    if len(kshape) != len(shape):
        raise ValueError("q, k and v must have the same leading dims")
    heads_kv = kshape[-2]
    if not _ok(log_decay, torch.float32, gpu):
        _need(log_decay, "log_decay", torch.float32, dev)
    if log_decay.dim() != 1 or log_decay.numel() != heads_kv:
        raise ValueError(f"log_decay must be [{heads_kv}], got {list(log_decay.shape)}")
    sq = 0 if _ok(q, bf16, gpu) else _token_rows(q, "q", lead, shape[-2], dim, dev)
    dense = kshape[:-2] == lead and kshape[-1] == dim
    sk = 0 if dense and _ok(k, bf16, gpu) else _token_rows(k, "k", lead, heads_kv, dim, dev)
    sv = 0 if dense and v.shape == kshape and _ok(v, bf16, gpu) else _token_rows(v, "v", lead, heads_kv, dim, dev)
    return heads_kv, sq, sk, sv


def _linear_problem(q, k, v, log_decay, scale, cu_seqlens, error_word, dout=None):
    gpu, dev = _gpu_of(q, "q")
    shape = q.shape
    tokens, n, length, cu = _lead(shape, cu_seqlens, gpu, dev)
    heads_kv, sq, sk, sv = _linear_heads(q, k, v, log_decay, gpu, dev)
    sd = 0
    if dout is not None and (dout.shape != shape or not _ok(dout, torch.bfloat16, gpu)):
        sd = _token_rows(dout, "dout", shape[:-2], shape[-2], shape[-1], dev)
    dim = shape[-1]
    return _LinearProblem(n, length, tokens, shape[-2], heads_kv, dim,
                          float(scale) if scale is not None else 1.0 / math.sqrt(dim), sq, sk, sv, sd,
                          cu, log_decay.data_ptr(), _word(error_word, gpu, dev)), gpu, dev


def _linear_state(t, name, p, gpu, dev):
    if not _ok(t, torch.float32, gpu):
        _need(t, name, torch.float32, dev)
    if t.shape != (p.num_seqs, p.heads_kv, p.head_dim, p.head_dim):
        raise ValueError(f"{name} must be {[p.num_seqs, p.heads_kv, p.head_dim, p.head_dim]}, got {list(t.shape)}")


def _linear_work(size, p, workspace, like):
    """A call's workspace and its bytes, allocated where none is given."""
    if workspace is not None:
        return workspace, workspace.numel()
    n = size(ctypes.byref(p))
    return (torch.empty(n, dtype=torch.uint8, device=like.device) if n else None), n


def linear_attn_fwd_workspace_size(q, k, v, log_decay, *, cu_seqlens=None) -> int:
    p, _, dev = _linear_problem(q, k, v, log_decay, None, cu_seqlens, None)
    with torch.cuda.device(dev):
        return int(lib().linear_attn_fwd_workspace_size(ctypes.byref(p)))


def linear_attn_bwd_workspace_size(q, k, v, log_decay, *, cu_seqlens=None) -> int:
    p, _, dev = _linear_problem(q, k, v, log_decay, None, cu_seqlens, None)
    with torch.cuda.device(dev):
        return int(lib().linear_attn_bwd_workspace_size(ctypes.byref(p)))


def linear_attn_fwd(q, k, v, log_decay, *, scale=None, cu_seqlens=None, initial_state=None,
                    want_final_state=False, final_state=None, out=None, workspace=None,
                    error_word=None, stream=None):
    """Linear attention with a decay for each KV head, in chunks: q bf16
    [B, S, Hq, D], k, v [B, S, Hkv, D], or packed [T, H, D] with cu_seqlens;
    log_decay fp32 [Hkv], at most 0; initial_state fp32 [n, Hkv, D, D] or None.
    Returns (o, final_state), the latter None unless wanted or given.  A workspace
    is allocated here when none is given."""
    p, gpu, dev = _linear_problem(q, k, v, log_decay, scale, cu_seqlens, error_word)
    if initial_state is not None:
        _linear_state(initial_state, "initial_state", p, gpu, dev)
    if final_state is not None:
        _linear_state(final_state, "final_state", p, gpu, dev)
    if out is not None:
        _out_like(out, "out", q, gpu, dev)
    if workspace is not None:
        _need(workspace, "workspace", torch.uint8, dev)
    ctx, s = _on(dev, stream)
    if ctx is None:
        return _linear_fwd_here(p, q, k, v, initial_state, want_final_state, final_state, out, workspace, s)
    with ctx:
        return _linear_fwd_here(p, q, k, v, initial_state, want_final_state, final_state, out, workspace, s)


def _linear_fwd_here(p, q, k, v, initial_state, want_final_state, final_state, out, workspace, s):
    L = _LIB or lib()
    if out is None:
        out = _new_like(q, p.q_stride)
    if final_state is None and want_final_state:
        final_state = torch.empty((p.num_seqs, p.heads_kv, p.head_dim, p.head_dim), dtype=torch.float32,
                                  device=q.device)
    workspace, n = _linear_work(L.linear_attn_fwd_workspace_size, p, workspace, q)
    code = L.linear_attn_fwd(ctypes.byref(p), q.data_ptr(), k.data_ptr(), v.data_ptr(), _at(initial_state),
                             out.data_ptr(), _at(final_state), _at(workspace), n, s)
    if code:
        raise AttnError("linear_attn_fwd", code)
    return out, final_state


def linear_attn_bwd(q, k, v, dout, log_decay, *, scale=None, cu_seqlens=None, initial_state=None,
                    dfinal_state=None, want_dinitial_state=False, dinitial_state=None, dq=None,
                    dk=None, dv=None, workspace=None, error_word=None, stream=None):
    """Backward of linear_attn_fwd from its inputs, dout and dfinal_state (fp32
    [n, Hkv, D, D], the final state's gradient, or None).  Returns (dq, dk, dv,
    dinitial_state), the last None unless wanted or given; bitwise reproducible."""
    p, gpu, dev = _linear_problem(q, k, v, log_decay, scale, cu_seqlens, error_word, dout)
    for t, name in ((initial_state, "initial_state"), (dfinal_state, "dfinal_state"),
                    (dinitial_state, "dinitial_state")):
        if t is not None:
            _linear_state(t, name, p, gpu, dev)
    for t, name, like in ((dq, "dq", q), (dk, "dk", k), (dv, "dv", v)):
        if t is not None:
            _out_like(t, name, like, gpu, dev)
    if workspace is not None:
        _need(workspace, "workspace", torch.uint8, dev)
    args = (p, q, k, v, dout, initial_state, dfinal_state, want_dinitial_state, dinitial_state, dq, dk, dv, workspace)
    ctx, s = _on(dev, stream)
    if ctx is None:
        return _linear_bwd_here(*args, s)
    with ctx:
        return _linear_bwd_here(*args, s)


def _linear_bwd_here(p, q, k, v, dout, initial_state, dfinal_state, want_dinitial_state, dinitial_state, dq, dk, dv,
                     workspace, s):
    L = _LIB or lib()
    dq = _new_like(q, p.q_stride) if dq is None else dq
    dk = _new_like(k, p.k_stride) if dk is None else dk
    dv = _new_like(v, p.v_stride) if dv is None else dv
    if dinitial_state is None and want_dinitial_state:
        dinitial_state = torch.empty((p.num_seqs, p.heads_kv, p.head_dim, p.head_dim), dtype=torch.float32,
                                     device=q.device)
    workspace, n = _linear_work(L.linear_attn_bwd_workspace_size, p, workspace, q)
    code = L.linear_attn_bwd(ctypes.byref(p), q.data_ptr(), k.data_ptr(), v.data_ptr(), dout.data_ptr(),
                             _at(initial_state), _at(dfinal_state), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
                             _at(dinitial_state), _at(workspace), n, s)
    if code:
        raise AttnError("linear_attn_bwd", code)
    return dq, dk, dv, dinitial_state


def linear_attn_step(q, k, v, log_decay, state, *, slots=None, scale=None, out=None,
                     error_word=None, stream=None):
    """One token for each sequence: q bf16 [n, Hq, D], k, v [n, Hkv, D]; state fp32
    [slots, Hkv, D, D], updated in place; slots int32 [n], the state of each
    sequence (-1: padding; None: sequence n's is state[n]).  Returns o."""
    gpu, dev = _gpu_of(q, "q")
    shape = q.shape
    if len(shape) != 3:
        raise ValueError("q, k and v must be [num_seqs, heads, head_dim]")
    n, heads, dim = shape
    heads_kv, sq, sk, sv = _linear_heads(q, k, v, log_decay, gpu, dev)
    if not _ok(state, torch.float32, gpu):
        _need(state, "state", torch.float32, dev)
    st = state.shape
    if len(st) != 4 or st[1] != heads_kv or st[2] != dim or st[3] != dim:
        raise ValueError(f"state must be [slots, {heads_kv}, {dim}, {dim}], got {list(st)}")
    at = None
    if slots is not None:
        if not _ok(slots, torch.int32, gpu):
            _need(slots, "slots", torch.int32, dev)
        if slots.dim() != 1 or slots.numel() != n:
            raise ValueError(f"slots must be [{n}], got {list(slots.shape)}")
        at = slots.data_ptr()
    if out is not None:
        _out_like(out, "out", q, gpu, dev)
    p = _LinearStep(_size(n, "sequences"), _size(st[0], "states"), heads, heads_kv, dim,
                    float(scale) if scale is not None else 1.0 / math.sqrt(dim), sq, sk, sv, at, log_decay.data_ptr(), _word(error_word, gpu, dev))
    ctx, s = _on(dev, stream)
    if ctx is None:
        return _linear_step_here(p, q, k, v, state, out, s)
    with ctx:
        return _linear_step_here(p, q, k, v, state, out, s)


def _linear_step_here(p, q, k, v, state, out, s):
    if out is None:
        out = _new_like(q, p.q_stride)
    code = (_LIB or lib()).linear_attn_step(ctypes.byref(p), q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                            state.data_ptr(), out.data_ptr(), s)
    if code:
        raise AttnError("linear_attn_step", code)
    return out
