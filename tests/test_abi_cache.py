"""Host-only checks of the paged cache's C ABI and binding: invalid calls are
rejected before the GPU is touched (no kernel is launched here)."""
import ctypes

import pytest
import torch

import softmax_attention_backward_gb300 as A
from softmax_attention_backward_gb300 import build as B

FAKE = 0x10000   # aligned; never dereferenced


@pytest.fixture(scope="module")
def L():
    B.build()
    return A.lib()


def _p(**kw):
    p = A._CacheProblem()
    d = dict(num_seqs=4, tokens=4, heads_q=8, heads_kv=2, head_dim=128, cache_type=0, page_size=16, num_pages=100,
             max_pages=32, max_new=1, causal=1, scale=0.1, cu_seqlens=FAKE, seqlens_kv=FAKE, page_table=FAKE)
    d.update(kw)
    for k, v in d.items():
        setattr(p, k, v)
    return p


def _ptrs(n, **at):
    v = [FAKE] * n
    for i, x in at.items():
        v[int(i[1:])] = x
    return [ctypes.c_void_p(x) for x in v]


def _append(L, p, **at):   # q k v cos_sin q_out k_cache v_cache k_scale v_scale
    return L.attn_cache_append(ctypes.byref(p), *_ptrs(9, **at), None)


def _fwd(L, p, ws=1 << 30, **at):   # q k_cache v_cache k_scale v_scale o lse workspace
    return L.attn_cache_fwd(ctypes.byref(p), *_ptrs(8, **at), ws, None)


BAD = [(dict(num_seqs=0), 1), (dict(tokens=-1), 1), (dict(heads_q=0), 1), (dict(heads_q=7), 1), (dict(heads_kv=0), 1),
       (dict(num_pages=0), 1), (dict(max_pages=0), 1), (dict(max_new=0), 1), (dict(max_new=-1), 1), (dict(cache_type=2), 1),
       (dict(scale=float("inf")), 1), (dict(scale=float("nan")), 1), (dict(cu_seqlens=None), 1), (dict(seqlens_kv=None), 1),
       (dict(page_table=None), 1), (dict(head_dim=96), 2), (dict(page_size=8), 2), (dict(page_size=48), 2),
       (dict(page_size=256), 2), (dict(heads_q=1 << 17), 2), (dict(tokens=1 << 29), 2), (dict(num_pages=1 << 27), 2),
       (dict(cu_seqlens=FAKE + 2), 3), (dict(seqlens_kv=FAKE + 1), 3), (dict(page_table=FAKE + 2), 3),
       (dict(error_word=FAKE + 2), 3), (dict(q_stride=512), 1), (dict(q_stride=1028), 1), (dict(q_stride=-1024), 1)]


@pytest.mark.parametrize("kw,code", BAD)
def test_both_refuse(L, kw, code):
    assert _append(L, _p(**kw)) == code
    assert _fwd(L, _p(**kw)) == code
    if "stride" not in next(iter(kw)):
        assert L.attn_cache_fwd_workspace_size(ctypes.byref(_p(**kw))) == 0


def test_null_problem(L):
    assert L.attn_cache_append(None, *_ptrs(9), None) == 1
    assert L.attn_cache_fwd(None, *_ptrs(8), 0, None) == 1
    assert L.attn_cache_fwd_workspace_size(None) == 0


def test_append_refusals(L):
    for i in (1, 2, 5, 6):
        assert _append(L, _p(), **{f"i{i}": 0}) == 1                 # k, v, the pools
        assert _append(L, _p(), **{f"i{i}": FAKE + 8}) == 3
    assert _append(L, _p(), i0=0) == 1 and _append(L, _p(), i4=0) == 1   # q and q_out go together
    assert _append(L, _p(cache_type=1), i7=0) == 1 and _append(L, _p(cache_type=1), i8=0) == 1
    assert _append(L, _p(cache_type=1), i7=FAKE + 2) == 3
    assert _append(L, _p(rot_dim=24, max_position=9)) == 1           # not a multiple of 16
    assert _append(L, _p(rot_dim=144, max_position=9)) == 1          # more than head_dim
    assert _append(L, _p(rot_dim=-16, max_position=9)) == 1
    assert _append(L, _p(rot_dim=64, max_position=0)) == 1
    assert _append(L, _p(rot_dim=64, max_position=9), i3=0) == 1     # no table
    assert _append(L, _p(rot_dim=64, max_position=9), i3=FAKE + 4) == 3
    assert _append(L, _p(k_stride=128)) == 1 and _append(L, _p(v_stride=260)) == 1
    # q_out over a q whose tokens lie apart
    assert _append(L, _p(q_stride=2048)) == 1
    assert _append(L, _p(tokens=0)) == 0                             # nothing enqueued


def test_fwd_refusals_and_workspace(L):
    for i in (0, 1, 2, 5, 6):
        assert _fwd(L, _p(), **{f"i{i}": 0}) == 1
        assert _fwd(L, _p(), **{f"i{i}": FAKE + 8}) == 3
    assert _fwd(L, _p(cache_type=1), i3=0) == 1 and _fwd(L, _p(cache_type=1), i4=0) == 1
    n = L.attn_cache_fwd_workspace_size(ctypes.byref(_p()))
    # per CTA: a part of 8 rows x 128 fp32 for each of 8 warps, and two parts with (maximum,
    # sum) of their rows and 16 bytes of meta data
    assert n == 152 * (8 * 8 * 128 * 4 + 2 * (8 * 128 * 4 + 8 * 8 + 16))
    assert L.attn_cache_fwd_workspace_size(ctypes.byref(_p(max_new=3))) == 152 * (
        8 * 16 * 128 * 4 + 2 * (16 * 128 * 4 + 16 * 8 + 16))
    assert _fwd(L, _p(), ws=n - 1) == 5 and _fwd(L, _p(), i7=0) == 5
    assert _fwd(L, _p(), i7=FAKE + 4) == 3
    assert _fwd(L, _p(tokens=0), ws=0) == 0


def test_binding_refusals():
    bf = torch.bfloat16
    with pytest.raises(TypeError, match="float8_e4m3fn"):
        A.attn_cache_empty(4, 1, 16, 64, dtype=torch.float16, device="cpu")
    k, v, ks, vs = A.attn_cache_empty(4, 1, 16, 64, dtype=torch.float8_e4m3fn, device="cpu")
    assert k.shape == v.shape == (4, 1, 16, 64) and ks.shape == vs.shape == (4, 1)
    k, v, ks, vs = A.attn_cache_empty(4, 1, 16, 64, device="cpu")
    assert k.dtype == bf and ks is None and vs is None
    i32 = dict(dtype=torch.int32)
    kw = dict(page_table=torch.zeros(1, 4, **i32), seqlens_kv=torch.ones(1, **i32), cu_seqlens=torch.zeros(2, **i32),
              max_new=1)
    q = torch.zeros(1, 2, 64, dtype=bf)
    with pytest.raises(ValueError, match="CUDA"):
        A.attn_cache_fwd(q, k, v, **kw)
    with pytest.raises(TypeError, match="k_cache"):
        A.attn_cache_fwd(q, k.float(), v.float(), **kw)
    with pytest.raises(ValueError, match="without q"):
        A.attn_cache_append(None, q, q, k, v, q_out=q, **kw)
