"""Host-only checks of the rotation's and linear attention's C ABI and binding: invalid
calls are rejected before the GPU is touched (no kernel is launched here)."""
import ctypes

import pytest
import torch

import softmax_attention_backward_gb300 as A
from softmax_attention_backward_gb300 import build as B

FAKE = 0x10000   # aligned; never dereferenced
BF = torch.bfloat16


@pytest.fixture(scope="module")
def L():
    B.build()
    return A.lib()


def _make(cls, base, kw):
    p = cls()
    for k, v in {**base, **kw}.items():
        setattr(p, k, v)
    return p


def _ptrs(n, at):
    v = [FAKE + (i << 24) for i in range(n)]
    for i, x in at.items():
        v[i] = x
    return [ctypes.c_void_p(x) for x in v]


def _table(L, out=FAKE, **kw):
    base = dict(max_position=8, rot_dim=64, base=10000.0, scaling=0, factor=1.0, original=0, fast=32.0, slow=1.0, magnitude=1.0)
    return L.attn_rotary_table(ctypes.byref(_make(A._RotaryTable, base, kw)), ctypes.c_void_p(out), None)


@pytest.mark.parametrize("kw,code", [
    (dict(max_position=-1), 1), (dict(rot_dim=0), 1), (dict(rot_dim=8), 2), (dict(rot_dim=24), 2), (dict(rot_dim=272), 2),
    (dict(base=0.0), 1), (dict(base=-1.0), 1), (dict(base=float("inf")), 1), (dict(base=float("nan")), 1),
    (dict(magnitude=float("inf")), 1), (dict(magnitude=1e300), 1), (dict(scaling=4), 1), (dict(scaling=-1), 1), (dict(scaling=1, factor=0.0), 1),
    (dict(scaling=2, factor=float("nan")), 1), (dict(scaling=3, factor=2.0), 1),
    (dict(scaling=3, factor=2.0, original=64, fast=1.0), 1), (dict(scaling=3, factor=2.0, original=64, fast=float("inf")), 1),
    (dict(out=0), 1), (dict(out=FAKE + 8), 3), (dict(max_position=0), 0)])
def test_table_refusals(L, kw, code):
    assert _table(L, **kw) == code
    assert L.attn_rotary_table(None, None, None) == 1


ROT = dict(tokens=4, heads_q=8, heads_k=2, head_dim=128, rot_dim=64, rot_offset=0, interleaved=0, max_position=16, seqlen=4,
           num_seqs=0, q_stride=0, k_stride=0, cu_seqlens=None, positions=None)


@pytest.mark.parametrize("fn", ["attn_rotary_fwd", "attn_rotary_bwd"])
@pytest.mark.parametrize("kw,at,code", [
    (dict(tokens=-1), {}, 1), (dict(heads_q=0), {}, 1), (dict(heads_k=-1), {}, 1), (dict(head_dim=0), {}, 1),
    (dict(rot_dim=0), {}, 1), (dict(max_position=0), {}, 1), (dict(rot_offset=-8), {}, 1), (dict(seqlen=0), {}, 1),
    (dict(cu_seqlens=FAKE), {}, 1), (dict(head_dim=132), {}, 2), (dict(head_dim=1032), {}, 2), (dict(rot_dim=40), {}, 2),
    (dict(rot_offset=4), {}, 2), (dict(rot_offset=72), {}, 1), (dict(rot_dim=144), {}, 1), (dict(heads_k=0), {}, 1),
    (dict(heads_q=1 << 24), {}, 2), (dict(tokens=(1 << 31) - 1), {}, 2),
    ({}, {0: 0}, 1), ({}, {1: 0}, 1), ({}, {2: 0}, 1), ({}, {3: 0}, 1), ({}, {4: 0}, 1), ({}, {1: 0, 4: 0}, 1),
    ({}, {0: FAKE + 8}, 3), ({}, {1: FAKE + 8}, 3), ({}, {2: FAKE + 4}, 3), ({}, {3: FAKE + 2}, 3), ({}, {4: FAKE + 2}, 3),
    (dict(positions=FAKE + 2), {}, 3), (dict(error_word=FAKE + 1), {}, 3), (dict(q_stride=1020), {}, 1),
    (dict(q_stride=1028), {}, 3), (dict(k_stride=128), {}, 1), (dict(q_stride=2048), {3: FAKE}, 1), (dict(tokens=0), {}, 0)])
def test_rotation_refusals(L, fn, kw, at, code):
    # q k cos_sin q_out k_out
    assert getattr(L, fn)(ctypes.byref(_make(A._RotaryProblem, ROT, kw)), *_ptrs(5, at), None) == code
    assert getattr(L, fn)(None, *_ptrs(5, {}), None) == 1


LIN = dict(num_seqs=2, seqlen=3, tokens=6, heads_q=8, heads_kv=2, head_dim=128, scale=0.1, cu_seqlens=None, log_decay=FAKE)


def _fwd(L, kw={}, at={}, ws=1 << 34):   # q k v initial o final workspace
    return L.linear_attn_fwd(ctypes.byref(_make(A._LinearProblem, LIN, kw)), *_ptrs(7, at), ws, None)


def _bwd(L, kw={}, at={}, ws=1 << 34):   # q k v dout initial dfinal dq dk dv dinitial workspace
    return L.linear_attn_bwd(ctypes.byref(_make(A._LinearProblem, LIN, kw)), *_ptrs(11, at), ws, None)


BAD = [(dict(num_seqs=0), 1), (dict(tokens=-1), 1), (dict(tokens=7), 1), (dict(seqlen=-1), 1), (dict(heads_q=0), 1),
       (dict(heads_q=7), 1), (dict(heads_kv=0), 1), (dict(head_dim=0), 1), (dict(head_dim=96), 2), (dict(head_dim=256), 2),
       (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(log_decay=None), 1), (dict(log_decay=FAKE + 2), 3),
       (dict(cu_seqlens=FAKE + 2), 3), (dict(error_word=FAKE + 2), 3), (dict(heads_q=1 << 17), 2),
       (dict(cu_seqlens=FAKE, tokens=1 << 28), 2), (dict(cu_seqlens=FAKE, num_seqs=1 << 26), 2)]


@pytest.mark.parametrize("kw,code", BAD)
def test_linear_refuses(L, kw, code):
    assert _fwd(L, kw) == code
    assert _bwd(L, kw) == code
    p = _make(A._LinearProblem, LIN, kw)
    assert L.linear_attn_fwd_workspace_size(ctypes.byref(p)) == 0
    assert L.linear_attn_bwd_workspace_size(ctypes.byref(p)) == 0


def test_linear_pointers(L):
    assert L.linear_attn_fwd(None, *_ptrs(7, {}), 0, None) == 1
    assert L.linear_attn_bwd(None, *_ptrs(11, {}), 0, None) == 1
    assert L.linear_attn_fwd_workspace_size(None) == 0 and L.linear_attn_bwd_workspace_size(None) == 0
    for i in (0, 1, 2, 4):
        assert _fwd(L, at={i: 0}) == 1 and _fwd(L, at={i: FAKE + 8}) == 3
    for i in (0, 1, 2, 3, 6, 7, 8):
        assert _bwd(L, at={i: 0}) == 1 and _bwd(L, at={i: FAKE + 8}) == 3
    for i in (3, 5):
        assert _fwd(L, at={i: FAKE + 8}) == 3
    for i in (4, 5, 9):
        assert _bwd(L, at={i: FAKE + 8}) == 3
    far = {i: (i + 1) << 24 for i in range(11)}      # states of 256 KB, apart
    for x in (0, 16, 0x3fff0, -0x3fff0):              # the final state over the initial one
        assert _fwd(L, at={**{i: far[i] for i in range(7)}, 5: far[3] + x}, ws=0) == 1
        assert _bwd(L, at={**far, 9: far[5] + x}, ws=0) == 1 and _bwd(L, at={**far, 9: far[4] + x}, ws=0) == 1
    for s in ("q_stride", "k_stride", "v_stride"):
        for x in (8, 1028, -1024):
            assert _fwd(L, {s: x}) == 1 and _bwd(L, {s: x}) == 1
    assert _bwd(L, dict(dout_stride=1028)) == 1
    assert _fwd(L, dict(num_seqs=0, seqlen=0, tokens=0)) == 0 and _bwd(L, dict(num_seqs=0, seqlen=0, tokens=0)) == 0
    # without a token and without a state wanted, nothing is enqueued
    assert _fwd(L, dict(seqlen=0, tokens=0), {i: 0 for i in range(7)}) == 0
    assert _bwd(L, dict(seqlen=0, tokens=0), {i: 0 for i in range(11)}) == 0


STEP = dict(num_seqs=3, num_slots=5, heads_q=8, heads_kv=2, head_dim=64, scale=0.1, slots=FAKE, log_decay=FAKE)


@pytest.mark.parametrize("kw,at,code", [
    (dict(num_seqs=-1), {}, 1), (dict(num_slots=0), {}, 1), (dict(heads_q=0), {}, 1), (dict(heads_q=7), {}, 1),
    (dict(heads_kv=0), {}, 1), (dict(head_dim=0), {}, 1), (dict(head_dim=32), {}, 2), (dict(scale=float("inf")), {}, 1),
    (dict(slots=None, num_seqs=6), {}, 1), (dict(log_decay=None), {}, 1), (dict(heads_q=1 << 17), {}, 2),
    (dict(slots=FAKE + 2), {}, 3), (dict(log_decay=FAKE + 2), {}, 3), (dict(error_word=FAKE + 2), {}, 3),
    (dict(q_stride=8), {}, 1), (dict(k_stride=132), {}, 1), (dict(v_stride=-128), {}, 1),
    *[({}, {i: 0}, 1) for i in range(5)], *[({}, {i: FAKE + 8}, 3) for i in range(5)], (dict(num_seqs=0), {}, 0)])
def test_step_refusals(L, kw, at, code):
    # q k v state o
    assert L.linear_attn_step(ctypes.byref(_make(A._LinearStep, STEP, kw)), *_ptrs(5, at), None) == code
    assert L.linear_attn_step(None, *_ptrs(5, {}), None) == 1


def test_binding_refusals():
    q, g = torch.zeros(1, 4, 2, 64, dtype=BF), torch.zeros(2)
    with pytest.raises(ValueError, match="CUDA"):
        A.linear_attn_fwd(q, q, q, g)
    with pytest.raises(ValueError, match="CUDA"):
        A.linear_attn_bwd(q, q, q, q, g)
    with pytest.raises(ValueError, match="CUDA"):
        A.linear_attn_step(q[0], q[0], q[0], g, torch.zeros(4, 2, 64, 64))
    with pytest.raises(ValueError, match="CUDA"):
        A.attn_rotary_fwd(q, q, torch.zeros(4, 64))
    with pytest.raises(ValueError, match="scaling"):
        A.attn_rotary_table(8, 64, scaling="other")
    with pytest.raises(ValueError, match="CUDA"):
        A.attn_rotary_table(8, 64, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        A.attn_rotary_table(8, 64, out=torch.zeros(8, 64))


def test_outputs_that_share_memory_are_refused(L):
    # rows of 4 x 1024 and 4 x 256 bf16 (rotation), 6 x 1024 and 6 x 256 bf16 and states of 256 KB (linear)
    far = [(i + 1) << 24 for i in range(11)]
    for fn in ("attn_rotary_fwd", "attn_rotary_bwd"):
        for i, x in ((3, far[0] + 16), (3, far[0] - 16), (3, far[1]), (4, far[0]), (4, far[1] + 2032), (4, far[3] + 8176)):
            at = {**dict(enumerate(far[:5])), i: x}
            assert getattr(L, fn)(ctypes.byref(_make(A._RotaryProblem, ROT, {})), *_ptrs(5, at), None) == 1
    for out, n, call in (((4, 5), 6, _fwd), ((6, 7, 8, 9), 10, _bwd)):
        for i in out:
            for k in range(n):
                if k != i:
                    assert call(L, at={**dict(enumerate(far[:n + 1])), i: far[k]}, ws=0) == 1
    at = dict(enumerate(far[:7]))
    assert _fwd(L, at={**at, 4: far[0] + 16}, ws=0) == 1 and _fwd(L, at={**at, 4: far[1] - 16}, ws=0) == 1
    assert _fwd(L, dict(k_stride=4096), {**at, 4: far[1] + 5 * 8192 + 496}, ws=0) == 1   # the last row's last bytes
    for i in (3, 4):
        for k in range(5):
            if k != i:
                at = {**dict(enumerate(far[:5])), i: far[k]}
                assert L.linear_attn_step(ctypes.byref(_make(A._LinearStep, STEP, {})), *_ptrs(5, at), None) == 1
