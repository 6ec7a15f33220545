"""Host-only checks of calls at the edges of the rotation's and linear attention's contracts: outputs
over the small arrays and the workspace, sizes that 32 bits do not hold."""
import ctypes

import pytest
import torch

import softmax_attention_backward_gb300 as A
from test_abi_linear import LIN, ROT, STEP, L, _bwd, _fwd, _make, _ptrs   # noqa: F401 (L is a fixture)

FAR = [(i + 1) << 24 for i in range(12)]   # arguments apart from each other; never dereferenced


@pytest.mark.parametrize("small", ["log_decay", "cu_seqlens", "error_word"])
def test_outputs_over_small_arrays_are_refused(L, small):
    # (2 sequences: cu_seqlens has 12 bytes; log_decay of 2 heads 8)
    size = dict(log_decay=8, cu_seqlens=12, error_word=4)[small]
    for out, n, call in (((4, 5), 7, _fwd), ((6, 7, 8, 9), 11, _bwd)):
        at = dict(enumerate(FAR[:n]))
        for i in out:
            for x in (FAR[i], FAR[i] + 64, FAR[i] - size + 4):
                assert call(L, {"log_decay": 8, small: x}, at, ws=0) == 1
        # a final state without a token
        assert call(L, {"log_decay": 8, "seqlen": 0, "tokens": 0, small: FAR[out[-1]] + 64}, at, ws=0) == 1


def test_a_workspace_over_another_argument_is_refused(L):
    # one long sequence, which is cut; the rows take 16 MB of 8 heads of 128
    kw = dict(num_seqs=1, seqlen=8192, tokens=8192, heads_q=8, heads_kv=8, log_decay=FAR[11] << 4)
    for n, call, size in ((7, _fwd, L.linear_attn_fwd_workspace_size), (11, _bwd, L.linear_attn_bwd_workspace_size)):
        need = size(ctypes.byref(_make(A._LinearProblem, LIN, kw)))
        assert need > 0
        at = {i: x << 4 for i, x in enumerate(FAR[:n])}
        assert call(L, kw, at, ws=need - 1) == 5                     # (too small, and nothing else is wrong)
        for i in range(n - 1):
            for x in (at[i], at[i] - need + 16):
                assert call(L, kw, {**at, n - 1: x}, ws=need) == 1
        assert call(L, {**kw, "log_decay": at[n - 1] + need - 16}, at, ws=need) == 1


def test_a_step_over_its_slots_or_decays_is_refused(L):
    # states of 5 x 2 x 64 x 64 fp32, outputs of 3 x 8 x 64 bf16
    for name in ("slots", "log_decay", "error_word"):
        for i in (3, 4):
            for x in (FAR[i], FAR[i] + 64, FAR[i] - 4 if name != "error_word" else FAR[i]):
                kw = dict(slots=4, log_decay=8, error_word=None)
                assert L.linear_attn_step(ctypes.byref(_make(A._LinearStep, STEP, {**kw, name: x})),
                                          *_ptrs(5, dict(enumerate(FAR[:5]))), None) == 1


@pytest.mark.parametrize("fn", ["attn_rotary_fwd", "attn_rotary_bwd"])
def test_a_rotation_over_its_table_or_positions_is_refused(L, fn):
    # q_out of 4 x 8 x 128 and k_out of 4 x 2 x 128 bf16; a table of 16 x 64 fp32
    for i in (3, 4):
        for kw, at in ((dict(), {2: FAR[i]}), (dict(), {2: FAR[i] - 4080}), (dict(), {2: FAR[i] + 1024}),
                       (dict(positions=FAR[i] - 12), {}), (dict(positions=FAR[i] + 1024), {}),
                       (dict(cu_seqlens=FAR[i] - 4, num_seqs=1), {}), (dict(error_word=FAR[i] + 8), {})):
            p = _make(A._RotaryProblem, ROT, kw)
            assert getattr(L, fn)(ctypes.byref(p), *_ptrs(5, {**dict(enumerate(FAR[:5])), **at}), None) == 1


def test_sizes_past_32_bits_are_refused():
    # (cut off to 32 bits they would be other sizes: 2^32 + 8 positions a table of 8)
    for kw in (dict(max_position=(1 << 32) + 8), dict(max_position=1 << 31), dict(max_position=8 - (1 << 32)), dict(rot_dim=(1 << 32) + 64),
               dict(scaling="parts", factor=2.0, original=(1 << 32) + 64)):
        with pytest.raises(ValueError, match="at most"):
            A.attn_rotary_table(**{**dict(max_position=8, rot_dim=64, device="cuda:0"), **kw})
    for shape in ((1 << 16, 1 << 16, 1, 16), (1 << 32, 0, 1, 16), (0, 1 << 32, 1, 16)):
        with pytest.raises(ValueError, match="at most"):
            A._lead(torch.Size(shape), None, 0, None)
    assert A._lead(torch.Size((1 << 15, 1 << 15, 1, 16)), None, 0, None)[:3] == (1 << 30, 1 << 15, 1 << 15)
