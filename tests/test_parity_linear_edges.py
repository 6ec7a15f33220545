"""GPU tests of linear attention's edges: arrays of lengths that break their contract at sizes that
are cut into segments."""
import pytest
import torch

import softmax_attention_backward_gb300 as A
from _linear_util import BF, DEV

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32, device=DEV)


def _inside(n, margin=16 << 20):
    """A workspace of n bytes, and the margins on both sides of it that a call leaves as they are."""
    all_ = torch.full((n + 2 * margin,), 0x5A, dtype=torch.uint8, device=DEV)
    return all_[margin:margin + n], (all_[:margin], all_[margin + n:])


@pytest.mark.parametrize("D,hq,hkv", [(128, 2, 2), (128, 4, 1), (64, 2, 2), (64, 4, 2)])
@pytest.mark.parametrize("T,cu", [(4096, [0, 4096, 0, 4096]), (8192, [0, 8192, 0, 8192, 0, 8192]),
                                  (8192, [0, 8192, *[0] * 38, 8192]), (8192, [0, 3000, 2000, 8192, 100, 8192]),
                                  (4096, [4096, 0, 4096]), (4096, [0, 1 << 30, -7, 4096])])
def test_decreasing_ends_stay_within_the_workspace(D, hq, hkv, T, cu):
    g = torch.Generator().manual_seed(T + len(cu))
    q, k, v, do = (torch.randn(T, h, D, generator=g).to(BF).to(DEV) for h in (hq, hkv, hkv, hq))
    decay = -torch.exp2(-10 * torch.rand(hkv, generator=g)).to(DEV)
    good = torch.tensor(cu).clamp(0, T).cummax(0).values.to(**I32)   # each begins where the one before ends
    cu = torch.tensor(cu, **I32)
    for states in (False, True):
        kw = dict(initial_state=torch.ones(len(cu) - 1, hkv, D, D, device=DEV) if states else None)
        for backward in (False, True):
            size = A.linear_attn_bwd_workspace_size if backward else A.linear_attn_fwd_workspace_size
            n = size(q, k, v, decay, cu_seqlens=cu)
            assert n > 0
            ws, around = _inside(n)

            def call(cu, err):
                if backward:
                    return A.linear_attn_bwd(q, k, v, do, decay, cu_seqlens=cu, want_dinitial_state=states, workspace=ws,
                                             error_word=err, **kw)
                return A.linear_attn_fwd(q, k, v, decay, cu_seqlens=cu, want_final_state=states, workspace=ws, error_word=err,
                                         **kw)

            err = torch.zeros(1, **I32)
            got = call(cu, err)
            torch.cuda.synchronize()
            assert err.item() == 4
            for m in around:
                assert (m == 0x5A).all()
            err.zero_()
            want = call(good, err)
            assert err.item() == (4 if good[0] else 0)
            live = slice(int(good[0]), T)          # rows of sequences, which are those of `good`
            for x, y in zip(got, want):
                if x is not None:
                    assert torch.equal(x, y) if x.dim() == 4 else torch.equal(x[live], y[live])
