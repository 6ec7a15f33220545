"""GPU tests of linear attention's edges: arrays of lengths that break their contract at sizes that
are cut into segments."""
import pytest
import torch

import softmax_attention_backward_gb300 as A
from _linear_util import BF, DEV, F64, Rows
from oracle import linear as OL

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


# A rounding to bf16 of normally distributed values is off by 0.736 2^-8 / sqrt 3 of them in the mean
# square (0.541 the ratio of 4^e to the values' square, 0.46 to 0.55 over mixtures of scales).  Two
# independent ones, the output's and that of a score or of a decayed key or state on the way, are off by
# sqrt(1 + 0.55 / 0.46) = 1.48 times the output's alone at most; three by 1.7, where the rows see
# far more of the states than of their own chunk, as here: memories of 500 to 4000 tokens.
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,hq,hkv", [([4096], 4, 4), ([4096], 8, 2), ([384] * 16, 10, 10), ([1500, 700, 900], 4, 2),
                                         ([2500, 1900, 800, 600, 500, 400, 300, 200, 150, 100, 90, 60], 16, 16)])
@pytest.mark.parametrize("states", [False, True])
def test_two_roundings_and_no_more(D, lens, hq, hkv, states):
    s = Rows(lens, hq, hkv, D, states=states, seed=40, decay=-torch.exp2(-9 - 3 * torch.linspace(0, 1, hkv)))
    got = s.call(states=states)
    want = [OL.linear_forward(s.q, s.k, s.v, s.g, s.scale, lens, s.init)[0],
            *OL.linear_backward(s.q, s.k, s.v, s.do, s.g, s.scale, lens, s.init, s.dfin)[:3]]
    ratio = {}
    for name, x, w in zip(("o", "dq", "dk", "dv"), (got[0], *got[2:5]), want):
        once = (w.to(BF).to(F64) - w).square().mean().sqrt()
        ratio[name] = ((x.to(F64) - w).square().mean().sqrt() / once).item()
    assert max(ratio.values()) <= 1.5, ratio


def test_thousands_of_steps_keep_the_decay():
    # Each step rounds a state once to fp32 (2^-24 of it at most, 1 / sqrt 3 of that in the mean square, in directions
    # that do not follow from each other: 1 - l is at least 800 steps of fp32).  6000 of them add up to 77 of
    # one; twice that is allowed.  One fp32 number for the decay is off by the same in every step,
    # 1.4e-4 of the state after all of them.
    N, D = 6000, 64
    g = torch.tensor([-2.0 ** -11, -3e-4, -1e-3, -1e-4])
    l = torch.exp(g.to(F64))
    once = 2.0 ** -24 / 3 ** 0.5
    bound = 2 * N ** 0.5 * once
    assert (N * (l.float().to(F64) / l - 1).abs()).max() > 4 * bound      # (what the test is to tell apart)
    gen = torch.Generator().manual_seed(50)
    k, v = (torch.randn(16, 2, 4, D, generator=gen).to(BF) for _ in range(2))
    k[:, 0] = 0                                           # one sequence keeps its first state alone
    state = torch.randn(2, 4, D, D, generator=gen)
    st, gd, kd, vd = state.to(DEV), g.to(DEV), k.to(DEV), v.to(DEV)
    want = state.to(F64)
    kv = k.to(F64)[..., :, None] * v.to(F64)[..., None, :]
    for i in range(N):
        A.linear_attn_step(kd[i % 16], kd[i % 16], vd[i % 16], gd, st)
        want = l[:, None, None] * want + kv[i % 16]
    rms = ((st.cpu().to(F64) - want).square().mean((2, 3)) / want.square().mean((2, 3))).sqrt()
    assert (rms <= bound).all(), rms
