"""The linear-attention oracle against autograd through the quadratic form, and the
frequencies' closed forms (CPU)."""
import math

import pytest
import torch

from oracle import linear as OL

F64 = torch.float64


def quadratic(q, k, v, g, scale, initial):
    """One sequence: o_i = scale sum_{j <= i} l^(i - j) <q_i, k_j> v_j + scale l^(i + 1) S_0^T q_i."""
    T, hq, D = q.shape
    hkv = k.shape[1]
    i = torch.arange(T, dtype=F64)
    far = i[:, None] - i
    o = []
    for h in range(hq):
        a = h * hkv // hq
        w = torch.where(far >= 0, torch.exp(g[a] * far.clamp(min=0)), torch.zeros((), dtype=F64))
        s0 = torch.exp(g[a] * (i + 1))[:, None] * (q[:, h] @ initial[a])
        o.append(scale * ((q[:, h] @ k[:, a].T * w) @ v[:, a] + s0))
    left = torch.exp(g[:, None] * (T - 1 - i))
    final = torch.exp(g * T)[:, None, None] * initial + torch.einsum("thr,thc->hrc", left.T[..., None] * k, v)
    return torch.stack(o, 1), final


@pytest.mark.parametrize("hq,hkv,D,lens", [(2, 2, 3, [5]), (6, 2, 4, [7, 1, 4]), (3, 1, 2, [0, 9])])
def test_oracle_against_autograd(hq, hkv, D, lens):
    gen = torch.Generator().manual_seed(hq + D)
    T = sum(lens)

    def randn(*s):
        return torch.randn(*s, generator=gen, dtype=F64)

    q, k, v, do = randn(T, hq, D), randn(T, hkv, D), randn(T, hkv, D), randn(T, hq, D)
    init, dfin = randn(len(lens), hkv, D, D), randn(len(lens), hkv, D, D)
    g = -torch.rand(hkv, generator=gen, dtype=F64)
    o, fin = OL.linear_forward(q, k, v, g, 0.7, lens, init)
    got = OL.linear_backward(q, k, v, do, g, 0.7, lens, init, dfin)
    for n, at, m in OL.rows_of(lens, T):
        x = [t[at:at + m].clone().requires_grad_() for t in (q, k, v)] + [init[n].clone().requires_grad_()]
        ro, rf = quadratic(*x[:3], g, 0.7, x[3])
        torch.testing.assert_close(o[at:at + m], ro.detach())
        torch.testing.assert_close(fin[n], rf.detach())
        want = torch.autograd.grad((ro * do[at:at + m]).sum() + (rf * dfin[n]).sum(), x)
        for a, b in zip([t[at:at + m] for t in got[:3]] + [got[3][n]], want):
            torch.testing.assert_close(a, b)


def test_no_decay_and_full_decay():
    gen = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(6, 2, 3, generator=gen, dtype=F64) for _ in range(3))
    o, fin = OL.linear_forward(q, k, v, torch.tensor([0.0, -math.inf]), 1.0, [6])
    torch.testing.assert_close(fin[0, 0], k[:, 0].T @ v[:, 0])          # everything is kept
    torch.testing.assert_close(fin[0, 1], torch.outer(k[5, 1], v[5, 1]))  # only the last token
    torch.testing.assert_close(o[:, 1], (q[:, 1] * k[:, 1]).sum(-1, keepdim=True) * v[:, 1])


def test_frequencies():
    f = OL.frequencies(64, 10000.0)
    assert f[0] == 1.0 and abs(f[-1] - 10000.0 ** (-62 / 64)) < 1e-18
    assert OL.frequencies(64, scaling="linear", factor=4.0) == [x / 4 for x in f]
    b = OL.frequencies(64, scaling="base", factor=4.0)
    assert b[0] == 1.0 and abs(b[-1] / f[-1] - 0.25) < 1e-12            # the lowest is divided, the highest kept
    p = OL.frequencies(64, scaling="parts", factor=4.0, original=2048)
    assert p[0] == f[0] and abs(p[-1] - f[-1] / 4) < 1e-18
    assert all(x / 4 - 1e-18 <= y <= x for x, y in zip(f, p))
