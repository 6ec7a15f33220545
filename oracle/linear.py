"""fp64 CPU oracle for the rotation by position and for linear attention with a decay per head.

TEST INFRASTRUCTURE ONLY, like the rest of this package.

Table: cos_sin[p, a] = m cos(p f_a), cos_sin[p, r/2 + a] = m sin(p f_a), f_a = base^(-2a/r),
scaled: linear, f / factor; base, base * factor^(r / (r - 2)) for base; parts, f (w + (1 - w) /
factor), w the ramp from 0 to 1 of original f / 2 pi between slow and fast.

Linear attention of one sequence and KV head, l = exp(log_decay), token by token:
  S_t = l S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t   (q of every query head of the KV head)
and backwards, D_t = dL/dS_t:
  D_t = (D_{t+1} l, or dL/d(final state) past the last token) + scale sum_q q_t dout_t^T,
  dq_t = scale S_t dout_t, dk_t = D_t v_t, dv_t = D_t^T k_t, dL/d(initial state) = l D_first.
"""
from __future__ import annotations

import math

import torch

F64 = torch.float64


def frequencies(rot, base=10000.0, scaling="none", factor=1.0, original=0, fast=32.0, slow=1.0):
    if scaling == "base":
        base = base * factor ** (rot / (rot - 2.0))
    f = [base ** (-2.0 * a / rot) for a in range(rot // 2)]
    if scaling == "linear":
        f = [x / factor for x in f]
    if scaling == "parts":
        w = [min(1.0, max(0.0, (original * x / (2 * math.pi) - slow) / (fast - slow))) for x in f]
        f = [x * (u + (1 - u) / factor) for x, u in zip(f, w)]
    return f


def rows_of(lens, rows):
    """[(sequence, its first row, its tokens)] of a packing; rows behind are padding."""
    out, at = [], 0
    for n, m in enumerate(lens):
        out.append((n, at, m))
        at += m
    assert at <= rows
    return out


def linear_forward(q, k, v, log_decay, scale, lens, initial=None):
    """q [T, Hq, D], k, v [T, Hkv, D] -> o fp64 [T, Hq, D], final states [n, Hkv, D, D]."""
    T, hq, D = q.shape
    hkv = k.shape[1]
    g = hq // hkv
    q, k, v = (x.to(F64) for x in (q, k, v))
    l = torch.exp(log_decay.to(F64))[:, None, None]
    o = torch.zeros(T, hq, D, dtype=F64)
    final = torch.zeros(len(lens), hkv, D, D, dtype=F64)
    for n, at, m in rows_of(lens, T):
        S = torch.zeros(hkv, D, D, dtype=F64) if initial is None else initial[n].to(F64).clone()
        for t in range(at, at + m):
            S = l * S + k[t, :, :, None] * v[t, :, None, :]
            o[t] = scale * torch.einsum("hgr,hrc->hgc", q[t].view(hkv, g, D), S).reshape(hq, D)
        final[n] = S
    return o, final


def linear_backward(q, k, v, dout, log_decay, scale, lens, initial=None, dfinal=None):
    """dq [T, Hq, D], dk, dv [T, Hkv, D], dinitial [n, Hkv, D, D], fp64."""
    T, hq, D = q.shape
    hkv = k.shape[1]
    g = hq // hkv
    q, k, v, dout = (x.to(F64) for x in (q, k, v, dout))
    l = torch.exp(log_decay.to(F64))[:, None, None]
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dinitial = torch.zeros(len(lens), hkv, D, D, dtype=F64)
    for n, at, m in rows_of(lens, T):
        S = torch.zeros(hkv, D, D, dtype=F64) if initial is None else initial[n].to(F64).clone()
        for t in range(at, at + m):
            S = l * S + k[t, :, :, None] * v[t, :, None, :]
            dq[t] = scale * torch.einsum("hgc,hrc->hgr", dout[t].view(hkv, g, D), S).reshape(hq, D)
        G = torch.zeros(hkv, D, D, dtype=F64) if dfinal is None else dfinal[n].to(F64).clone()
        for t in range(at + m - 1, at - 1, -1):
            G = G + scale * torch.einsum("hgr,hgc->hrc", q[t].view(hkv, g, D), dout[t].view(hkv, g, D))
            dk[t] = torch.einsum("hrc,hc->hr", G, v[t])
            dv[t] = torch.einsum("hrc,hr->hc", G, k[t])
            G = l * G
        dinitial[n] = G
    return dq, dk, dv, dinitial
