"""fp64 CPU oracle for the paged key/value cache: append with rotation, attention.

TEST INFRASTRUCTURE ONLY, like the rest of this package.

Rotation of a row x at position p, with c, s = cos_sin[p, :r/2], cos_sin[p, r/2:]:
pair a = (x, y) -> (x c_a - y s_a, y c_a + x s_a); the pair is (x[a], x[a + r/2]),
or (x[2a], x[2a + 1]) when interleaved; dims at or past r stay.

An e4m3 page and head has one scale 2^e: the least integer e >= -100 with
amax <= 448 2^e over the finite new values; a page that already holds keys keeps
the larger of its scale and this one.

Attention of new token i (of m) of a sequence of length L, position L - m + i: the
softmax over the keys j < L, and j <= position when causal; no visible key: o = 0,
lse = -inf.
"""
from __future__ import annotations

import math

import torch

F64 = torch.float64
E4M3_MAX = 448.0


def rotate(x, pos, cos_sin, interleaved=False):
    """x [T, H, D], pos [T] -> fp64, one row at a time."""
    y = x.to(F64).clone()
    if cos_sin is None:
        return y
    r = cos_sin.shape[1]
    for t in range(x.shape[0]):
        for a in range(r // 2):
            i, j = (2 * a, 2 * a + 1) if interleaved else (a, a + r // 2)
            c, s = float(cos_sin[pos[t], a]), float(cos_sin[pos[t], r // 2 + a])
            u, w = y[t, :, i].clone(), y[t, :, j].clone()
            y[t, :, i] = u * c - w * s
            y[t, :, j] = w * c + u * s
    return y


def page_scale(amax: float) -> float:
    e = -100
    while amax > E4M3_MAX * 2.0 ** e:
        e += 1
    return 2.0 ** e


class Cache:
    """What a cache should hold: the unrounded value of every (sequence, position),
    and for e4m3 the scale of every (page, head)."""

    def __init__(self, heads, dim, page_size, e4m3):
        self.heads, self.dim, self.page_size, self.e4m3 = heads, dim, page_size, e4m3
        self.rows = {}     # (page, slot) -> [heads, dim]
        self.scale = {}    # (page, head) -> float

    def append(self, values, start, pages):
        """values fp64 [m, heads, dim] of positions start ..; pages: the sequence's page list."""
        ps, end = self.page_size, start + values.shape[0]
        lo = start
        while lo < end:
            hi = min(end, (lo // ps + 1) * ps)
            page = int(pages[lo // ps])
            part = values[lo - start:hi - start]
            if self.e4m3:
                for h in range(self.heads):
                    x = part[:, h]
                    x = x[torch.isfinite(x)].abs()
                    s = page_scale(x.max().item() if x.numel() else 0.0)
                    if lo % ps:
                        s = max(s, self.scale[page, h])
                    self.scale[page, h] = s
            for j in range(lo, hi):
                self.rows[page, j % ps] = part[j - lo]
            lo = hi


def attention(q, k, v, scale, causal=True):
    """One sequence: q [m, Hq, D], k, v [L, Hkv, D] -> o [m, Hq, D], lse [Hq, m], and
    for error bounds: wabs = softmax |v| and smax = max_j scale sum_d |q_d k_jd|."""
    q, k, v = (t.to(F64) for t in (q, k, v))
    m, hq, d = q.shape
    L, hkv = k.shape[0], k.shape[1]
    o, wabs = torch.zeros(m, hq, d, dtype=F64), torch.zeros(m, hq, d, dtype=F64)
    lse, smax = torch.full((hq, m), -math.inf, dtype=F64), torch.zeros(hq, m, dtype=F64)
    for h in range(hq):
        g = h // (hq // hkv)
        for i in range(m):
            n = min(L, L - m + i + 1) if causal else L
            if n <= 0:
                continue
            x = scale * (k[:n, g] @ q[i, h])
            top = x.max()
            e = torch.exp(x - top)
            lse[h, i] = top + torch.log(e.sum())
            p = e / e.sum()
            o[i, h] = p @ v[:n, g]
            wabs[i, h] = p @ v[:n, g].abs()
            smax[h, i] = (abs(scale) * (k[:n, g].abs() @ q[i, h].abs())).max()
    return o, lse, wabs, smax
