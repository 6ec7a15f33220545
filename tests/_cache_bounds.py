"""Error bounds of the paged cache's attention that count, for each row, only what the
row sees, and steps whose values' page scales are chosen."""
import torch

from _cache_util import F8, Step

F64 = torch.float64


class ScaledStep(Step):
    """An e4m3 step with its values' (or keys') page scales set by the test."""

    def set_scales(self, i, exponents):
        """exponents: {(sequence, column): e}, the scale 2^e for every KV head; i: 0 keys, 1 values."""
        for (n, c), e in exponents.items():
            self.scales[i][self.table[n, c]] = 2.0 ** e
        self.refresh(i)

    def set_rows(self, i, n, rows, x):
        """Keys or values `rows` (positions) of sequence n become the codes nearest to x [rows, Hkv, D]."""
        for j, r in enumerate(rows):
            page, slot = int(self.table[n, r // self.ps]), r % self.ps
            code = (x[j].float() / self.scales[i][page][:, None]).clamp(-448, 448).to(F8)
            self.pools[i].view(torch.uint8)[page, :, slot] = code.view(torch.uint8)
        self.refresh(i)

    def refresh(self, i):
        self.true[i] = self.pools[i].float().double() * self.scales[i].double()[..., None, None]


def answer(s, p_bits, causal=True, scale=None):
    """o [T, Hq, D], lse [Hq, T] in fp64, and their bounds.

    A logit's error es is as in _cache_util.bounds; a probability's relative to itself is
    twice that.  P is then rounded to 2^-p_bits of itself.  An e4m3 cache's P (p_bits 11)
    is multiplied by its page's scale and by a power 2^(8 - R) first, R (log2) at most the
    largest p_j scale_j (over the largest p) of the keys that the row sees, and is off by
    half of fp16's least subnormal, 2^-25, at the small end: 2^-33 of that largest product
    for each unit of code that the row sees.  The powers are fp32 exponentials (2^-22
    each, a few dozen of them where R rises) of differences of at most 2^7 (2^-17 each):
    2^-14 together.  Then one rounding to bf16, 2^-8."""
    scale = s.D ** -0.5 if scale is None else scale
    g, e4m3 = s.hq // s.hkv, s.cache != "bf16"
    o = torch.zeros(s.T, s.hq, s.D, dtype=F64)
    o_tol = torch.full_like(o, 1e-37)
    lse = torch.full((s.hq, s.T), -float("inf"), dtype=F64)
    lse_tol = torch.zeros_like(lse)
    for n, (L, m) in enumerate(s.seqs):
        if not m or not L:
            continue
        k, v = s.keys(n)
        t0 = int(s.cu[n])
        pos = L - m + torch.arange(m)
        seen = torch.arange(L)[None] <= (pos[:, None] if causal else torch.full((m, 1), L))
        if e4m3:
            vs = s.scales[1][s.table[n, :-(-L // s.ps)].long()].double().repeat_interleave(s.ps, 0)[:L]
        for h in range(s.hq):
            kh, vh = k[:, h // g], v[:, h // g]
            q = s.q[t0:t0 + m, h].double()
            x = (scale * q @ kh.T).masked_fill(~seen, -float("inf"))
            any_ = seen.any(1)
            p = torch.softmax(x, -1).masked_fill(~any_[:, None], 0)
            smax = (abs(scale) * q.abs() @ kh.abs().T).masked_fill(~seen, 0).amax(-1)
            es = (s.D + 8) * 2.0 ** -24 * smax.clamp(min=1) + 2.0 ** -19
            want, wabs = p @ vh, p @ vh.abs()
            err = (2 * es[:, None] + 2.0 ** -p_bits + (2.0 ** -14 if e4m3 else 0)) * wabs
            if e4m3:
                sc = vs[:, h // g]
                codes = seen.double() @ (vh.abs() / sc[:, None])
                err += 2.0 ** -33 * (p * sc).amax(-1, keepdim=True) * codes
            o[t0:t0 + m, h] = want
            o_tol[t0:t0 + m, h] += err * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs()
            lse[h, t0:t0 + m] = x.logsumexp(-1)
            lse_tol[h, t0:t0 + m] = es + 2.0 ** -22 * lse[h, t0:t0 + m].abs().nan_to_num(posinf=0)
    return dict(o=o, lse=lse, o_tol=o_tol, lse_tol=lse_tol)
