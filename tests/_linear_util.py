"""Inputs of the linear-attention tests, the call, and error bounds that count, for each
element, what its row sees."""
import torch

import softmax_attention_backward_gb300 as A
from oracle import linear as OL

F64, BF = torch.float64, torch.bfloat16
DEV = torch.device("cuda:0") if torch.cuda.is_available() else None
CHUNK = 128          # tokens of a chunk, as documented in include/linear.h
HALF = 2.0 ** -8     # half a step of bf16, relative


class Rows:
    """A problem: lens of the sequences, `pad` rows behind them (NaN), the decays."""

    def __init__(self, lens, hq, hkv, D, *, pad=0, seed=0, decay=None, states=False, scale=None):
        g = torch.Generator().manual_seed(seed + 1000 * len(lens) + sum(lens))
        self.lens, self.hq, self.hkv, self.D, self.pad = lens, hq, hkv, D, pad
        self.T = sum(lens) + pad
        self.scale = D ** -0.5 if scale is None else scale

        def rows(h):
            x = torch.randn(self.T, h, D, generator=g).to(BF)
            x[self.T - pad:] = float("nan")
            return x

        self.q, self.k, self.v, self.do = rows(hq), rows(hkv), rows(hkv), rows(hq)
        self.g = torch.as_tensor(decay, dtype=torch.float32).expand(hkv).contiguous() if decay is not None else \
            -torch.exp2(-10 * torch.rand(hkv, generator=g))
        n = len(lens)
        self.init = 2 * torch.randn(n, hkv, D, D, generator=g) if states else None
        self.dfin = torch.randn(n, hkv, D, D, generator=g) if states else None
        self.cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32)

    @property
    def live(self):
        return slice(0, self.T - self.pad)

    def shaped(self, t):
        """Dense where all sequences are as long and no row is padding, packed otherwise."""
        return t.unflatten(0, (len(self.lens), -1)) if self.dense else t

    @property
    def dense(self):
        return not self.pad and len(set(self.lens)) == 1 and self.lens[0] > 0

    def call(self, packed=None, states=True, **kw):
        """(o, final, dq, dk, dv, dinitial) of the library, flat rows, on the CPU."""
        if packed is not None and packed:
            shaped, cu = (lambda t: t), self.cu
        else:
            shaped, cu = self.shaped, None if self.dense else self.cu
        x = [shaped(t).to(DEV) for t in (self.q, self.k, self.v, self.do)]
        g = self.g.to(DEV)
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        kw = dict(cu_seqlens=None if cu is None else cu.to(DEV), scale=self.scale, error_word=err,
                  initial_state=None if self.init is None else self.init.to(DEV), **kw)
        o, fin = A.linear_attn_fwd(*x[:3], g, want_final_state=states, **kw)
        d = A.linear_attn_bwd(*x, g, dfinal_state=None if self.dfin is None else self.dfin.to(DEV),
                              want_dinitial_state=states, **kw)
        torch.cuda.synchronize()
        assert err.item() == 0
        flat = [t.view(self.T, -1, self.D).cpu() for t in (o, *d[:3])]
        return flat[0], None if fin is None else fin.cpu(), flat[1], flat[2], flat[3], None if d[3] is None else d[3].cpu()

    def answer(self):
        """The same in fp64, and for each output a bound."""
        live = self.live
        q, k, v, do = (t[live].to(F64) for t in (self.q, self.k, self.v, self.do))
        o, fin = OL.linear_forward(q, k, v, self.g, self.scale, self.lens, self.init)
        d = OL.linear_backward(q, k, v, do, self.g, self.scale, self.lens, self.init, self.dfin)
        # All products' magnitudes: the same formulas of absolute values.
        ini, dfi = (None if t is None else t.abs() for t in (self.init, self.dfin))
        oa, fa = OL.linear_forward(q.abs(), k.abs(), v.abs(), self.g, abs(self.scale), self.lens, ini)
        da = OL.linear_backward(q.abs(), k.abs(), v.abs(), do.abs(), self.g, abs(self.scale), self.lens, ini, dfi)
        return (o, fin, *d), (oa, fa, *da)


def check(s, got, *, states=True):
    """Every element within the bound of its own products, relative to their magnitudes' sum.
    bf16 outputs: three roundings to bf16 meet a product at most (a decayed key of the state, the
    state that a row meets or a score, the output), 2^-8 each, and the rest (fp32 sums and
    exponentials) stays below 2^-11.  States: keys in three bf16 terms (2^-24); a decay l^m is
    the exponential of m log l, whose rounding 2^-24 |m log l| weighs l^m |m log l| <= 1 / e
    against the newest products', with 2^-22 of the exponential's own, for each chunk that it
    crosses, 2^-18 in all up to 20 chunks; sums of 128 terms and one for each chunk, 2^-17."""
    want, size = s.answer()
    bf = (0, 2, 3, 4)
    for i, name in enumerate(("o", "final", "dq", "dk", "dv", "dinitial")):
        x = got[i]
        if x is None:
            assert not states and i in (1, 5)
            continue
        x = x.to(F64)
        if i in bf:
            pad = x[s.T - s.pad:]
            assert not pad.any(), f"{name}: padding rows"
            x = x[s.live]
        assert torch.isfinite(x).all(), f"{name}: non-finite values"
        tol = size[i] * (3.1 * HALF if i in bf else 2.0 ** -16) + 1e-37
        err = (x - want[i]).abs()
        assert (err <= tol).all(), f"{name}: {(err / tol).max():.2f} of the bound"
        # roundings of independent terms: a rounding to bf16 is off by at most 2^-8 / sqrt 3 of the
        # value in the mean square; four of them over random terms stay below 2 2^-8 / sqrt 3.
        if x.numel() >= 4096 and i in bf:
            rms = err.square().mean().sqrt() / want[i].square().mean().sqrt().clamp(min=1e-30)
            assert rms <= 2 * HALF / 3 ** 0.5, f"{name}: rms error {rms:.2e}"
        if x.numel() >= 4096 and i not in bf:
            rms = err.square().mean().sqrt() / want[i].square().mean().sqrt().clamp(min=1e-30)
            assert rms <= 2.0 ** -17, f"{name}: rms error {rms:.2e}"
