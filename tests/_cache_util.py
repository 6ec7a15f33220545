"""Steps over a paged cache for the tests: inputs, page lists, the oracle's answer
and error bounds."""
import torch

from oracle import cache as OC

F8 = torch.float8_e4m3fn


def table(positions, rot):
    freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    ang = torch.arange(positions, dtype=torch.float64)[:, None] * freq
    return torch.cat([ang.cos(), ang.sin()], 1).float()


class Step:
    """A cache of random values under random pages, and new tokens' queries.  What
    no sequence's length reaches is NaN: unused rows, unused pages, their scales.

    seqs: (length, new tokens) of each sequence."""

    def __init__(self, cache, D, hq, hkv, ps, seqs, seed=0, pad_tokens=3, extra_cols=2, amp=1.0):
        g = torch.Generator().manual_seed(seed)
        self.cache, self.D, self.hq, self.hkv, self.ps, self.seqs = cache, D, hq, hkv, ps, seqs
        need = [-(-l // ps) for l, _ in seqs]
        pages = sum(need) + 2
        perm = torch.randperm(pages, generator=g).tolist()
        self.cols = max(need) + extra_cols
        self.table = torch.full((len(seqs), self.cols), -7, dtype=torch.int32)   # unused: not a page
        at = 0
        for n, k in enumerate(need):
            self.table[n, :k] = torch.tensor(perm[at:at + k], dtype=torch.int32)
            at += k
        self.T = sum(m for _, m in seqs) + pad_tokens
        self.q = (amp * torch.randn(self.T, hq, D, generator=g)).to(torch.bfloat16)
        self.cu = torch.tensor([0] + [m for _, m in seqs]).cumsum(0).to(torch.int32)
        self.kv = torch.tensor([l for l, _ in seqs], dtype=torch.int32)
        self.max_new = max(1, max(m for _, m in seqs))
        self.pools, self.scales, self.true = [], [], []
        for _ in range(2):
            x = torch.randn(pages, hkv, ps, D, generator=g)
            if cache == "bf16":
                pool, scale = x.to(torch.bfloat16), None
                val = pool.double()
            else:
                scale = torch.exp2(torch.randint(-9, -4, (pages, hkv), generator=g).float())
                pool = (x / scale[..., None, None]).clamp(-448, 448).to(F8)
                val = pool.float().double() * scale.double()[..., None, None]
            live = torch.zeros(pages, ps, dtype=torch.bool)
            for n, (l, _) in enumerate(seqs):
                for c in range(need[n]):
                    live[self.table[n, c], :min(ps, l - c * ps)] = True
            dead = ~live[:, None, :, None].expand_as(pool)
            if cache == "bf16":
                pool[dead] = float("nan")
            else:
                pool.view(torch.uint8)[dead] = 0x7f
                scale[~live.any(1)] = float("nan")
            self.pools.append(pool)
            self.scales.append(scale)
            self.true.append(val)

    def to(self, dev):
        kw = dict(page_table=self.table.to(dev), seqlens_kv=self.kv.to(dev), cu_seqlens=self.cu.to(dev),
                  max_new=self.max_new)
        if self.cache != "bf16":
            kw.update(k_scale=self.scales[0].to(dev), v_scale=self.scales[1].to(dev))
        return (self.q.to(dev), self.pools[0].to(dev), self.pools[1].to(dev)), kw

    def keys(self, n, l=None):
        """True fp64 keys and values [L, Hkv, D] of sequence n."""
        l = self.seqs[n][0] if l is None else l
        c = -(-l // self.ps)
        out = []
        for t in self.true:
            x = t[self.table[n, :c].long()].permute(0, 2, 1, 3).reshape(-1, self.hkv, self.D)
            out.append(x[:l])
        return out

    def answer(self, causal=True, scale=None):
        """o [T, Hq, D], lse [Hq, T] and the bounds on their errors."""
        scale = self.D ** -0.5 if scale is None else scale
        o = torch.zeros(self.T, self.hq, self.D, dtype=torch.float64)
        wabs, vsum = torch.zeros_like(o), torch.zeros_like(o)
        lse = torch.full((self.hq, self.T), -float("inf"), dtype=torch.float64)
        smax = torch.zeros(self.hq, self.T, dtype=torch.float64)
        for n, (l, m) in enumerate(self.seqs):
            if m == 0:
                continue
            k, v = self.keys(n)
            r = slice(int(self.cu[n]), int(self.cu[n + 1]))
            o[r], lse[:, r], wabs[r], smax[:, r] = OC.attention(self.q[r], k, v, scale, causal)
            if self.cache != "bf16":
                sc = self.scales[1][self.table[n, :-(-l // self.ps)].long()].double()      # [pages, Hkv]
                codes = v.abs() / sc.repeat_interleave(self.ps, 0)[:l, :, None]
                vs = codes.sum(0) * (sc.max(0).values[:, None] if l else 0)
                vsum[r] = vs.repeat_interleave(self.hq // self.hkv, 0)
        rows = self.max_new * (self.hq // self.hkv)
        return dict(o=o, lse=lse, wabs=wabs, **bounds(o, lse, wabs, vsum, smax, self.D, self.cache, rows))


def bounds(o, lse, wabs, vsum, smax, D, cache, rows):
    """Error bounds of attn_cache_fwd.

    A logit is D exact products summed in fp32 (in any order within (D + 2) half steps
    of the sum of their magnitudes, which is at most smax), one fp32 product with the
    scale and one subtraction of the maximum, both on numbers of at most a few smax:
    its error is at most (D + 8) 2^-24 smax, in natural units; smax >= 1 covers the
    exponential's own 2^-22 and the fp32 sums and joins (a few dozen of them: 2^-19).
    The error of a probability relative to itself is twice that (numerator and sum).
    P is rounded: bf16 caches, to two bf16 (2^-16) for at most 16 query rows per KV head and
    to bf16 (2^-8) by the tcgen05 kernel for more rows; e4m3, by both to fp16: 2^-11, and
    2^-25 absolute below its normal range, over a sum of at least 1.  Each of these scales
    |v|, the last one |code| times the largest page scale (vsum).  Then one rounding to
    bf16, 2^-8."""
    es = (D + 8) * 2.0 ** -24 * smax.clamp(min=1) + 2.0 ** -19
    pr = 2.0 ** -11 if cache != "bf16" else 2.0 ** -16 if rows <= 16 else 2.0 ** -8
    err = (2 * es.t()[..., None] + pr) * wabs + (2.0 ** -25 * vsum if cache != "bf16" else 0)
    return dict(o_tol=err * (1 + 2.0 ** -8) + 2.0 ** -8 * o.abs() + 1e-37,
                lse_tol=es + 2.0 ** -22 * lse.abs().nan_to_num(posinf=0))


def check(ref, o, lse):
    o, lse = o.double().cpu(), lse.double().cpu()
    assert torch.equal(torch.isneginf(lse), torch.isneginf(ref["lse"]))
    seen = torch.isfinite(ref["lse"])
    assert torch.isfinite(o).all() and torch.isfinite(lse[seen]).all()
    over = ((o - ref["o"]).abs() / ref["o_tol"]).max().item() if o.numel() else 0.0
    assert over <= 1, f"o is {over:.2f} times its bound off"
    if seen.any():
        over = ((lse[seen] - ref["lse"][seen]).abs() / ref["lse_tol"][seen]).max().item()
        assert over <= 1, f"lse is {over:.2f} times its bound off"
    empty = ~seen.t()
    assert (o[empty] == 0).all()
