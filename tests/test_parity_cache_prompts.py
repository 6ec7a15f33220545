"""GPU tests of large appends, in which a thread goes over several heads (rows) or several
units of a page (e4m3), against the definition in 64 bits."""
import pytest
import torch

import softmax_attention_backward_gb300 as A
from _cache_util import F8, table

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0") if torch.cuda.is_available() else None
F64 = torch.float64


def unit_loop(D, ps, new, hkv):
    """Units that a thread of the e4m3 path goes over, by the library's rule."""
    wide = 256 // max(32, ps * (D // 16) // 4)
    n = len(new)
    items = min(((max(new) - 1 + ps - 1) // ps + 1) * n, sum(new) // ps + 2 * n)
    loop = 8
    while loop > 1 and items * 2 * hkv // (wide * loop) < 152:
        loop //= 2
    return loop, wide


def head_block(D, T, heads):
    blocks, hb = -(-T // (256 // (D // 16))), 8
    while hb > 1 and blocks * heads // hb < 304:
        hb //= 2
    return hb


def rotate(x, pos, cs, interleaved):
    y = x.to(F64).clone()
    if cs is None:
        return y
    r = cs.shape[1]
    c, s = (cs[pos, a:b].to(F64)[:, None] for a, b in ((0, r // 2), (r // 2, r)))
    i, j = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
    u, w = y[..., i].clone(), y[..., j].clone()
    y[..., i], y[..., j] = u * c - w * s, w * c + u * s
    return y


def page_exponents(amax):
    """The least integer e >= -100 with amax <= 448 2^e."""
    m, e = torch.frexp(amax)
    return torch.where(amax > 0, torch.where(m <= 0.875, e - 9, e - 8), torch.full_like(e, -100)).clamp(min=-100)


def append_and_check(cache, D, hq, hkv, ps, calls, rot, interleaved, seed, specials=False, fused=False):
    g = torch.Generator().manual_seed(seed)
    n = len(calls[0])
    most = [sum(c[i] for c in calls) for i in range(n)]
    cols = max(-(-m // ps) for m in most) + 1
    pages = n * cols + 1
    tab = torch.randperm(pages, generator=g)[:n * cols].view(n, cols).to(torch.int32)
    kc, vc, ks, vs = A.attn_cache_empty(pages, hkv, ps, D, dtype=torch.bfloat16 if cache == "bf16" else F8, device=DEV)
    for t in (kc, vc):
        t.view(torch.uint8).fill_(0x5a)
    if ks is not None:
        ks.fill_(float("nan")), vs.fill_(float("nan"))
    cs = table(max(most) + 3, rot) if rot else None
    want = [torch.zeros(pages, ps, hkv, D, dtype=F64) for _ in range(2)]
    live = torch.zeros(pages, ps, dtype=torch.bool)
    scale = [torch.zeros(pages, hkv, dtype=F64) for _ in range(2)]
    lens = torch.zeros(n, dtype=torch.int64)
    for call, new in enumerate(calls):
        T = sum(new) + 2
        x = [(torch.randn(T, h, D, generator=g) * 3.0 ** (call % 3)).to(torch.bfloat16) for h in (hq, hkv, hkv)]
        if specials:     # finite maxima beside infinities and NaN, a page of zeros
            for t in x[1:]:
                t[::97, :, 3] = float("inf")
                t[5::131, :, 7] = float("nan")
                t[3::211, 0] = -float("inf")
                t[20 * ps:22 * ps, -1] = 0
        m = torch.tensor(new)
        cu = torch.cat([torch.zeros(1, dtype=torch.int64), m.cumsum(0)])
        lens += m
        seq = torch.repeat_interleave(torch.arange(n), m)
        pos = lens[seq] - m[seq] + torch.arange(len(seq)) - cu[seq]
        page, slot = tab[seq, pos // ps].long(), pos % ps
        dev = [t.to(DEV) for t in x]
        if fused:
            wide = torch.full((T, hq + 2 * hkv + 1, D), float("nan"), dtype=torch.bfloat16, device=DEV)
            at = 0
            for i, h in enumerate((hq, hkv, hkv)):
                wide[:, at:at + h] = dev[i]
                dev[i] = wide[:, at:at + h]
                at += h
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        q = A.attn_cache_append(*dev, kc, vc, page_table=tab.to(DEV), k_scale=ks, v_scale=vs, max_new=max(new),
                                seqlens_kv=lens.to(torch.int32).to(DEV), cu_seqlens=cu.to(torch.int32).to(DEV),
                                cos_sin=None if cs is None else cs.to(DEV), interleaved=interleaved, error_word=err)
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        rows = slice(0, len(seq))
        # three fp32 roundings on magnitudes of at most sqrt(2) max |x|, then bf16's half step
        qw = rotate(x[0][rows], pos, cs, interleaved)
        tol = 2.0 ** -8 * qw.abs() + 2.0 ** -21 * x[0][rows].double().abs().amax(-1, keepdim=True)
        assert ((q[rows].double().cpu() - qw).abs() <= tol).all()
        assert (q[len(seq):] == 0).all()
        live[page, slot] = True
        for i, y in enumerate((rotate(x[1][rows], pos, cs, interleaved), x[2][rows].to(F64))):
            want[i][page, slot] = y
            if cache != "bf16":
                fin = torch.where(torch.isfinite(y), y.abs(), torch.zeros_like(y)).float().amax(-1)
                amax = torch.zeros(pages, hkv).scatter_reduce_(0, page[:, None].expand(-1, hkv), fin, "amax")
                sc = torch.exp2(page_exponents(amax).double())
                first = torch.full((pages,), ps).scatter_reduce_(0, page, slot, "amin")
                touched = first < ps
                sc = torch.where(first[:, None] > 0, torch.maximum(sc, scale[i]), sc)
                scale[i] = torch.where(touched[:, None], sc, scale[i])
                # an infinity is stored as the largest code, and is a value like others from then on
                top = (torch.sign(y) * 448 * scale[i][page][..., None])
                want[i][page, slot] = torch.where(torch.isinf(y), top, y)
    for i, (pool, dev_scale) in enumerate(((kc, ks), (vc, vs))):
        assert (pool.view(torch.uint8).cpu()[~live[:, None, :].expand(pages, hkv, ps)] == 0x5a).all()
        got = pool.float().double().cpu().transpose(1, 2)[live]
        w = want[i][live]
        big = torch.where(torch.isfinite(w), w.abs(), torch.zeros_like(w)).amax(-1, keepdim=True)
        if cache == "bf16":
            assert ((got - w).abs() <= 2.0 ** -8 * w.abs() + 2.0 ** -21 * big).all()
            continue
        used = live.any(1)
        assert torch.equal(dev_scale.double().cpu()[used], scale[i][used])
        assert dev_scale.cpu()[~used].isnan().all()
        sc = scale[i][:, None, :, None].expand(pages, ps, hkv, 1)[live]
        got = got * sc
        nan = w.isnan()
        assert torch.equal(got.isnan(), nan)
        # a code's half step, relative 2^-4 or half the least subnormal 2^-9 (twice: rounded again when the scale grew)
        tol = 2.0 ** -4 * w.abs() + 2 * 2.0 ** -10 * sc + 2.0 ** -21 * big
        assert ((got - w).abs() <= tol)[~nan].all()


def lengths(n, top, seed):
    g = torch.Generator().manual_seed(seed)
    return tuple(int(x) for x in torch.randint(1, top, (n,), generator=g))


@pytest.mark.parametrize("D,hkv,ps,n,top,loop", [
    (128, 5, 32, 40, 300, 2),     # 10 units in groups of four: a ragged last turn
    (128, 5, 32, 200, 120, 8),
    (64, 9, 16, 150, 130, 4),     # 18 units in groups of eight
    (128, 3, 128, 60, 700, 8),    # a whole block to a unit
    (64, 7, 64, 90, 400, 8),
    (64, 3, 128, 100, 500, 4),
])
@pytest.mark.parametrize("rot", ["all", "half"])
def test_e4m3_threads_over_several_units(D, hkv, ps, n, top, loop, rot):
    # pages begun by an earlier call (few tokens, then a smaller magnitude's), then prompts of every length
    first, new = lengths(n, ps + 9, 1), lengths(n, top, 2)
    got, wide = unit_loop(D, ps, new, hkv)
    assert got >= loop and 2 * hkv > wide * 1
    half = rot == "half"
    append_and_check("e4m3", D, 2 * hkv, hkv, ps, [first, new], D // 2 if half else D, half, seed=D + ps)


def test_e4m3_several_units_with_special_values():
    n = 60
    new = lengths(n, 300, 3)
    assert unit_loop(128, 32, new, 5)[0] > 1
    append_and_check("e4m3", 128, 5, 5, 32, [lengths(n, 20, 4), new], 0, False, seed=5, specials=True)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("D,hq,hkv,n,top,hb", [(128, 7, 7, 12, 700, 4), (64, 10, 5, 40, 900, 4), (128, 12, 3, 60, 600, 8),
                                               (64, 21, 7, 60, 500, 8)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rows_over_several_heads(cache, D, hq, hkv, n, top, hb, interleaved):
    # heads of q, k and v that do not divide by the group; a quarter of the dims rotated; fused projections
    new = lengths(n, top, 6)
    heads = hq + (2 * hkv if cache == "bf16" else 0)
    got = head_block(D, sum(new) + 2, heads)
    assert got >= (hb if cache == "bf16" else 2) and (hq % got or hkv % got)
    append_and_check(cache, D, hq, hkv, 32, [lengths(n, 12, 7), new], D // 4, interleaved, seed=D, fused=True)
