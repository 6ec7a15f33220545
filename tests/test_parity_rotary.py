"""GPU tests of the rotation by position: table, forward, backward, refusals only the
device sees, graphs."""
import math

import pytest
import torch

import softmax_attention_backward_gb300 as A
from oracle import cache as OC
from oracle import linear as OL

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0") if torch.cuda.is_available() else None
F64, BF = torch.float64, torch.bfloat16


def exact_table(n, f, magnitude=1.0, first=0):
    angle = torch.arange(first, first + n, dtype=F64)[:, None] * torch.tensor(f, dtype=F64)
    return torch.cat([angle.cos(), angle.sin()], 1) * magnitude


# An entry's phase is exact to fp32's resolution; the series' last steps round its value at most four
# times and the magnitude once, 2^-24 of at most 1 each: 6 2^-24 with the phase's own.
TABLE_TOL = 6 * 2.0 ** -24


@pytest.mark.parametrize("kw", [dict(), dict(scaling="linear", factor=4.0), dict(scaling="base", factor=3.5),
                                dict(scaling="parts", factor=16.0, original=2048),
                                dict(scaling="parts", factor=8.0, original=512, fast=4.0, slow=1.0, base=500000.0)])
@pytest.mark.parametrize("n,rot", [(1, 16), (700, 64), (301, 128), (33, 256), (1000, 48)])
def test_table(n, rot, kw):
    got = A.attn_rotary_table(n, rot, magnitude=1.25, device=DEV, **kw)
    want = exact_table(n, OL.frequencies(rot, **kw), 1.25)
    assert got.shape == (n, rot) and got.dtype == torch.float32
    assert (got.cpu().double() - want).abs().max() <= 1.25 * TABLE_TOL


def test_table_far_positions_and_small_bases():
    n = 1 << 20
    got = A.attn_rotary_table(n, 16, device=DEV)[-4096:].cpu().double()
    # the fp64 angle itself is off by 2^-53 of 2^20, far below the bound
    assert (got - exact_table(4096, OL.frequencies(16), first=n - 4096)).abs().max() <= TABLE_TOL
    got = A.attn_rotary_table(64, 16, base=0.01, device=DEV).cpu().double()   # frequencies above one turn
    assert (got - exact_table(64, OL.frequencies(16, base=0.01))).abs().max() <= TABLE_TOL + 64 * 100 * 2.0 ** -53 * 2


def test_table_small_angles_keep_their_precision():
    got = A.attn_rotary_table(64, 64, base=1e9, device=DEV).cpu().double()
    want = exact_table(64, OL.frequencies(64, base=1e9))
    s, w = got[1:, 32:], want[1:, 32:]
    assert ((s - w).abs() <= 8 * 2.0 ** -24 * w.abs()).all()


# (x c - y s) in fp32: three roundings, 2^-24 of |x c| + |y s| each, then one to bf16
def check_rotated(got, x, pos, cs, interleaved, offset, inverse=False):
    """got, x [T, H, D] on the CPU; pos [T], -1 for rows of zeros."""
    r = cs.shape[1]
    sign = torch.cat([torch.ones(r // 2), -torch.ones(r // 2)]) if inverse else torch.ones(r)
    live = pos >= 0
    part = x[..., offset:offset + r]
    want = x.to(F64).clone()
    want[..., offset:offset + r] = OC.rotate(part, pos.clamp(min=0), cs * sign, interleaved)
    want[~live] = 0
    size = OC.rotate(part.abs(), pos.clamp(min=0), torch.cat([cs[:, :r // 2].abs(), -cs[:, r // 2:].abs()], 1), interleaved)
    other = OC.rotate(part.abs(), pos.clamp(min=0), cs.abs(), interleaved)
    tol = torch.zeros_like(want)
    tol[..., offset:offset + r] = 3 * 2.0 ** -24 * torch.maximum(size.abs(), other.abs())
    tol = tol + 2.0 ** -8 * (want.abs() + tol) * (tol > 0)
    assert ((got.to(F64) - want).abs() <= tol).all()


SHAPES = [(64, 64, 0), (128, 128, 0), (128, 64, 64), (64, 32, 8), (576, 64, 512), (192, 48, 16), (1024, 256, 768), (16, 16, 0)]


@pytest.mark.parametrize("D,rot,offset", SHAPES)
@pytest.mark.parametrize("hq,hk", [(1, 0), (4, 1), (9, 3), (5, 5)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation(D, rot, offset, hq, hk, interleaved):
    g = torch.Generator().manual_seed(D + hq)
    cs = A.attn_rotary_table(300, rot, device=DEV)
    q = torch.randn(2, 37, hq, D, generator=g).to(BF)
    k = torch.randn(2, 37, hk, D, generator=g).to(BF) if hk else None
    pos = torch.arange(37).repeat(2)
    for call, inverse in ((A.attn_rotary_fwd, False), (A.attn_rotary_bwd, True)):
        out = call(q.to(DEV), None if k is None else k.to(DEV), cs, interleaved=interleaved, rot_offset=offset)
        assert (out[1] is None) == (k is None)
        for o, x in zip(out, (q, k)):
            if x is not None:
                assert o.shape == x.shape
                check_rotated(o.cpu().flatten(0, 1), x.flatten(0, 1), pos, cs.cpu(), interleaved, offset, inverse)


@pytest.mark.parametrize("lens,pad", [([1], 0), ([5, 0, 17, 1, 0], 3), ([40] * 33, 7), ([0, 0], 4)])
def test_packed_positions_and_padding(lens, pad):
    T = sum(lens) + pad
    g = torch.Generator().manual_seed(T)
    q, k = (torch.randn(T, h, 64, generator=g).to(BF) for h in (4, 2))
    q[T - pad:] = float("nan")
    cs = A.attn_rotary_table(64, 64, device=DEV)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    pos = torch.cat([torch.arange(m) for m in lens] + [torch.full((pad,), -1)])
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = A.attn_rotary_fwd(q.to(DEV), k.to(DEV), cs, cu_seqlens=cu.to(DEV), error_word=err)
    for o, x in zip(out, (q.nan_to_num(), k)):
        check_rotated(o.cpu(), x, pos, cs.cpu(), False, 0)
    assert err.item() == 0


def test_given_positions_and_flags():
    g = torch.Generator().manual_seed(2)
    q, k = (torch.randn(2, 4, h, 128, generator=g).to(BF) for h in (8, 2))
    cs = A.attn_rotary_table(100, 64, device=DEV)
    given = torch.tensor([[0, 99, -1, 7], [100, -2, 7, 1 << 30]], dtype=torch.int32)
    pos = torch.where((given >= 0) & (given < 100), given, -1).flatten()
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = A.attn_rotary_fwd(q.to(DEV), k.to(DEV), cs, positions=given.to(DEV), interleaved=True, error_word=err)
    for o, x in zip(out, (q, k)):
        check_rotated(o.cpu().flatten(0, 1), x.flatten(0, 1), pos, cs.cpu(), True, 0)
    assert err.item() == 1
    err.zero_()
    A.attn_rotary_fwd(q.to(DEV), k.to(DEV), cs, positions=given[:1].expand(2, 4).contiguous().to(DEV), error_word=err)
    assert err.item() == 0
    A.attn_rotary_fwd(q.to(DEV), k.to(DEV), cs[:3].contiguous(), error_word=err)    # a sequence past the table
    assert err.item() == 4
    assert not A.attn_rotary_fwd(q.to(DEV), k.to(DEV), cs[:3].contiguous())[0][:, 3].any()


@pytest.mark.parametrize("interleaved", [False, True])
def test_in_place_and_fused_projection(interleaved):
    g = torch.Generator().manual_seed(4)
    cs = A.attn_rotary_table(64, 64, device=DEV)
    fused = torch.randn(2, 30, 12 * 128, generator=g).to(BF).to(DEV)
    q, k = fused[..., :1024].unflatten(-1, (8, 128)), fused[..., 1024:1280].unflatten(-1, (2, 128))
    dense = [t.contiguous() for t in (q, k)]
    want = A.attn_rotary_fwd(*dense, cs, interleaved=interleaved, rot_offset=32)
    got = A.attn_rotary_fwd(q, k, cs, interleaved=interleaved, rot_offset=32)
    both = A.attn_rotary_fwd(*dense, cs, interleaved=interleaved, rot_offset=32, q_out=dense[0], k_out=dense[1])
    for a, b, c in zip(want, got, both):
        assert torch.equal(a, b) and torch.equal(a, c) and a.is_contiguous() and b.is_contiguous()
    # the transposed rotation undoes it up to the roundings: |c^2 + s^2 - 1| and two of 2^-8, and
    # each of a pair's values takes part of the other's error
    back = A.attn_rotary_bwd(*got, cs, interleaved=interleaved, rot_offset=32)
    for x, y in zip((q, k), back):
        assert ((x.double() - y.double()).abs() <= 2.0 ** -8 * (2 * x.abs().double().amax() + 1e-3)).all()
    with pytest.raises(A.AttnError):
        A.attn_rotary_fwd(q, k, cs, q_out=q[:, :, :].as_strided(q.shape, (30 * 1024, 1024, 128, 1)))


def test_the_same_rotation_as_the_cache_append():
    g = torch.Generator().manual_seed(5)
    T, D = 40, 128
    q, k, v = (torch.randn(T, h, D, generator=g).to(BF).to(DEV) for h in (8, 2, 2))
    cs = A.attn_rotary_table(64, D, device=DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    kc, vc, _, _ = A.attn_cache_empty(4, 2, 16, D, device=DEV)
    step = dict(page_table=torch.arange(4, **i32)[None], seqlens_kv=torch.tensor([T], **i32),
                cu_seqlens=torch.tensor([0, T], **i32), max_new=T)
    for interleaved in (False, True):
        want = A.attn_cache_append(q, k, v, kc, vc, cos_sin=cs, interleaved=interleaved, **step)
        got, kr = A.attn_rotary_fwd(q, k, cs, cu_seqlens=step["cu_seqlens"], interleaved=interleaved)
        assert torch.equal(got, want)
        assert torch.equal(kr, kc.transpose(1, 2).reshape(64, 2, D)[:T])


def test_no_tokens_and_many():
    cs = A.attn_rotary_table(16, 16, device=DEV)
    q = torch.empty(0, 4, 64, dtype=BF, device=DEV)
    assert A.attn_rotary_fwd(q, q, cs, positions=torch.empty(0, dtype=torch.int32, device=DEV))[0].shape == q.shape
    T = 1 << 16
    assert not A.attn_rotary_fwd(torch.zeros(T, 4, 16, dtype=BF, device=DEV), None, cs,
                                 positions=torch.zeros(T, dtype=torch.int32, device=DEV))[0].any()


@pytest.mark.slow
def test_offsets_past_32_bits():
    cs = A.attn_rotary_table(128, 64, device=DEV)
    T, H = (1 << 18) + 3, 128                      # 2^32 elements and a few rows
    q = torch.empty(T, H, 128, dtype=BF, device=DEV)
    q[:] = torch.randn(1, 1, 128, generator=torch.Generator().manual_seed(1)).to(BF).to(DEV)
    pos = torch.arange(T, dtype=torch.int32, device=DEV) % 128
    A.attn_rotary_fwd(q, None, cs, positions=pos, q_out=q)
    few = torch.randn(1, 1, 128, generator=torch.Generator().manual_seed(1)).to(BF).to(DEV).expand(128, 1, 128)
    want = A.attn_rotary_fwd(few.contiguous(), None, cs, positions=pos[:128].contiguous())[0][:, 0]
    for rows in (slice(0, 128), slice(T - 200, T)):
        assert (q[rows] == want[pos[rows].long()][:, None]).all()


def test_captured_and_replayed():
    g = torch.Generator().manual_seed(6)
    q, k = (torch.randn(50, h, 64, generator=g).to(BF).to(DEV) for h in (4, 2))
    cs = torch.empty(64, 64, device=DEV)
    cu = torch.tensor([0, 20, 50], dtype=torch.int32, device=DEV)
    qo, ko = torch.empty_like(q), torch.empty_like(k)

    def step():
        A.attn_rotary_table(64, 64, out=cs)
        A.attn_rotary_fwd(q, k, cs, cu_seqlens=cu, q_out=qo, k_out=ko)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for lens in ([20, 30], [0, 45], [50, 0]):
        cu.copy_(torch.tensor([0] + lens).cumsum(0).to(torch.int32))
        graph.replay()
        want = A.attn_rotary_fwd(q, k, cs, cu_seqlens=cu)
        assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])


def test_binding_refusals():
    cs = A.attn_rotary_table(64, 64, device=DEV)
    q = torch.zeros(2, 8, 4, 64, dtype=BF, device=DEV)
    p = torch.zeros(2, 8, dtype=torch.int32, device=DEV)
    bad = [dict(q=q.float()), dict(q=q[..., ::2]), dict(k=q[:1]), dict(k=q[0]), dict(cos_sin=cs.double()), dict(cos_sin=cs[0]),
           dict(positions=p[:1]), dict(positions=p.long()), dict(positions=p, cu_seqlens=p[0]), dict(q_out=q[:1]),
           dict(cu_seqlens=p[0]), dict(q=q[0]), dict(q=q.expand(2, 8, 4, 64)[:, :1].expand(2, 8, 4, 64)),
           dict(q=q.transpose(1, 2)), dict(cos_sin=cs.cpu()), dict(k_out=q, k=None)]
    for kw in bad:
        a = dict(q=q, k=q, cos_sin=cs)
        a.update(kw)
        with pytest.raises((TypeError, ValueError)):
            A.attn_rotary_fwd(a.pop("q"), a.pop("k"), a.pop("cos_sin"), **a)
    with pytest.raises(A.AttnError):
        A.attn_rotary_fwd(q, None, cs, rot_offset=8)
    assert math.isfinite(A.attn_rotary_fwd(q, None, cs)[0].sum().item())


def test_magnitude_between_two_fp32_numbers():
    # Held in fp32 it would be 1: off by 2^-24 everywhere.  Two roundings (sine or cosine, product) and the
    # series' own error stay below 1.8 times one rounding in the mean square.
    m = 1.0 + 2.0 ** -24
    f = [10000.0 ** (-2.0 * a / 64) for a in range(32)]
    want = exact_table(3000, f, m)
    got = A.attn_rotary_table(3000, 64, magnitude=m, device=DEV).cpu().double()
    once = (want.float().double() - want).square().mean().sqrt()
    assert (got - want).square().mean().sqrt() <= 1.8 * once
