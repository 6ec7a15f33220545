"""GPU tests of linear attention with a decay per head: forward and backward over lengths,
heads, decays and states, the recurrent step, and runs of them together."""
import math

import pytest
import torch

import softmax_attention_backward_gb300 as A
from _linear_util import BF, DEV, F64, HALF, Rows, check
from oracle import linear as OL

pytestmark = pytest.mark.gpu
I32 = dict(dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens", [[1], [2], [31], [32], [33], [127], [128], [129], [255], [257], [640]])
@pytest.mark.parametrize("states", [False, True])
def test_lengths(D, lens, states):
    s = Rows(lens, 2, 2, D, states=states)
    check(s, s.call(states=states), states=states)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (6, 2), (12, 1), (40, 2)])
@pytest.mark.parametrize("lens,pad", [([1], 0), ([2, 2, 2], 0), ([7] * 5, 0), ([8] * 3, 0), ([9] * 3, 0), ([3, 0, 1, 2], 2),
                                      ([0, 8], 0), ([0], 3), ([5, 1], 3)])
@pytest.mark.parametrize("decay", [None, -math.inf])
def test_few_tokens(D, hq, hkv, lens, pad, decay):
    # Up to 8 tokens (packed: in all) nothing but an output is rounded to bf16: half a step of it, and
    # fp32 sums and products, of 8 tokens' 40 / 2 heads and 128 dims in chains of 160 and 32 at most, 2^-24 each.
    for packed in (False, True):
        for states in (False, True):
            s = Rows(lens, hq, hkv, D, pad=pad, decay=decay, states=states, seed=31)
            got = s.call(packed=packed, states=states)
            check(s, got, states=states)
            if s.T > 8 if packed or not s.dense else max(lens) > 8:
                continue
            for x, w, m in zip(got, *s.answer()):
                if x is not None:
                    x = x.to(F64)[s.live] if x.dtype == BF else x.to(F64)
                    tol = (HALF * 1.01 * w.abs() if x.dim() == 3 else 0) + 2.0 ** -16 * m + 1e-37
                    assert ((x - w).abs() <= tol).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 1), (6, 2), (3, 3), (10, 5), (16, 1)])
@pytest.mark.parametrize("states", [False, True])
def test_heads(D, hq, hkv, states):
    s = Rows([150, 150], hq, hkv, D, states=states, seed=1)
    check(s, s.call(states=states), states=states)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,pad", [([5, 0, 130, 1], 0), ([0], 5), ([0, 0, 300], 60), ([129, 127, 128], 3), ([3] * 40, 9),
                                      ([700, 2, 400], 130)])
@pytest.mark.parametrize("states", [False, True])
def test_packed(D, lens, pad, states):
    s = Rows(lens, 4, 2, D, pad=pad, states=states, seed=2)
    check(s, s.call(packed=True, states=states), states=states)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("decay", [0.0, -1e-4, -0.05, -1.0, -30.0, -200.0, -1e9, -math.inf])
def test_decays(D, decay):
    s = Rows([300, 200], 2, 1, D, pad=7, decay=decay, states=True, seed=3)
    check(s, s.call())


@pytest.mark.parametrize("D", [64, 128])
def test_one_long_sequence_is_cut_into_segments(D):
    s = Rows([2500], 4, 2, D, states=True, seed=4)
    check(s, s.call())


def test_many_long_sequences():
    s = Rows([1100, 900, 1300, 40, 777], 8, 4, 128, pad=50, states=True, seed=5)
    check(s, s.call())


@pytest.mark.parametrize("hq,hkv", [(2, 2), (3, 1)])
def test_more_packed_sequences_than_a_warp_holds(hq, hkv):
    # 70 sequences of 0 to 900 tokens: the order of the walks by length, and places of the segments
    lens = [(i * i * 37 + 11 * i) % 901 if i % 7 else 0 for i in range(70)]
    s = Rows(lens, hq, hkv, 64, pad=21, states=True, seed=6)
    check(s, s.call())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("states", [False, True])
def test_many_short_walks(D, states):
    # more walks than SMs, of one to three chunks: two on an SM at a time where head_dim is 64
    s = Rows([300, 7, 130, 257, 64, 128, 0, 1, 31, 200], 40, 20, D, pad=3, states=states, seed=7)
    got = s.call(states=states)
    check(s, got, states=states)
    again = s.call(states=states)
    for x, y in zip(got, again):
        assert x is None and y is None or torch.equal(x, y)


def test_scales():
    for scale in (0.0, -0.25, 3.0):
        s = Rows([200], 2, 1, 64, states=True, scale=scale, seed=6)
        check(s, s.call())


@pytest.mark.parametrize("D", [64, 128])
def test_magnitudes(D):
    s = Rows([200, 131], 2, 2, D, states=True, seed=7)
    for t, e in ((s.q, 40), (s.k, -50), (s.v, 30), (s.do, -45), (s.init, -20), (s.dfin, -5)):
        t *= 2.0 ** e
    check(s, s.call())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("packed", [False, True])
def test_bitwise_reproducible_and_every_element_written(D, packed):
    s = Rows([1000, 1000], 4, 2, D, states=True, seed=8)
    first = s.call(packed=packed)
    x = [(t if packed else s.shaped(t)).to(DEV) for t in (s.q, s.k, s.v, s.do)]
    g, kw = s.g.to(DEV), dict(cu_seqlens=s.cu.to(DEV) if packed else None, scale=s.scale, initial_state=s.init.to(DEV))
    for junk in (0xFF, 0x7F):
        nan = [torch.full_like(t, float("nan")) for t in (x[0], x[0], x[1], x[2])]
        fin, dini = (torch.full(s.init.shape, float("nan"), device=DEV) for _ in range(2))
        wf, wb = (torch.full((f(*x[:3], g, cu_seqlens=kw["cu_seqlens"]),), junk, dtype=torch.uint8, device=DEV)
                  for f in (A.linear_attn_fwd_workspace_size, A.linear_attn_bwd_workspace_size))
        o, f = A.linear_attn_fwd(*x[:3], g, out=nan[0], final_state=fin, workspace=wf, **kw)
        d = A.linear_attn_bwd(*x, g, dfinal_state=s.dfin.to(DEV), dq=nan[1], dk=nan[2], dv=nan[3], dinitial_state=dini,
                              workspace=wb, **kw)
        assert o is nan[0] and f is fin and d[0] is nan[1] and d[3] is dini
        for a, b in zip((o, f, *d), first):
            assert torch.equal(a.cpu().view(b.shape), b)


@pytest.mark.parametrize("D", [64, 128])
def test_gradients_against_differences(D):
    # of L = <o, dout> + <final, dfinal>, along random directions, in the library's own forward: both
    # passes' roundings enter, so the comparison is against fp64 differences of the oracle's forward
    s = Rows([140], 2, 1, D, states=True, seed=9)
    _, _, dq, dk, dv, dinit = (None if t is None else t.to(F64) for t in s.call())
    g = torch.Generator().manual_seed(1)

    def loss(q, k, v, init):
        o, fin = OL.linear_forward(q, k, v, s.g, s.scale, s.lens, init)
        return (o * s.do.to(F64)).sum() + (fin * s.dfin.to(F64)).sum()

    x = [s.q.to(F64), s.k.to(F64), s.v.to(F64), s.init.to(F64)]
    size = s.answer()[1]
    for i, (grad, bound) in enumerate(zip((dq, dk, dv, dinit), (size[2], size[3], size[4], size[5]))):
        u = torch.randn(x[i].shape, generator=g, dtype=F64)
        h = 1e-4    # the loss is quadratic at most in one input along a line: central differences are exact
        a, b = list(x), list(x)
        a[i], b[i] = x[i] + h * u, x[i] - h * u
        slope = (loss(*a) - loss(*b)) / (2 * h)
        # independent errors of at most 3.1 2^-8 of each element's bound, along u
        tol = 3.1 * HALF * (u * bound).square().sum().sqrt() * 4
        assert (slope - (grad * u).sum()).abs() <= tol


def test_rows_and_sequences_keep_to_themselves():
    # NaN in one sequence and in a head: no other one sees it, nor rows of earlier chunks
    s = Rows([200, 333, 129], 4, 2, 64, pad=20, states=True, seed=10)
    clean = s.call()
    for t in (s.q, s.k, s.v, s.do):
        t[200 + 150, 0 if t.shape[1] == 2 else slice(0, 2)] = float("nan")
    got = s.call()
    for i, (a, b) in enumerate(zip(got, clean)):
        if i in (1, 5):
            assert torch.equal(a[[0, 2]], b[[0, 2]]) and torch.equal(a[:, 1], b[:, 1])
        else:
            half = a.shape[1] // 2
            rows = torch.ones(s.T, dtype=torch.bool)
            rows[200:533] = False
            assert torch.equal(a[rows], b[rows]) and torch.equal(a[:, half:], b[:, half:])
    assert torch.equal(got[0][200:328], clean[0][200:328])          # the forward's chunk before
    assert got[0][350, 0].isnan().any()


def test_decay_out_of_range_is_flagged():
    s = Rows([50], 2, 2, 64, decay=torch.tensor([0.0, -0.5]))
    want = s.call(states=False)
    for bad in (0.25, math.nan, math.inf):
        err = torch.zeros(1, **I32)
        g = torch.tensor([bad, -0.5], device=DEV)
        x = [s.shaped(t).to(DEV) for t in (s.q, s.k, s.v, s.do)]
        o, _ = A.linear_attn_fwd(*x[:3], g, error_word=err)
        assert err.item() == 0x10 and torch.equal(o.cpu().view(want[0].shape), want[0])
        err.zero_()
        A.linear_attn_bwd(*x, g, error_word=err)
        assert err.item() == 0x10


def test_bad_cu_seqlens_is_flagged():
    s = Rows([60, 60], 2, 2, 64, pad=8, seed=11)
    x = [t.nan_to_num().to(DEV) for t in (s.q, s.k, s.v, s.do)]
    for cu in ([0, 60, 200], [0, 100, 60], [-5, 60, 120], [0, 1 << 30, 120], [5, 60, 120]):
        err = torch.zeros(1, **I32)
        kw = dict(cu_seqlens=torch.tensor(cu, **I32), error_word=err)
        A.linear_attn_fwd(*x[:3], s.g.to(DEV), **kw)
        torch.cuda.synchronize()
        assert err.item() == 4
        err.zero_()
        A.linear_attn_bwd(*x, s.g.to(DEV), **kw)
        torch.cuda.synchronize()
        assert err.item() == 4


def test_no_tokens():
    init = torch.randn(2, 3, 64, 64, device=DEV)
    q = torch.empty(2, 0, 3, 64, dtype=BF, device=DEV)
    g = torch.zeros(3, device=DEV)
    o, fin = A.linear_attn_fwd(q, q, q, g, initial_state=init, want_final_state=True)
    assert o.shape == q.shape and torch.equal(fin, init)
    assert not A.linear_attn_fwd(q, q, q, g, want_final_state=True)[1].any()
    d = A.linear_attn_bwd(q, q, q, q, g, dfinal_state=init, want_dinitial_state=True)
    assert torch.equal(d[3], init)
    q = torch.empty(0, 9, 3, 64, dtype=BF, device=DEV)                      # no sequence
    o, fin = A.linear_attn_fwd(q, q, q, g, want_final_state=True)
    assert o.shape == q.shape and fin.shape == (0, 3, 64, 64)
    assert A.linear_attn_step(q[:, 0], q[:, 0], q[:, 0], g, init).shape == (0, 3, 64)
    assert A.attn_rotary_fwd(q, q, A.attn_rotary_table(9, 64, device=DEV))[0].shape == q.shape


def test_fused_projection_and_another_stream():
    s = Rows([190, 190], 4, 2, 128, states=True, seed=12)
    fused = torch.cat([t.flatten(1) for t in (s.q, s.k, s.v)], 1).to(DEV)
    for lead in ((380,), (2, 190)):
        want = s.call(packed=len(lead) == 1)
        q, k, v = (t.unflatten(-1, (-1, 128)) for t in fused.view(*lead, -1).split([512, 256, 256], -1))
        assert not q.is_contiguous()
        side = torch.cuda.Stream(DEV)
        side.wait_stream(torch.cuda.current_stream())
        kw = dict(cu_seqlens=s.cu.to(DEV) if len(lead) == 1 else None, initial_state=s.init.to(DEV), stream=side)
        do = torch.cat([s.do.view(380, 4, 128), s.do.view(380, 4, 128)], 1).to(DEV).view(*lead, 8, 128)[..., :4, :]
        side.wait_stream(torch.cuda.current_stream())
        o, fin = A.linear_attn_fwd(q, k, v, s.g.to(DEV), want_final_state=True, **kw)
        d = A.linear_attn_bwd(q, k, v, do, s.g.to(DEV), dfinal_state=s.dfin.to(DEV), want_dinitial_state=True, **kw)
        torch.cuda.synchronize()
        for a, b in zip((o, fin, *d), want):
            assert torch.equal(a.cpu().view(b.shape), b)


def test_captured_and_replayed_with_other_lengths():
    s = Rows([300, 180, 40], 4, 2, 64, pad=60, states=True, seed=13)
    x = [t.nan_to_num().to(DEV) for t in (s.q, s.k, s.v, s.do)]
    g, cu, init, dfin = (t.to(DEV) for t in (s.g, s.cu, s.init, s.dfin))
    side = torch.cuda.Stream(DEV)

    def step():
        kw = dict(cu_seqlens=cu, initial_state=init)
        return (*A.linear_attn_fwd(*x[:3], g, want_final_state=True, **kw),
                *A.linear_attn_bwd(*x, g, dfinal_state=dfin, want_dinitial_state=True, **kw))

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for lens in ([300, 180, 40], [0, 580, 0], [1, 2, 3], [193, 193, 194]):
        cu.copy_(torch.tensor([0] + lens).cumsum(0).to(torch.int32))
        for t in out:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, step()):
            assert torch.equal(a, b)
    del side


@pytest.mark.parametrize("D,hq,hkv", [(64, 4, 2), (64, 24, 24), (128, 4, 1)])
def test_calls_in_a_row_of_one_workspace(D, hq, hkv):
    # Long sequences, so that each call's walks start while its pass over the states runs: their inputs
    # come from the kernel before, their outputs go to the one behind, and the next call's pass
    # writes the same workspace.  Eager and replayed.
    s = Rows([3000, 1500], hq, hkv, D, states=True, seed=14)
    x = [t.to(DEV) for t in (s.q, s.k, s.v, s.do)]
    cu, g, dfin = s.cu.to(DEV), s.g.to(DEV), s.dfin.to(DEV)
    cs = A.attn_rotary_table(3000, D, device=DEV)
    ws = torch.empty(max(f(*x[:3], g, cu_seqlens=cu) for f in
                         (A.linear_attn_fwd_workspace_size, A.linear_attn_bwd_workspace_size)), dtype=torch.uint8, device=DEV)
    assert ws.numel() > 0
    kw = dict(cu_seqlens=cu, workspace=ws)

    def run(initial):
        q, k = A.attn_rotary_fwd(x[0], x[1], cs, cu_seqlens=cu)
        o, state = A.linear_attn_fwd(q, k, x[2], g, initial_state=initial, want_final_state=True, **kw)
        o2, state2 = A.linear_attn_fwd(q, k, o[:, :hkv].contiguous(), g, initial_state=state, want_final_state=True, **kw)
        dq, dk, dv, dini = A.linear_attn_bwd(q, k, x[2], o2, g, initial_state=initial, dfinal_state=dfin,
                                             want_dinitial_state=True, **kw)
        return o, state, o2, state2, *A.attn_rotary_bwd(dq, dk, cs, cu_seqlens=cu), dv, dini

    initial = s.init.to(DEV)
    want = []
    for t in run(initial):
        torch.cuda.synchronize()
        want.append(t.clone())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(initial)
    for i in range(6):
        for t in out:
            t.fill_(float("nan"))
        ws.fill_(0xFF)
        graph.replay()
        ws.fill_(0xFF)       # (behind the replay: nothing of it may still want the workspace)
        for a, b, c in zip(out, want, run(initial)):
            assert torch.equal(a, b) and torch.equal(c, b)


def test_two_calls_at_once():
    a, b = Rows([900], 4, 2, 128, states=True, seed=14), Rows([700, 650], 4, 4, 128, states=True, seed=15)
    wa, wb = a.call(packed=True), b.call(packed=True)
    streams = [torch.cuda.Stream(DEV) for _ in range(2)]
    for _ in range(3):
        got = []
        for s, st in zip((a, b), streams):
            with torch.cuda.stream(st):
                x = [t.to(DEV) for t in (s.q, s.k, s.v, s.do)]
                kw = dict(cu_seqlens=s.cu.to(DEV), initial_state=s.init.to(DEV))
                got.append((*A.linear_attn_fwd(*x[:3], s.g.to(DEV), want_final_state=True, **kw),
                            *A.linear_attn_bwd(*x, s.g.to(DEV), dfinal_state=s.dfin.to(DEV), want_dinitial_state=True, **kw)))
        torch.cuda.synchronize()
        for g, w in zip(got, (wa, wb)):
            for p, r in zip(g, w):
                assert torch.equal(p.cpu().view(r.shape), r)


# ---------------------------------------------------------------------------
# the step
# ---------------------------------------------------------------------------
def step_inputs(n, slots, hq, hkv, D, seed=0):
    g = torch.Generator().manual_seed(seed + n)
    q, k, v = (torch.randn(n, h, D, generator=g).to(BF) for h in (hq, hkv, hkv))
    return q, k, v, -torch.exp2(-10 * torch.rand(hkv, generator=g)), 2 * torch.randn(slots, hkv, D, D, generator=g)


def check_step(q, k, v, g, state, slots, got, got_state, scale):
    """fp32 throughout: two roundings of 2^-24 and one of the decay (2^-22) in a state, D + 1 more
    in a sum, then one to bf16."""
    want = state.to(F64)
    n, hq, D = q.shape
    hkv = k.shape[1]
    l = torch.exp(g.to(F64))[:, None, None]
    o, size = torch.zeros(n, hq, D, dtype=F64), torch.zeros(n, hq, D, dtype=F64)
    touched = set()
    mag = state.to(F64).abs()
    for i, at in enumerate(slots):
        if at < 0 or at >= state.shape[0] or at in touched:
            continue
        touched.add(at)
        kv = k[i].to(F64)[:, :, None] * v[i].to(F64)[:, None, :]
        want[at] = l * want[at] + kv
        mag[at] = l * mag[at] + kv.abs()
        for x, s, y in ((o, want, q), (size, mag, q.abs())):
            x[i] = torch.einsum("hgr,hrc->hgc", y[i].to(F64).view(hkv, -1, D), s[at]).reshape(hq, D)
    assert ((got_state.to(F64) - want).abs() <= mag * 2.0 ** -21).all()
    same = [i for i in range(state.shape[0]) if i not in touched]
    assert torch.equal(got_state[same], state[same])
    tol = abs(scale) * size * (D + 16) * 2.0 ** -24
    assert ((got.to(F64) - scale * o).abs() <= tol + HALF * (scale * o).abs() * (1 + 2.0 ** -8)).all()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 8), (6, 2), (5, 1), (16, 2), (32, 1)])
@pytest.mark.parametrize("n", [1, 3, 40])
def test_step(D, hq, hkv, n):
    q, k, v, g, state = step_inputs(n, n + 4, hq, hkv, D)
    slots = torch.randperm(n + 4, generator=torch.Generator().manual_seed(n))[:n].to(torch.int32)
    st, err = state.to(DEV), torch.zeros(1, **I32)
    o = A.linear_attn_step(q.to(DEV), k.to(DEV), v.to(DEV), g.to(DEV), st, slots=slots.to(DEV), error_word=err)
    assert err.item() == 0
    check_step(q, k, v, g, state, slots.tolist(), o.cpu(), st.cpu(), D ** -0.5)


def test_step_padding_bad_and_repeated_slots():
    q, k, v, g, state = step_inputs(9, 6, 4, 2, 64, seed=1)
    slots = [3, -1, 6, 3, 0, -2, 0, 5, 3]
    st, err = state.to(DEV), torch.zeros(1, **I32)
    call = lambda sl, e: A.linear_attn_step(q.to(DEV), k.to(DEV), v.to(DEV), g.to(DEV), st, scale=0.3,
                                            slots=torch.tensor(sl, **I32), error_word=e)
    o = call(slots, err)
    assert err.item() == 1
    check_step(q, k, v, g, state, slots, o.cpu(), st.cpu(), 0.3)
    st.copy_(state)
    err.zero_()
    slots = [3, -1, -1, 5, -1, 0, -1, 1, -1]                      # padding alone is no error
    o = call(slots, err)
    assert err.item() == 0
    check_step(q, k, v, g, state, slots, o.cpu(), st.cpu(), 0.3)


def test_step_many_sequences_and_repeats_far_apart():
    n = 700
    q, k, v, g, state = step_inputs(n, n, 2, 1, 64, seed=2)
    slots = list(range(n))
    slots[699], slots[650], slots[300] = 2, 2, 299
    st, err = state.to(DEV), torch.zeros(1, **I32)
    o = A.linear_attn_step(q.to(DEV), k.to(DEV), v.to(DEV), g.to(DEV), st, slots=torch.tensor(slots, **I32), error_word=err)
    assert err.item() == 1
    check_step(q, k, v, g, state, slots, o.cpu(), st.cpu(), 0.125)


@pytest.mark.parametrize("decay", [0.0, -math.inf, -200.0])
def test_step_decays_and_no_slots(decay):
    q, k, v, g, state = step_inputs(5, 7, 4, 2, 128, seed=3)
    g[:] = decay
    st = state.to(DEV)
    o = A.linear_attn_step(q.to(DEV), k.to(DEV), v.to(DEV), g.to(DEV), st)
    check_step(q, k, v, g, state, list(range(5)), o.cpu(), st.cpu(), 128 ** -0.5)


def test_step_fused_projection_graph_and_flags():
    q, k, v, g, state = step_inputs(6, 8, 8, 2, 128, seed=4)
    fused = torch.cat([t.flatten(1) for t in (q, k, v)], 1).to(DEV)
    qs, ks, vs = (t.unflatten(-1, (-1, 128)) for t in fused.split([1024, 256, 256], 1))
    slots = torch.tensor([1, 0, 7, 5, 4, -1], **I32)
    st, gd = state.to(DEV), g.to(DEV)
    out = torch.empty(6, 8, 128, dtype=BF, device=DEV)
    A.linear_attn_step(qs, ks, vs, gd, st, slots=slots, out=out)
    check_step(q, k, v, g, state, slots.tolist(), out.cpu(), st.cpu(), 128 ** -0.5)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        A.linear_attn_step(qs, ks, vs, gd, st, slots=slots, out=out)
    for sl in ([1, 0, 7, 5, 4, -1], [3, 2, -1, 0, 1, 6]):
        st.copy_(state)
        slots.copy_(torch.tensor(sl))
        graph.replay()
        check_step(q, k, v, g, state, sl, out.cpu(), st.cpu(), 128 ** -0.5)
    err = torch.zeros(1, **I32)
    A.linear_attn_step(qs, ks, vs, torch.full_like(gd, 0.5), st, slots=slots, error_word=err)
    assert err.item() == 0x10


def test_binding_refusals():
    q, k = (torch.zeros(2, 8, h, 64, dtype=BF, device=DEV) for h in (4, 2))
    g, cu, st = torch.zeros(2, device=DEV), torch.tensor([0, 8], **I32), torch.zeros(2, 2, 64, 64, device=DEV)
    for kw in (dict(q=q.float()), dict(q=q[0]), dict(k=k[:1]), dict(v=k[:, :4]), dict(v=q), dict(log_decay=g.double()),
               dict(log_decay=g[:1]), dict(cu_seqlens=cu), dict(initial_state=st[:1]), dict(initial_state=st.half()),
               dict(final_state=st.transpose(2, 3)), dict(out=q[:1]), dict(workspace=g), dict(error_word=g), dict(q=q.transpose(1, 2)),
               dict(k=k[..., :32]), dict(log_decay=g.cpu()), dict(v=k[:, :1].expand(2, 8, 2, 64))):
        a = dict(q=q, k=k, v=k, log_decay=g)
        a.update(kw)
        with pytest.raises((TypeError, ValueError)):
            A.linear_attn_fwd(a.pop("q"), a.pop("k"), a.pop("v"), a.pop("log_decay"), **a)
    for kw in (dict(dout=k), dict(dfinal_state=st[:1]), dict(dq=k), dict(dk=q), dict(dinitial_state=st.double())):
        a = dict(dout=q)
        a.update(kw)
        with pytest.raises((TypeError, ValueError)):
            A.linear_attn_bwd(q, k, k, a.pop("dout"), g, **a)
    with pytest.raises(A.AttnError):
        A.linear_attn_fwd(q, k, k, g, initial_state=st, final_state=st)
    q, k = q[:, 0], k[:, 0]
    for kw in (dict(state=st[..., :32]), dict(state=st.double()), dict(state=st[0]), dict(slots=cu.long()), dict(slots=cu[:1]),
               dict(out=k), dict(log_decay=g[:1]), dict(q=q.float()), dict(q=q[:1]), dict(v=k[:1])):
        a = dict(q=q, k=k, v=k, log_decay=g, state=st)
        a.update(kw)
        with pytest.raises((TypeError, ValueError)):
            A.linear_attn_step(a.pop("q"), a.pop("k"), a.pop("v"), a.pop("log_decay"), a.pop("state"), **a)
    with pytest.raises(A.AttnError):
        A.linear_attn_step(q, k, k, g, st[:1])                      # more sequences than states


# ---------------------------------------------------------------------------
# runs of them together
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("D,rot,interleaved", [(64, 32, True), (128, 128, False)])
def test_training_step_of_a_rotated_layer(D, rot, interleaved):
    s = Rows([210, 75], 4, 2, D, seed=20)
    cs = A.attn_rotary_table(256, rot, device=DEV)
    cu, g = s.cu.to(DEV), s.g.to(DEV)
    kw = dict(cu_seqlens=cu, interleaved=interleaved)
    q, k = A.attn_rotary_fwd(s.q.to(DEV), s.k.to(DEV), cs, **kw)
    o, _ = A.linear_attn_fwd(q, k, s.v.to(DEV), g, cu_seqlens=cu)
    dq, dk, dv, _ = A.linear_attn_bwd(q, k, s.v.to(DEV), s.do.to(DEV), g, cu_seqlens=cu)
    dq, dk = A.attn_rotary_bwd(dq, dk, cs, **kw)
    # the same in fp64 from the unrotated rows: rotation, layer, gradients through both
    from oracle import cache as OC
    pos = torch.cat([torch.arange(m) for m in s.lens])
    c64 = cs.cpu().double()
    rq, rk = (OC.rotate(t, pos, c64, interleaved) for t in (s.q, s.k))
    ro, _ = OL.linear_forward(rq, rk, s.v, s.g, s.scale, s.lens)
    rd = OL.linear_backward(rq, rk, s.v, s.do, s.g, s.scale, s.lens)
    inv = torch.cat([c64[:, :rot // 2], -c64[:, rot // 2:]], 1)
    want = (ro, OC.rotate(rd[0], pos, inv, interleaved), OC.rotate(rd[1], pos, inv, interleaved), rd[2])
    for name, a, b in zip(("o", "dq", "dk", "dv"), (o, dq, dk, dv), want):
        # q and k rounded after the rotation, scores, states and keys, the outputs, the gradients after
        # the rotation back: seven roundings of 2^-8 / sqrt 3 at most in the mean square
        rms = (a.cpu().double() - b).square().mean().sqrt() / b.square().mean().sqrt()
        assert rms <= 7 ** 0.5 * HALF / 3 ** 0.5, f"{name}: {rms:.2e}"


@pytest.mark.parametrize("D", [64, 128])
def test_prompt_in_chunks_then_tokens(D):
    n, T, hq, hkv = 2, 330, 4, 2
    s = Rows([T] * n, hq, hkv, D, seed=21)
    q, k, v = (s.shaped(t).to(DEV) for t in (s.q, s.k, s.v))
    g = s.g.to(DEV)
    want, fin = OL.linear_forward(s.q, s.k, s.v, s.g, s.scale, s.lens)
    size, fsize = OL.linear_forward(s.q.abs(), s.k.abs(), s.v.abs(), s.g, s.scale, s.lens)
    pool = torch.full((5, hkv, D, D), float("nan"), device=DEV)
    slots = torch.tensor([4, 1], **I32)
    out, state, at = [], None, 0
    for m in (100, 1, 128, 71):
        rows = slice(at, at + m)
        o, state = A.linear_attn_fwd(q[:, rows].contiguous(), k[:, rows].contiguous(), v[:, rows].contiguous(), g,
                                     initial_state=state, want_final_state=True)
        out.append(o)
        at += m
    pool[slots.long()] = state
    for t in range(at, T):
        out.append(A.linear_attn_step(q[:, t], k[:, t], v[:, t], g, pool, slots=slots)[:, None])
    got = torch.cat(out, 1).flatten(0, 1).cpu().double()
    assert ((got - want).abs() <= 3.1 * HALF * size + 1e-37).all()
    assert ((pool[slots.long()].cpu().double() - fin).abs() <= 2.0 ** -16 * fsize).all()
    assert pool[[0, 2, 3]].isnan().all()


def test_batch_entries_agree_with_single_calls():
    s = Rows([260, 70, 1, 129], 4, 2, 64, states=True, seed=22)
    both = s.call()
    at = 0
    for n, m in enumerate(s.lens):
        one = Rows([m], 4, 2, 64, states=True)
        for t in ("q", "k", "v", "do"):
            setattr(one, t, getattr(s, t)[at:at + m].clone())
        one.g, one.init, one.dfin = s.g, s.init[n:n + 1], s.dfin[n:n + 1]
        check(one, one.call())
        want, size = one.answer()
        for i in (0, 2, 3, 4):
            assert ((both[i][at:at + m].double() - want[i]).abs() <= 3.1 * HALF * size[i] + 1e-37).all()
        at += m
