"""GPU tests of the paged cache at its edges: extreme magnitudes, offsets past 32 bits,
odd groups of heads, captured graphs of every kernel, calls at once, flags."""
import pytest
import torch

import softmax_attention_backward_gb300 as A
from _cache_util import F8, Step, check, table
from test_parity_cache import run_fwd

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0") if torch.cuda.is_available() else None
CACHES = ["bf16", "e4m3"]
I32 = dict(dtype=torch.int32, device=DEV)

# steps that the kernel for few rows serves, the tcgen05 kernel, and (e4m3) both together
FEW = dict(D=128, hq=8, hkv=2, ps=32, seqs=[(500, 1), (1300, 2), (31, 1)])
MANY = dict(D=128, hq=8, hkv=2, ps=32, seqs=[(500, 90), (1300, 120), (31, 7)])
MIXED = dict(D=64, hq=8, hkv=2, ps=16, seqs=[(40 + 37 * n, 1) for n in range(29)] + [(700, 90)])


# ---------------------------------------------------------------------------
# magnitudes
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("D,m", [(64, 1), (128, 1), (64, 60), (128, 60)])
@pytest.mark.parametrize("down", [30, 80])
def test_small_values(D, m, down):
    # values of 2^-down, and lengths whose last chunk has pages missing at its end
    s = Step("e4m3", D, 4, 2, 16, [(130, m), (80, m), (77, m)], seed=61)
    s.scales[1] *= 2.0 ** -down
    s.true[1] = s.pools[1].float().double() * s.scales[1].double()[..., None, None]
    check(s.answer(), *run_fwd(s))


@pytest.mark.parametrize("D,m", [(64, 2), (128, 2), (64, 60), (128, 60)])
@pytest.mark.parametrize("scale", [None, 0.0, -0.1])
def test_zero_queries_over_zero_pages(D, m, scale):
    # an appended page of zeros has the scale 2^-100
    s = Step("e4m3", D, 4, 2, 16, [(130, m), (64, m)], seed=62)
    s.q[::2] = 0
    s.q[1::4] *= 2.0 ** -60
    for i in range(2):
        for page in s.table[:, 1::2].flatten().tolist():
            if page >= 0:
                real = ~s.pools[i][page].float().isnan()
                s.pools[i].view(torch.uint8)[page][real] = 0
                s.scales[i][page] = 2.0 ** -100
        s.true[i] = s.pools[i].float().double() * s.scales[i].double()[..., None, None]
    check(s.answer(scale=scale), *run_fwd(s, scale=scale))


@pytest.mark.parametrize("m", [1, 60])
def test_zero_values_count_in_the_sum(m):
    # all pages but the first hold zero values, under a scale of 2^-100, and keys at the same logit
    s = Step("e4m3", 64, 2, 1, 16, [(160, m)], seed=63)
    s.q[:] = 0
    s.q[:, :, 0] = 1.0
    for page in s.table[0, :10].tolist():
        for i in range(2):
            s.pools[i].view(torch.uint8)[page] = 0
            s.scales[i][page] = 2.0 ** -100
    s.scales[1][s.table[0, 0]] = 2.0 ** -8
    s.pools[1][s.table[0, 0]] = torch.randn(1, 16, 64, generator=torch.Generator().manual_seed(1)).to(F8)
    for i in range(2):
        s.true[i] = s.pools[i].float().double() * s.scales[i].double()[..., None, None]
    check(s.answer(scale=1.0), *run_fwd(s, scale=1.0))


@pytest.mark.parametrize("D", [64, 128])
def test_query_magnitudes_and_page_scales_many_rows(D):
    s = Step("e4m3", D, 4, 2, 16, [(300, 64), (150, 33)], seed=64)
    s.q[:20] *= 2.0 ** -60
    s.q[20:40] *= 2.0 ** 4
    s.q[40] = 0
    for i in range(2):
        g = torch.Generator().manual_seed(i)
        e = torch.randint(*((-12, -4) if i == 0 else (-40, 20)), s.scales[i].shape, generator=g)
        live = ~s.scales[i].isnan()
        s.scales[i][live] = torch.exp2(e[live].float())
        s.true[i] = s.pools[i].float().double() * s.scales[i].double()[..., None, None]
    check(s.answer(scale=0.01), *run_fwd(s, scale=0.01))


# ---------------------------------------------------------------------------
# shapes
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("D,hq,hkv", [(64, 10, 2), (128, 14, 2), (64, 24, 1), (128, 128, 1), (128, 130, 1)])
def test_groups_with_many_rows(cache, D, hq, hkv):
    s = Step(cache, D, hq, hkv, 32, [(150, 30), (70, 2), (9, 9)], seed=65)
    check(s.answer(), *run_fwd(s))


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("causal", [True, False])
def test_sequences_of_many_row_blocks(cache, causal):
    # blocks of 16 tokens: 44, 19, 1 and 18 of them
    s = Step(cache, 64, 16, 1, 32, [(900, 700), (350, 300), (40, 3), (600, 280)], seed=73)
    check(s.answer(causal), *run_fwd(s, causal))


@pytest.mark.parametrize("cache", CACHES)
def test_more_sequences_than_threads_with_prompts_among_them(cache):
    seqs = [(400, 300) if n % 100 == 50 else (20 + n % 7, n % 3) for n in range(520)]
    s = Step(cache, 64, 16, 1, 16, seqs, seed=74)
    check(s.answer(), *run_fwd(s))


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("case", [FEW, MANY, MIXED], ids=["few", "many", "mixed"])
def test_pool_past_32_bit_offsets(cache, case):
    # the same step with its pages at the end of a pool of more than 2^32 bytes: the same bits
    s = Step(cache, seed=66, **case)
    (q, k, v), kw = s.to(DEV)
    o, lse = A.attn_cache_fwd(q, k, v, **kw)
    check(s.answer(), o, lse)
    per = k[0].numel()
    pages = (2 ** 32 + 2 ** 28) // per
    assert pages * s.hkv * s.ps < 2 ** 31
    base = pages - k.shape[0]
    big = [torch.empty((pages,) + tuple(k.shape[1:]), dtype=k.dtype, device=DEV) for _ in range(2)]
    for t, small in zip(big, (k, v)):
        t[base:] = small
    kw["page_table"] = torch.where(kw["page_table"] >= 0, kw["page_table"] + base, -7)
    for name in ("k_scale", "v_scale"):
        if name in kw:
            t = torch.full((pages, s.hkv), float("nan"), device=DEV)
            t[base:] = kw[name]
            kw[name] = t
    o2, lse2 = A.attn_cache_fwd(q, *big, **kw)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("new", [(3, 1), (70, 20)])
def test_append_past_32_bit_offsets(cache, new):
    D, H, ps, cols = 128, 2, 32, 4
    g = torch.Generator().manual_seed(67)
    T = sum(new)
    x = [torch.randn(T, h, D, generator=g).to(torch.bfloat16).to(DEV) for h in (4, H, H)]
    dtype = torch.bfloat16 if cache == "bf16" else F8
    per = H * ps * D
    pages = (2 ** 32 + 2 ** 28) // per
    lens = [m + 10 for m in new]
    got = []
    for count in (2 * cols, pages):
        pools = [torch.empty((count, H, ps, D), dtype=dtype, device=DEV) for _ in range(2)]
        sc = [torch.full((count, H), 2.0 ** -100, device=DEV) for _ in range(2)] if cache != "bf16" else [None, None]
        for t in pools:
            t[-2 * cols:].view(torch.uint8).zero_()
        tab = (torch.arange(2 * cols, **I32) + (count - 2 * cols)).view(2, cols)
        q = A.attn_cache_append(*x, *pools, page_table=tab, k_scale=sc[0], v_scale=sc[1],
                                seqlens_kv=torch.tensor(lens, **I32), max_new=max(new),
                                cu_seqlens=torch.tensor([0, new[0], T], **I32), cos_sin=table(200, D).to(DEV))
        got.append([q] + [t[-2 * cols:].view(torch.uint8).clone() for t in pools] +
                   [t[-2 * cols:].clone() for t in sc if t is not None])
    for a, b in zip(*got):
        assert torch.equal(a, b)


# ---------------------------------------------------------------------------
# graphs, calls at once
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("case", [FEW, MANY, MIXED], ids=["few", "many", "mixed"])
def test_step_captured_and_replayed(cache, case):
    # an append with the attention that reads it, captured once and replayed over a text that grows
    D, hq, hkv, ps = case["D"], case["hq"], case["hkv"], case["ps"]
    new = [m for _, m in case["seqs"]]
    n, T = len(new), sum(new) + 2
    steps, g = 3, torch.Generator().manual_seed(68)
    cols = -(-steps * max(new) // ps) + 1
    dtype = torch.bfloat16 if cache == "bf16" else F8

    def fresh():
        kc, vc, ks, vs = A.attn_cache_empty(n * cols, hkv, ps, D, dtype=dtype, device=DEV)
        for t in (kc, vc):
            t.view(torch.uint8).fill_(0x7f)
        return (kc, vc), dict(k_scale=ks, v_scale=vs,
                              page_table=torch.arange(n * cols, **I32).flip(0).contiguous().view(n, cols),
                              seqlens_kv=torch.zeros(n, **I32), cu_seqlens=torch.zeros(n + 1, **I32), max_new=max(new))

    cs = table(steps * max(new), D).to(DEV)
    x = [torch.empty(T, h, D, dtype=torch.bfloat16, device=DEV) for h in (hq, hkv, hkv)]
    rot, o = torch.empty_like(x[0]), torch.empty_like(x[0])
    lse = torch.empty(hq, T, device=DEV)
    err = torch.zeros(1, **I32)

    def step(pools, kw, ws):
        A.attn_cache_append(*x, *pools, cos_sin=cs, q_out=rot, error_word=err, **kw)
        A.attn_cache_fwd(rot, *pools, out=o, lse=lse, workspace=ws, error_word=err, **kw)

    def feed(kw, i):
        # the last step has fewer new tokens: the rest of the rows is padding
        m = new if i + 1 < steps else [max(1, y // 2) for y in new]
        kw["seqlens_kv"].add_(torch.tensor(m, **I32))
        kw["cu_seqlens"].copy_(torch.tensor([0] + m).cumsum(0))
        for t, y in zip(x, data[i]):
            t.copy_(y)

    data = [[torch.randn(T, h, D, generator=g).to(torch.bfloat16) for h in (hq, hkv, hkv)] for _ in range(steps)]
    pools, kw = fresh()
    ws = torch.empty(A.attn_cache_fwd_workspace_size(x[0], *pools, **kw), dtype=torch.uint8, device=DEV)
    want = []
    for i in range(steps):
        feed(kw, i)
        step(pools, kw, ws)
        want.append((rot.clone(), o.clone(), lse.clone()))
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    pools, kw = fresh()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(pools, kw, ws)
    for i in range(steps):
        feed(kw, i)
        for t in (rot, o, lse):
            t.fill_(float("nan"))
        ws.fill_(0xff)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want[i], (rot, o, lse)):
            assert torch.equal(a, b), i
        assert torch.isfinite(o).all()
    assert int(err.item()) == 0


@pytest.mark.parametrize("cache", CACHES)
def test_two_graphs_that_share_a_workspace_one_after_another(cache):
    steps = [Step(cache, seed=76, **FEW), Step(cache, seed=77, **MANY)]
    calls = [x.to(DEV) for x in steps]
    size = max(A.attn_cache_fwd_workspace_size(*x, **kw) for x, kw in calls)
    ws = torch.empty(size, dtype=torch.uint8, device=DEV)
    outs = [A.attn_cache_fwd(*x, workspace=ws, **kw) for x, kw in calls]
    graphs = []
    for (x, kw), (o, lse) in zip(calls, outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            A.attn_cache_fwd(*x, out=o, lse=lse, workspace=ws, **kw)
    for o, lse in outs:
        o.fill_(float("nan")), lse.fill_(float("nan"))
    for i in (0, 1, 1, 0, 0, 1):
        graphs[i].replay()
    torch.cuda.synchronize()
    for s, (o, lse) in zip(steps, outs):
        check(s.answer(), o, lse)


@pytest.mark.parametrize("cache", CACHES)
def test_many_rows_two_calls_at_once(cache):
    a, b = Step(cache, seed=69, **MANY), Step(cache, seed=70, **MIXED)
    (xa, ka), (xb, kb) = a.to(DEV), b.to(DEV)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [(A.attn_cache_fwd(*xa, stream=s1, **ka), A.attn_cache_fwd(*xb, stream=s2, **kb)) for _ in range(5)]
    torch.cuda.synchronize()
    ra, rb = a.answer(), b.answer()
    for x, y in got:
        check(ra, *x)
        check(rb, *y)


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("case", [MANY, MIXED], ids=["many", "mixed"])
def test_query_stride_and_workspace_contents_many_rows(cache, case):
    s = Step(cache, seed=71, **case)
    (q, k, v), kw = s.to(DEV)
    wide = torch.full((s.T, s.hq + 5, s.D), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide[:, 2:2 + s.hq] = q
    ws = torch.full((A.attn_cache_fwd_workspace_size(q, k, v, **kw),), 0xff, dtype=torch.uint8, device=DEV)
    o, lse = A.attn_cache_fwd(wide[:, 2:2 + s.hq], k, v, workspace=ws, **kw)
    check(s.answer(), o, lse)
    o2, lse2 = A.attn_cache_fwd(q, k, v, **kw)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("case", [FEW, MANY], ids=["few", "many"])
def test_sequences_that_share_pages(cache, case):
    # both read the first sequence's pages, the second as a prefix
    s = Step(cache, seed=72, **case)
    full = s.seqs[0][0] // s.ps
    s.table[1, :full] = s.table[0, :full]
    check(s.answer(), *run_fwd(s))


# ---------------------------------------------------------------------------
# flags
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("max_new", [4, 40])
def test_append_without_queries_flags_positions(cache, max_new):
    # the last sequence's new tokens all lie past the rotation table
    D = 64
    x = torch.randn(8, 1, D).to(torch.bfloat16).to(DEV)
    dtype = torch.bfloat16 if cache == "bf16" else F8
    kc, vc, ks, vs = A.attn_cache_empty(6, 1, 16, D, dtype=dtype, device=DEV)
    err = torch.zeros(1, **I32)
    A.attn_cache_append(None, x, x, kc, vc, k_scale=ks, v_scale=vs, cos_sin=table(16, D).to(DEV), error_word=err,
                        page_table=torch.tensor([[0, 1], [2, 3]], **I32), max_new=max_new,
                        seqlens_kv=torch.tensor([4, 24], **I32), cu_seqlens=torch.tensor([0, 4, 8], **I32))
    torch.cuda.synchronize()
    assert int(err.item()) == 4
