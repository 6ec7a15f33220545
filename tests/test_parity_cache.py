"""GPU parity of the paged cache (append, attention) against the fp64 oracle, at the
sizes and contents where it can go wrong, and its contracts."""
import pytest
import torch

import softmax_attention_backward_gb300 as A
from oracle import cache as OC
from _cache_util import F8, Step, bounds, check, table

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0") if torch.cuda.is_available() else None
CACHES = ["bf16", "e4m3"]


def _err():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def run_fwd(s, causal=True, scale=None, expect=0):
    (q, k, v), kw = s.to(DEV)
    err = _err()
    o = torch.full_like(q, float("nan"))
    lse = torch.full((s.hq, s.T), float("nan"), device=DEV)
    A.attn_cache_fwd(q, k, v, causal=causal, scale=scale, out=o, lse=lse, error_word=err, **kw)
    torch.cuda.synchronize()
    assert int(err.item()) == expect
    return o, lse


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ps", [16, 64, 128])
def test_decode_lengths(cache, D, ps):
    # one token each, lengths around the chunk of 16 keys, the page and the warp
    lens = [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 300]
    s = Step(cache, D, 8, 2, ps, [(l, 1) for l in lens], seed=D + ps)
    check(s.answer(), *run_fwd(s))


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("D,hq,hkv", [(64, 4, 4), (128, 3, 1), (64, 10, 2), (128, 8, 1), (64, 12, 1), (128, 16, 1),
                                      (64, 34, 2), (128, 40, 1)])
def test_head_groups(cache, D, hq, hkv):
    # groups of 1 to 40 query heads: every number of rows and row blocks
    s = Step(cache, D, hq, hkv, 32, [(70, 1), (200, 1), (5, 1)], seed=hq)
    check(s.answer(), *run_fwd(s))


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("D,hq,hkv", [(64, 4, 2), (128, 6, 2)])
def test_several_new_tokens(cache, causal, D, hq, hkv):
    seqs = [(100, 3), (9, 9), (40, 17), (0, 0), (257, 70), (130, 1), (33, 2)]
    s = Step(cache, D, hq, hkv, 16, seqs, seed=5)
    check(s.answer(causal), *run_fwd(s, causal))


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("causal", [True, False])
def test_rows_that_see_nothing(cache, causal):
    # sequences without keys; more queries than keys (the first see none when causal)
    s = Step(cache, 128, 4, 2, 16, [(0, 1), (3, 5), (20, 1), (0, 2), (1, 3)], seed=6)
    (q, k, v), kw = s.to(DEV)
    check(s.answer(causal), *run_fwd(s, causal, expect=4))   # flagged: more tokens than keys


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("D", [64, 128])
def test_items_without_keys_between_others(cache, D):
    # many rows: items that have no chunk at all before, between and after items of one chunk and more
    for seqs in ([(0, 20), (100, 40), (0, 20), (0, 33), (64, 30), (0, 40)], [(0, 40)], [(30, 30), (0, 25)],
                 [(20, 20)] * 3 + [(0, 30)] * 3 + [(20, 20)] * 2, [(0, 30)] * 40 + [(10, 10)] * 40 + [(0, 18)] * 3):
        s = Step(cache, D, 4, 2, 16, seqs, seed=61)
        check(s.answer(), *run_fwd(s, expect=4))


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("D", [64, 128])
def test_long_axis_is_split_and_joined(cache, D):
    # one sequence over every CTA, and lengths that put range borders inside items
    s = Step(cache, D, 4, 1, 64, [(12345, 1)], seed=7)
    check(s.answer(), *run_fwd(s))
    s = Step(cache, D, 4, 2, 16, [(5000, 1), (3, 1), (1700, 1), (900, 1), (16, 1)], seed=8)
    check(s.answer(), *run_fwd(s))
    s = Step(cache, D, 8, 1, 32, [(4000, 3), (2500, 2)], seed=9)
    check(s.answer(), *run_fwd(s))


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("D,hq,hkv,ps", [(64, 2, 1, 16), (128, 3, 1, 32), (64, 8, 8, 64), (128, 8, 2, 128), (128, 4, 1, 16)])
def test_chunks_of_prompts(cache, D, hq, hkv, ps):
    # several row tiles and blocks; tiles of an odd number of rows (groups of 3); prefixes of every kind;
    # decoding sequences, empty ones and short drafts among them
    seqs = [(700, 300), (129, 129), (2, 1), (513, 1), (0, 0), (400, 90), (130, 7), (64, 64), (33, 20)]
    s = Step(cache, D, hq, hkv, ps, seqs, seed=ps + D)
    check(s.answer(), *run_fwd(s))


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("D", [64, 128])
def test_chunk_over_a_long_prefix_is_split_and_joined(cache, D):
    s = Step(cache, D, 4, 1, 64, [(9000, 40)], seed=41)
    check(s.answer(), *run_fwd(s))
    s = Step(cache, D, 4, 2, 16, [(3000, 70), (20, 20), (1500, 1), (800, 5)], seed=42)
    check(s.answer(False), *run_fwd(s, False))


@pytest.mark.parametrize("cache", CACHES)
def test_chunk_with_bad_pages(cache):
    # pages missing at the start, in the middle and at the end of a chunk's keys
    for ps, cols in ((16, (0, 2, 7)), (64, (1,)), (128, (0,))):
        s = Step(cache, 64, 4, 2, ps, [(230, 40), (90, 60)], seed=43)
        keep = torch.ones(230, dtype=torch.bool)
        for c in cols:
            s.table[0, c] = -3 if c else 10 ** 6
            keep[c * ps:(c + 1) * ps] = False
        o, lse = run_fwd(s, causal=False, expect=1)
        t = s.table.clone()
        s.table[0].clamp_(0, s.pools[0].shape[0] - 1)
        k, v = s.keys(0)
        r = slice(0, 40)
        ro, rl, wabs, smax = OC.attention(s.q[r], k[keep], v[keep], 64 ** -0.5, causal=False)
        b = bounds(ro, rl, wabs, 2.0 ** -5 * 230 * 448, smax, 64, cache, 120)
        check(dict(o=ro, lse=rl, **b), o[r], lse[:, r])
        ref = s.answer(False)
        r = slice(40, 100)
        check({n: x[:, r] if n.startswith("lse") else x[r] for n, x in ref.items()}, o[r], lse[:, r])


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("D,hq,hkv", [(64, 4, 2), (128, 12, 1)])
def test_prompts_among_many_decoding_sequences(cache, D, hq, hkv):
    # e4m3: both kernels in one call; rows on both sides of the border, empty sequences, padding
    seqs = [((37 * n) % 200 + 1, 1) for n in range(40)]
    seqs[3], seqs[17], seqs[20], seqs[30], seqs[39] = (300, 200), (0, 0), (90, 8), (100, 9), (70, 60)
    s = Step(cache, D, hq, hkv, 16, seqs, seed=71)
    check(s.answer(), *run_fwd(s))


@pytest.mark.parametrize("cache", CACHES)
def test_many_short_sequences(cache):
    # more sequences than threads of a CTA, empty ones among them, all within few chunks
    seqs = [((7 * n) % 41, 1 if (7 * n) % 41 else 0) for n in range(700)]
    s = Step(cache, 64, 4, 2, 16, seqs, seed=10)
    check(s.answer(), *run_fwd(s))


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
def test_scales_and_peaked_rows(cache, scale):
    s = Step(cache, 64, 4, 2, 16, [(500, 1), (77, 4)], seed=11, amp=3.0)
    check(s.answer(scale=scale), *run_fwd(s, scale=scale))


def test_query_magnitudes_e4m3():
    # q is scaled by a power of two per row: tiny, huge, zero and mixed rows
    s = Step("e4m3", 128, 4, 2, 16, [(100, 4), (50, 1)], seed=12)
    s.q[0] *= 2.0 ** -60
    s.q[1] *= 2.0 ** 20
    s.q[2] = 0
    s.q[3, :, 0] = 2.0 ** 14
    s.q[3, :, 1:] *= 2.0 ** -12
    scale = torch.tensor([2.0 ** -8])
    check(s.answer(scale=2.0 ** -24), *run_fwd(s, scale=2.0 ** -24))


def test_page_scales_far_apart():
    s = Step("e4m3", 64, 2, 1, 16, [(200, 1), (90, 2)], seed=13)
    for i in range(2):
        g = torch.Generator().manual_seed(i)
        # keys within logits' reach, values over 60 powers of two
        e = torch.randint(*((-12, -4) if i == 0 else (-40, 20)), s.scales[i].shape, generator=g)
        live = ~s.scales[i].isnan()
        s.scales[i][live] = torch.exp2(e[live].float())
        s.true[i] = s.pools[i].float().double() * s.scales[i].double()[..., None, None]
    check(s.answer(), *run_fwd(s))


@pytest.mark.parametrize("D,m", [(64, 1), (128, 1), (64, 40), (128, 40)])
def test_subnormal_codes_and_odd_scales(D, m):
    # codes below the normal range (tiny values under large scales), scales past the range of
    # the fast conversion and, for values, scales that are no powers of two
    s = Step("e4m3", D, 4, 2, 16, [(120, m), (77, m)], seed=51)
    g = torch.Generator().manual_seed(3)
    for i in range(2):
        live = ~s.scales[i].isnan()
        x = 0.02 * torch.randn(s.pools[i].shape, generator=g)
        ok = ~s.pools[i].float().isnan()
        s.pools[i].view(torch.uint8)[ok] = x.to(F8).view(torch.uint8)[ok]
        e = torch.randint(0, 12, s.scales[i].shape, generator=g).float()
        s.scales[i][live] = (torch.exp2(e) * (1.0 if i == 0 else 1.37))[live]
        s.true[i] = s.pools[i].float().double() * s.scales[i].double()[..., None, None]
    check(s.answer(scale=2.0 ** -8), *run_fwd(s, scale=2.0 ** -8))


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("m", [1, 40])
def test_nan_of_a_seen_key_stays_nan(cache, m):
    s = Step(cache, 64, 4, 2, 16, [(100, m), (100, m)], seed=52)
    (q, k, v), kw = s.to(DEV)
    page = int(s.table[0, 1])
    v.view(torch.uint8 if cache == "e4m3" else torch.int16)[page, 0, 3, 5] = 0x7f if cache == "e4m3" else 0x7fc0
    o, lse = A.attn_cache_fwd(q, k, v, causal=False, **kw)
    bad = o[:m, :2, 5].isnan()
    assert bad.all() and int(o.isnan().sum()) == bad.numel() and torch.isfinite(lse[:, :2 * m]).all()
    k.view(torch.uint8 if cache == "e4m3" else torch.int16)[page, 1, 3, 5] = 0x7f if cache == "e4m3" else 0x7fc0
    o, lse = A.attn_cache_fwd(q, k, v, causal=False, **kw)
    assert o[:m, 2:].isnan().all() and lse[2:, :m].isnan().all() and torch.isfinite(o[m:2 * m].float()).all()


def test_lowest_and_infinite_keys():
    # a key whose logit is -inf or the type's lowest drops out; values are not touched
    s = Step("bf16", 64, 2, 2, 16, [(40, 1)], seed=14)
    s.q[0] = s.q[0].abs() + 0.5
    page = int(s.table[0, 1])
    for pool, true in ((s.pools[0], s.true[0]),):
        pool[page, :, 3] = -float("inf")
        pool[page, :, 5] = torch.finfo(torch.bfloat16).min
        true[page, :, 3] = -1e30
        true[page, :, 5] = -1e30
    ref = s.answer()
    t = s.answer(scale=s.D ** -0.5)
    # smax is meaningless with such keys: the others' logits bound the error
    for p in (3, 5):
        s.true[0][page, :, p] = 0
    ref["o_tol"], ref["lse_tol"] = s.answer()["o_tol"], s.answer()["lse_tol"]
    o, lse = run_fwd(s)
    check(ref, o, lse)


def test_bad_page_is_flagged_and_its_keys_left_out():
    for cache in CACHES:
        s = Step(cache, 64, 2, 1, 16, [(100, 1), (64, 1)], seed=15)
        good = s.answer()
        s.table[0, 2] = 10 ** 6
        o, lse = run_fwd(s, expect=1)
        k, v = s.keys(1)
        # sequence 1 untouched; sequence 0 attends the other pages' keys
        assert (o[1].double().cpu() - good["o"][1]).abs().le(good["o_tol"][1]).all()
        keep = [c for c in range(7) if c != 2]
        rows = [t[s.table[0, keep].long()].permute(0, 2, 1, 3).reshape(-1, 1, 64) for t in s.true]
        rows = [r[:84] for r in rows]   # 100 keys less 16
        ro, rl, wabs, smax = OC.attention(s.q[:1], *rows, 64 ** -0.5)
        b = bounds(ro, rl, wabs, 2.0 ** -5 * 84 * 448, smax, 64, cache, 2)   # scales of 2^-5 at most
        check(dict(o=ro, lse=rl, **b), o[:1], lse[:, :1])


def test_length_past_the_page_table_is_flagged():
    s = Step("bf16", 64, 2, 1, 16, [(64, 1)], seed=16, extra_cols=0)
    ref = s.answer()
    s.kv[0] = 10 ** 9
    check(ref, *run_fwd(s, expect=4))


def test_more_new_tokens_than_max_new_is_flagged_and_still_right():
    s = Step("bf16", 64, 2, 1, 16, [(64, 20), (30, 1)], seed=17)
    s.max_new = 1
    check(s.answer(), *run_fwd(s, expect=4))


@pytest.mark.parametrize("cache", CACHES)
def test_query_stride_side_stream_and_workspace_contents(cache):
    s = Step(cache, 128, 4, 2, 32, [(600, 2), (100, 1)], seed=18)
    (q, k, v), kw = s.to(DEV)
    wide = torch.full((s.T, 9, 128), float("nan"), dtype=torch.bfloat16, device=DEV)
    wide[:, 2:6] = q
    ws = torch.full((A.attn_cache_fwd_workspace_size(q, k, v, **kw),), 0xff, dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    o, lse = A.attn_cache_fwd(wide[:, 2:6], k, v, workspace=ws, stream=side, **kw)
    side.synchronize()
    check(s.answer(), o, lse)
    o2, lse2 = A.attn_cache_fwd(q, k, v, **kw)      # other workspace: the same bits
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_two_calls_at_once():
    a = Step("bf16", 64, 4, 2, 16, [(3000, 1)], seed=19)
    b = Step("e4m3", 128, 8, 2, 32, [(2000, 3), (50, 1)], seed=20)
    (xa, ka), (xb, kb) = a.to(DEV), b.to(DEV)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [(A.attn_cache_fwd(*xa, stream=s1, **ka), A.attn_cache_fwd(*xb, stream=s2, **kb)) for _ in range(5)]
    torch.cuda.synchronize()
    for ra, rb in got:
        check(a.answer(), *ra)
        check(b.answer(), *rb)


@pytest.mark.parametrize("cache", CACHES)
def test_captured_and_replayed_with_other_lengths(cache):
    s = Step(cache, 64, 4, 2, 16, [(400, 1), (300, 2), (50, 1)], seed=21)
    (q, k, v), kw = s.to(DEV)
    o, lse = A.attn_cache_fwd(q, k, v, **kw)
    ws = torch.empty(A.attn_cache_fwd_workspace_size(q, k, v, **kw), dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        A.attn_cache_fwd(q, k, v, out=o, lse=lse, workspace=ws, **kw)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        A.attn_cache_fwd(q, k, v, out=o, lse=lse, workspace=ws, **kw)
    for seqs in ([(400, 1), (300, 2), (50, 1)], [(17, 2), (299, 1), (1, 1)], [(1, 1), (0, 0), (33, 1)]):
        s.seqs = seqs
        s.kv.copy_(torch.tensor([l for l, _ in seqs]))
        s.cu.copy_(torch.tensor([0] + [m for _, m in seqs]).cumsum(0))
        kw["seqlens_kv"].copy_(s.kv)
        kw["cu_seqlens"].copy_(s.cu)
        o.fill_(float("nan"))
        lse.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        check(s.answer(), o, lse)


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------
def _append_case(cache, D, hq, hkv, ps, seqs, rot, interleaved, seed, calls=1, amp=1.0):
    """`calls` appends in a row, each of seqs[n] = new tokens per call; checks the cache
    after each against the oracle, and that nothing else was written."""
    g = torch.Generator().manual_seed(seed)
    n = len(seqs[0])
    most = [sum(c[i] for c in seqs) for i in range(n)]
    cols = max(1, max(-(-m // ps) for m in most)) + 1
    pages = n * cols + 1
    tab = torch.randperm(pages, generator=g)[:n * cols].view(n, cols).to(torch.int32)
    dtype = torch.bfloat16 if cache == "bf16" else F8
    kc, vc, ks, vs = A.attn_cache_empty(pages, hkv, ps, D, dtype=dtype, device=DEV)
    mark = 0x5a
    for t in (kc, vc):
        t.view(torch.uint8).fill_(mark)
    if ks is not None:
        ks.fill_(float("nan")), vs.fill_(float("nan"))
    models = [OC.Cache(hkv, D, ps, cache != "bf16") for _ in range(2)]
    cs = table(max(most) + 5, rot) if rot else None
    lens = [0] * n
    for call, new in enumerate(seqs):
        T = sum(new) + 2
        x = [(amp * 10.0 ** (call % 3) * torch.randn(T, h, D, generator=g)).to(torch.bfloat16) for h in (hq, hkv, hkv)]
        cu = torch.tensor([0] + list(new)).cumsum(0).to(torch.int32)
        lens = [l + m for l, m in zip(lens, new)]
        err = _err()
        q = A.attn_cache_append(*(t.to(DEV) for t in x), kc, vc, page_table=tab.to(DEV), k_scale=ks, v_scale=vs,
                                seqlens_kv=torch.tensor(lens, dtype=torch.int32, device=DEV), cu_seqlens=cu.to(DEV),
                                max_new=max(1, max(new)), cos_sin=None if cs is None else cs.to(DEV),
                                interleaved=interleaved, error_word=err)
        torch.cuda.synchronize()
        assert int(err.item()) == 0
        for i, m in enumerate(new):
            r = slice(int(cu[i]), int(cu[i + 1]))
            pos = list(range(lens[i] - m, lens[i]))
            want = OC.rotate(x[0][r], pos, cs, interleaved)
            # fp32 products and sum of magnitudes at most sqrt(2) max|x|, then bf16
            tol = 2.0 ** -8 * want.abs() + 2.0 ** -21 * x[0][r].double().abs().amax(-1, keepdim=True)
            assert ((q[r].double().cpu() - want).abs() <= tol).all()
            models[0].append(OC.rotate(x[1][r], pos, cs, interleaved), lens[i] - m, tab[i])
            models[1].append(x[2][r].double(), lens[i] - m, tab[i])
        assert (q[int(cu[-1]):] == 0).all()
        for pool, scale, model in ((kc, ks, models[0]), (vc, vs, models[1])):
            raw, val = pool.view(torch.uint8).cpu(), pool.cpu().float().double()
            untouched = torch.ones(pages, ps, dtype=torch.bool)
            for (page, slot), want in model.rows.items():
                untouched[page, slot] = False
                got = val[page, :, slot]
                if scale is None:
                    tol = 2.0 ** -8 * want.abs() + 2.0 ** -21 * want.abs().amax(-1, keepdim=True)
                else:
                    s = torch.tensor([model.scale[page, h] for h in range(hkv)], dtype=torch.float64)[:, None]
                    got = got * s
                    # a code's half step, relative 2^-4 or half the least subnormal 2^-9 (twice: a
                    # code may have been rounded again when the scale grew)
                    tol = 2.0 ** -4 * want.abs() + 2 * 2.0 ** -10 * s + 2.0 ** -21 * want.abs().amax(-1, keepdim=True)
                assert ((got - want).abs() <= tol).all(), (call, page, slot)
            if scale is not None:
                sc = scale.cpu().double()
                for (page, h), want in model.scale.items():
                    assert sc[page, h].item() == want
                written = {page for page, _ in model.scale}
                rest = [p for p in range(pages) if p not in written]
                assert sc[rest].isnan().all()
            assert (raw[untouched[:, None, :].expand(pages, hkv, ps)] == mark).all()
    return kc, vc, ks, vs, tab, lens


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("D,rot,interleaved", [(64, 64, False), (64, 32, True), (128, 128, False), (128, 64, False),
                                               (128, 128, True), (128, 16, False), (64, 0, False)])
def test_append_rotations(cache, D, rot, interleaved):
    _append_case(cache, D, 3, 1, 16, [(5, 1, 0, 18), (1, 1, 1, 1)], rot, interleaved, seed=rot + D)


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("ps", [16, 32, 64, 128])
def test_append_across_pages(cache, ps):
    # prompts that end inside, at and past a page; then tokens one by one; then a chunk over several pages
    calls = [(ps - 1, ps, ps + 1, 3 * ps + 5)] + [(1, 1, 1, 1)] * 3 + [(2, 8, 0, 7), (2 * ps, 9, 1, 0)]
    _append_case(cache, 128, 4, 2, ps, calls, 32, False, seed=ps)


@pytest.mark.parametrize("cache", CACHES)
def test_append_many_sequences(cache):
    # a scan over more sequences than a block has threads, some without new tokens
    new = tuple((5 * n) % 23 if n % 3 else 0 for n in range(300))
    _append_case(cache, 64, 2, 1, 16, [new, tuple(min(m, 1) for m in new)], 16, False, seed=3)


def test_append_magnitudes_and_growth():
    # growing, shrinking, tiny and zero values: the page's scale only grows
    g = torch.Generator().manual_seed(4)
    kc, vc, ks, vs = A.attn_cache_empty(2, 1, 16, 64, dtype=F8, device=DEV)
    tab = torch.tensor([[1]], dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    amps = [0.0, 1e-3, 1.0, 0.5, 300.0, 1e4, 0.0, 1e-30, 1e30, 448.0]
    seen, want_scale = [], 0.0
    for i, a in enumerate(amps):
        x = (a * torch.randn(1, 1, 64, generator=g)).to(torch.bfloat16)
        seen.append(x[0, 0].double())
        want_scale = max(want_scale, OC.page_scale(x.double().abs().max().item()))
        A.attn_cache_append(None, x.to(DEV), x.to(DEV), kc, vc, page_table=tab, cu_seqlens=cu, max_new=1, k_scale=ks,
                            seqlens_kv=torch.tensor([i + 1], dtype=torch.int32, device=DEV), v_scale=vs)
        assert ks[1, 0].item() == want_scale and vs[1, 0].item() == want_scale
        got = kc[1, 0, :i + 1].float().double().cpu() * want_scale
        want = torch.stack(seen)
        assert ((got - want).abs() <= 2.0 ** -4 * want.abs() + 2 * 2.0 ** -10 * want_scale).all()
        assert torch.equal(kc.view(torch.uint8)[1], vc.view(torch.uint8)[1])


def test_append_scale_border_and_specials():
    # exactly 448 2^e keeps e; the next bf16 above takes e + 1; infinities saturate, NaN stays
    kc, vc, ks, vs = A.attn_cache_empty(3, 1, 16, 64, dtype=F8, device=DEV)
    x = torch.zeros(3, 1, 64, dtype=torch.bfloat16)
    x[0, 0, 5] = 448.0 / 64
    x[1, 0, 5] = 450.0 / 64
    x[2, 0, 0], x[2, 0, 1], x[2, 0, 2], x[2, 0, 3] = float("inf"), float("nan"), -float("inf"), 7.0
    A.attn_cache_append(None, x.to(DEV), x.to(DEV), kc, vc, k_scale=ks, v_scale=vs, max_new=1,
                        page_table=torch.tensor([[0], [1], [2]], dtype=torch.int32, device=DEV),
                        seqlens_kv=torch.ones(3, dtype=torch.int32, device=DEV),
                        cu_seqlens=torch.arange(4, dtype=torch.int32, device=DEV))
    assert ks[:, 0].tolist() == [2.0 ** -6, 2.0 ** -5, 2.0 ** -6]
    row = kc[2, 0, 0].float()
    assert row[0] == 448 and row[1].isnan() and row[2] == -448 and row[3] == 448


@pytest.mark.parametrize("cache", CACHES)
@pytest.mark.parametrize("new", [(2, 3), (40, 9)])
def test_append_strides_in_place_stream(cache, new):
    # slices of one fused projection, the rotated q over its own dense buffer, another stream
    D, hq, hkv, ps, T = 64, 4, 2, 16, sum(new)
    g = torch.Generator().manual_seed(9)
    fused = torch.randn(T, hq + 2 * hkv, D, generator=g).to(torch.bfloat16).to(DEV)
    q, k, v = fused[:, :hq], fused[:, hq:hq + hkv], fused[:, hq + hkv:]
    cs = table(64, 64).to(DEV)
    kw = dict(page_table=torch.arange(6, dtype=torch.int32, device=DEV).view(2, 3), cos_sin=cs, max_new=max(new),
              seqlens_kv=torch.tensor(new, dtype=torch.int32, device=DEV),
              cu_seqlens=torch.tensor([0, new[0], T], dtype=torch.int32, device=DEV))
    outs = []
    side = torch.cuda.Stream()
    for way in range(2):
        kc, vc, ks, vs = A.attn_cache_empty(6, hkv, ps, D, dtype=torch.bfloat16 if cache == "bf16" else F8, device=DEV)
        for t in (kc, vc):
            t.view(torch.uint8).zero_()
        torch.cuda.synchronize()
        if way == 0:
            qo = A.attn_cache_append(q, k, v, kc, vc, k_scale=ks, v_scale=vs, stream=side, **kw)
        else:
            dense = q.contiguous()
            qo = A.attn_cache_append(dense, k.contiguous(), v.contiguous(), kc, vc, k_scale=ks, v_scale=vs, q_out=dense,
                                     **kw)
            assert qo is dense
        torch.cuda.synchronize()
        outs.append((qo, kc.view(torch.uint8), vc.view(torch.uint8)) + (() if ks is None else (ks, vs)))
    for x, y in zip(*outs):
        assert torch.equal(x, y)


def test_append_flags_and_skips():
    D, T = 64, 6
    x = torch.randn(T, 1, D).to(torch.bfloat16).to(DEV)
    cs = table(20, 64).to(DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    for tab, kv, cu, max_new, bit, written in (
            ([[0], [99]], [3, 3], [0, 3, 6], 3, 1, 3),        # a bad page
            ([[0], [1]], [17, 3], [0, 3, 6], 3, 4, 5),        # past the page table
            ([[0], [1]], [2, 3], [0, 3, 6], 3, 4, 5),         # more tokens than the length
            ([[0], [1]], [3, 3], [0, 3, 6], 2, 4, 4),         # more tokens than max_new
            ([[0, 2], [1, 3]], [22, 3], [0, 3, 6], 3, 4, 4)):  # past the rotation table
        kc, vc, _, _ = A.attn_cache_empty(4, 1, 16, D, device=DEV)
        kc.fill_(float("nan")), vc.fill_(float("nan"))
        err = _err()
        A.attn_cache_append(x, x, x, kc, vc, page_table=torch.tensor(tab, **i32), max_new=max_new, cos_sin=cs,
                            seqlens_kv=torch.tensor(kv, **i32), cu_seqlens=torch.tensor(cu, **i32), error_word=err)
        torch.cuda.synchronize()
        assert int(err.item()) == bit, (kv, max_new)
        assert int((~kc[..., 0].isnan()).sum()) == written, (kv, max_new)


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("D,hq,hkv", [(64, 4, 2), (128, 8, 2)])
def test_generation_matches_the_forward_over_the_whole_text(D, hq, hkv):
    """A text appended as a prompt, a chunk and token by token into a bf16 cache gives
    the rows that attn_fwd gives over the whole text."""
    S, parts = 200, [90, 60] + [1] * 50
    g = torch.Generator().manual_seed(31)
    q, k, v = (torch.randn(S, h, D, generator=g).to(torch.bfloat16).to(DEV) for h in (hq, hkv, hkv))
    cs = table(S, D).to(DEV)
    kc, vc, _, _ = A.attn_cache_empty(16, hkv, 16, D, device=DEV)
    tab = torch.randperm(16, generator=g).to(torch.int32).to(DEV)[None]
    outs, lses, qs, at = [], [], [], 0
    for m in parts:
        r = slice(at, at + m)
        at += m
        kw = dict(page_table=tab, seqlens_kv=torch.tensor([at], dtype=torch.int32, device=DEV), max_new=m,
                  cu_seqlens=torch.tensor([0, m], dtype=torch.int32, device=DEV))
        qr = A.attn_cache_append(q[r], k[r], v[r], kc, vc, cos_sin=cs, **kw)
        o, lse = A.attn_cache_fwd(qr, kc, vc, **kw)
        outs.append(o), lses.append(lse), qs.append(qr)
    o, lse, qr = torch.cat(outs), torch.cat(lses, 1), torch.cat(qs)
    kr = kc[tab[0].long()].transpose(1, 2).reshape(-1, hkv, D)[:S]
    wo, wl = A.attn_fwd(qr[None], kr[None].contiguous(), v[None], causal=True)
    ro, rl, wabs, smax = OC.attention(qr.cpu(), kr.cpu(), v.cpu(), D ** -0.5)
    b = bounds(ro, rl, wabs, torch.zeros_like(ro), smax, D, "bf16", 1000)   # its prompt and chunk: many rows
    check(dict(o=ro, lse=rl, **b), o, lse)
    # both within their bounds of the same rows: at most twice the bound apart
    assert ((o.double() - wo[0].double()).abs().cpu() <= 2 * b["o_tol"]).all()
    assert ((lse.double() - wl[0].double()).abs().cpu() <= 2e-4 * rl.abs().clamp(min=1)).all()


def test_generation_e4m3_hardly_depends_on_the_cuts():
    """The e4m3 cache of a text, appended at once and token by token: the same values
    up to codes that were subnormal under the smaller scale."""
    S, D, hkv = 150, 64, 2
    g = torch.Generator().manual_seed(32)
    k, v = (torch.randn(S, hkv, D, generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
    tab = torch.arange(10, dtype=torch.int32, device=DEV)[None]
    vals = []
    for parts in ([S], [1] * S, [70, 1, 79]):
        kc, vc, ks, vs = A.attn_cache_empty(10, hkv, 16, D, dtype=F8, device=DEV)
        at = 0
        for m in parts:
            A.attn_cache_append(None, k[at:at + m], v[at:at + m], kc, vc, k_scale=ks, v_scale=vs, page_table=tab, max_new=m,
                                seqlens_kv=torch.tensor([at + m], dtype=torch.int32, device=DEV),
                                cu_seqlens=torch.tensor([0, m], dtype=torch.int32, device=DEV))
            at += m
        vals.append([(c.float() * s[..., None, None]).transpose(1, 2).reshape(-1, hkv, D)[:S].double()
                     for c, s in ((kc, ks), (vc, vs))] + [ks, vs])
    for other in vals[1:]:
        assert torch.equal(other[2], vals[0][2]) and torch.equal(other[3], vals[0][3])
        for x, y, s in zip(vals[0][:2], other[:2], (vals[0][2], vals[0][3])):
            step = s.repeat_interleave(16, 0)[:S, :, None].double() * 2.0 ** -9
            assert ((x - y).abs() <= step).all()
            assert (x == y)[(x.abs() >= 2 * step * 2 ** 3)].all()
