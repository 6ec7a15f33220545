"""GPU tests of the e4m3 cache's attention where the values' page scales lie far apart and
where probabilities are small: a row's precision goes by what the row sees and weighs.
`m` new tokens: few rows per KV head, or as many as the tcgen05 kernel takes."""
import pytest
import torch

from _cache_bounds import ScaledStep, answer
from _cache_util import check
from test_parity_cache import run_fwd

pytestmark = pytest.mark.gpu

ROWS = [(64, 1), (128, 1), (64, 5), (64, 40), (128, 40)]
INF = float("inf")


def one_sink(L, D, m, nats, sink_value, ps=16, seed=81, seqs=None):
    """q picks out dim 0, in which key 0 alone is not zero: its logit is `nats` above all the others', its
    value sink_value."""
    s = ScaledStep("e4m3", D, 4, 2, ps, seqs or [(L, m)], seed=seed, pad_tokens=0)
    s.q[:] = 0
    s.q[:, :, 0] = 1.0
    for n, (l, _) in enumerate(s.seqs):
        cols = -(-l // ps)
        s.set_scales(0, {(n, c): 0 for c in range(cols)})
        s.set_scales(1, {(n, c): -7 for c in range(cols)})
        for i in range(2):
            pool = s.pools[i]
            for c in range(cols):
                page = int(s.table[n, c])
                rows = min(ps, l - c * ps)
                if i == 0:
                    pool.view(torch.uint8)[page, :, :rows] = 0
                else:
                    g = torch.Generator().manual_seed(seed + c)
                    x = torch.randn(s.hkv, rows, D, generator=g) * 2.0 ** 7
                    pool[page, :, :rows] = x.clamp(-448, 448).to(pool.dtype)
            s.refresh(i)
        key = torch.zeros(1, s.hkv, D)
        key[..., 0] = 16.0
        s.set_rows(0, n, [0], key)
        s.set_rows(1, n, [0], torch.full((1, s.hkv, D), sink_value))
    return s, nats / 16.0


@pytest.mark.parametrize("D,m", ROWS)
@pytest.mark.parametrize("L,nats", [(300, 8.0), (8191, 12.0), (8191, 16.0), (8191, 16.6), (8191, 20.0), (20000, 17.4)])
def test_long_tail_below_a_sink(D, m, L, nats):
    # the sink's value is zero: all of the output is the tail's
    s, scale = one_sink(L, D, m, nats, 0.0)
    check(answer(s, 11, scale=scale), *run_fwd(s, scale=scale))


@pytest.mark.parametrize("D,m", ROWS)
@pytest.mark.parametrize("ratio", [12, 16, 20, 24, 60])
@pytest.mark.parametrize("at", ["first", "middle", "last"])
def test_large_scale_page_of_no_weight(D, m, ratio, at):
    # one page under a scale 2^ratio times the others', its keys far below all others (by 30 nats or more)
    L, ps = 2000, 16
    s = ScaledStep("e4m3", D, 4, 2, ps, [(L, m)], seed=82)
    cols = -(-L // ps)
    page = {"first": 0, "middle": cols // 2, "last": cols - 2 - m // ps}[at]
    s.set_scales(1, {(0, c): -7 for c in range(cols)})
    s.set_scales(1, {(0, page): -7 + ratio})
    s.set_scales(0, {(0, page): -2})
    s.q[:, :, 0] = 8.0
    depth = 30.0 + 0.7 * max(0, ratio - 24)     # its products stay below the others'
    x = torch.zeros(ps, s.hkv, D)
    x[..., 0] = -depth * D ** 0.5 / 8.0
    s.set_rows(0, 0, range(page * ps, (page + 1) * ps), x)
    other = [r for r in range(0, L) if r // ps != page]
    # the others' dim 0 holds nothing that could outweigh their own spread
    for c in range(cols):
        if c != page:
            s.pools[0].view(torch.uint8)[s.table[0, c], :, :min(ps, L - c * ps), 0] = 0
    s.refresh(0)
    assert len(other) == L - ps
    check(answer(s, 11), *run_fwd(s))


@pytest.mark.parametrize("ps", [16, 32, 128])
@pytest.mark.parametrize("D,m", [(64, 3), (128, 3), (64, 40), (128, 40)])
@pytest.mark.parametrize("ratio", [16, 24, 80])
def test_large_scale_page_behind_the_diagonal(ps, D, m, ratio):
    # the newest page's values are 2^ratio times the others'; rows whose positions lie before it do not see it
    lens = [(4 * ps + 2, m), (10 * ps + 2, m), (2 * ps + 1, min(m, 2 * ps + 1))]
    s = ScaledStep("e4m3", D, 4, 2, ps, lens, seed=83)
    for n, (l, _) in enumerate(lens):
        last = (l - 1) // ps
        s.set_scales(1, {(n, c): -7 for c in range(last)})
        s.set_scales(1, {(n, last): -7 + ratio})
    check(answer(s, 11), *run_fwd(s))


@pytest.mark.parametrize("ps", [16, 64])
@pytest.mark.parametrize("D,m", ROWS)
def test_scales_and_weights_at_random(ps, D, m):
    # value scales over 60 powers of two, logits spread over some 40 nats, several sequences, CTAs' parts joined
    s = ScaledStep("e4m3", D, 4, 2, ps, [(1500, m), (333, m), (40, m), (5000, m)], seed=84, amp=4.0)
    g = torch.Generator().manual_seed(7)
    for n, (l, _) in enumerate(s.seqs):
        s.set_scales(1, {(n, c): int(torch.randint(-50, 10, (1,), generator=g)) for c in range(-(-l // ps))})
    check(answer(s, 11, scale=0.3 * 8 / D ** 0.5), *run_fwd(s, scale=0.3 * 8 / D ** 0.5))


@pytest.mark.parametrize("D,m", ROWS)
@pytest.mark.parametrize("lo,hi", [(-100, 0), (-100, -90), (0, 90), (-60, 60), (-118, -112)])
def test_scales_at_the_ends_of_their_range(D, m, lo, hi):
    # alternating pages; values whose products with a probability cross fp16's range both ways
    s = ScaledStep("e4m3", D, 4, 2, 16, [(600, m), (45, m)], seed=85)
    for n, (l, _) in enumerate(s.seqs):
        s.set_scales(1, {(n, c): (lo, hi)[c % 2] for c in range(-(-l // 16))})
    check(answer(s, 11), *run_fwd(s))


@pytest.mark.parametrize("D,m", ROWS)
def test_rising_weights(D, m):
    # logits that rise along the keys by half a nat each, values that fall: every chunk brings a new maximum
    s, _ = one_sink(400, D, m, 1.0, 0.0)
    x = torch.zeros(400, s.hkv, D)
    x[..., 0] = torch.arange(400)[:, None] / 2.0
    s.set_rows(0, 0, range(400), x)
    for c in range(25):
        s.set_scales(1, {(0, c): -7 - c})
    for scale in (1.0, -1.0, 0.05):
        check(answer(s, 11, scale=scale), *run_fwd(s, scale=scale))


@pytest.mark.parametrize("m", [1, 40])
@pytest.mark.parametrize("ps", [16, 64])
def test_missing_pages_beside_far_scales(m, ps):
    # a bad page (flagged, left out) between pages of far scales, rows without keys, a last page half full
    s = ScaledStep("e4m3", 64, 4, 2, ps, [(10 * ps + 3, m), (0, 0), (3 * ps, m)], seed=86)
    for n, (l, _) in enumerate(s.seqs):
        s.set_scales(1, {(n, c): (-30, 5, -7)[c % 3] for c in range(-(-l // ps))})
    ref = answer(s, 11, causal=False)
    s.table[0, 4] = 10 ** 6
    o, lse = run_fwd(s, causal=False, expect=1)
    r = slice(m, 2 * m)
    check({k: x[:, r] if k.startswith("lse") else x[r] for k, x in ref.items()}, o[r], lse[:, r])
    # the first sequence without the page's keys: one with the page's columns closed up
    t = ScaledStep("e4m3", 64, 4, 2, ps, [(9 * ps + 3, m)], seed=0, pad_tokens=0)
    t.q, t.table, t.cols = s.q[:m].clone(), s.table[:1, [c for c in range(s.table.shape[1]) if c != 4]], s.cols - 1
    t.pools, t.scales, t.true = s.pools, s.scales, s.true
    check(answer(t, 11, causal=False), o[:m], lse[:, :m])


@pytest.mark.parametrize("D,m", ROWS)
@pytest.mark.parametrize("bits", [16, 22, 24, 25, 30, 40])
@pytest.mark.parametrize("e", [-40, -7, 9, 30])
def test_logits_whose_rounding_is_whole_powers(D, m, bits, e):
    # logits up to 2^bits (log2 units), each a single product, so far apart that one key has all the weight: o is its
    # value, whatever scale its page has; the other pages' scales lie on both sides of it.  The tcgen05 kernel takes
    # the maximum off the unrounded product: from 2^26 on that alone is several powers of two
    if m == 40 and bits > 25:
        bits = 25
    L, top = 130, 2.0 ** bits
    s, _ = one_sink(L, D, m, 1.0, 0.0, seqs=[(L, m)])
    x = torch.zeros(L, s.hkv, D)
    x[..., 0] = (torch.arange(L) % 13).float()[:, None]
    for win in (5, 70, L - m):
        y = x.clone()
        y[win, :, 0] = 14.0
        s.set_rows(0, 0, range(L), y)
        for c in range(-(-L // 16)):
            s.set_scales(1, {(0, c): e - 12 if c % 2 else e + 12})
        s.set_scales(1, {(0, win // 16): e})
        scale = top / 1.4426950408889634 / 14.0
        o, lse = run_fwd(s, scale=scale)
        v = s.keys(0)[1][win].repeat_interleave(s.hq // s.hkv, 0)
        # P of the key is 1 within 2^-11 and a few exponentials' 2^-22, the row sum too, then bf16
        assert ((o[:m].double().cpu() - v).abs() <= (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -18) * v.abs()).all()
        want = scale * 14.0
        assert ((lse[:, :m].double().cpu() - want).abs() <= 2.0 ** -21 * want).all()


@pytest.mark.parametrize("D,m", ROWS)
@pytest.mark.parametrize("bits", [20, 28, 31])
def test_small_elements_beside_a_large_one_in_a_query(D, m, bits):
    # an element 2^bits times the others, where the keys hold zeros: the others, of three bits each, make the logits.
    # q is held in fp16 times a power of two, exact for bf16 elements of at least 2^-31 of the row's largest
    s = ScaledStep("e4m3", D, 4, 2, 16, [(300, m), (70, m)], seed=87)
    g = torch.Generator().manual_seed(9)
    sign = 1.0 - 2.0 * torch.randint(0, 2, s.q.shape, generator=g)
    s.q = (sign * (1.0 + torch.randint(0, 8, s.q.shape, generator=g) / 8.0)).to(torch.bfloat16)
    s.q[:, :, 9] = 2.0 ** bits
    live = ~s.pools[0].float().isnan()
    live[..., :9] = False
    live[..., 10:] = False
    s.pools[0].view(torch.uint8)[live] = 0
    s.refresh(0)
    check(answer(s, 11), *run_fwd(s))
