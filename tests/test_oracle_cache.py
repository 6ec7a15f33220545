"""The paged-cache oracle against independent forms: library attention, complex
rotation, closed forms of the scale."""
import math

import pytest
import torch

from oracle import cache as OC
from _cache_util import table

F64 = torch.float64


@pytest.mark.parametrize("m,L,hq,hkv", [(1, 7, 4, 2), (5, 5, 2, 2), (3, 20, 6, 1)])
@pytest.mark.parametrize("causal", [True, False])
def test_attention_is_the_library_one(m, L, hq, hkv, causal):
    g = torch.Generator().manual_seed(m * L)
    q, k, v = (torch.randn(n, h, 16, generator=g, dtype=F64) for n, h in ((m, hq), (L, hkv), (L, hkv)))
    o, lse, wabs, smax = OC.attention(q, k, v, 0.3, causal)
    kk, vv = (t.repeat_interleave(hq // hkv, 1).transpose(0, 1) for t in (k, v))
    mask = torch.arange(L)[None] <= L - m + torch.arange(m)[:, None] if causal else torch.ones(m, L, dtype=torch.bool)
    want = torch.nn.functional.scaled_dot_product_attention(q.transpose(0, 1), kk, vv, attn_mask=mask, scale=0.3)
    assert torch.allclose(o, want.transpose(0, 1), atol=1e-12)
    x = (0.3 * q.transpose(0, 1) @ kk.transpose(1, 2)).masked_fill(~mask, -math.inf)
    assert torch.allclose(lse, x.logsumexp(-1), atol=1e-12)
    assert (wabs >= o.abs() - 1e-12).all() and (smax >= x.masked_fill(~mask, 0).abs().amax(-1) - 1e-12).all()


def test_attention_rows_without_keys():
    q, k, v = torch.ones(3, 1, 4), torch.ones(2, 1, 4), torch.ones(2, 1, 4)
    o, lse, _, _ = OC.attention(q, k, v, 1.0)
    assert (o[0] == 0).all() and lse[0, 0] == -math.inf and torch.allclose(o[1:], torch.ones(2, 1, 4, dtype=F64))


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_a_complex_product(interleaved):
    g = torch.Generator().manual_seed(1)
    x = torch.randn(6, 2, 16, generator=g, dtype=F64)
    cs, pos = table(40, 8), [3, 0, 39, 7, 7, 12]
    y = OC.rotate(x, pos, cs, interleaved)
    z = torch.complex(x[..., 0:8:2], x[..., 1:8:2]) if interleaved else torch.complex(x[..., :4], x[..., 4:8])
    w = torch.complex(cs[pos, :4].double(), cs[pos, 4:].double())[:, None] * z
    got = torch.complex(y[..., 0:8:2], y[..., 1:8:2]) if interleaved else torch.complex(y[..., :4], y[..., 4:8])
    assert torch.allclose(got, w, atol=1e-12) and torch.equal(y[..., 8:], x[..., 8:])
    assert torch.equal(OC.rotate(x, pos, None), x)


def test_page_scale():
    assert OC.page_scale(0.0) == 2.0 ** -100
    for a in (1e-20, 0.3, 1.0, 7.0, 7.01, 448.0, 449.0, 3e38):
        s = OC.page_scale(a)
        assert a <= 448 * s and a > 448 * s / 2 and math.log2(s) == int(math.log2(s))


def test_append_pages_and_scales():
    c = OC.Cache(1, 2, 4, True)
    x = torch.tensor([[[448.0, 1.0]], [[2.0, 3.0]], [[900.0, 0.0]]], dtype=F64)
    c.append(x[:1], 0, [5, 6])
    assert c.scale == {(5, 0): 1.0}
    c.append(x[1:].repeat(2, 1, 1), 1, [5, 6])     # positions 1 .. 4: two pages
    assert c.scale == {(5, 0): 4.0, (6, 0): 4.0} and set(c.rows) == {(5, 0), (5, 1), (5, 2), (5, 3), (6, 0)}
    c.append(x[1:2], 5, [5, 6])                    # smaller values: the scale stays
    assert c.scale[6, 0] == 4.0
    c.append(x[1:2], 4, [5, 6])                    # a page begun anew: the scale starts anew
    assert c.scale[6, 0] == 2.0 ** -7
