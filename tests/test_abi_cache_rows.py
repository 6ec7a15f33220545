"""Host-only checks of the rows that the paged cache's calls take: which token strides
are passed on, and calls without a token."""
import pytest
import torch

import softmax_attention_backward_gb300 as A

BF = torch.bfloat16


def _stride(t, heads, dim):
    return A._need_rows(t, "q", heads, dim, t.device)


def test_strides_that_are_passed_on():
    fused = torch.zeros(5, 12, 64, dtype=BF)
    assert _stride(fused, 12, 64) == 0                      # dense
    assert _stride(fused[:, 2:6], 4, 64) == 12 * 64         # a slice of a fused projection
    assert _stride(fused[::2], 12, 64) == 2 * 12 * 64       # every second token
    assert _stride(fused[:1, 2:6], 4, 64) == 0              # one token: no stride to speak of
    assert _stride(fused[:, 3:4], 1, 64) == 12 * 64


@pytest.mark.parametrize("heads", [1, 2])
@pytest.mark.parametrize("tokens", [2, 7])
def test_tokens_that_lie_over_each_other_are_refused(heads, tokens):
    # a stride of 0 stands for dense rows behind the binding: a broadcast token would be read
    # past its end
    one = torch.zeros(1, heads, 64, dtype=BF)
    wide = one.expand(tokens, heads, 64)
    assert wide.stride(0) == 0
    with pytest.raises(ValueError, match="tokens"):
        _stride(wide, heads, 64)
    windows = torch.zeros(64 * heads + 16 * tokens, dtype=BF).as_strided((tokens, heads, 64), (16, 64, 1))
    with pytest.raises(ValueError, match="tokens"):
        _stride(windows, heads, 64)


def test_heads_that_lie_apart_or_over_each_other_are_refused():
    for t in (torch.zeros(3, 1, 64, dtype=BF).expand(3, 4, 64), torch.zeros(3, 8, 64, dtype=BF)[:, ::2],
              torch.zeros(3, 64, 4, dtype=BF).transpose(1, 2), torch.zeros(3, 4, 1, dtype=BF).expand(3, 4, 64)):
        with pytest.raises(ValueError, match="heads"):
            _stride(t, 4, 64)


# ---------------------------------------------------------------------------
# a step to which no sequence brings a token
# ---------------------------------------------------------------------------
def test_calls_without_a_token_need_no_rows():
    from test_abi_cache import FAKE, _append, _fwd, _p
    from softmax_attention_backward_gb300 import build
    build.build()
    L = A.lib()
    none = {f"i{i}": 0 for i in (0, 1, 2, 4)}                       # q, k, v, q_out
    assert _append(L, _p(tokens=0, max_new=0), **none) == 0
    assert _append(L, _p(tokens=0), **none) == 0
    assert _append(L, _p(tokens=0, cache_type=1), **none) == 0
    assert _fwd(L, _p(tokens=0), ws=0, i0=0, i5=0, i6=0, i7=0) == 0   # q, o, lse, workspace
    # the cache is still asked for
    assert _append(L, _p(tokens=0), i5=0) == 1 and _fwd(L, _p(tokens=0), i1=0) == 1
    assert _append(L, _p(tokens=0, cache_type=1), i7=0) == 1
    assert _append(L, _p(tokens=0), i5=FAKE + 8) == 3


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, torch.float8_e4m3fn])
def test_step_without_a_token(dtype):
    dev = torch.device("cuda:0")
    kc, vc, ks, vs = A.attn_cache_empty(4, 2, 16, 64, dtype=dtype, device=dev)
    before = [t.view(torch.uint8).clone() for t in (kc, vc)]
    err = torch.zeros(1, dtype=torch.int32, device=dev)
    kw = dict(page_table=torch.arange(4, dtype=torch.int32, device=dev).view(2, 2), max_new=1, k_scale=ks, v_scale=vs,
              seqlens_kv=torch.tensor([20, 3], dtype=torch.int32, device=dev),
              cu_seqlens=torch.zeros(3, dtype=torch.int32, device=dev), error_word=err)
    q, k = torch.empty(0, 4, 64, dtype=BF, device=dev), torch.empty(0, 2, 64, dtype=BF, device=dev)
    got = A.attn_cache_append(q, k, k, kc, vc, **kw)
    o, lse = A.attn_cache_fwd(got, kc, vc, **kw)
    torch.cuda.synchronize()
    assert got.shape == (0, 4, 64) and o.shape == (0, 4, 64) and lse.shape == (4, 0) and int(err.item()) == 0
    for a, b in zip(before, (kc, vc)):
        assert torch.equal(a, b.view(torch.uint8))
