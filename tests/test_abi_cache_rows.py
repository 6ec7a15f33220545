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
