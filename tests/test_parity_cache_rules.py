"""GPU tests of the bf16 cache's attention on both sides of the border between its two
kernels, each within its own rounding of P."""
import pytest

from _cache_bounds import answer
from _cache_util import Step, check
from test_parity_cache import run_fwd

pytestmark = pytest.mark.gpu

# (hq, hkv, sequences, bits of P): the kernel for few rows holds P in two bf16, 2^-16, the tcgen05 kernel in one, 2^-8
FEW, MANY = 16, 8


@pytest.mark.parametrize("D,hq,hkv,seqs,bits", [
    (64, 8, 2, [(900, 4), (50, 4), (300, 4)], FEW),                      # 16 rows each
    (128, 8, 2, [(900, 4), (50, 4), (300, 4)], FEW),
    (64, 8, 2, [(900, 8), (50, 1), (300, 1)] + [(77, 4)] * 2, FEW),      # 32 at most, 14 on average
    (64, 4, 1, [(2000, 8), (500, 4), (300, 4), (20, 4)], MANY),          # 32 at most, 20 on average
    (128, 8, 2, [(900, 5)] + [(300 + n, 2) for n in range(7)], FEW),     # 20 at most, 9 on average
    (128, 8, 2, [(900, 8), (50, 1), (300, 1)] + [(77, 1)] * 2, FEW),     # 32 at most, 9 on average
    (128, 4, 1, [(2000, 8), (500, 1), (300, 1), (20, 1)], MANY),         # 32 at most, 11 on average
    (64, 8, 2, [(900, 5), (50, 5), (300, 5)], MANY),                     # 20 each
    (128, 8, 2, [(900, 5), (50, 5), (300, 5)], MANY),
    (64, 8, 2, [(900, 9)] + [(300 + n, 1) for n in range(20)], MANY),    # 36 at most
    (128, 8, 2, [(900, 9)] + [(300 + n, 1) for n in range(20)], MANY),
])
def test_each_kernel_within_its_own_rounding(D, hq, hkv, seqs, bits):
    s = Step("bf16", D, hq, hkv, 16, seqs, seed=91, pad_tokens=0)
    check(answer(s, bits), *run_fwd(s))
