"""The bounds of token_reference against what the kernels do.

_relative counts the additions of 256 threads and references that rise once in a round of six vectors, which are the figures of
the kernel for more than 32 alternatives.  The kernel for fewer runs blocks of 128, 256 or 512 threads with rounds of five or
four.  Counted here for it, from the rules of its launch, is what a row's sum goes through:

  * additions, half a step u each: two a vector of eight bf16 elements to each partial sum, one a vector of four fp32 ones;
    one a rise, where the old largest element joins; fifteen more until one sum is left (a thread's halves 2, the element
    outside the vectors 1, the warp's 5, an own largest element 1, the parts' 1 + 5);
  * rises, an exponential and two products each: one a round but the first, one for the elements outside the vectors, one
    into the row's sum.

The bound's 160 additions and 6 rises beside the loops' leave room for the difference: nothing up to the headline vocabulary needs
more than it has.  Batches of some hundred bf16 rows of more than 870000 columns would need up to 2% more; none is tested.
"""

import math

import pytest

from test_policy_loss import SIZES as POLICY_SIZES
from test_token_logprobs import SIZES
from token_reference import EX2, U, _relative

SMS = 152


def _launch(N, V, bf16, n):
    """(threads, loads in a round, blocks a row) of the scoring kernel, n <= 32."""
    size, G = (2, 8) if bf16 else (4, 4)
    if N > 2 * SMS and V * size <= 64 * 1024:
        return 128, 5, 1
    if n and SMS < N <= 2 * SMS and V * size > 64 * 1024:
        return 512, 4, 1
    cs, fill = 1, 4 if n else 5
    while cs < 8 and N * cs * 2 <= fill * SMS and V >= 2 * cs * 256 * 4 * G:
        cs *= 2
    return 256, 5, cs


def _needed(N, V, bf16, n):
    """Relative error of the sum over the elements, without that of the exponents' arguments (counted by size elsewhere)."""
    threads, loads, cs = _launch(N, V, bf16, n)
    vectors = math.ceil(V / (8 if bf16 else 4) / cs)
    rounds = math.ceil(vectors / (threads * loads))
    additions = math.ceil(vectors / threads) * (2 if bf16 else 1) + rounds + 15
    rises = max(rounds - 1, 0) + 2
    return EX2 + additions * U + rises * (EX2 + 2 * U)


OTHERS = [(15000, 151936), (70001, 3), (70001, 5), (2000, 4003), (500, 151936), (700, 5000), (700, 100000), (20, 40000), (40 * 12, 20011), (20 * 12, 40009),
          (12, 151936), (30, 20011), (14, 30001), (13, 100001), (20, 500001), (16, 400001), (400, 1999), (200, 1001), (6, 1 << 20), (70, 32000)]


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("n", [0, 1, 32])
def test_bounds_cover_the_launches(n, bf16):
    for N, V in OTHERS + [s[:2] for s in SIZES] + POLICY_SIZES:
        assert _needed(N, V, bf16, n) <= _relative(V, bf16), (N, V)
    # every size up to the headline vocabulary, whatever the batch
    for N in (1, 20, 100, 160, 300, 400, 100000):
        for V in [1, 7, 100, 1000, 5000, 8192, 16384, 16385, 20000, 32000, 32768, 32769, 50001, 65536, 128256, 151936]:
            assert _needed(N, V, bf16, n) <= _relative(V, bf16), (N, V)


def test_where_they_end():
    assert 1.0 < _needed(4096, 1 << 20, True, 0) / _relative(1 << 20, True) < 1.02
    assert _needed(4096, 870000, True, 0) <= _relative(870000, True)
    assert _needed(4096, 1 << 20, False, 0) <= _relative(1 << 20, False)
