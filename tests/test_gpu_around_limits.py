"""The calls around the decode step at the ends of their ranges: the most rows and channels of a product,
millions of short rows, and counts of sequences around the look-up's powers of 32."""

import pytest
import torch

from mla_latent_kv_28_b200 import binding
from tests.test_gpu_append_rows import check as check_append
from tests.test_gpu_linear_q8 import codes_of, expected, same, scales_of
from tests.test_gpu_rows_q8 import check as check_rows, gamma_of, rows_of

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
MOST = 1 << 20


@pytest.fixture(scope="module")
def handle():
    with binding.MlaDecode(1, 1, 64) as h:
        yield h
        h.check_device_errors()


@pytest.mark.parametrize("rows,k,n", [(MOST, 16, 24), (MOST, 520, 9), (MOST - 1, 33, 40), (1, 48, MOST), (65, 16, MOST),
                                      (300, 130, MOST - 3)])
def test_the_largest_products(handle, rows, k, n):
    a, w, sa, sw = codes_of(rows, k, 1), codes_of(n, k, 2), scales_of(rows, 3), scales_of(n, 4)
    out = handle.linear_q8(a, sa, w, sw)
    step = 1 << 16
    for i in range(0, max(rows, n), step):   # by parts: the definition's fp64 sums are large
        if rows > n:
            assert same(out[i:i + step], expected(a[i:i + step], sa[i:i + step], w, sw, BF))
        else:
            assert same(out[:, i:i + step].contiguous(), expected(a, sa, w[i:i + step], sw[i:i + step], BF))


def test_products_past_the_limits_are_refused(handle):
    a = torch.zeros((MOST + 1, 16), dtype=torch.int8, device=DEV)
    s, one = torch.zeros(MOST + 1, device=DEV), torch.zeros((1, 16), dtype=torch.int8, device=DEV)
    for call in (lambda: handle.linear_q8(a, s, one, s[:1]), lambda: handle.linear_q8(one, s[:1], a, s)):
        with pytest.raises(binding.MlaError, match="UNSUPPORTED"):
            call()


@pytest.mark.parametrize("rows,d", [((1 << 22) + 3, 1), ((1 << 21) + 1, 3), (1_000_003, 8), (400_001, 24)])
@pytest.mark.parametrize("x_type", [BF, F32])
def test_millions_of_short_rows(handle, rows, d, x_type):
    x = rows_of(rows, d, x_type, 5)
    check_rows(handle, x)
    check_rows(handle, x, gamma_of(d), rows_of(rows, d, BF, 6))


@pytest.mark.parametrize("batch", [2, 31, 32, 33, 63, 64, 65, 1023, 1024])
@pytest.mark.parametrize("many", [False, True])
def test_counts_of_sequences(batch, many):
    """Some without rows, the last one among them or not; a padded tail; rows alone in a warp and two to one."""
    least = 32 * torch.cuda.get_device_properties(0).multi_processor_count + 1
    for empty_last in (False, True):
        new = [(b * 7 + 1) % 3 for b in range(batch)]
        new[0], new[-1] = 1, 0 if empty_last else 2
        if many:
            middle = batch // 2
            new[middle] += max(0, least - sum(new))
        cached = [(11 * b) % 100 for b in range(batch)]
        check_append(new, cached, True, many != empty_last, BF, tail=3, seed=200 + batch)
