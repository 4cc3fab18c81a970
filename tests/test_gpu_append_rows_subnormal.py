"""append_rows(_fp8) without an eps on rows so small that 1 / rms leaves fp32."""

import pytest
import torch

from tests.test_gpu_append_rows import check, inputs

pytestmark = pytest.mark.gpu

F32 = torch.float32


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("factor", [1e-36, 1e-39, 1e-42])
def test_rows_whose_inverse_norm_leaves_fp32(fp8, factor):
    """Without an eps a row of subnormal values is normalised like any other."""
    x, gamma = inputs(5, F32, 53)
    x[:, :512] *= factor
    x[2], x[4, :512] = inputs(1, F32, 54)[0][0], 0.0
    x[4, 17] = 2.0 ** -149          # the smallest value alone
    check([5], [3], False, fp8, F32, seed=55, eps=0.0, x_gamma=(x, gamma))
