"""append_rows_fp8 where the fp32 maximum of a row does not tell its exponent: latent and rotated values
a few fp32 steps from the border, at far positions, rows alone in a warp and two to a warp."""

import numpy as np
import pytest
import torch

import oracle
from mla_latent_kv_28_b200 import binding
from tests._borders import BORDER, EPS, border_rows, exponents, rows_in

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("yarn", [False, True])
def test_exponents_next_to_their_border(many, yarn):
    n = 32 * torch.cuda.get_device_properties(0).multi_processor_count + 1 if many else 501
    first = 100_000
    y = oracle.Yarn(factor=40.0, original_len=4096, alpha=1.0, beta=32.0, mscale_coef=0.0707) if yarn else None
    kw = dict(yarn_factor=40.0, yarn_original_len=4096, yarn_alpha=1.0, yarn_beta=32.0, yarn_mscale_coef=0.0707) if yarn else {}
    theta = oracle.rope_theta(64, 10000.0, y)
    x, gamma = border_rows(n, first, theta, 2 + many)
    rows = rows_in(np.float64, x, gamma, first, theta)
    want = exponents(rows)
    # the fp64 angle of a position p is off by p theta 2^-53 < 2^-36 here and there: rows that are no
    # farther from the border than that have no exponent to be held to
    clear = np.abs(np.abs(rows).max(axis=1) / BORDER - 1) > 2.0 ** -33
    assert clear.mean() > 0.99
    lens = torch.tensor([first + n], dtype=torch.int32, device=DEV)
    starts = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    pages = -(-(first + n) // 64)
    used = pages - first // 64
    table = torch.full((1, pages), -1, dtype=torch.int32, device=DEV)
    table[0, pages - used:] = torch.arange(used, dtype=torch.int32, device=DEV)
    codes = torch.zeros((used, 64, 576), dtype=torch.uint8, device=DEV)
    exps = torch.zeros((used, 64), dtype=torch.int8, device=DEV)
    with binding.MlaDecode(1, 1, first + n, page_size=64, **kw) as h:
        h.append_rows_fp8(torch.from_numpy(x).to(DEV), torch.from_numpy(gamma).to(torch.bfloat16).to(DEV), codes, exps,
                          lens, starts, table, eps=EPS)
        h.check_device_errors()
    got = exps.flatten()[first % 64:first % 64 + n].cpu().numpy().astype(np.int64)
    assert np.array_equal(got[clear], want[clear])
    assert (exponents(rows_in(np.float32, x, gamma, first, theta)) != want).sum() >= 10
