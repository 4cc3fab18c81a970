"""add_norm_q8 without an eps on rows so small that 1 / rms leaves fp32: normalised like any other."""

import numpy as np
import pytest
import torch

from mla_latent_kv_28_b200 import binding
from tests.test_gpu_rows_q8 import STAT, expected_codes, gamma_of, rows_of

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


# widths: eight lanes a row, a warp, odd ones, blocks with one and with two vectors a thread
@pytest.mark.parametrize("d", [64, 48, 777, 1024, 2049, 5120, 16384])
@pytest.mark.parametrize("x_type,res_type", [(BF, None), (F32, None), (F32, F32), (BF, BF)])
def test_subnormal_rows(d, x_type, res_type):
    x = rows_of(9, d, F32, 61)
    for r, factor in enumerate((1.0, 1e-30, 1e-38, 1e-39, 1e-40, 1e-41, 0.0, 0.0, 1.0)):
        x[r] *= factor
    x[6, d // 2] = 2.0 ** -149 if x_type == F32 else 2.0 ** -133    # the type's smallest value alone
    x[7, 3], x[7, 5] = 2.0 ** -130, -(2.0 ** -131)
    x, gamma = x.to(x_type), gamma_of(d)
    res = None if res_type is None else (x * 2).to(res_type)
    with binding.MlaDecode(1, 1, 64) as h:
        codes, scales, _, y = h.add_norm_q8(x, gamma, res, eps=0.0, want_y=True)
        h.check_device_errors()
    r = x.float().cpu().numpy()
    if res is not None:
        r = r + res.float().cpu().numpy()
    t = r * gamma.float().cpu().numpy()[None]
    want, m = expected_codes(t)
    assert np.array_equal(codes.cpu().numpy(), want)
    kept = m > 0     # (bf16 rounds some rows to zeros: codes and scale 0, and no 1 / rms)
    assert kept.sum() >= 8 and bool((scales.cpu()[torch.from_numpy(~kept)] == 0).all())
    r, t, m, y, scales = r[kept], t[kept], m[kept], y.cpu()[torch.from_numpy(kept)], scales.cpu()[torch.from_numpy(kept)]
    rstd = 1.0 / np.sqrt((r.astype(np.float64) ** 2).mean(axis=1))
    s = m.astype(np.float64) * rstd / 127.0
    assert np.all(np.abs(scales.double().numpy() - s) <= STAT * s)
    ref = t.astype(np.float64) * rstd[:, None]
    assert np.all(np.abs(y.double().numpy() - ref) <= np.abs(ref) * (2.0 ** -8 + STAT) + 2.0 ** -134)
