"""append_rows(_fp8) on rows that hold infinities or NaN: what the formula gives, the exponents as
append_kv_fp8 chooses them, and rows beside them as without them."""

import numpy as np
import pytest
import torch

import oracle
from mla_latent_kv_28_b200 import binding
from tests.test_gpu_append_rows import inputs

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
INF, NAN = float("inf"), float("nan")
ROWS, FIRST = 9, 3   # positions 3 .. 11 of one sequence


def special_rows(x_type):
    """Rows 0, 2, 6 and 8 as drawn; an infinity in the key part (1), a NaN in the latent part (3), a
    NaN in the key part (4), an infinity in the latent part (5), a negative one in the key part (7)."""
    x, gamma = inputs(ROWS, x_type, 51)
    x[1, 512 + 4] = INF
    x[3, 100] = NAN
    x[4, 575] = NAN
    x[5, 7] = INF
    x[7, 512 + 9] = -INF
    return x, gamma


def append(x, gamma, fp8):
    n = x.shape[0]
    lens = torch.tensor([FIRST + n], dtype=torch.int32, device=DEV)
    starts = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    cache = torch.zeros((1, 64, 576), dtype=torch.uint8 if fp8 else BF, device=DEV)
    exps = torch.full((1, 64), 99, dtype=torch.int8, device=DEV)
    with binding.MlaDecode(1, 1, 64) as h:
        if fp8:
            h.append_rows_fp8(x, gamma, cache, exps, lens, starts)
        else:
            h.append_rows(x, gamma, cache, lens, starts)
        h.check_device_errors()
    return cache[0, FIRST:FIRST + n].cpu(), exps[0, FIRST:FIRST + n].cpu()


def by_formula(x, gamma):
    """The rows in fp64; infinities and NaN go where the formula takes them."""
    v, g = x.double().cpu().numpy(), gamma.double().cpu().numpy()
    theta = oracle.rope_theta(64, 10000.0)
    with np.errstate(all="ignore"):
        c = v[:, :512] * (1 / np.sqrt((v[:, :512] ** 2).mean(axis=1, keepdims=True) + 1e-6)) * g
        a = (FIRST + np.arange(len(v)))[:, None] * theta[None]
        even, odd = v[:, 512::2], v[:, 513::2]
        k = np.stack([even * np.cos(a) - odd * np.sin(a), even * np.sin(a) + odd * np.cos(a)], axis=2)
    return np.concatenate([c, k.reshape(len(v), 64)], axis=1)


@pytest.mark.parametrize("x_type", [BF, F32])
def test_bf16_rows(x_type):
    x, gamma = special_rows(x_type)
    got, _ = append(x, gamma, False)
    want = by_formula(x, gamma)
    got = got.double().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(np.isinf(got), np.isinf(want))
    assert np.array_equal(np.sign(got[np.isinf(got)]), np.sign(want[np.isinf(want)]))
    clean, _ = append(inputs(ROWS, x_type, 51)[0], gamma, False)
    for r in (0, 2, 6, 8):
        assert np.array_equal(clean[r].double().numpy(), got[r])


@pytest.mark.parametrize("x_type", [BF, F32])
def test_quantised_rows(x_type):
    """A NaN is a NaN code and counts for no exponent; a row with an infinity has exponent 127, the
    infinity the largest code and every other value that is under 2^116 the code of 0."""
    x, gamma = special_rows(x_type)
    codes, exps = append(x, gamma, True)
    want = by_formula(x, gamma)
    assert [int(exps[r]) for r in (1, 7)] == [127, 127]
    values = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(values), np.isnan(want))
    for r in (1, 7):
        assert np.array_equal(values[r], np.where(np.isinf(want[r]), np.sign(want[r]) * 448.0, 0.0))
    for r in (3, 4, 5):
        fine = np.where(np.isnan(want[r]), 0.0, want[r])
        assert int(exps[r]) == oracle.fp8_row_exponent(fine)
        scaled = fine / 2.0 ** int(exps[r])
        # half a step of a normal or of a subnormal code, and the fp32 value's own error
        room = np.maximum(np.abs(scaled) * 2.0 ** -4, 2.0 ** -10) + 2.0 ** -19 * np.abs(scaled).max()
        assert np.all(np.abs(np.nan_to_num(values[r]) - scaled) <= room)
    clean, clean_exps = append(inputs(ROWS, x_type, 51)[0], gamma, True)
    for r in (0, 2, 6, 8):
        assert torch.equal(clean[r], codes[r]) and clean_exps[r] == exps[r]


def test_infinite_row_as_append_kv_fp8_writes_it():
    """The projection's sum leaves fp32 for one key value: both calls store the same row."""
    d, token = 512, 5
    hidden = torch.zeros((1, d), dtype=BF, device=DEV)
    hidden[0, 0], hidden[0, 300] = 2.0 ** 64, 1.0
    w_dkv, w_kr = torch.zeros((512, d), dtype=BF, device=DEV), torch.zeros((64, d), dtype=BF, device=DEV)
    g = torch.Generator().manual_seed(52)
    w_dkv[:, 300] = torch.randn(512, generator=g).to(BF).to(DEV)
    w_kr[:, 300] = torch.randn(64, generator=g).to(BF).to(DEV)
    w_kr[10, 0] = 2.0 ** 100          # 2^164
    gamma = torch.ones(512, dtype=BF, device=DEV)
    lens = torch.tensor([token + 1], dtype=torch.int32, device=DEV)
    caches = [torch.zeros((1, 64, 576), dtype=torch.uint8, device=DEV) for _ in range(2)]
    exps = [torch.full((1, 64), 99, dtype=torch.int8, device=DEV) for _ in range(2)]
    x = torch.cat([w_dkv[:, 300], w_kr[:, 300]]).float()[None]
    x[0, 512 + 10] = INF
    with binding.MlaDecode(1, 1, 64) as h:
        h.append_kv_fp8(hidden, w_dkv, w_kr, gamma, caches[0], exps[0], lens)
        h.append_rows_fp8(x, gamma, caches[1], exps[1], lens)
        h.check_device_errors()
    assert int(exps[0][0, token]) == 127 and torch.equal(exps[0], exps[1])
    assert torch.equal(caches[0], caches[1])


def test_smallest_exponent():
    """Rows whose exponent would lie under -126 get -126."""
    x = torch.zeros((3, 576), device=DEV)
    x[0, 512] = 2.0 ** -126
    x[1, 512], x[1, 514] = 1.75 * 2.0 ** -118, 2.0 ** -124       # -126 by itself
    x[2, 513] = -(2.0 ** -140)                                  # a subnormal alone
    gamma = torch.ones(512, dtype=BF, device=DEV)
    lens, starts = torch.ones(3, dtype=torch.int32, device=DEV), torch.arange(4, dtype=torch.int32, device=DEV)
    codes, exps = torch.zeros((3, 64, 576), dtype=torch.uint8, device=DEV), torch.zeros((3, 64), dtype=torch.int8, device=DEV)
    with binding.MlaDecode(1, 3, 64) as h:
        h.append_rows_fp8(x, gamma, codes, exps, lens, starts)   # position 0: the key part as it is
        h.check_device_errors()
    assert exps[:, 0].tolist() == [-126] * 3
    want = (x.double() * 2.0 ** 126).float().to(torch.float8_e4m3fn).float()   # 1; 448 and 4; 2^-14, nearest to 0
    assert torch.equal(codes[:, 0].view(torch.float8_e4m3fn).float(), want)
