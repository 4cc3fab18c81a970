"""add_norm_q8 and quantize_rows over the widths, alignments and row counts at which another kernel takes
the rows, each against the definition (codes and sums exactly)."""

import pytest
import torch

from mla_latent_kv_28_b200 import binding
from tests.test_gpu_rows_q8 import check, gamma_of, rows_of

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
TYPES = [(BF, None), (F32, None), (BF, BF), (BF, F32), (F32, BF), (F32, F32)]


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


@pytest.fixture(scope="module")
def handle():
    with binding.MlaDecode(1, 1, 64) as h:
        yield h
        h.check_device_errors()


def norm_and_quantise(h, rows, d, x_type, res_type, seed, pad=0):
    x = rows_of(rows, d, x_type, seed, pad)
    check(h, x, gamma_of(d), None if res_type is None else rows_of(rows, d, res_type, seed + 1, pad))
    if res_type is None:
        check(h, x)


# two, four and one value at a time: up to 256, 512 and 1024 values a row for a warp, then for blocks with one
# vector a thread (bf16, up to 4096) or two
@pytest.mark.parametrize("d", [2, 10, 254, 258, 510, 514, 1022, 1026, 2050, 4094, 4098, 5122, 16382,
                               4, 12, 252, 260, 508, 516, 1020, 1028, 2052, 4092, 4100, 5124, 16380,
                               255, 257, 511, 513, 1023, 1025, 2049, 4095, 4097])
@pytest.mark.parametrize("x_type,res_type", TYPES)
def test_narrow_widths(handle, d, x_type, res_type):
    norm_and_quantise(handle, 5, d, x_type, res_type, 100 + d)


# eight at a time: eight and sixteen lanes and a warp a row, blocks with one vector (few rows) and two
@pytest.mark.parametrize("rows,d", [(1, 8), (67, 56), (67, 64), (35, 72), (35, 128), (9, 136), (9, 256), (9, 264), (9, 512),
                                    (9, 520), (9, 768), (9, 776), (9, 1024), (9, 1032), (9, 1280), (9, 8192), (9, 8200),
                                    (9, 16384), (301, 1032), (301, 1288), (301, 2048), (301, 4104)])
@pytest.mark.parametrize("x_type,res_type", TYPES)
def test_whole_vectors(handle, rows, d, x_type, res_type):
    norm_and_quantise(handle, rows, d, x_type, res_type, 200 + d)


@pytest.mark.parametrize("values", [2, 4, 6])
@pytest.mark.parametrize("x_type,res_type", TYPES)
def test_rows_that_start_between_vectors(handle, values, x_type, res_type):
    """A width of whole vectors whose rows start 2, 4 or 6 values off; codes likewise."""
    rows, d = 7, 1536
    wide = rows_of(rows, d + 8, x_type, 300 + values)
    x = wide[:, values:values + d]
    res = None if res_type is None else rows_of(rows, d, res_type, 310)
    codes = torch.full((rows, d + 8), 99, dtype=torch.int8, device=DEV)
    check(handle, x, gamma_of(d), res, codes=codes[:, values:values + d])
    assert bool((codes[:, :values] == 99).all()) and bool((codes[:, values + d:] == 99).all())
    check(handle, x)


# Five vectors a lane: 1025 to 1280 values and 32 rows for each SM; the last block's groups lie behind the rows.
@pytest.mark.parametrize("d", [1032, 1200, 1280])
@pytest.mark.parametrize("x_type", [BF, F32])
def test_five_vectors_a_lane(handle, d, x_type):
    norm_and_quantise(handle, 32 * sms() + 1, d, x_type, None, 400 + d)
    x = rows_of(32 * sms() + 3, d, x_type, 410, pad=8)
    codes = torch.full((x.shape[0], d + 16), 99, dtype=torch.int8, device=DEV)
    check(handle, x, codes=codes[:, :d])
    assert bool((codes[:, d:] == 99).all())


# Four vectors a thread: from 2048 values, 81920 values for each SM; the last vectors of a row partly filled.
@pytest.mark.parametrize("d", [2048, 2056, 5128, 8192, 16376])
@pytest.mark.parametrize("x_type,res_type", [(BF, None), (F32, None), (BF, BF)])
def test_four_vectors_a_thread(handle, d, x_type, res_type):
    rows = -(-sms() * 81920 // d) + 1
    norm_and_quantise(handle, rows, d, x_type, res_type, 500 + d)


@pytest.mark.parametrize("res_type", [None, BF])
def test_four_vectors_a_thread_with_special_rows(handle, res_type):
    """Apart rows, in place, with zeros, infinities, NaN and magnitudes whose squares leave fp32."""
    d = 4104
    rows = -(-sms() * 81920 // d) + 3
    wide = rows_of(rows, d + 8, BF, 600, 0)
    x, g = wide[:, :d], gamma_of(d)
    for r, factor in ((1, 0.0), (5, 1e-25), (6, 1e18), (rows - 1, 1e25)):
        x[r] *= factor
    res = None if res_type is None else (x * 0.5).clone()
    check(handle, x, g, res)
    want = handle.add_norm_q8(x, g, res, want_y=True)
    x[2, 17], x[7, d - 1], x[rows - 2, 0] = float("inf"), float("nan"), -float("inf")
    bad = torch.zeros(rows, dtype=torch.bool, device=DEV)
    bad[[2, 7, rows - 2]] = True
    got = handle.add_norm_q8(x, g, res, residual_out=res, y=x)
    assert got[3] is x and (res is None or got[2] is res)
    assert bool((got[0][bad] == 0).all()) and bool(got[1][bad].isnan().all())
    for a, b in zip(want, got):
        assert (a is None and b is None) or torch.equal(a[~bad], b[~bad])
