"""linear_q8 bit for bit against its definition: the integer sum (exact in fp64), one rounding to
fp32, one at each scale, one to the output's type."""

import numpy as np
import pytest
import torch

from mla_latent_kv_28_b200 import binding

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def handle():
    with binding.MlaDecode(1, 1, 64) as h:
        yield h
        h.check_device_errors()


def codes_of(rows, k, seed, pad=0, lo=-128):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randint(lo, 128, (rows, (k + 15) // 16 * 16 + pad), generator=g, device=DEV, dtype=torch.int8)[:, :k]


def scales_of(n, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.exp(torch.randn(n, generator=g, device=DEV)) * 0.01


def expected(a, sa, w, sw, dtype):
    acc = a.double() @ w.double().T     # integers under 2^31: exact
    return ((acc.float() * sw[None]) * sa[:, None]).to(dtype)


def same(a, b):
    bits = torch.int16 if a.dtype == BF else torch.int32
    return a.shape == b.shape and a.dtype == b.dtype and torch.equal(a.contiguous().view(bits), b.contiguous().view(bits))


SHAPES = [(1, 1, 1), (1, 64, 16), (1, 5120, 2112), (2, 128, 128), (3, 17, 5), (16, 256, 130), (17, 1000, 777),
          (33, 4096, 512), (64, 1536, 1024), (65, 129, 64), (100, 130, 96), (128, 16384, 256), (128, 64, 300),
          (129, 128, 32), (130, 64, 1), (200, 5120, 96), (256, 512, 256), (257, 1000, 300), (333, 1000, 777),
          (513, 2048, 2112), (1000, 640, 4096), (4096, 256, 4096), (5000, 130, 1000)]


@pytest.mark.parametrize("rows,k,n", SHAPES)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_shapes(handle, rows, k, n, dtype):
    a, w, sa, sw = codes_of(rows, k, 1), codes_of(n, k, 2), scales_of(rows, 3), scales_of(n, 4)
    out = handle.linear_q8(a, sa, w, sw, out_dtype=dtype)
    handle.check_device_errors()
    assert same(out, expected(a, sa, w, sw, dtype))


@pytest.mark.parametrize("rows,k,n", [(129, 5120, 33), (191, 9921, 65), (200, 16384, 130), (300, 9920, 64),
                                      (486, 10284, 417), (1025, 8192, 48), (2319, 11392, 17)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_long_sums_of_several_tiles_of_tokens(handle, rows, k, n, dtype):
    a, w, sa, sw = codes_of(rows, k, 31), codes_of(n, k, 32), scales_of(rows, 33), scales_of(n, 34)
    block = torch.full((rows + 2, n + 3), 7.0, dtype=dtype, device=DEV)
    handle.linear_q8(a, sa, w, sw, out=block[1:rows + 1, 1:n + 1])
    handle.check_device_errors()
    assert same(block[1:rows + 1, 1:n + 1], expected(a, sa, w, sw, dtype))
    block[1:rows + 1, 1:n + 1] = 7.0
    assert bool((block == 7.0).all())


@pytest.mark.parametrize("rows", [1, 7, 128, 129, 300])
def test_largest_sums(handle, rows):
    """The longest sum of the largest products, and of the largest negative ones."""
    k, n = 131071, 40
    a, w = codes_of(rows, k, 5), codes_of(n, k, 6)
    a[0] = -128
    w[0] = -128
    w[1] = 127
    sa, sw = scales_of(rows, 7), scales_of(n, 8)
    out = handle.linear_q8(a, sa, w, sw, out_dtype=F32)
    handle.check_device_errors()
    assert same(out, expected(a, sa, w, sw, F32))


@pytest.mark.parametrize("rows", [5, 200])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("pad", [1, 4, 8, 640])
def test_strides(handle, rows, dtype, pad):
    """Codes whose rows lie apart, an output inside a wider one; nothing outside it is written."""
    k, n = 320, 261
    a, w, sa, sw = codes_of(rows, k, 9, 64), codes_of(n, k, 10, 16), scales_of(rows, 11), scales_of(n, 12)
    whole = torch.full((rows + 2, n + pad), 3.0, dtype=dtype, device=DEV)
    out = whole[1:rows + 1, pad // 2:pad // 2 + n]
    handle.linear_q8(a, sa, w, sw, out=out)
    assert same(out, expected(a, sa, w, sw, dtype))
    mask = torch.ones_like(whole, dtype=torch.bool)
    mask[1:rows + 1, pad // 2:pad // 2 + n] = False
    assert bool((whole[mask] == 3).all())


@pytest.mark.parametrize("rows", [3, 150])
def test_codes_behind_a_row_do_not_count(handle, rows):
    """k inside wider rows: what stands behind a row's end is not summed."""
    k, n = 200, 48
    wide_a, wide_w = codes_of(rows, 256, 13), codes_of(n, 256, 14)
    a, w = wide_a[:, :k], wide_w[:, :k]
    sa, sw = scales_of(rows, 15), scales_of(n, 16)
    assert same(handle.linear_q8(a, sa, w, sw), expected(a, sa, w, sw, BF))


@pytest.mark.parametrize("rows", [4, 140])
def test_non_finite_and_zero_scales(handle, rows):
    k, n = 96, 70
    a, w, sa, sw = codes_of(rows, k, 17, lo=1), codes_of(n, k, 18, lo=1), scales_of(rows, 19), scales_of(n, 20)
    clean = handle.linear_q8(a, sa, w, sw, out_dtype=F32)
    sa[1], sa[2], sw[3], sw[5] = float("nan"), 0.0, float("inf"), 0.0
    out = handle.linear_q8(a, sa, w, sw, out_dtype=F32)
    assert bool(out[1].isnan().all()) and bool((out[2, 6:] == 0).all())
    assert bool(out[0, 3].isinf()) and bool((out[3:, 5] == 0).all())
    rest = [j for j in range(n) if j not in (3, 5)]
    assert torch.equal(out[3:][:, rest], clean[3:][:, rest]) and torch.equal(out[0, rest], clean[0, rest])


@pytest.mark.parametrize("rows", [3, 130])
def test_rows_far_apart(handle, rows):
    """Offsets of rows past 2^31 in the codes and, in values, in the output."""
    k, n = 200, 40
    far = (2 ** 31 // (rows - 1) // 16 + 4) * 16
    a = torch.zeros((rows - 1) * far + 256, dtype=torch.int8, device=DEV).as_strided((rows, k), (far, 1))
    a.copy_(codes_of(rows, k, 60))
    w, sa, sw = codes_of(n, k, 61), scales_of(rows, 62), scales_of(n, 63)
    out = torch.zeros((rows - 1) * far + n, dtype=BF, device=DEV).as_strided((rows, n), (far, 1))
    handle.linear_q8(a, sa, w, sw, out=out)
    assert same(out, expected(a, sa, w, sw, BF))


def test_no_rows(handle):
    w, sw = codes_of(8, 32, 21), scales_of(8, 22)
    assert handle.linear_q8(codes_of(0, 32, 23), torch.empty(0, device=DEV), w, sw).shape == (0, 8)


@pytest.mark.parametrize("rows", [1, 64, 700])
def test_quantised_product(handle, rows):
    """quantize_rows on both sides: off the real product by the two quantisations at most. With
    codes a, w exact to half a code, each product is off by s_a |w| / 2 + s_w |a| / 2 + s_a s_w / 4."""
    g = torch.Generator(device=DEV).manual_seed(24)
    x = torch.randn((rows, 512), generator=g, device=DEV)
    wt = torch.randn((96, 512), generator=g, device=DEV) * 0.05
    a, sa = handle.quantize_rows(x)
    w, sw = handle.quantize_rows(wt)
    out = handle.linear_q8(a, sa, w, sw, out_dtype=F32).double()
    ref = x.double() @ wt.double().T
    bound = 0.5 * sa[:, None] * wt.abs().sum(1)[None] + 0.5 * sw[None] * x.abs().sum(1)[:, None] + \
        0.25 * 512 * sa[:, None] * sw[None]
    assert bool(((out - ref).abs() <= bound.double() * 1.001).all())


def test_two_streams_and_graphs(handle):
    """Calls on two streams at once, and a captured one replayed with other inputs beside an eager one."""
    cases = []
    for i, (rows, k, n) in enumerate([(8, 2048, 512), (300, 512, 768)]):
        cases.append((codes_of(rows, k, 30 + i), scales_of(rows, 32 + i), codes_of(n, k, 34 + i), scales_of(n, 36 + i)))
    want = [expected(*c, BF) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(20):
        for i, c in enumerate(cases):
            outs[i].append(torch.empty_like(want[i]))
            handle.linear_q8(*c, out=outs[i][-1], stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(same(o, want[i]) for o in outs[i])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = [handle.linear_q8(*c) for c in cases]
    for c in cases:
        c[0].copy_(codes_of(c[0].shape[0], c[0].shape[1], 40))
    graph.replay()
    torch.cuda.synchronize()
    assert all(same(o, expected(*c, BF)) for o, c in zip(captured, cases))
    handle.check_device_errors()


def test_refusals(handle):
    a, w, sa, sw = codes_of(4, 64, 50), codes_of(8, 64, 51), scales_of(4, 52), scales_of(8, 53)
    for args in ((a.cpu(), sa, w, sw), (a.float(), sa, w, sw), (a, sa[:3], w, sw), (a, sa, w[:, :32], sw),
                 (a, sa.double(), w, sw), (a, sa, w, sw[:7]), (a[0], sa, w, sw), (a.t(), sa, w, sw)):
        with pytest.raises(ValueError):
            handle.linear_q8(*args)
    with pytest.raises(ValueError):
        handle.linear_q8(a, sa, w, sw, out=torch.empty((4, 9), device=DEV))
    with pytest.raises((ValueError, KeyError)):
        handle.linear_q8(a, sa, w, sw, out_dtype=torch.float16)
    odd = torch.zeros((4, 65), dtype=torch.int8, device=DEV)
    for args in ((odd[:, :64], sa, w, sw), (odd.view(-1)[1:257].view(4, 64), sa, w, sw)):
        with pytest.raises(binding.MlaError, match="INVALID_ARG"):
            handle.linear_q8(*args)
    long = torch.zeros((1, 131072), dtype=torch.int8, device=DEV)
    with pytest.raises(binding.MlaError, match="UNSUPPORTED"):
        handle.linear_q8(long, sa[:1], long, sw[:1])
    handle.check_device_errors()
