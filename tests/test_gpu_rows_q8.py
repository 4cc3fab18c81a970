"""add_norm_q8 and quantize_rows against their definition: codes and the residual's sum exactly
(they depend on no rounding but the defined ones), scales and the normalised row to the rounding of
their fp32 statistics."""

import threading

import numpy as np
import pytest
import torch

from mla_latent_kv_28_b200 import binding

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24
# The sum of squares: at most 16 additions in a thread, 5 in a warp, 5 over the warps (26 u); the
# mean and eps 2 u; the root halves that (14 u); root and reciprocal 2 u; a product and a quotient
# more in a scale, two products in y (2 u).
STAT = 18 * U


@pytest.fixture(scope="module")
def handle():
    with binding.MlaDecode(1, 1, 64) as h:
        yield h


def rows_of(rows, d, dtype, seed, pad=0, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, d + pad), generator=g) * torch.exp(spread * torch.randn((rows, 1), generator=g))
    x[:, : d : max(1, d // 5)] *= 9.0
    return x.to(dtype).to(DEV)[:, :d]


def expected_codes(t):
    """t [rows, d] fp32 (numpy) -> codes and max|t| by the definition. The quotient of a 31-bit by a
    24-bit number lies at least 2^-33 off a border it is not on, so fp64 decides every border."""
    m = np.abs(t).max(axis=1, keepdims=True)
    fine = np.isfinite(m) & (m > 0)
    with np.errstate(all="ignore"):
        q = np.rint(t.astype(np.float64) * 127.0 / m.astype(np.float64))
    return np.where(fine, q, 0).astype(np.int8), m[:, 0]


def check(h, x, gamma=None, residual=None, eps=1e-6, want_y=True, **kw):
    if gamma is None:
        codes, scales = h.quantize_rows(x, **kw)
        residual_out = y = None
    else:
        res_before = None if residual is None else residual.clone()
        codes, scales, residual_out, y = h.add_norm_q8(x, gamma, residual, eps=eps, want_y=want_y, **kw)
    torch.cuda.synchronize()
    assert codes.dtype == torch.int8 and codes.shape == x.shape and scales.shape == x.shape[:1]
    r = x.float().cpu().numpy()
    if gamma is not None and residual is not None:
        r = r + res_before.float().cpu().numpy()
        want = torch.from_numpy(r).to(residual.dtype)
        assert torch.equal(residual_out.cpu(), want)
    t = r if gamma is None else r * gamma.float().cpu().numpy()[None]
    want_codes, m = expected_codes(t)
    assert np.array_equal(codes.cpu().numpy(), want_codes)
    rstd = np.ones(len(r))
    if gamma is not None:
        rstd = 1.0 / np.sqrt((r.astype(np.float64) ** 2).mean(axis=1) + eps)
    s = m.astype(np.float64) * rstd / 127.0
    assert np.all(np.abs(scales.cpu().numpy() - s) <= STAT * s)
    if want_y and gamma is not None:
        ref = r.astype(np.float64) * rstd[:, None] * gamma.double().cpu().numpy()[None]
        err = np.abs(y.double().cpu().numpy() - ref)
        assert np.all(err <= np.abs(ref) * (2.0 ** -8 + 2 * STAT) + 2.0 ** -134)
    return codes, scales, residual_out, y


def gamma_of(d, seed=3):
    return (1 + 0.1 * torch.randn(d, generator=torch.Generator().manual_seed(seed))).to(BF).to(DEV)


@pytest.mark.parametrize("rows,d", [(1, 1), (3, 7), (2, 8), (1, 64), (5, 100), (4, 256), (9, 1000), (64, 1536),
                                    (7, 2112), (33, 5120), (2, 5121), (3, 8192), (3, 8200), (2, 11111), (2, 16384),
                                    (1, 16383), (700, 48)])
@pytest.mark.parametrize("x_type,res_type", [(BF, None), (F32, None), (BF, BF), (BF, F32), (F32, BF), (F32, F32)])
def test_norm(handle, rows, d, x_type, res_type):
    x = rows_of(rows, d, x_type, 1)
    res = None if res_type is None else rows_of(rows, d, res_type, 2)
    check(handle, x, gamma_of(d), res)


@pytest.mark.parametrize("rows,d", [(1, 1), (3, 9), (17, 128), (5, 777), (40, 5120), (3, 16384), (2, 16383)])
@pytest.mark.parametrize("x_type", [BF, F32])
def test_quantize(handle, rows, d, x_type):
    check(handle, rows_of(rows, d, x_type, 5))


@pytest.mark.parametrize("pad", [1, 5, 8, 576])
def test_strides_and_offsets(handle, pad):
    """Rows that lie apart, start anywhere, and outputs of the caller's own strides."""
    rows, d = 6, 1536
    x = rows_of(rows, d, F32, 6, pad)
    res = rows_of(rows, d, BF, 7, pad)
    codes = torch.full((rows, d + pad), 99, dtype=torch.int8, device=DEV)
    y = torch.full((rows, d + pad), 7.0, dtype=BF, device=DEV)
    out = torch.full((rows, d + pad), 7.0, dtype=BF, device=DEV)
    scales = torch.empty(rows, device=DEV)
    check(handle, x, gamma_of(d), res, codes=codes[:, :d], y=y[:, :d], residual_out=out[:, :d], scales=scales)
    assert bool((codes[:, d:] == 99).all()) and bool((y[:, d:] == 7).all()) and bool((out[:, d:] == 7).all())
    flat = rows_of(rows, d + 8, BF, 8)
    check(handle, flat[:, 1:d + 1], gamma_of(d + 3)[3:], rows_of(rows, d + 1, F32, 9)[:, 1:])


def test_in_place(handle):
    """residual_out may be the residual, y may be x."""
    x, res = rows_of(5, 640, BF, 10), rows_of(5, 640, BF, 11)
    x2, res2 = x.clone(), res.clone()
    codes, scales, r, y = handle.add_norm_q8(x, gamma_of(640), res, want_y=True)
    c2, s2, r2, y2 = handle.add_norm_q8(x2, gamma_of(640), res2, residual_out=res2, y=x2)
    assert r2 is res2 and y2 is x2
    for a, b in ((codes, c2), (scales, s2), (r, r2), (y, y2)):
        assert torch.equal(a, b)


def test_borders_between_codes(handle):
    """Values on, just over and just under (j + 1/2) m / 127: ties go to the even code."""
    d = 1024
    m = np.float32(1.27)
    j = np.arange(-127, 127, dtype=np.float64)
    exact = ((j + 0.5) * float(m) / 127.0).astype(np.float32)
    t = np.concatenate([exact, np.nextafter(exact, np.float32(9)), np.nextafter(exact, np.float32(-9)), [m]])
    t = np.pad(t.astype(np.float32), (0, d - len(t)))
    ties = np.pad(np.concatenate([(j + 0.5), [127.0]]).astype(np.float32), (0, d - 255))   # m = 127: exact ties
    x = torch.from_numpy(np.stack([t, -t, ties, 2.0 ** -60 * ties, 2.0 ** 60 * ties])).to(DEV)
    check(handle, x)
    check(handle, x, torch.ones(d, dtype=BF, device=DEV), want_y=False)


def test_empty_zero_and_non_finite_rows(handle):
    d = 300
    x = rows_of(7, d, F32, 12)
    x[1] = 0.0
    x[2, 17] = float("inf")
    x[3, 299] = float("nan")
    x[4, 0] = -float("inf")
    x[5] = 0.0
    x[5, 5] = 1e-42     # a subnormal alone
    keep = [0, 1, 5, 6]
    for gamma in (None, gamma_of(d)):
        out = handle.quantize_rows(x) if gamma is None else handle.add_norm_q8(x, gamma)[:2]
        codes, scales = out
        assert bool(codes[2:5].eq(0).all()) and bool(scales[2:5].isnan().all())
        assert bool(codes[1].eq(0).all()) and float(scales[1]) == 0.0
        assert bool(scales[keep].isfinite().all())
        clean = handle.quantize_rows(x[keep].contiguous()) if gamma is None else \
            handle.add_norm_q8(x[keep].contiguous(), gamma)[:2]
        assert torch.equal(clean[0], codes[keep]) and torch.equal(clean[1], scales[keep])
    assert int(codes[5, 5]) == 127   # its own largest value
    empty = torch.empty((0, d), device=DEV)
    codes, scales, res, y = handle.add_norm_q8(empty, gamma_of(d), empty, want_y=True)
    assert codes.shape == (0, d) and scales.shape == (0,) and y.shape == (0, d) and res.shape == (0, d)


@pytest.mark.parametrize("factor", [1e-25, 1e-12, 1e18, 1e25])
def test_magnitudes_whose_squares_leave_fp32(handle, factor):
    x = (rows_of(3, 513, F32, 13) * factor).contiguous()
    check(handle, x, gamma_of(513), eps=0.0)


def test_eps_and_only_y(handle):
    x, g = rows_of(4, 384, BF, 14), gamma_of(384)
    check(handle, x, g, eps=0.7)
    y = torch.empty_like(x)
    args = binding.NORM_ARGS.pack(4, 384, 0, x.data_ptr(), 384, 0, 0, 0, 0, g.data_ptr(), y.data_ptr(), 384, 0, 0, 0, 0, 1e-6)
    assert handle._lib.mla_add_norm_q8(handle._h, args, torch.cuda.current_stream().cuda_stream) == binding.MLA_OK
    assert torch.equal(y, handle.add_norm_q8(x, g, want_y=True)[3])


def test_codes_do_not_depend_on_layout_or_run(handle):
    x, g = rows_of(11, 2048, F32, 15), gamma_of(2048)
    one = handle.add_norm_q8(x, g)
    wide = torch.empty((11, 2049), device=DEV)
    wide[:, 1:] = x
    other = handle.add_norm_q8(wide[:, 1:], g)
    again = handle.add_norm_q8(x, g)
    assert torch.equal(one[0], other[0]) and torch.equal(one[0], again[0]) and torch.equal(one[1], again[1])


def test_rows_more_than_32_bits_apart(handle):
    """Offsets of rows past 2^31 values, in the inputs and in the outputs."""
    far, d = 1_100_000_008, 640
    big = torch.zeros(2 * far + d, dtype=BF, device=DEV)
    x = big.as_strided((3, d), (far, 1))
    x.copy_(rows_of(3, d, BF, 25))
    codes = torch.zeros(2 * far + d, dtype=torch.int8, device=DEV).as_strided((3, d), (far, 1))
    want = handle.add_norm_q8(x.contiguous(), gamma_of(d), want_y=True)
    got = handle.add_norm_q8(x, gamma_of(d), codes=codes, y=x)   # in place, far apart
    assert torch.equal(want[0], codes) and torch.equal(want[1], got[1]) and torch.equal(want[3], x)


def test_calls_from_two_threads(handle):
    """The calls share nothing: two threads with a stream each, on one handle."""
    data = [(rows_of(300, 1536, BF, 26 + i), gamma_of(1536, 28 + i)) for i in range(2)]
    want = [handle.add_norm_q8(*a, want_y=True) for a in data]
    torch.cuda.synchronize()
    got = [[], []]

    def work(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(30):
                got[i].append(handle.add_norm_q8(*data[i], want_y=True))
        stream.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    for i in range(2):
        assert len(got[i]) == 30
        for out in got[i]:
            assert all(torch.equal(want[i][j], out[j]) for j in (0, 1, 3))


def test_other_stream_and_graph(handle):
    x, g, res = rows_of(8, 1536, BF, 16), gamma_of(1536), rows_of(8, 1536, F32, 17)
    want = handle.add_norm_q8(x, g, res, want_y=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = handle.add_norm_q8(x, g, res, want_y=True, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = handle.add_norm_q8(x, g, res, want_y=True)
        q = handle.quantize_rows(out[3])
    x.copy_(rows_of(8, 1536, BF, 18))
    graph.replay()
    want = handle.add_norm_q8(x, g, res, want_y=True)
    assert all(torch.equal(a, b) for a, b in zip(want, out))
    assert torch.equal(q[0], handle.quantize_rows(want[3])[0])


@pytest.mark.parametrize("call", ["norm", "quantize", "linear"])
def test_new_outputs_belong_to_the_stream_that_writes_them(handle, call):
    """Memory that the current stream has freed but still writes is not the other stream's output."""
    rows, d = 256, 1024
    x, g = rows_of(rows, d, BF, 31), gamma_of(d)
    codes, scales = handle.quantize_rows(x)
    run = {"norm": lambda s: handle.add_norm_q8(x, g, want_y=True, stream=s)[3],
           "quantize": lambda s: handle.quantize_rows(x, stream=s)[0],
           "linear": lambda s: handle.linear_q8(codes, scales, codes, scales, out_dtype=F32, stream=s)}[call]
    want = run(None).clone()
    big, s = torch.empty(1 << 28, device="cuda"), torch.cuda.Stream()
    torch.cuda.synchronize()
    taken = torch.empty_like(want)
    for _ in range(20):
        big.fill_(1.0)
    taken.fill_(5)
    del taken
    got = run(s)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_refusals(handle):
    x, g = rows_of(4, 64, BF, 19), gamma_of(64)
    for call in (lambda: handle.add_norm_q8(x.cpu(), g), lambda: handle.add_norm_q8(x.half(), g),
                 lambda: handle.add_norm_q8(x, g[:63]), lambda: handle.add_norm_q8(x, g.float()),
                 lambda: handle.add_norm_q8(x.t(), g), lambda: handle.add_norm_q8(x[0], g),
                 lambda: handle.add_norm_q8(x, g, x[:3]), lambda: handle.add_norm_q8(x, g, residual_out=x),
                 lambda: handle.add_norm_q8(x, g, y=x.float()), lambda: handle.quantize_rows(x[:1].expand(4, 64)),
                 lambda: handle.quantize_rows(x, scales=torch.empty(3, device=DEV))):
        with pytest.raises(ValueError):
            call()
    for call, name in ((lambda: handle.add_norm_q8(x, g, eps=-1.0), "INVALID_ARG"),
                       (lambda: handle.add_norm_q8(x, g, eps=float("nan")), "INVALID_ARG"),
                       (lambda: handle.quantize_rows(torch.empty((1, 16385), device=DEV)), "UNSUPPORTED")):
        with pytest.raises(binding.MlaError, match=name):
            call()
