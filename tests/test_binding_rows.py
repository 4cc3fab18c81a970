"""What the binding passes on for the calls around the decode step, and what it refuses, without a GPU:
a stand-in library records the packed arguments, and tensors live on the CPU (device index -1)."""

import pytest
import torch

from mla_latent_kv_28_b200 import binding

BF, F32 = torch.bfloat16, torch.float32
CALLS = {"mla_add_norm_q8": binding.NORM_ARGS, "mla_quantize_rows": binding.QUANTIZE_ARGS,
         "mla_linear_q8": binding.LINEAR_ARGS, "mla_append_rows": binding.ROWS_ARGS,
         "mla_append_rows_fp8": binding.ROWS_ARGS}


class Library:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(h, args, stream):
            self.calls.append((name, CALLS[name].unpack(args), stream))
            return binding.MLA_OK
        return call


@pytest.fixture
def handle():
    h = object.__new__(binding.MlaDecode)
    h._lib, h._h, h.device, h.q_len = Library(), None, -1, 1
    h.cfg = binding.make_config(1, 8, 100)
    h._here = lambda stream: 77
    return h


def test_norm_arguments(handle):
    x, g = torch.zeros((3, 48), dtype=BF)[:, :40], torch.zeros(40, dtype=BF)
    res = torch.zeros((3, 41))[:, 1:]
    codes, scales, out, y = handle.add_norm_q8(x, g, res, eps=0.5, want_y=True)
    assert codes.shape == (3, 40) and codes.stride() == (48, 1) and codes.dtype == torch.int8
    assert scales.shape == (3,) and out.dtype == F32 and out.stride() == (40, 1) and y.dtype == BF
    assert handle._lib.calls == [("mla_add_norm_q8", (
        3, 40, 0, x.data_ptr(), 48, res.data_ptr(), 41, out.data_ptr(), 40, g.data_ptr(), y.data_ptr(), 40,
        codes.data_ptr(), 48, scales.data_ptr(), 1, 0.5), 77)]
    handle.add_norm_q8(x.float(), g)
    assert handle._lib.calls[1][1][2] == 1 and handle._lib.calls[1][1][5:9] == (0, 0, 0, 0)
    assert handle._lib.calls[1][1][10] == 0   # no y
    same = handle.add_norm_q8(x, g, out, residual_out=out, y=x, codes=codes, scales=scales)
    assert same[0] is codes and same[1] is scales and same[2] is out and same[3] is x
    args = handle._lib.calls[2][1]
    assert args[5] == args[7] == out.data_ptr() and args[3] == args[10] == x.data_ptr()


def test_linear_arguments(handle):
    a, w = torch.zeros((2, 32), dtype=torch.int8)[:, :20], torch.zeros((5, 64), dtype=torch.int8)[:, :20]
    sa, sw = torch.zeros(2), torch.zeros(5)
    out = handle.linear_q8(a, sa, w, sw, out_dtype=F32)
    wide = torch.zeros((2, 9), dtype=BF)
    handle.linear_q8(a, sa, w, sw, out=wide[:, 3:8])
    (_, first, _), (_, second, _) = handle._lib.calls
    assert first == (2, 20, 5, 1, a.data_ptr(), 32, sa.data_ptr(), w.data_ptr(), 64, sw.data_ptr(), out.data_ptr(), 5)
    assert second[3] == 0 and second[10:] == (wide.data_ptr() + 6, 9)
    one = torch.zeros((1, 20), dtype=torch.int8)   # one row: any stride of 16 bytes will do
    handle.linear_q8(one, torch.zeros(1), w, sw)
    assert handle._lib.calls[2][1][5] == 32


def test_append_arguments(handle):
    x = torch.zeros((6, 2112))[:, 1536:]
    g, cache = torch.zeros(512, dtype=BF), torch.zeros((2, 120, 640), dtype=BF)[:, :, :576]
    lens, starts = torch.zeros(2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    assert handle.append_rows(x, g, cache, lens, starts) is cache
    p = cache.data_ptr()
    name, args, _ = handle._lib.calls[0]
    assert name == "mla_append_rows"
    assert args[:3] == (2, 6, 1) and args[4:] == (x.data_ptr(), 2112, g.data_ptr(), p, p + 1024, 0, 640, 120,
                                                  lens.data_ptr(), starts.data_ptr(), 0, 0, 0)
    handle.cfg = binding.make_config(1, 8, 100, page_size=64)
    codes, exps = torch.zeros((9, 64, 576), dtype=torch.uint8), torch.zeros((9, 64), dtype=torch.int8)
    table = torch.zeros((2, 3), dtype=torch.int32)
    handle.append_rows_fp8(x, g, codes, exps, lens, starts, table)
    name, args, _ = handle._lib.calls[1]
    assert name == "mla_append_rows_fp8"
    assert args[7:] == (codes.data_ptr(), 0, exps.data_ptr(), 576, 0, lens.data_ptr(), starts.data_ptr(),
                        table.data_ptr(), 3, 9)


def test_no_rows_make_no_call(handle):
    handle.quantize_rows(torch.zeros((0, 8)))
    handle.add_norm_q8(torch.zeros((0, 8)), torch.zeros(8, dtype=BF))
    handle.linear_q8(torch.zeros((0, 16), dtype=torch.int8), torch.zeros(0), torch.zeros((3, 16), dtype=torch.int8), torch.zeros(3))
    handle.append_rows(torch.zeros((0, 576)), torch.zeros(512, dtype=BF), torch.zeros((1, 100, 576), dtype=BF),
                       torch.zeros(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32))
    assert handle._lib.calls == []


def refused(handle, calls):
    for i, call in enumerate(calls):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")
    assert handle._lib.calls == []


def test_norm_refusals(handle):
    x, g = torch.zeros((4, 64), dtype=BF), torch.zeros(64, dtype=BF)
    n = handle.add_norm_q8
    refused(handle, [
        lambda: n(x.half(), g), lambda: n(x[0], g), lambda: n(x.t(), g), lambda: n(x[None], g),
        lambda: n(x[:1].expand(4, 64), g), lambda: n(torch.zeros(4 * 32 + 32).as_strided((4, 64), (32, 1)), g),
        lambda: n(x, g[:63]), lambda: n(x, g.float()), lambda: n(x, torch.zeros(128, dtype=BF)[::2]),
        lambda: n(x, g, x[:3]), lambda: n(x, g, x.half()), lambda: n(x, g, x.t()), lambda: n(x, g, residual_out=x),
        lambda: n(x, g, x, residual_out=x.float()), lambda: n(x, g, y=x.float()), lambda: n(x, g, y=x[:2]),
        lambda: n(x, g, codes=torch.zeros((4, 63), dtype=torch.int8)), lambda: n(x, g, codes=x),
        lambda: n(x, g, scales=torch.zeros(3)), lambda: n(x, g, scales=torch.zeros(8)[::2]),
    ])


def test_linear_refusals(handle):
    a, w, sa, sw = torch.zeros((4, 32), dtype=torch.int8), torch.zeros((8, 32), dtype=torch.int8), torch.zeros(4), torch.zeros(8)
    f = handle.linear_q8
    refused(handle, [
        lambda: f(a.float(), sa, w, sw), lambda: f(a[0], sa, w, sw), lambda: f(a.t(), sa, w, sw), lambda: f(a, sa, w[:, :16], sw),
        lambda: f(a, sa[:3], w, sw), lambda: f(a, sa, w, sw[:3]), lambda: f(a, sa.double(), w, sw), lambda: f(a, sa, w.float(), sw),
        lambda: f(a, sa, w, sw, out_dtype=torch.float16), lambda: f(a, sa, w, sw, out=torch.zeros((4, 9))),
        lambda: f(a, sa, w, sw, out=torch.zeros((8, 4)).t()), lambda: f(a, sa, w, sw, out=torch.zeros((4, 8), dtype=torch.half)),
        lambda: f(a, sa[:, None], w, sw),
    ])


def test_append_refusals(handle):
    x, g, cache = torch.zeros((5, 576)), torch.zeros(512, dtype=BF), torch.zeros((2, 100, 576), dtype=BF)
    lens, starts = torch.zeros(2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    codes, exps = torch.zeros((2, 100, 576), dtype=torch.uint8), torch.zeros((2, 100), dtype=torch.int8)
    table = torch.zeros((2, 2), dtype=torch.int32)
    f, q = handle.append_rows, handle.append_rows_fp8
    refused(handle, [
        lambda: f(x[:, :575], g, cache, lens, starts), lambda: f(x.half(), g, cache, lens, starts),
        lambda: f(x, g[:511], cache, lens, starts), lambda: f(x, g.float(), cache, lens, starts),
        lambda: f(x, g, cache.float(), lens, starts), lambda: f(x, g, cache[0], lens, starts),
        lambda: f(x, g, cache[:, :99], lens, starts), lambda: f(x, g, cache[:1], lens, starts),
        lambda: f(x, g, cache[:, :, :575], lens, starts), lambda: f(x, g, codes, lens, starts),
        lambda: f(x, g, cache, lens.long(), starts), lambda: f(x, g, cache, lens[None], starts),
        lambda: f(x, g, cache, lens, starts[:2]), lambda: f(x, g, cache, lens, starts.float()),
        lambda: f(x, g, cache, lens, starts, table),          # pages on a contiguous handle
        lambda: q(x, g, cache, exps, lens, starts), lambda: q(x, g, codes, exps[:, :99], lens, starts),
        lambda: q(x, g, codes, exps.to(torch.uint8), lens, starts),
        lambda: f(x, g, torch.zeros(2 * 100 * 576 + 600, dtype=BF).as_strided((2, 100, 576), (57608, 576, 1)), lens, starts),
    ])
    handle.cfg = binding.make_config(1, 8, 100, page_size=64)
    pages = torch.zeros((7, 64, 576), dtype=BF)
    refused(handle, [
        lambda: f(x, g, pages[:, :63], lens, starts, table), lambda: f(x, g, pages, lens, starts, table.long()),
        lambda: f(x, g, pages, lens, starts, table[:1]), lambda: f(x, g, pages, lens, starts, table[0]),
        lambda: f(x, g, pages, lens, starts, torch.zeros((2, 4), dtype=torch.int32)[:, ::2]),
        lambda: f(x, g, pages[::2], lens, starts, table),
    ])


def test_tensors_of_another_device_are_refused(handle):
    handle.device = 0
    x, g, lens = torch.zeros((2, 576)), torch.zeros(512, dtype=BF), torch.zeros(2, dtype=torch.int32)
    a, s = torch.zeros((2, 16), dtype=torch.int8), torch.zeros(2)
    refused(handle, [
        lambda: handle.add_norm_q8(x, torch.zeros(576, dtype=BF)), lambda: handle.quantize_rows(x),
        lambda: handle.linear_q8(a, s, a, s), lambda: handle.append_rows(x, g, torch.zeros((2, 100, 576), dtype=BF), lens),
    ])


def test_streams_of_another_device_are_refused(handle):
    class Stream:
        device, cuda_stream = torch.device("cuda", 3), 5
    a, s = torch.zeros((2, 16), dtype=torch.int8), torch.zeros(2)
    refused(handle, [
        lambda: handle.add_norm_q8(torch.zeros((2, 16)), torch.zeros(16, dtype=BF), stream=Stream()),
        lambda: handle.quantize_rows(torch.zeros((2, 16)), stream=Stream()),
        lambda: handle.linear_q8(a, s, a, s, stream=Stream()),
    ])
