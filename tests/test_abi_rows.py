"""Argument checks of the calls around the decode step without a GPU (CPU only). The checks read
nothing of a handle but its configuration, its first member, so a zeroed block that starts with one
stands in for it; a call that passes every check ends at the device, which is absent."""

import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

from mla_latent_kv_28_b200 import binding

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="the stand-in handle must never reach a GPU")

OK, ARG, UNSUPPORTED, CUDA = binding.MLA_OK, binding.MLA_ERR_INVALID_ARG, binding.MLA_ERR_UNSUPPORTED, binding.MLA_ERR_CUDA
P = 0x10000   # an aligned address; nothing reads it


@pytest.fixture(scope="module")
def lib():
    from mla_latent_kv_28_b200 import build
    build.build()
    return binding.load_library()


def stand_in(**kw):
    block = (ctypes.c_char * 8192)()
    cfg = binding.make_config(16, 8, 300, **kw)
    ctypes.memmove(block, ctypes.byref(cfg), ctypes.sizeof(cfg))
    return block


def call(fn, layout, names, defaults, **kw):
    args = dict(defaults, **kw)
    h, stream = args.pop("h"), args.pop("stream")
    packed = None if args.get("args", 0) is None else layout.pack(*[args[n] or 0 for n in names])
    return fn(None if h is None else ctypes.addressof(h), packed, stream)


def test_structs_are_packed_as_declared(lib):
    """The binding's layouts against the header's, compiled."""
    gcc = shutil.which("gcc")
    if gcc is None:
        pytest.skip("gcc not available")
    names = {"mla_add_norm_q8_t": binding.NORM_ARGS, "mla_quantize_rows_t": binding.QUANTIZE_ARGS,
             "mla_linear_q8_t": binding.LINEAR_ARGS, "mla_append_rows_t": binding.ROWS_ARGS}
    text = open(os.path.join(os.path.dirname(__file__), "..", "include", "mla_decode.h")).read()
    kinds = {"int64_t": "q", "int32_t": "i", "float": "f"}
    for name, layout in names.items():
        fields = re.findall(r"typedef struct \{([^}]*)\} " + name, text)[0]
        fields = re.sub(r"/\*.*?\*/", "", fields)
        want = "".join("Q" if "*" in f else kinds[f.split()[0]] for f in fields.split(";") if f.strip())
        assert want == layout.format, name
    source = '#include "mla_decode.h"\n' + "".join(
        f"_Static_assert(sizeof({n}) == {layout.size}, \"{n}\");\n" for n, layout in names.items())
    run = subprocess.run([gcc, "-xc", "-fsyntax-only", "-I", os.path.join(os.path.dirname(__file__), "..", "include"), "-"],
                         input=source, text=True, capture_output=True)
    assert run.returncode == 0, run.stderr


NORM = ["n_rows", "d", "x_type", "x", "x_stride", "residual", "residual_stride", "residual_out",
        "residual_out_stride", "gamma", "y", "y_stride", "codes", "codes_stride", "scales", "residual_type", "eps"]
NORM_OK = dict(n_rows=4, d=64, x=P, x_type=0, x_stride=64, residual=P, residual_stride=64, residual_out=P,
               residual_out_stride=64, residual_type=1, gamma=P, eps=1e-6, y=P, y_stride=64, codes=P,
               codes_stride=64, scales=P, stream=None)


@pytest.mark.parametrize("change,status", [
    ({}, CUDA), ({"n_rows": 0}, OK), ({"residual": None, "residual_out": None, "residual_type": 9}, CUDA),
    ({"y": None}, CUDA), ({"codes": None, "scales": None}, CUDA), ({"codes": P + 1, "codes_stride": 65}, CUDA),
    ({"x": P + 2, "x_stride": 65}, CUDA), ({"d": 16384, **{f"{n}_stride": 16384 for n in ("x", "residual", "residual_out", "y", "codes")}}, CUDA),
    ({"args": None}, ARG), ({"h": None}, ARG), ({"x": None}, ARG), ({"gamma": None}, ARG), ({"scales": None}, ARG), ({"codes": None}, ARG),
    ({"y": None, "codes": None, "scales": None}, ARG), ({"residual_out": None}, ARG), ({"residual": None}, ARG),
    ({"n_rows": -1}, ARG), ({"d": 0}, ARG), ({"x_type": 2}, ARG), ({"residual_type": -1}, ARG), ({"x_stride": 63}, ARG),
    ({"residual_stride": 63}, ARG), ({"residual_out_stride": 1}, ARG), ({"y_stride": 0}, ARG), ({"codes_stride": 63}, ARG),
    ({"x": P + 1}, ARG), ({"residual": P + 2}, ARG), ({"gamma": P + 1}, ARG), ({"y": P + 1}, ARG), ({"scales": P + 2}, ARG),
    ({"eps": -1.0}, ARG), ({"eps": float("inf")}, ARG), ({"eps": float("nan")}, ARG),
    ({"d": 16385, **{f"{n}_stride": 16385 for n in ("x", "residual", "residual_out", "y", "codes")}}, UNSUPPORTED),
    ({"n_rows": 2 ** 31}, UNSUPPORTED),
])
def test_add_norm_q8(lib, change, status):
    assert call(lib.mla_add_norm_q8, binding.NORM_ARGS, NORM, dict(NORM_OK, h=stand_in()), **change) == status


QUANT = ["n_rows", "d", "x_type", "x", "x_stride", "codes", "codes_stride", "scales"]
QUANT_OK = dict(n_rows=4, d=64, x=P, x_type=1, x_stride=70, codes=P, codes_stride=64, scales=P, stream=None)


@pytest.mark.parametrize("change,status", [
    ({}, CUDA), ({"n_rows": 0}, OK), *[({n: None}, ARG) for n in ("args", "h", "x", "codes", "scales")],
    ({"d": -3}, ARG), ({"x_type": 7}, ARG), ({"x": P + 2}, ARG), ({"x_stride": 60}, ARG), ({"codes_stride": 60}, ARG),
])
def test_quantize_rows(lib, change, status):
    assert call(lib.mla_quantize_rows, binding.QUANTIZE_ARGS, QUANT, dict(QUANT_OK, h=stand_in()), **change) == status


LINEAR = ["n_rows", "k", "n", "out_type", "codes", "codes_stride", "scales", "w_codes", "w_stride", "w_scales", "out",
          "out_stride"]
LINEAR_OK = dict(n_rows=4, k=60, n=9, codes=P, codes_stride=64, scales=P, w_codes=P, w_stride=64, w_scales=P, out=P,
                 out_type=0, out_stride=9, stream=None)


@pytest.mark.parametrize("change,status", [
    ({}, CUDA), ({"n_rows": 0}, OK), ({"out": P + 2, "out_stride": 11}, CUDA), ({"n_rows": 500}, CUDA),
    ({"k": 131071, "codes_stride": 131072, "w_stride": 131072}, CUDA),
    *[({n: None}, ARG) for n in ("args", "h", "codes", "scales", "w_codes", "w_scales", "out")],
    ({"n_rows": -1}, ARG), ({"k": 0}, ARG), ({"n": 0}, ARG), ({"out_type": 2}, ARG), ({"codes_stride": 48}, ARG),
    ({"codes_stride": 72}, ARG), ({"w_stride": 72}, ARG), ({"out_stride": 8}, ARG), ({"codes": P + 8}, ARG),
    ({"w_codes": P + 4}, ARG), ({"out": P + 1}, ARG), ({"out_type": 1, "out": P + 2}, ARG), ({"scales": P + 1}, ARG),
    ({"k": 131072, "codes_stride": 131072, "w_stride": 131072}, UNSUPPORTED), ({"n_rows": 2 ** 20 + 1}, UNSUPPORTED),
    ({"n": 2 ** 20 + 1, "out_stride": 2 ** 21}, UNSUPPORTED), ({"codes_stride": 2 ** 32 + 16}, UNSUPPORTED),
])
def test_linear_q8(lib, change, status):
    assert call(lib.mla_linear_q8, binding.LINEAR_ARGS, LINEAR, dict(LINEAR_OK, h=stand_in()), **change) == status


ROWS = ["batch", "n_rows", "x_type", "eps", "x", "x_stride", "gamma", "c_kv", "k_r", "kv_exp", "row_stride",
        "seq_stride", "kv_lens", "row_starts", "page_table", "max_pages", "num_pages"]
ROWS_OK = dict(batch=3, n_rows=40, x=P, x_type=0, x_stride=576, gamma=P, eps=1e-6, c_kv=P, k_r=P + 1024, kv_exp=P + 1,
               row_stride=576, seq_stride=300, kv_lens=P, row_starts=P, page_table=None, max_pages=0, num_pages=0,
               stream=None)
ROWS_BAD = [
    *[({n: None}, ARG) for n in ("args", "h", "x", "gamma", "c_kv", "kv_lens")],
    ({"batch": 0}, ARG), ({"batch": 9}, ARG), ({"n_rows": -1}, ARG), ({"row_starts": None}, ARG), ({"x_type": 5}, ARG),
    ({"x_stride": 568}, ARG), ({"x_stride": 580}, ARG), ({"x": P + 8}, ARG), ({"gamma": P + 8}, ARG), ({"c_kv": P + 8}, ARG),
    ({"eps": -1.0}, ARG), ({"eps": float("inf")}, ARG), ({"kv_lens": P + 2}, ARG), ({"row_starts": P + 2}, ARG),
    ({"seq_stride": 299}, ARG), ({"row_stride": 580}, ARG), ({"row_stride": 500}, ARG), ({"page_table": P}, ARG),
]


@pytest.mark.parametrize("change,status", [
    ({}, CUDA), ({"n_rows": 0}, OK), ({"x_type": 1, "x_stride": 580}, CUDA), ({"row_stride": 640, "seq_stride": 400}, CUDA),
    ({"kv_exp": None}, CUDA), ({"k_r": None}, ARG), ({"k_r": P + 8}, ARG), *ROWS_BAD])
def test_append_rows(lib, change, status):
    assert call(lib.mla_append_rows, binding.ROWS_ARGS, ROWS, dict(ROWS_OK, h=stand_in()), **change) == status


@pytest.mark.parametrize("change,status", [
    ({}, CUDA), ({"n_rows": 0}, OK), ({"kv_exp": None}, ARG), ({"k_r": None}, CUDA), ({"row_stride": 584}, ARG),
    ({"row_stride": 592}, CUDA), ({"row_stride": 560}, ARG), *ROWS_BAD])
def test_append_rows_fp8(lib, change, status):
    assert call(lib.mla_append_rows_fp8, binding.ROWS_ARGS, ROWS, dict(ROWS_OK, h=stand_in()), **change) == status


@pytest.mark.parametrize("change,status", [
    ({}, CUDA), ({"page_table": None}, ARG), ({"max_pages": 4}, ARG), ({"num_pages": 0}, ARG), ({"page_table": P + 2}, ARG)])
def test_append_rows_paged(lib, change, status):
    defaults = dict(ROWS_OK, h=stand_in(page_size=64), page_table=P, max_pages=5, num_pages=2, seq_stride=0)
    assert call(lib.mla_append_rows, binding.ROWS_ARGS, ROWS, defaults, **change) == status
