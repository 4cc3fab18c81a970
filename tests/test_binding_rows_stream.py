"""The cache write of projected rows on streams, without a GPU: which stream is passed on, and that
streams of another device are refused as by the other calls around the decode step."""

import pytest
import torch

from mla_latent_kv_28_b200 import binding


class Library:
    def __init__(self):
        self.streams = []

    def __getattr__(self, name):
        return lambda h, args, stream: self.streams.append((name, stream)) or binding.MLA_OK


class Stream:
    def __init__(self, index, value):
        self.device, self.cuda_stream = torch.device("cuda", index), value


@pytest.fixture
def handle():
    h = object.__new__(binding.MlaDecode)
    h._lib, h._h, h.device, h.q_len = Library(), None, -1, 1   # CPU tensors are on device -1
    h.cfg = binding.make_config(1, 8, 100)
    return h


def calls(h, rows, stream):
    x, g = torch.zeros((rows, 576)), torch.zeros(512, dtype=torch.bfloat16)
    lens, starts = torch.zeros(2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    codes, exps = torch.zeros((2, 100, 576), dtype=torch.uint8), torch.zeros((2, 100), dtype=torch.int8)
    return [lambda: h.append_rows(x, g, torch.zeros((2, 100, 576), dtype=torch.bfloat16), lens, starts, stream=stream),
            lambda: h.append_rows_fp8(x, g, codes, exps, lens, starts, stream=stream)]


@pytest.mark.parametrize("rows", [0, 5])
def test_streams_of_another_device_are_refused(handle, rows):
    for index, value in ((3, 5), (0, 0)):     # 0: the default stream has the same value on every device
        for call in calls(handle, rows, Stream(index, value)):
            with pytest.raises(ValueError, match="stream"):
                call()
    assert handle._lib.streams == []


def test_the_given_stream_is_passed_on(handle):
    class Here:
        class device:
            index = -1
        cuda_stream = 41
    for call in calls(handle, 5, Here):
        call()
    assert handle._lib.streams == [("mla_append_rows", 41), ("mla_append_rows_fp8", 41)]
