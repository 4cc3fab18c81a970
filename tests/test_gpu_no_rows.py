"""No rows are no error: the C calls of the cache write without row_starts, whatever q_len says."""

import pytest
import torch

from mla_latent_kv_28_b200 import binding

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("q_len", [1, 3])
@pytest.mark.parametrize("fp8", [False, True])
def test_append_rows_without_rows(q_len, fp8):
    x = torch.zeros((6, 576), dtype=torch.bfloat16, device="cuda")
    gamma = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    cache = torch.full((2, 64, 576), 3, dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda")
    exps = torch.full((2, 64), 3, dtype=torch.int8, device="cuda")
    lens = torch.tensor([5, 6], dtype=torch.int32, device="cuda")
    with binding.MlaDecode(1, 2, 64, q_len=q_len) as h:
        call = h._lib.mla_append_rows_fp8 if fp8 else h._lib.mla_append_rows
        p = cache.data_ptr()

        def status(n):
            args = binding.ROWS_ARGS.pack(2, n, 0, 1e-6, x.data_ptr(), 576, gamma.data_ptr(), p, 0 if fp8 else p + 1024,
                                          exps.data_ptr() if fp8 else 0, 576, 64, lens.data_ptr(), 0, 0, 0, 0)
            return call(h._h, args, torch.cuda.current_stream().cuda_stream)

        assert status(0) == binding.MLA_OK
        assert status(-1) == binding.MLA_ERR_INVALID_ARG and status(5) == binding.MLA_ERR_INVALID_ARG
        h.check_device_errors()
    assert bool((cache == 3).all()) and bool((exps == 3).all())
