"""A handle is made beside the device's running work: it waits for nobody else's."""

import pytest
import torch

from mla_latent_kv_28_b200 import binding

pytestmark = pytest.mark.gpu


def test_create_does_not_wait_for_other_work():
    """About a second of work is queued on the default stream; the handle is there before it ends, and
    its tables are whole for a stream that does not wait for the default one."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((5, 576), generator=gen, device="cuda")
    gamma = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    lens = torch.tensor([900], dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, 5], dtype=torch.int32, device="cuda")
    cache, want = (torch.zeros((1, 1000, 576), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    side = torch.cuda.Stream()
    with binding.MlaDecode(1, 1, 1000) as h:      # kernels and modules are loaded
        h.append_rows(x, gamma, want, lens, starts)
        h.check_device_errors()
        torch.cuda.synchronize()
        ended = torch.cuda.Event()
        torch.cuda._sleep(1000)
        torch.cuda.synchronize()
        torch.cuda._sleep(2_000_000_000)
        ended.record()
        other = binding.MlaDecode(1, 1, 1000)
        early = not ended.query()
        other.append_rows(x, gamma, cache, lens, starts, stream=side)
        side.synchronize()
        also_early = not ended.query()
        torch.cuda.synchronize()
        other.close()
    assert early and also_early
    assert torch.equal(cache, want) and bool((want != 0).any())
