"""One attention layer around the decode step as a server runs it: residual addition and norm into
int8, the fused down-projection, c^Q's norm and the two up-projections, the cache write of the other
576 columns, the decode step, and W^O. Every stage is checked against its definition on what the stage
before it left on the GPU, and the whole run, captured into a graph and replayed on other inputs,
against the same run call by call."""

import numpy as np
import pytest
import torch

import oracle
from mla_latent_kv_28_b200 import binding
from tests._parity import assert_close, f64
from tests.test_gpu_append_rows import expected_rows
from tests.test_gpu_linear_q8 import expected, same
from tests.test_gpu_rows_q8 import expected_codes

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
B, D, RANK, HEADS, PAGE = 13, 1024, 768, 16, 64
LENS = [1, 2, 63, 64, 65, 127, 128, 129, 200, 7, 1, 64, 190]


class Layer:
    def __init__(self, fp8, seed):
        g = torch.Generator().manual_seed(seed)
        self.fp8 = fp8
        self.h = binding.MlaDecode(HEADS, B, max(LENS), page_size=PAGE)
        pages = [-(-n // PAGE) for n in LENS]
        self.table = torch.full((B, max(pages)), -1, dtype=torch.int32)
        order = torch.randperm(sum(pages), generator=g)
        at = 0
        for b, n in enumerate(pages):
            self.table[b, :n] = order[at:at + n].to(torch.int32)
            at += n
        self.table = self.table.to(DEV)
        self.lens = torch.tensor(LENS, dtype=torch.int32, device=DEV)
        if fp8:
            self.cache = torch.randint(0, 0x70, (sum(pages), PAGE, 576), generator=g, dtype=torch.uint8).to(DEV)
            self.exps = torch.randint(-9, -5, (sum(pages), PAGE), generator=g, dtype=torch.int8).to(DEV)
        else:
            self.cache = torch.randn((sum(pages), PAGE, 576), generator=g).to(BF).to(DEV)
        self.gammas = [(1 + 0.1 * torch.randn(n, generator=g)).to(BF).to(DEV) for n in (D, RANK, 512)]
        weight = lambda n, k: self.h.quantize_rows((torch.randn((n, k), generator=g) / k ** 0.5).to(DEV))
        self.w_down, self.w_uq, self.w_qr = weight(RANK + 576, D), weight(HEADS * 128, RANK), weight(HEADS * 64, RANK)
        self.w_o = weight(D, HEADS * 128)
        self.w_uk, self.w_uv = ((torch.randn((HEADS, 128, 512), generator=g) / 23).to(BF).to(DEV) for _ in range(2))
        self.x, self.residual = self.draw(seed + 1)

    def draw(self, seed):
        g = torch.Generator().manual_seed(seed)
        return torch.randn((B, D), generator=g).to(BF).to(DEV), (3 * torch.randn((B, D), generator=g)).to(DEV)

    def run(self):
        h, s = self.h, {}
        s["a"], s["sa"], s["res"], _ = h.add_norm_q8(self.x, self.gammas[0], self.residual)
        s["down"] = h.linear_q8(s["a"], s["sa"], *self.w_down, out_dtype=F32)
        s["q"], s["sq"], _, _ = h.add_norm_q8(s["down"][:, :RANK], self.gammas[1])
        s["q_c"] = h.linear_q8(s["q"], s["sq"], *self.w_uq).view(B, HEADS, 128)
        s["q_r"] = h.linear_q8(s["q"], s["sq"], *self.w_qr).view(B, HEADS, 64)
        rows = s["down"][:, RANK:]
        if self.fp8:
            h.append_rows_fp8(rows, self.gammas[2], self.cache, self.exps, self.lens, None, self.table)
            q_abs = h.absorb_q(s["q_c"], s["q_r"], self.w_uk, self.lens)
            latent, _ = h.decode_attn_fp8(q_abs, self.cache, self.exps, self.lens, self.table)
            s["o"] = h.apply_wuv(latent, self.w_uv)
        else:
            h.append_rows(rows, self.gammas[2], self.cache, self.lens, None, self.table)
            s["o"] = h.step(s["q_c"], s["q_r"], self.w_uk, self.w_uv, self.cache, self.lens, self.table)
        s["oq"], s["so"] = h.quantize_rows(s["o"].view(B, HEADS * 128))
        s["out"] = h.linear_q8(s["oq"], s["so"], *self.w_o)
        return s

    def cache64(self):
        if not self.fp8:
            return f64(self.cache)
        values = self.cache.view(torch.float8_e4m3fn).double() * torch.exp2(self.exps.double())[..., None]
        return values.cpu().numpy()


@pytest.mark.parametrize("fp8", [False, True])
def test_layer_stage_by_stage(fp8):
    layer = Layer(fp8, 60)
    s = layer.run()
    layer.h.check_device_errors()
    g0, g1, g2 = (g.float().cpu().numpy() for g in layer.gammas)
    r = layer.x.float().cpu().numpy() + layer.residual.cpu().numpy()
    assert np.array_equal(s["res"].cpu().numpy(), r)
    assert np.array_equal(s["a"].cpu().numpy(), expected_codes(r * g0[None])[0])
    assert same(s["down"], expected(s["a"], s["sa"], *layer.w_down, F32))
    down = s["down"].cpu().numpy()
    assert np.array_equal(s["q"].cpu().numpy(), expected_codes(down[:, :RANK] * g1[None])[0])
    for name, w in (("q_c", layer.w_uq), ("q_r", layer.w_qr)):
        assert same(s[name].reshape(B, -1), expected(s["q"], s["sq"], *w, BF))
    pos = np.array(LENS) - 1
    ref, slack = expected_rows(s["down"][:, RANK:], layer.gammas[2], pos, oracle.rope_theta(64, 10000.0), 1e-6)
    table, cache = layer.table.cpu().numpy(), layer.cache64()
    got = np.stack([cache[table[b, p // PAGE], p % PAGE] for b, p in enumerate(pos)])
    if fp8:   # half a step of E4M3: 2^-4 of a value, 2^-10 of the row's scale
        scale = 2.0 ** np.array([layer.exps[table[b, p // PAGE], p % PAGE].item() for b, p in enumerate(pos)])[:, None]
        assert np.all(np.abs(got - ref) <= np.maximum(np.abs(ref) * 2.0 ** -4, scale * 2.0 ** -10) + 1.07 * slack)
    else:
        assert np.all(np.abs(got - ref) <= np.abs(ref) * 2.0 ** -8 + 1.01 * slack)
    heads = oracle.mla_decode_nonabsorbed(f64(s["q_c"]), f64(s["q_r"]), f64(layer.w_uk), f64(layer.w_uv), cache,
                                          np.array(LENS), oracle.default_scale(), 10000.0, table, PAGE)
    assert_close(f64(s["o"]), heads, "the heads' outputs")
    assert np.array_equal(s["oq"].cpu().numpy(), expected_codes(s["o"].float().view(B, -1).cpu().numpy())[0])
    assert same(s["out"], expected(s["oq"], s["so"], *layer.w_o, BF))
    layer.h.close()


@pytest.mark.parametrize("fp8", [False, True])
def test_layer_captured_and_replayed(fp8):
    layer, other = Layer(fp8, 61), Layer(fp8, 61)
    layer.run()
    layer.cache.copy_(other.cache)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer.run()
    for seed in (70, 71):
        for a in (layer, other):
            x, residual = a.draw(seed)
            a.x.copy_(x)
            a.residual.copy_(residual)
        graph.replay()
        want = other.run()
        layer.h.check_device_errors()
        for name in want:
            assert torch.equal(out[name], want[name]), name
        assert torch.equal(layer.cache.view(torch.uint8), other.cache.view(torch.uint8))
    layer.h.close()
    other.h.close()
