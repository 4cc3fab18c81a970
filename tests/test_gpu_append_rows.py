"""append_rows and append_rows_fp8 against the definition in fp64: the rows written, element by
element, every other cache row left bit for bit as it was."""

import numpy as np
import pytest
import torch

import oracle
from mla_latent_kv_28_b200 import binding
from mla_latent_kv_28_b200 import workloads as wl

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32
PAGE = 64
U = 2.0 ** -24
# Latent values: the sum of 512 squares takes 16 + 5 additions (21 u), eps 1 u, halved by the root
# (11 u), root and reciprocal 2 u, two products 2 u.
LATENT = 15 * U
# Rotated values: half a step of the fp32 turn (2^-26, times 2 pi), 2 steps of a sine of at most 1
# (2^-23), two products and a sum (3 u): under 2^-21 of |x0| + |x1|.
ROTATED = 2.0 ** -21


def inputs(rows, x_type, seed, pad=0, spread=0.5):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, 576 + pad), generator=g) * torch.exp(spread * torch.randn((rows, 1), generator=g))
    gamma = (1 + 0.1 * torch.randn(512, generator=g)).to(BF)
    return x.to(x_type).to(DEV)[:, :576], gamma.to(DEV)


def layout(new, cached, paged, seed, fp8, extra=0):
    """kv_lens, row_starts, page table and a cache with random bytes for these sequences."""
    g = torch.Generator().manual_seed(seed)
    lens = [a + b for a, b in zip(new, cached)]
    starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    longest = max(1, max(lens))
    if paged:
        pages = [-(-n // PAGE) for n in lens]
        order = torch.randperm(sum(pages) + 2, generator=g).tolist()
        table = torch.full((len(new), max(1, -(-longest // PAGE))), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(pages):
            table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
            at += n
        shape = (sum(pages) + 2, PAGE, 576)
    else:
        table, shape = None, (len(new), longest + extra, 576)
    if fp8:
        cache = torch.randint(0, 127, shape, generator=g, dtype=torch.uint8).to(DEV)
        exps = torch.randint(-9, 9, shape[:2], generator=g, dtype=torch.int8).to(DEV)
    else:
        cache, exps = torch.randn(shape, generator=g).to(BF).to(DEV), None
    return (torch.tensor(lens, dtype=torch.int32, device=DEV), torch.from_numpy(starts).to(DEV),
            None if table is None else table.to(DEV), cache, exps, longest)


def expected_rows(x, gamma, pos, theta, eps):
    x, gamma = x.double().cpu().numpy(), gamma.double().cpu().numpy()
    c = x[:, :512] / np.sqrt((x[:, :512] ** 2).mean(axis=1, keepdims=True) + eps) * gamma
    a = np.asarray(pos, dtype=np.float64)[:, None] * theta[None]
    e, o = x[:, 512::2], x[:, 513::2]
    k = np.stack([e * np.cos(a) - o * np.sin(a), e * np.sin(a) + o * np.cos(a)], axis=2).reshape(len(x), 64)
    size = np.repeat(np.abs(e) + np.abs(o), 2, axis=1)
    return np.concatenate([c, k], axis=1), np.concatenate([np.abs(c) * LATENT, size * ROTATED], axis=1)


def where(new, cached, table):
    """(first index, second index, position) of every row, in order."""
    out = []
    for b, (n, c) in enumerate(zip(new, cached)):
        for pos in range(c, c + n):
            out.append((b, pos, pos) if table is None else (int(table[b, pos // PAGE]), pos % PAGE, pos))
    return out


def check(new, cached, paged, fp8, x_type, pad=0, tail=0, seed=0, eps=1e-6, base=10000.0, spread=0.5, starts=True,
          q_len=1, extra=0, x_gamma=None):
    rows = sum(new)
    x, gamma = inputs(rows + tail, x_type, seed + 1, pad, spread) if x_gamma is None else x_gamma
    lens, row_starts, table, cache, exps, longest = layout(new, cached, paged, seed, fp8, extra)
    before, exps_before = cache.clone(), None if exps is None else exps.clone()
    with binding.MlaDecode(1, len(new), longest, page_size=PAGE if paged else 0, rope_base=base, q_len=q_len) as h:
        args = (lens, row_starts if starts else None, table)
        if fp8:
            got = h.append_rows_fp8(x, gamma, cache, exps, *args, eps=eps)
            assert got[0] is cache and got[1] is exps
        else:
            assert h.append_rows(x, gamma, cache, *args, eps=eps) is cache
        h.check_device_errors()
    at = where(new, cached, None if table is None else table.cpu())
    mask = torch.ones(cache.shape[:2], dtype=torch.bool, device=DEV)
    first, second = [a for a, _, _ in at], [b for _, b, _ in at]
    if at:
        mask[first, second] = False
    bits = torch.uint8 if fp8 else torch.int16
    assert torch.equal(cache.view(bits)[mask], before.view(bits)[mask])
    if fp8:
        assert torch.equal(exps[mask], exps_before[mask])
    if rows == 0:
        return
    theta = oracle.rope_theta(64, base) if base > 0 else np.zeros(32)
    ref, slack = expected_rows(x[:rows], gamma, [p for _, _, p in at], theta, eps)
    if not fp8:
        got = cache[first, second].double().cpu().numpy()
        assert np.all(np.abs(got - ref) <= np.abs(ref) * 2.0 ** -8 + 1.01 * slack + 2.0 ** -134)
        return
    e = exps[first, second].cpu().numpy().astype(np.int64)
    want_e = np.array([oracle.fp8_row_exponent(r) for r in ref])
    assert np.array_equal(e, want_e)
    codes = cache[first, second].view(torch.float8_e4m3fn).float().cpu().numpy().astype(np.float64)
    scaled, room = ref / 2.0 ** e[:, None], slack / 2.0 ** e[:, None]
    # half a step: 2^-4 of a normal value, 2^-10 of the subnormal ones
    assert np.all(np.abs(codes - scaled) <= np.maximum(np.abs(scaled) * 2.0 ** -4, 2.0 ** -10) + 1.07 * room)


LAYOUTS = {
    "one token": ([1], [0]),
    "one token, far": ([1], [9000]),
    "decode batch": ([1] * 70, [(37 * i) % 300 for i in range(70)]),
    "prompts": ([65, 128, 1, 63, 64], [0, 0, 0, 0, 0]),
    "ragged with nothing in between": ([0, 3, 0, 0, 130, 1, 0, 17, 0], [5, 60, 0, 64, 1, 127, 0, 200, 63]),
    "nothing": ([0, 0], [3, 0]),
    "one thousand sequences": ([i % 3 for i in range(1000)], [i % 70 for i in range(1000)]),
}


@pytest.mark.parametrize("name", list(LAYOUTS))
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("x_type", [BF, F32])
def test_layouts(name, paged, fp8, x_type):
    new, cached = LAYOUTS[name]
    check(new, cached, paged, fp8, x_type, seed=len(name))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("pad,tail", [(8, 0), (64, 5), (1536, 1)])
def test_strides_and_rows_behind_the_last(fp8, pad, tail):
    check([4, 0, 9], [3, 2, 1], True, fp8, F32, pad=pad, tail=tail, seed=21)
    check([4, 0, 9], [3, 2, 1], False, fp8, BF, pad=pad, tail=tail, seed=22, extra=7)


@pytest.mark.parametrize("fp8", [False, True])
def test_without_row_starts(fp8):
    """q_len rows per sequence, as the other calls of the handle take them."""
    check([1] * 5, [7, 0, 63, 64, 100], True, fp8, BF, seed=23, starts=False)
    check([4] * 3, [7, 0, 62], False, fp8, F32, seed=24, starts=False, q_len=4)


@pytest.mark.parametrize("fp8", [False, True])
def test_rope_off_eps_and_magnitudes(fp8):
    check([3, 2], [10, 20], False, fp8, F32, seed=25, base=0.0, eps=0.5)
    check([30], [131000], False, fp8, F32, seed=26, spread=3.0)
    x, gamma = inputs(6, F32, 27)
    for factor in (1e-22, 1e-3, 1e17):
        y = x.clone()
        y[:, :512] *= factor
        check([6], [1], False, fp8, F32, seed=28, eps=0.0, x_gamma=(y, gamma))


def test_zero_rows():
    """A row of zeros is written as zeros (exponent 0 where it is quantised)."""
    x, gamma = torch.zeros((2, 576), device=DEV), inputs(1, F32, 29)[1]
    for fp8 in (False, True):
        check([2], [3], False, fp8, F32, seed=30, x_gamma=(x, gamma))


def test_exponent_at_its_border():
    """The row's largest value on, just over and just under 448 * 2^e: the exponent is the
    definition's. Position 0 leaves the key part as it is, so the border is met exactly."""
    edge = np.float32(448.0)
    values = [edge, np.nextafter(edge, np.float32(0)), np.nextafter(edge, np.float32(999)), np.float32(7.0),
              np.nextafter(np.float32(7), np.float32(9)), np.float32(3.5), np.float32(1e-3)]
    x = torch.zeros((len(values), 576), device=DEV)
    x[:, :512] = torch.randn((len(values), 512), generator=torch.Generator().manual_seed(31)).to(DEV) * 0.1
    x[:, 512] = torch.tensor(values, device=DEV)
    gamma = torch.full((512,), 2.0 ** -6, dtype=BF, device=DEV)
    check([1] * len(values), [0] * len(values), False, True, F32, seed=32, x_gamma=(x, gamma))


def test_same_rows_as_append_kv():
    """The projection outside: append_rows of what append_kv projects gives its rows to a rounding
    of the projection's fp32 sum order (bf16 results may differ by one step)."""
    w = wl.make_workload(9, 16, ("uniform", 1, 300), page_size=64, seed=33, max_kv_len=300)
    inp = {k: v.to(DEV) for k, v in wl.draw_append_inputs(9, 512, seed=34).items()}
    g = w.to(DEV)
    other = g.cache.clone()
    with binding.MlaDecode(16, 9, 300, page_size=64, rope_base=w.rope_base) as h:
        h.append_kv(inp["hidden"], inp["w_dkv"], inp["w_kr"], inp["gamma"], g.cache, g.kv_lens, g.page_table)
        x = (inp["hidden"].double() @ torch.cat([inp["w_dkv"], inp["w_kr"]]).double().T).float()
        h.append_rows(x, inp["gamma"], other, g.kv_lens, None, g.page_table)
        h.check_device_errors()
    a, b = g.cache.nan_to_num().double(), other.nan_to_num().double()
    # fp32 sums of 512 products: off by 512 u of the products' magnitudes S at most; the norm passes
    # that on once through the value and once through the statistic; then two half steps of bf16
    size = (inp["hidden"].double().abs() @ torch.cat([inp["w_dkv"], inp["w_kr"]]).double().abs().T).max()
    rstd = 1 / x[:, :512].double().square().mean(dim=1).sqrt().min()
    room = 512 * U * size * max(1.0, float(rstd * inp["gamma"].double().abs().max())) * 2
    assert bool(((a - b).abs() <= 2.0 ** -7 * b.abs() + room + b.abs() * room).all())


def test_bad_rows_set_error_bits_and_the_others_are_written():
    """A kv_lens entry without room for its rows, one over max_kv_len, and a bad page: skipped."""
    new, cached = [3, 2, 2, 2], [0, 5, 100, 62]
    lens, starts, table, cache, _, _ = layout(new, cached, True, 35, False)
    x, gamma = inputs(9, F32, 36)
    good, before = cache.clone(), cache.clone()
    with binding.MlaDecode(1, 4, 128, page_size=PAGE) as h:
        table = torch.nn.functional.pad(table, (0, 2 - table.shape[1]), value=-1)
        h.append_rows(x, gamma, good, lens, starts, table)
        h.check_device_errors()
        lens[0] = 2                       # row 0 would lie at position -1
        lens[1] = 129                     # over max_kv_len
        table[3, 1] = cache.shape[0]      # a page that positions 62 and 63 do not reach
        h.append_rows(x, gamma, cache, lens, starts, table)
        with pytest.raises(binding.MlaError) as e:
            h.check_device_errors()
        assert e.value.detail == 0b100
        for page in (-1, cache.shape[0], 2 ** 31 - 1):
            wrong, same = table.clone(), cache.clone()
            wrong[3, 0] = page
            h.append_rows(x, gamma, same, lens, starts, wrong)
            with pytest.raises(binding.MlaError) as e:
                h.check_device_errors()
            assert e.value.detail == 0b101 and torch.equal(same, cache)
        # descending starts: no row may be written outside a sequence
        bad = starts.clone()
        bad[1:4] = torch.tensor([5, 1, 9], dtype=torch.int32, device=DEV)
        scratch = cache.clone()
        h.append_rows(x, gamma, scratch, lens, bad, table)
        try:
            h.check_device_errors()
        except binding.MlaError as err:
            assert err.detail & ~0b101 == 0
    t = table.cpu()
    written = (cache.view(torch.int16) != before.view(torch.int16)).any(dim=-1)
    expect = torch.zeros_like(written)
    expect[t[0, 0], 0] = expect[t[0, 0], 1] = True      # rows 1 and 2 of sequence 0, at positions 0 and 1
    expect[t[2, 1], 100 - 64] = expect[t[2, 1], 101 - 64] = True
    expect[t[3, 0], 62] = expect[t[3, 0], 63] = True
    assert torch.equal(written, expect)
    assert torch.equal(cache[t[2, 1], 36:38], good[t[2, 1], 36:38])


def test_cache_past_32_bits():
    """Rows behind 2^31 values of the pool, and positions of a long sequence."""
    pages, length = 60_000, 3_000_000
    cache = torch.zeros((pages, PAGE, 576), dtype=BF, device=DEV)
    table = torch.arange(pages - length // PAGE - 1, pages, dtype=torch.int32, device=DEV)[None]
    x, gamma = inputs(70, BF, 43)
    lens, starts = torch.tensor([length], dtype=torch.int32, device=DEV), torch.tensor([0, 70], dtype=torch.int32, device=DEV)
    with binding.MlaDecode(1, 1, length, page_size=PAGE) as h:
        h.append_rows(x, gamma, cache, lens, starts, table)
        h.check_device_errors()
    pos = np.arange(length - 70, length)
    theta = oracle.rope_theta(64, 10000.0)
    ref, slack = expected_rows(x, gamma, pos, theta, 1e-6)
    t = table[0].cpu().numpy()
    got = cache[t[pos // PAGE].tolist(), (pos % PAGE).tolist()].double().cpu().numpy()
    # the fp64 angle of a position p itself is off by p theta 2^-53: 3e6 * 2^-53 < 2^-31
    assert np.all(np.abs(got - ref) <= np.abs(ref) * 2.0 ** -8 + 1.01 * slack + 2.0 ** -30)
    assert int((cache != 0).any(dim=-1).sum()) == 70


@pytest.mark.parametrize("fp8", [False, True])
def test_graph_and_stream(fp8):
    new, cached = [5, 0, 70], [1, 2, 3]
    lens, starts, table, cache, exps, longest = layout(new, cached, True, 37, fp8)
    x, gamma = inputs(80, BF, 38)
    with binding.MlaDecode(1, 3, longest, page_size=PAGE) as h:
        def call(c, e, stream=None):
            if fp8:
                h.append_rows_fp8(x, gamma, c, e, lens, starts, table, stream=stream)
            else:
                h.append_rows(x, gamma, c, lens, starts, table, stream=stream)
        graph = torch.cuda.CUDAGraph()
        mine, mine_e = cache.clone(), None if exps is None else exps.clone()
        call(mine.clone(), None if exps is None else exps.clone())
        with torch.cuda.graph(graph):
            call(mine, mine_e)
        x.copy_(inputs(80, BF, 39)[0])
        starts.copy_(torch.tensor([0, 4, 6, 75], dtype=torch.int32))   # other rows per sequence
        lens.copy_(torch.tensor([6, 2, 73], dtype=torch.int32))
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        call(cache, exps, s)
        s.synchronize()
        graph.replay()
        h.check_device_errors()
    assert torch.equal(mine.view(torch.uint8), cache.view(torch.uint8))
    assert exps is None or torch.equal(mine_e, exps)


def test_refusals():
    lens, starts, table, cache, _, longest = layout([2, 3], [4, 5], False, 40, False)
    x, gamma = inputs(5, BF, 41)
    codes, exps = torch.zeros(cache.shape, dtype=torch.uint8, device=DEV), torch.zeros(cache.shape[:2], dtype=torch.int8, device=DEV)
    with binding.MlaDecode(1, 2, longest) as h:
        bad = [
            lambda: h.append_rows(x.cpu(), gamma, cache, lens, starts),
            lambda: h.append_rows(x[:, :575], gamma, cache, lens, starts),
            lambda: h.append_rows(x.half(), gamma, cache, lens, starts),
            lambda: h.append_rows(x, gamma.float(), cache, lens, starts),
            lambda: h.append_rows(x, gamma, cache.float(), lens, starts),
            lambda: h.append_rows(x, gamma, cache[:, :-1], lens, starts),     # shorter than max_kv_len
            lambda: h.append_rows(x, gamma, cache[:1], lens, starts),         # fewer sequences
            lambda: h.append_rows(x, gamma, cache, lens.long(), starts),
            lambda: h.append_rows(x, gamma, cache, lens, starts[:2]),
            lambda: h.append_rows_fp8(x, gamma, codes, exps[:, :-1], lens, starts),
            lambda: h.append_rows_fp8(x, gamma, cache, exps, lens, starts),
        ]
        for call in bad:
            with pytest.raises(ValueError):
                call()
        for call in (lambda: h.append_rows(x, gamma, cache, lens, starts, eps=-1.0),
                     lambda: h.append_rows(x, gamma, cache, lens),                       # 5 rows, 2 sequences
                     lambda: h.append_rows(inputs(5, BF, 42, 4)[0], gamma, cache, lens, starts),   # rows not 16-byte aligned
                     lambda: h.append_rows(x, gamma, cache, lens, starts, eps=float("inf"))):
            with pytest.raises(binding.MlaError, match="INVALID_ARG"):
                call()
        with pytest.raises((ValueError, binding.MlaError)):
            h.append_rows(x, gamma, cache, lens, starts, torch.zeros((2, 1), dtype=torch.int32, device=DEV))
        h.check_device_errors()
    assert bool((codes == 0).all())
