"""append_rows(_fp8) at the row counts from which two rows share a warp: element by element against
fp64, at the places where such a pair differs from a row alone (a window of sequences that ends
between its rows, an odd last row, a tail that begins with its second row, one row of it skipped)."""

import numpy as np
import pytest
import torch

import oracle
from mla_latent_kv_28_b200 import binding
from tests.test_gpu_append_rows import PAGE, check, expected_rows, inputs, layout, where

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, F32 = torch.bfloat16, torch.float32


def least():
    """An odd count of rows just above the least that run two to a warp."""
    return 32 * torch.cuda.get_device_properties(0).multi_processor_count + 1


def spread(new, rows, last):
    """Adds rows to the last `last` sequences until there are `rows`."""
    new = list(new)
    assert sum(new) <= rows
    i = 0
    while sum(new) < rows:
        new[-1 - i % last] += 1
        i += 1
    return new


def borders(rows):
    """Sequences 31 and 32, and 63 and 64, meet between the two rows of a warp."""
    new = [2] + [1] * 31 + [3] + [1] * 30 + [1] + [1] * 40
    starts = np.concatenate([[0], np.cumsum(new)])
    assert starts[32] % 2 == 1 and starts[64] % 2 == 1
    return spread(new, rows, 40)


def empties(rows):
    """After such a meeting come sequences without rows: to the window's end, past it, past two."""
    new = [2] + [1] * 31 + [0] * 40 + [1] * 20 + [0] * 5 + [4] + [0] * 100 + [1] * 60
    starts = np.concatenate([[0], np.cumsum(new)])
    assert starts[32] % 2 == 1
    return spread(new, rows, 60)


def thousand(rows):
    return spread([i % 7 for i in range(1000)], rows, 500)


LAYOUTS = {"borders": borders, "empty sequences": empties, "one thousand": thousand}


@pytest.mark.parametrize("name", list(LAYOUTS))
@pytest.mark.parametrize("paged,fp8,x_type", [(True, False, BF), (True, True, F32), (False, True, BF), (False, False, F32)])
def test_layouts(name, paged, fp8, x_type):
    new = LAYOUTS[name](least())
    cached = [(29 * b) % 150 for b in range(len(new))]
    check(new, cached, paged, fp8, x_type, seed=70 + len(name))


@pytest.mark.parametrize("paged,fp8,x_type", [(True, False, F32), (True, True, BF)])
@pytest.mark.parametrize("tail", [1, 2, 37])
def test_a_tail_that_begins_with_a_warps_second_row(paged, fp8, x_type, tail):
    """A padded batch, rows apart."""
    new = borders(least())
    check(new, [5] * len(new), paged, fp8, x_type, pad=64, tail=tail, seed=80 + tail)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("x_type", [BF, F32])
def test_few_long_sequences(fp8, x_type):
    check([least() // 2, 0, least() // 2 + 2], [0, 3, 77], True, fp8, x_type, seed=84)


@pytest.mark.parametrize("fp8", [False, True])
def test_without_row_starts(fp8):
    batch = min(1024, least() // 5 + 3)
    check([5] * batch, [(31 * b) % 90 for b in range(batch)], True, fp8, BF, seed=85, starts=False, q_len=5)


@pytest.mark.parametrize("fp8", [False, True])
def test_eps_base_and_magnitudes(fp8):
    """No rotation; and rows of a pair on either side of the squares' range in fp32."""
    new = borders(least())
    check(new, [9] * len(new), True, fp8, F32, seed=86, base=0.0, eps=0.5)
    x, gamma = inputs(sum(new), F32, 87)
    x[1::4, :512] *= 1e-22
    x[2::4, :512] *= 1e17
    x[7] = 0.0
    x[7, 0] = 1.0
    check(new, [9] * len(new), True, fp8, F32, seed=88, eps=0.0, x_gamma=(x, gamma))


@pytest.mark.parametrize("fp8", [False, True])
def test_one_row_of_a_pair_is_skipped(fp8):
    """A length without room, one over max_kv_len, and a bad page, each for one row of a warp."""
    new = borders(least())
    starts_of = np.concatenate([[0], np.cumsum(new)])
    single = [b for b in range(len(new)) if new[b] == 1]
    first = [b for b in single if starts_of[b] % 2 == 0]
    second = [b for b in single if starts_of[b] % 2 == 1]
    cached = [20] * len(new)
    lens, starts, table, cache, exps, longest = layout(new, cached, True, 89, fp8)
    x, gamma = inputs(sum(new), BF, 90)
    good, good_e = cache.clone(), None if exps is None else exps.clone()
    before, before_e = cache.clone(), None if exps is None else exps.clone()

    def call(h, c, e):
        if fp8:
            h.append_rows_fp8(x, gamma, c, e, lens, starts, table)
        else:
            h.append_rows(x, gamma, c, lens, starts, table)

    with binding.MlaDecode(1, len(new), longest, page_size=PAGE) as h:
        call(h, good, good_e)
        h.check_device_errors()
        skipped = [first[0], second[1], first[2], second[3], second[4], first[5]]
        at = where(new, cached, table.cpu())
        lens[skipped[0]] = 0
        lens[skipped[1]] = -5
        lens[skipped[2]] = longest + 1
        lens[skipped[3]] = 2 ** 31 - 1
        table[skipped[4], 0] = -1
        table[skipped[5], 0] = cache.shape[0]
        call(h, cache, exps)
        with pytest.raises(binding.MlaError) as e:
            h.check_device_errors()
        assert e.value.detail == 0b101
    for b in skipped:
        p, r, _ = at[starts_of[b]]
        good[p, r] = before[p, r]
        if fp8:
            good_e[p, r] = before_e[p, r]
    bits = torch.uint8 if fp8 else torch.int16
    assert torch.equal(cache.view(bits), good.view(bits))
    assert exps is None or torch.equal(exps, good_e)


@pytest.mark.parametrize("fp8", [False, True])
def test_special_rows_beside_others(fp8):
    """Infinities, NaN and zeros in one row of a pair leave the other as it is."""
    n = least()
    x, gamma = inputs(n, F32, 91)
    y = x.clone()
    odd = torch.arange(1, n, 8, device=DEV)
    y[odd[0::4], 512 + 3] = float("inf")
    y[odd[1::4], 5] = float("nan")
    y[odd[2::4]] = 0.0
    y[odd[3::4], 575] = float("nan")
    even = torch.arange(4, n, 8, device=DEV)
    y[even[0::2], 511] = -float("inf")
    y[even[1::2], 512] = float("nan")
    changed = torch.zeros(n, dtype=torch.bool, device=DEV)
    changed[odd] = changed[even] = True
    lens, starts = torch.tensor([n], dtype=torch.int32, device=DEV), torch.tensor([0, n], dtype=torch.int32, device=DEV)
    out = []
    with binding.MlaDecode(1, 1, n) as h:
        for rows in (x, y):
            cache = torch.zeros((1, n, 576), dtype=torch.uint8 if fp8 else BF, device=DEV)
            exps = torch.zeros((1, n), dtype=torch.int8, device=DEV)
            if fp8:
                h.append_rows_fp8(rows, gamma, cache, exps, lens, starts)
            else:
                h.append_rows(rows, gamma, cache, lens, starts)
            out.append((cache[0].view(torch.uint8), exps[0]))
        h.check_device_errors()
    for a, b in zip(*out):
        assert torch.equal(a[~changed], b[~changed])
    zero = cache[0][odd[2::4]]
    assert bool(((zero.view(torch.float8_e4m3fn).float() if fp8 else zero) == 0).all())
    assert bool((exps[0][odd[2::4]] == 0).all())


def test_two_streams_and_a_graph():
    """A captured call replayed on one stream while the same handle is used on another."""
    new = thousand(least())
    cached = [b % 60 for b in range(len(new))]
    lens, starts, table, cache, _, longest = layout(new, cached, True, 92, False)
    x, gamma = inputs(sum(new), BF, 93)
    a, b, want = cache.clone(), cache.clone(), cache.clone()
    with binding.MlaDecode(1, len(new), longest, page_size=PAGE) as h:
        h.append_rows(x, gamma, want, lens, starts, table)
        h.check_device_errors()
        graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph):
            h.append_rows(x, gamma, a, lens, starts, table)
        torch.cuda.synchronize()
        for _ in range(5):
            graph.replay()
            h.append_rows(x, gamma, b, lens, starts, table, stream=side)
        torch.cuda.synchronize()
        h.check_device_errors()
    assert torch.equal(a.view(torch.int16), want.view(torch.int16))
    assert torch.equal(b.view(torch.int16), want.view(torch.int16))


def test_yarn_frequencies():
    """With YaRN's frequencies (s = 40 over a 4K context) at positions up to 131072, rows alone in a
    warp and two to a warp."""
    yarn = dict(yarn_factor=40.0, yarn_original_len=4096, yarn_alpha=1.0, yarn_beta=32.0, yarn_mscale_coef=0.0707)
    theta = oracle.rope_theta(64, 10000.0, oracle.Yarn(factor=40.0, original_len=4096, alpha=1.0, beta=32.0, mscale_coef=0.0707))
    length = 131072
    for n in (300, least()):
        x, gamma = inputs(n, F32, 94)
        lens, starts = torch.tensor([length], dtype=torch.int32, device=DEV), torch.tensor([0, n], dtype=torch.int32, device=DEV)
        pages = length // PAGE
        table = torch.full((1, pages), -1, dtype=torch.int32, device=DEV)
        used = -(-n // PAGE) + 1
        table[0, pages - used:] = torch.randperm(used, generator=torch.Generator().manual_seed(95)).to(torch.int32).to(DEV)
        pos = np.arange(length - n, length)
        ref, slack = expected_rows(x, gamma, pos, theta, 1e-6)
        plain, _ = expected_rows(x, gamma, pos, oracle.rope_theta(64, 10000.0), 1e-6)
        assert np.abs(plain - ref)[:, 512:].max() > 0.5
        t = table[0].cpu().numpy()
        at = (t[pos // PAGE].tolist(), (pos % PAGE).tolist())
        with binding.MlaDecode(1, 1, length, page_size=PAGE, **yarn) as h:
            cache = torch.zeros((used, PAGE, 576), dtype=BF, device=DEV)
            h.append_rows(x, gamma, cache, lens, starts, table)
            codes = torch.zeros((used, PAGE, 576), dtype=torch.uint8, device=DEV)
            exps = torch.zeros((used, PAGE), dtype=torch.int8, device=DEV)
            h.append_rows_fp8(x, gamma, codes, exps, lens, starts, table)
            h.check_device_errors()
        got = cache[at].double().cpu().numpy()
        # the fp64 angle of a position p itself is off by p theta 2^-53 <= 2^-36
        assert np.all(np.abs(got - ref) <= np.abs(ref) * 2.0 ** -8 + 1.01 * slack + 2.0 ** -34)
        e = exps[at].cpu().numpy().astype(np.int64)
        assert np.array_equal(e, np.array([oracle.fp8_row_exponent(r) for r in ref]))
        values = codes[at].view(torch.float8_e4m3fn).double().cpu().numpy()
        scaled, room = ref / 2.0 ** e[:, None], slack / 2.0 ** e[:, None]
        assert np.all(np.abs(values - scaled) <= np.maximum(np.abs(scaled) * 2.0 ** -4, 2.0 ** -10) + 1.07 * room + 2.0 ** -30)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("many", [False, True])
@pytest.mark.parametrize("ahead", [1, 6, 64])
def test_rows_before_the_first_sequence(fp8, many, ahead):
    """Rows before row_starts[0] belong to nobody, as those behind the last sequence do."""
    new = borders(least()) if many else [3, 0, 70, 1]
    cached = [(7 * b) % 80 for b in range(len(new))]
    lens, starts, table, cache, exps, longest = layout(new, cached, True, 96, fp8)
    rows = sum(new)
    x, gamma = inputs(ahead + rows + 5, F32, 97)
    only, only_e = cache.clone(), None if exps is None else exps.clone()
    with binding.MlaDecode(1, len(new), longest, page_size=PAGE) as h:
        for c, e, v, s in ((cache, exps, x, starts + ahead), (only, only_e, x[ahead:ahead + rows], starts)):
            if fp8:
                h.append_rows_fp8(v, gamma, c, e, lens, s, table)
            else:
                h.append_rows(v, gamma, c, lens, s, table)
        h.check_device_errors()
    assert torch.equal(cache.view(torch.uint8), only.view(torch.uint8))
    assert exps is None or torch.equal(exps, only_e)


@pytest.mark.parametrize("fp8", [False, True])
def test_descending_starts_write_where_they_say(fp8):
    """row_starts that decrease are the caller's mistake: a row goes to the last sequence that starts at or
    before it if it ends behind it, and nowhere else. Of [0, 5, 1, 9, 9] row 0 would lie before its
    sequence, and rows 1 .. 8 are the last ones of sequence 2."""
    new, cached = [3, 2, 2, 2], [0, 5, 100, 62]
    lens, _, table, cache, exps, _ = layout(new, cached, True, 98, fp8)
    table = torch.nn.functional.pad(table, (0, 2 - table.shape[1]), value=-1)
    lens[0] = 2
    x, gamma = inputs(9, F32, 99)
    bad = torch.tensor([0, 5, 1, 9, 9], dtype=torch.int32, device=DEV)
    before, before_e = cache.clone(), None if exps is None else exps.clone()
    with binding.MlaDecode(1, 4, 128, page_size=PAGE) as h:
        if fp8:
            h.append_rows_fp8(x, gamma, cache, exps, lens, bad, table)
        else:
            h.append_rows(x, gamma, cache, lens, bad, table)
        with pytest.raises(binding.MlaError) as e:
            h.check_device_errors()
        assert e.value.detail == 0b100
    page = int(table[2, 1])
    written = torch.zeros(cache.shape[:2], dtype=torch.bool, device=DEV)
    written[page, 94 - 64:102 - 64] = True
    bits = torch.uint8 if fp8 else torch.int16
    assert torch.equal((cache.view(bits) != before.view(bits)).any(dim=-1), written)
    assert exps is None or torch.equal(exps[~written], before_e[~written])
    ref, slack = expected_rows(x[1:], gamma, range(94, 102), oracle.rope_theta(64, 10000.0), 1e-6)
    if not fp8:
        got = cache[page, 30:38].double().cpu().numpy()
        assert np.all(np.abs(got - ref) <= np.abs(ref) * 2.0 ** -8 + 1.01 * slack)
