"""The operators around the latent attention, as cases that can be timed and compared: the residual
addition with RMSNorm and int8 output (and the int8 rows without a norm), the int8 projection with a
scale per token and per output channel, and the cache write of projected rows.

`run` computes a case in plain torch operations, or, where `own` is true, through the binding.
"""

import math
import random

import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
D_LATENT, D_ROPE = 512, 64
ROW = D_LATENT + D_ROPE
ROPE_BASE = 10000.0
EPS = 1e-6
PAGE = 64
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"none": 0, "bf16": 2, "f32": 4}


def listed():
    return [
        # the block's input norm for one decoded token of one request
        {"name": "norm_1x5120", "op": "norm", "rows": 1, "d": 5120, "x": "bf16", "residual": "bf16", "y": False, "pad": 0},
        # the same norm over a long prompt, residual stream kept in fp32, bf16 rows wanted as well
        {"name": "norm_4096x5120_f32", "op": "norm", "rows": 4096, "d": 5120, "x": "bf16", "residual": "f32", "y": True, "pad": 0},
        # c^Q's norm: 1536 of the 2112 columns of the fused down-projection of a ragged batch, in fp32
        {"name": "norm_777x1536_f32", "op": "norm", "rows": 777, "d": 1536, "x": "f32", "residual": "none", "y": False, "pad": 576},
        # the heads' outputs (128 heads x 128) of a 2048-token prompt on their way into W^O
        {"name": "quant_2048x16384", "op": "quant", "rows": 2048, "d": 16384, "x": "bf16", "pad": 0},
        # the fused down-projection [W^DQ; W^DKV; W^KR] of one token
        {"name": "linear_1_5120_2112", "op": "linear", "rows": 1, "k": 5120, "n": 2112, "out": "f32"},
        # W^UQ for a decode batch of 64
        {"name": "linear_64_1536_16384", "op": "linear", "rows": 64, "k": 1536, "n": 16384, "out": "bf16"},
        # W^O for a decode batch of 33
        {"name": "linear_33_16384_5120", "op": "linear", "rows": 33, "k": 16384, "n": 5120, "out": "bf16"},
        # W^O for a 2048-token prompt
        {"name": "linear_2048_16384_5120", "op": "linear", "rows": 2048, "k": 16384, "n": 5120, "out": "bf16"},
        # nothing a multiple of a tile: a short ragged batch through an odd projection
        {"name": "linear_333_1000_777", "op": "linear", "rows": 333, "k": 1000, "n": 777, "out": "f32"},
        # one new token for each of 64 sequences, paged bf16 cache
        {"name": "append_64_paged", "op": "append", "seqs": 64, "rows": 64, "tail": 0, "context": 4096, "paged": True, "fp8": False, "x": "f32", "pad": 0},
        # a ragged chunk of prompts and decoding sequences, paged E4M3 cache, padded batch
        {"name": "append_8192_paged_fp8", "op": "append", "seqs": 24, "rows": 8192, "tail": 37, "context": 1024, "paged": True, "fp8": True, "x": "bf16", "pad": 1536},
        # a few long prompts written into a contiguous bf16 cache
        {"name": "append_65536", "op": "append", "seqs": 3, "rows": 65536, "tail": 0, "context": 0, "paged": False, "fp8": False, "x": "bf16", "pad": 0},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "quant", "linear", "linear", "append"])
    if op in ("norm", "quant"):
        d = _log(rng, 64, 16384)
        d = d if rng.random() < 0.4 else max(64, d // 64 * 64)
        rows = _log(rng, 1, max(1, min(65536, 20_000_000 // d)))
        case = {"op": op, "rows": rows, "d": d, "x": rng.choice(["bf16", "f32"])}
        if op == "norm":
            case["residual"] = rng.choice(["none", "bf16", "f32"])
            case["y"] = rng.random() < 0.5
        case["pad"] = rng.choice([0, 0, 8, 64, 5])
        return case
    if op == "linear":
        rows, k, n = _log(rng, 1, 8192), _log(rng, 64, 16384), _log(rng, 16, 16384)
        if rng.random() < 0.5:
            k, n = max(64, k // 64 * 64), max(16, n // 16 * 16)
        while rows * k * n > 2048 * 16384 * 5120:
            rows, k, n = max(1, rows // 2), max(64, k * 3 // 4), max(16, n * 3 // 4)
        return {"op": op, "rows": rows, "k": k, "n": n, "out": rng.choice(["bf16", "f32"])}
    rows = _log(rng, 1, 32768)
    return {"op": op, "seqs": _log(rng, 1, 256), "rows": rows, "tail": rng.choice([0, 0, 1, 19]), "context": _log(rng, 1, 1024),
            "paged": rng.random() < 0.6, "fp8": rng.random() < 0.5, "x": rng.choice(["bf16", "f32"]), "pad": rng.choice([0, 64, 1536])}


def _padded(rows, width, pad, dtype, gen, outliers=True):
    """[rows, width] as a slice of rows that are `pad` values longer; each token has its own
    magnitude and a few channels stand out, as in a residual stream."""
    x = torch.randn((rows, width + pad), generator=gen, device=DEV)
    if outliers:
        x *= torch.exp(0.5 * torch.randn((rows, 1), generator=gen, device=DEV))
        x[:, : width : max(1, width // 6)] *= 12.0
    return x.to(dtype)[:, :width]


def _codes(rows, width, gen):
    """int8 codes [rows, width] of Gaussian rows, their rows 16-byte aligned."""
    c = torch.randn((rows, -(-width // 16) * 16), generator=gen, device=DEV).mul_(127 / 4.2).round_().clamp_(-127, 127)
    return c.to(torch.int8)[:, :width]


def _lengths(case, seed):
    """New rows and cached rows of each sequence: prompts of uneven lengths, single tokens, and
    sequences that get nothing. The seed sets which sequence has which of the case's lengths."""
    rng = random.Random(case["seqs"] * 1_000_003 + case["rows"])
    n, rows = case["seqs"], case["rows"]
    if rows == n:
        new = [1] * n
    else:
        share = [rng.choice([0.0, 0.01, rng.random()]) for _ in range(n)]
        share[rng.randrange(n)] = 1.0
        new = [int(rows * s / sum(share)) for s in share]
        new[max(range(n), key=lambda i: new[i])] += rows - sum(new)
    both = [(i, rng.randint(0, case["context"])) for i in new]
    random.Random(seed).shuffle(both)
    return [i for i, _ in both], [i for _, i in both]


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    s = {"case": case}
    handle = dict(n_heads=1, max_batch=1, max_kv_len=64)
    if case["op"] in ("norm", "quant"):
        s["x"] = _padded(case["rows"], case["d"], case["pad"], TYPES[case["x"]], gen)
        if case["op"] == "norm":
            s["gamma"] = (1.0 + 0.1 * torch.randn(case["d"], generator=gen, device=DEV)).to(torch.bfloat16)
            res = case["residual"]
            s["residual"] = None if res == "none" else _padded(case["rows"], case["d"], 0, TYPES[res], gen).contiguous()
    elif case["op"] == "linear":
        s["codes"] = _codes(case["rows"], case["k"], gen)
        s["scales"] = torch.exp(0.5 * torch.randn(case["rows"], generator=gen, device=DEV)) * (4.2 / 127)
        s["w_codes"] = _codes(case["n"], case["k"], gen)
        s["w_scales"] = (0.8 + 0.4 * torch.rand(case["n"], generator=gen, device=DEV)) * (4.2 / 127 / math.sqrt(case["k"]))
    else:
        new, cached = _lengths(case, seed)
        lens = [a + b for a, b in zip(new, cached)]
        longest = max(1, max(lens))
        starts = [sum(new[:i]) for i in range(len(new) + 1)]
        s["x"] = _padded(case["rows"] + case["tail"], ROW, case["pad"], TYPES[case["x"]], gen, outliers=False)
        s["gamma"] = (1.0 + 0.1 * torch.randn(D_LATENT, generator=gen, device=DEV)).to(torch.bfloat16)
        s["kv_lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        s["starts"] = torch.tensor(starts, dtype=torch.int32, device=DEV)
        s["table"] = None
        if case["paged"]:
            pages = [-(-n // PAGE) for n in lens]
            blocks, width = sum(pages) + 3, -(-longest // PAGE)
            order = torch.randperm(blocks, generator=gen, device=DEV).to(torch.int32)
            at = torch.tensor([sum(pages[:i]) for i in range(len(pages))], device=DEV)[:, None] + torch.arange(width, device=DEV)[None]
            used = torch.arange(width, device=DEV)[None] < torch.tensor(pages, device=DEV)[:, None]
            s["table"] = torch.where(used, order[at.clamp(max=blocks - 1)], torch.full_like(at, -1, dtype=torch.int32))
            shape = (blocks, PAGE)
        else:
            shape = (case["seqs"], longest)
        if case["fp8"]:
            s["cache"] = torch.randint(0, 0x7F, shape + (ROW,), generator=gen, device=DEV, dtype=torch.uint8)
            s["exps"] = torch.randint(-9, -4, shape, generator=gen, device=DEV, dtype=torch.int8)
        else:
            s["cache"] = torch.randn(shape + (ROW,), generator=gen, device=DEV, dtype=torch.bfloat16)
        handle = dict(n_heads=1, max_batch=case["seqs"], max_kv_len=longest, page_size=PAGE if case["paged"] else 0, rope_base=ROPE_BASE)
    if own:
        from mla_latent_kv_28_b200 import binding

        s["handle"] = binding.MlaDecode(**handle)
    return s


def _codes_and_scales(t, rstd):
    """int8 codes of the rows of t (fp32) and their scales: the nearest integers of 127 t / max|t|,
    in 64 bits since values lie on and next to the borders between two codes."""
    m = t.abs().amax(dim=-1, keepdim=True)
    fine = torch.isfinite(m) & (m > 0)
    codes = torch.where(fine, torch.round(t.double() * 127.0 / m.double()), 0.0).to(torch.int8)
    scale = torch.where(m > 0, m * rstd / 127.0, 0.0)
    return codes, torch.where(torch.isfinite(m), scale, math.nan).squeeze(-1)


def _run_plain(s):
    case = s["case"]
    if case["op"] == "norm":
        r = s["x"].float()
        if s["residual"] is not None:
            r = r + s["residual"].float()
        rstd = 1.0 / torch.sqrt((r * r).mean(dim=-1, keepdim=True) + EPS)
        codes, scales = _codes_and_scales(r * s["gamma"].float(), rstd)
        return {"codes": codes, "scales": scales,
                "residual": None if s["residual"] is None else r.to(s["residual"].dtype),
                "y": (r * rstd * s["gamma"].float()).to(torch.bfloat16) if case["y"] else None}
    if case["op"] == "quant":
        codes, scales = _codes_and_scales(s["x"].float(), 1.0)
        return {"codes": codes, "scales": scales}
    if case["op"] == "linear":
        out = s["codes"].float() @ s["w_codes"].float().T
        return {"out": (out * s["w_scales"][None] * s["scales"][:, None]).to(TYPES[case["out"]])}
    rows = case["rows"]
    x = s["x"][:rows].float()
    i = torch.arange(rows, device=x.device)
    b = torch.searchsorted(s["starts"][1:].contiguous(), i.to(torch.int32), right=True)
    pos = s["kv_lens"][b].long() - s["starts"][b + 1].long() + i
    c, k = x[:, :D_LATENT].double(), x[:, D_LATENT:].double()
    c = c / torch.sqrt((c * c).mean(dim=-1, keepdim=True) + EPS) * s["gamma"].double()
    theta = ROPE_BASE ** (-2.0 * torch.arange(D_ROPE // 2, device=x.device, dtype=torch.float64) / D_ROPE)
    angle = pos[:, None].double() * theta[None]
    even, odd, cos, sin = k[:, 0::2], k[:, 1::2], torch.cos(angle), torch.sin(angle)
    row = torch.cat([c, torch.stack([even * cos - odd * sin, even * sin + odd * cos], dim=-1).flatten(1)], dim=1)
    first, second = (b, pos) if s["table"] is None else (s["table"][b, pos // PAGE].long(), pos % PAGE)
    if not case["fp8"]:
        s["cache"][first, second] = row.to(torch.bfloat16)
        return {"cache": s["cache"]}
    most = row.abs().amax(dim=-1)
    e = torch.where(most > 0, torch.ceil(torch.log2(most / 448.0)), 0.0)
    e = e + (most > 448.0 * torch.exp2(e)).double()
    e = e - ((most > 0) & (most <= 448.0 * torch.exp2(e - 1))).double()
    s["exps"][first, second] = e.to(torch.int8)
    s["cache"][first, second] = (row / torch.exp2(e)[:, None]).float().to(torch.float8_e4m3fn).view(torch.uint8)
    return {"codes": s["cache"].view(torch.float8_e4m3fn), "exps": s["exps"]}


def _run_own(s):
    case, h = s["case"], s["handle"]
    if case["op"] == "norm":
        codes, scales, residual, y = h.add_norm_q8(s["x"], s["gamma"], s["residual"], eps=EPS, want_y=case["y"])
        return {"codes": codes, "scales": scales, "residual": residual, "y": y}
    if case["op"] == "quant":
        codes, scales = h.quantize_rows(s["x"])
        return {"codes": codes, "scales": scales}
    if case["op"] == "linear":
        return {"out": h.linear_q8(s["codes"], s["scales"], s["w_codes"], s["w_scales"], out_dtype=TYPES[case["out"]])}
    if case["fp8"]:
        h.append_rows_fp8(s["x"], s["gamma"], s["cache"], s["exps"], s["kv_lens"], s["starts"], s["table"], eps=EPS)
        return {"codes": s["cache"].view(torch.float8_e4m3fn), "exps": s["exps"]}
    h.append_rows(s["x"], s["gamma"], s["cache"], s["kv_lens"], s["starts"], s["table"], eps=EPS)
    return {"cache": s["cache"]}


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    if case["op"] in ("norm", "quant"):
        each = BYTES[case["x"]] + 1
        if case["op"] == "norm":
            each += 2 * BYTES[case["residual"]] + (2 if case["y"] else 0)
        n = case["rows"] * case["d"]
        return {"bytes": n * each + 4 * case["rows"] + (2 * case["d"] if case["op"] == "norm" else 0), "flops": 8 * n}
    if case["op"] == "linear":
        m, k, n = case["rows"], case["k"], case["n"]
        return {"bytes": m * k + n * k + m * n * BYTES[case["out"]] + 4 * (m + n), "flops": 2 * m * n * k}
    rows = case["rows"]
    each = ROW * BYTES[case["x"]] + (ROW + 1 if case["fp8"] else 2 * ROW)
    return {"bytes": rows * each + 2 * D_LATENT + 8 * case["seqs"], "flops": rows * (4 * D_LATENT + 6 * D_ROPE)}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("norm", "quant"):
        v = s["x"].to(torch.float64)
        out = {}
        inverse = torch.ones_like(v[:, :1])
        if case["op"] == "norm":
            if s["residual"] is not None:
                v = v + s["residual"].to(torch.float64)
            out["residual"] = None if s["residual"] is None else v
            inverse = torch.rsqrt(v.pow(2).sum(dim=1, keepdim=True) / case["d"] + EPS)
            out["y"] = v * inverse * s["gamma"].to(torch.float64) if case["y"] else None
            v = v * s["gamma"].to(torch.float64)
        largest = torch.linalg.vector_norm(v, ord=math.inf, dim=1, keepdim=True)
        out["codes"] = None
        out["scales"] = (largest * inverse / 127.0).flatten()
        return out
    if case["op"] == "linear":
        left = s["codes"].to(torch.float64) * s["scales"].to(torch.float64).unsqueeze(1)
        right = s["w_codes"].to(torch.float64) * s["w_scales"].to(torch.float64).unsqueeze(1)
        return {"out": torch.matmul(left, right.t())}
    starts, lens = s["starts"].tolist(), s["kv_lens"].tolist()
    cache = (s["cache"].view(torch.float8_e4m3fn) if case["fp8"] else s["cache"]).to(torch.float64)
    pair = torch.arange(D_ROPE // 2, device=DEV, dtype=torch.float64)
    turn = torch.exp(-pair * (2.0 / D_ROPE) * math.log(ROPE_BASE))
    for b in range(case["seqs"]):
        first, last = starts[b], starts[b + 1]
        if first == last:
            continue
        x = s["x"][first:last].to(torch.float64)
        at = torch.arange(lens[b] - (last - first), lens[b], device=DEV)
        latent = x[:, :D_LATENT]
        latent = latent * s["gamma"].to(torch.float64) / (latent.square().sum(dim=1, keepdim=True) / D_LATENT + EPS).sqrt()
        key = torch.view_as_complex(x[:, D_LATENT:].reshape(-1, D_ROPE // 2, 2).contiguous())
        key = torch.view_as_real(key * torch.polar(torch.ones_like(turn), at.unsqueeze(1) * turn)).reshape(-1, D_ROPE)
        row = torch.cat((latent, key), dim=1)
        if case["fp8"]:
            _, power = torch.frexp(row.abs().max(dim=1, keepdim=True).values / 448.0)
            scale = torch.ldexp(torch.ones_like(row[:, :1]), power)
            scale = torch.where(row.abs().max(dim=1, keepdim=True).values <= 224.0 * scale, scale / 2, scale)
            row = row / scale
        if s["table"] is None:
            cache[b, at] = row
        else:
            cache[s["table"][b][at // PAGE].long(), at % PAGE] = row
    return {"codes": cache, "exps": None} if case["fp8"] else {"cache": cache}
