"""What the FP8 products and the experts' operators are timed and compared on.

FP8 here is E4M3 with one FP32 scale for a block: 128 consecutive values of a row for activations, 128 x 128 values for
weights. A held value stands for code * scale. Five operators:

* quantize: rows (or silu(gate) * up of rows that hold both) and weights into that form;
* product:  out = A W^T of two such matrices, summed block by block;
* experts:  the same for rows sorted by expert, each expert's rows against the expert's own weights; the rows may be
            taken from the tokens through an index;
* dispatch: (token, choice) pairs sorted by expert, the tokens' rows gathered in that order, and the gather's gradient;
* combine:  the rows back to their tokens, each times its weight, summed; and the gradients of rows and weights.

Widths are those of the 27B-class model that the library's GEMM workloads use (5120 hidden, 17408 between, 6144 of QKV)
and generic ones for the experts.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
TOP = 448.0               # the largest E4M3 value
LEAST = 2.0 ** -100       # a block's maximum counts as at least this


# ------------------------------------------------------------------------------------------------------ the cases

def _quantize_case(name, rows, cols, form="rows", dtype="bf16", experts=1, pad=0):
    return dict(name=name, op="quantize", rows=rows, cols=cols, form=form, dtype=dtype, experts=experts, pad=pad)


def _product_case(name, rows, n, k, dtype="bf16"):
    return dict(name=name, op="product", rows=rows, n=n, k=k, dtype=dtype)


def _experts_case(name, tokens, top, experts, n, k, dtype="bf16", gathered=True, absent=0.0):
    return dict(name=name, op="experts", tokens=tokens, top=top, experts=experts, n=n, k=k, dtype=dtype,
                gathered=gathered, absent=absent)


def _rows_case(name, op, tokens, top, experts, width, dtype="bf16", back=False, absent=0.0, pad=0):
    return dict(name=name, op=op, tokens=tokens, top=top, experts=experts, width=width, dtype=dtype, back=back,
                absent=absent, pad=pad)


def listed():
    return [
        # the input of a decode step's products: 61 users, where latency is all
        _quantize_case("quantize_decode_61", 61, 5120),
        # between the two halves of a feed-forward block in a prefill chunk: gate and up lie side by side
        _quantize_case("quantize_gated_2048", 2048, 17408, "gated"),
        # a weight as it is loaded or updated
        _quantize_case("quantize_weight", 17408, 5120, "weight"),
        # one user's token through the down projection: bound by the weight's bytes
        _product_case("product_decode_1", 1, 5120, 17408),
        # a ragged middle-sized product in half precision; neither side is a multiple of the tiles
        _product_case("product_ragged_1013", 1013, 2059, 4112, "f16"),
        # the up projection of a prefill chunk: the largest case, bound by arithmetic
        _product_case("product_prefill_8192", 8192, 17408, 5120),
        # a decode step of 32 users, eight of 64 experts each: most experts are read for a few rows
        _experts_case("experts_decode_32", 32, 8, 64, 2560, 5120),
        # a prefill chunk through the same experts, unevenly loaded
        _experts_case("experts_prefill_4096", 4096, 8, 64, 2560, 5120),
        # sorting and gathering for a handful of users: launches are what costs
        _rows_case("dispatch_17", "dispatch", 17, 8, 64, 5120),
        # a training micro-batch: the rows there and their gradient back
        _rows_case("dispatch_train_4096", "dispatch", 4096, 8, 64, 5120, back=True),
        # back to the tokens of a decode step; a quarter of the choices belongs to experts of another device
        _rows_case("combine_33", "combine", 33, 8, 64, 5120, absent=0.25),
        # the training micro-batch's way back, with the gradients of rows and weights
        _rows_case("combine_train_4096", "combine", 4096, 8, 64, 5120, back=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "product", "product", "experts", "dispatch", "combine"])
    half = rng.choice(["bf16", "f16"])
    if op == "quantize":
        form = rng.choice(["rows", "gated", "weight"])
        c = _quantize_case("", _log_int(rng, 1, 8192), 16 * _log_int(rng, 1, 1088), form,
                           rng.choice(["bf16", "bf16", "f16", "f32"]), _log_int(rng, 1, 8) if form == "weight" else 1,
                           rng.choice([0, 8, 64]))
        while c["rows"] * c["cols"] * c["experts"] > 17408 * 5120:
            c["rows"] = c["rows"] // 2 + 1
    elif op == "product":
        c = _product_case("", _log_int(rng, 1, 8192), _log_int(rng, 32, 17408), 16 * _log_int(rng, 4, 1088), half)
        while c["rows"] * c["n"] * c["k"] > 8192 * 17408 * 5120:
            c["n"] = c["n"] * 2 // 3
    elif op == "experts":
        experts = rng.choice([4, 8, 16, 32, 64, 128, 160, 256])
        c = _experts_case("", _log_int(rng, 1, 4096), rng.randint(1, min(8, experts)), experts, _log_int(rng, 64, 5120),
                          16 * _log_int(rng, 8, 320), half, rng.random() < 0.5, rng.choice([0.0, 0.0, 0.3]))
        while experts * c["n"] * c["k"] > 64 * 2560 * 5120 or c["tokens"] * c["top"] * c["n"] * c["k"] > 32768 * 2560 * 5120:
            c["n"] = c["n"] * 2 // 3 + 1
            c["k"] = c["k"] // 32 * 16 + 64 if c["k"] > 1024 else c["k"]
    else:
        experts = rng.choice([4, 8, 16, 60, 64, 128, 160, 256, 384])
        c = _rows_case("", op, _log_int(rng, 1, 8192), rng.randint(1, min(10, experts)), experts,
                       rng.choice([_log_int(rng, 64, 8192), 8 * _log_int(rng, 8, 1024)]), rng.choice(["bf16", "f16", "f32"]),
                       rng.random() < 0.5, rng.choice([0.0, 0.0, 0.5]), rng.choice([0, 8]))
        while c["tokens"] * c["top"] * c["width"] > 4096 * 8 * 5120 * (1 if c["dtype"] != "f32" else 0.5):
            c["tokens"] = c["tokens"] * 2 // 3 + 1
    del c["name"]
    return c


def _blocks(n):
    return -(-n // 128)


def _size(c):
    return 4 if c["dtype"] == "f32" else 2


def work(case):
    c = case
    if c["op"] == "quantize":
        n = c["rows"] * c["cols"] * c["experts"]
        scales = c["experts"] * (_blocks(c["rows"]) if c["form"] == "weight" else c["rows"]) * _blocks(c["cols"])
        return {"bytes": n * (_size(c) * (2 if c["form"] == "gated" else 1) + 1) + 4 * scales,
                "flops": n * (8 if c["form"] == "gated" else 3)}
    if c["op"] == "product":
        m, n, k = c["rows"], c["n"], c["k"]
        return {"bytes": (m + n) * k + 4 * (m + _blocks(n)) * _blocks(k) + 2 * m * n, "flops": 2 * m * n * k}
    held = c["tokens"] * c["top"] * (1.0 - c["absent"])                    # rows that some expert has, on average
    if c["op"] == "experts":
        n, k = c["n"], c["k"]
        met = c["experts"] * (1.0 - (1.0 - 1.0 / c["experts"]) ** held)    # experts with a row, on average
        read = min(c["tokens"], held) if c["gathered"] else held
        return {"bytes": met * (n * k + 4 * _blocks(n) * _blocks(k)) + read * (k + 4 * _blocks(k)) + 2 * held * n,
                "flops": 2 * held * n * k}
    pairs = c["tokens"] * c["top"]
    row, tokens = c["width"] * _size(c), c["tokens"]
    if c["op"] == "dispatch":
        moved = (tokens + held) * row + 12 * pairs
        return {"bytes": moved * (2 if c["back"] else 1), "flops": held * c["width"] if c["back"] else 0}
    moved = (tokens + held) * row + 8 * pairs
    if c["back"]:
        moved += (tokens + 2 * held) * row + 12 * pairs
    return {"bytes": moved, "flops": held * c["width"] * (5 if c["back"] else 2)}


# ----------------------------------------------------------------------------------------------------- the inputs

def _quantize(x, tall):
    """[..][N][K] in 32 bits -> E4M3 codes and the scales of blocks of `tall` rows by 128 columns."""
    n, k = x.shape[-2:]
    rows, cols = -(-n // tall), _blocks(k)
    y = torch.nn.functional.pad(x, (0, cols * 128 - k, 0, rows * tall - n))
    y = y.unflatten(-1, (cols, 128)).unflatten(-3, (rows, tall))
    scales = y.abs().amax((-3, -1)).clamp(min=LEAST) / TOP
    codes = (y / scales[..., None, :, None]).to(torch.float8_e4m3fn)
    return codes.flatten(-4, -3).flatten(-2)[..., :n, :k].contiguous(), scales


def _values(codes, scales, tall):
    """What codes under the scales of such blocks stand for, in 32 bits."""
    n, k = codes.shape[-2:]
    wide = scales.repeat_interleave(tall, -2) if tall > 1 else scales
    return codes.float() * wide[..., :n, :].repeat_interleave(128, -1)[..., :k]


def _activations(shape, gen):
    """Rows as layers make them: a few strong channels, the same ones for every token."""
    strong = 1.0 + 9.0 * (torch.rand(shape[-1:], generator=gen, device="cuda") < 0.01).float()
    return torch.randn(shape, generator=gen, device="cuda") * strong


def _padded(x, pad, dtype):
    """The rows as columns of a wider matrix, when there is a pad."""
    wide = torch.zeros((*x.shape[:-1], x.shape[-1] + pad), dtype=dtype, device="cuda")
    wide[..., :x.shape[-1]] = x
    return wide[..., :x.shape[-1]]


def _route(c, gen):
    """Experts of each token, the likeliest first, with unevenly popular experts, and their weights. A choice of an
    expert that is not here has the id -1."""
    logits = torch.randn((c["tokens"], c["experts"]), generator=gen, device="cuda")
    logits += 0.5 * torch.randn((c["experts"],), generator=gen, device="cuda")
    best, ids = torch.topk(logits, c["top"], dim=1)
    weights = torch.softmax(best, 1)
    gone = torch.rand(ids.shape, generator=gen, device="cuda") < c["absent"]
    return torch.where(gone, -1, ids).int(), weights


def _sorted(ids, experts):
    """Pairs (token, choice) by expert, then by place; those of no expert last. Offsets of the experts, the token of
    each sorted pair (-1 past the last expert's), and each pair's place (-1 for none)."""
    top = ids.shape[1]
    flat = ids.flatten().long()
    here = (flat >= 0) & (flat < experts)
    key = torch.where(here, flat, experts)
    order = torch.argsort(key, stable=True)
    counts = torch.zeros(experts + 1, dtype=torch.long, device=ids.device).scatter_add_(0, key, torch.ones_like(key))
    offsets = torch.cat([torch.zeros_like(counts[:1]), counts[:experts].cumsum(0)])
    i = torch.arange(flat.shape[0], device=ids.device)
    places = torch.empty_like(i).scatter_(0, order, i)
    tokens = torch.where(i < offsets[-1], order // top, -1)
    return offsets.int(), tokens.int(), torch.where(here, places, -1).int().reshape(ids.shape)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=c)
    if c["op"] == "quantize":
        if c["form"] == "weight":
            x = torch.randn((c["experts"], c["rows"], c["cols"]), generator=gen, device="cuda") * c["cols"] ** -0.5
            x = x if c["experts"] > 1 else x[0]
        else:
            x = _activations((c["rows"], c["cols"] * (2 if c["form"] == "gated" else 1)), gen)
        return s | dict(x=_padded(x, c["pad"], DTYPES[c["dtype"]]))
    if c["op"] == "product":
        s["a"], s["a_scales"] = _quantize(_activations((c["rows"], c["k"]), gen), 1)
        s["w"], s["w_scales"] = _quantize(torch.randn((c["n"], c["k"]), generator=gen, device="cuda") * c["k"] ** -0.5, 128)
        return s
    ids, weights = _route(c, gen)
    offsets, tokens, places = _sorted(ids, c["experts"])
    pairs = ids.numel()
    if c["op"] == "experts":
        rows = c["tokens"] if c["gathered"] else pairs
        s["a"], s["a_scales"] = _quantize(_activations((rows, c["k"]), gen), 1)
        s["w"] = torch.empty((c["experts"], c["n"], c["k"]), dtype=torch.float8_e4m3fn, device="cuda")
        s["w_scales"] = torch.empty((c["experts"], _blocks(c["n"]), _blocks(c["k"])), device="cuda")
        for e in range(c["experts"]):
            w = torch.randn((c["n"], c["k"]), generator=gen, device="cuda") * c["k"] ** -0.5
            s["w"][e], s["w_scales"][e] = _quantize(w, 128)
        return s | dict(offsets=offsets, rows=tokens if c["gathered"] else None,
                        longest=int((offsets[1:] - offsets[:-1]).max()),
                        out=torch.zeros((pairs, c["n"]), dtype=DTYPES[c["dtype"]], device="cuda"))
    dtype, width = DTYPES[c["dtype"]], c["width"]
    s |= dict(ids=ids, rows=torch.zeros((pairs, width), dtype=dtype, device="cuda"))
    if c["op"] == "dispatch":
        s["x"] = _padded(_activations((c["tokens"], width), gen), c["pad"], dtype)
        if c["back"]:
            s["grad"] = _padded(torch.randn((pairs, width), generator=gen, device="cuda"), c["pad"], dtype)
        return s
    s |= dict(places=places, weights=weights, y=_padded(torch.randn((pairs, width), generator=gen, device="cuda"), c["pad"], dtype))
    if c["back"]:
        s["grad"] = _padded(torch.randn((c["tokens"], width), generator=gen, device="cuda"), c["pad"], dtype)
    return s


# ------------------------------------------------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return _own(op, state)
    return {"quantize": _plain_quantize, "product": _plain_product, "experts": _plain_experts,
            "dispatch": _plain_dispatch, "combine": _plain_combine}[op](state)


def _own(op, s):
    import nvfp4_block_scaled_amd as nv
    c = s["case"]
    if op == "quantize":
        if c["form"] == "weight":
            codes, scales = nv.nvfp4_fp8_quantize_weight(s["x"])
        else:
            codes, scales = nv.nvfp4_fp8_quantize(s["x"], gated=c["form"] == "gated")
        return {"codes": codes, "scales": scales}
    if op == "product":
        return {"out": nv.nvfp4_fp8_gemm(s["a"], s["a_scales"], s["w"], s["w_scales"], out_dtype=c["dtype"])}
    if op == "experts":
        return {"out": nv.nvfp4_fp8_gemm_grouped(s["a"], s["a_scales"], s["w"], s["w_scales"], s["offsets"],
                                                 rows=s["rows"], out_dtype=c["dtype"], out=s["out"])}
    if op == "dispatch":
        offsets, tokens, places = nv.nvfp4_moe_sort(s["ids"], c["experts"])
        out = {"offsets": offsets, "tokens": tokens, "places": places,
               "rows": nv.nvfp4_moe_gather(s["x"], places, out=s["rows"])}
        if c["back"]:
            out["grad_x"] = nv.nvfp4_moe_gather_backward(s["grad"], places)
        return out
    out = {"out": nv.nvfp4_moe_combine(s["y"], s["places"], s["weights"])}
    if c["back"]:
        out["grad_y"], out["grad_weights"] = nv.nvfp4_moe_combine_backward(s["grad"], s["y"], s["places"], s["weights"],
                                                                           grad_y=s["rows"])
    return out


def _plain_quantize(s):
    c = s["case"]
    x = s["x"].float()
    if c["form"] == "gated":
        gate, up = x.split(c["cols"], -1)
        x = gate / (1.0 + torch.exp(-gate)) * up
    codes, scales = _quantize(x, 128 if c["form"] == "weight" else 1)
    return {"codes": codes, "scales": scales}


def _plain_product(s):
    a, w = _values(s["a"], s["a_scales"], 1), _values(s["w"], s["w_scales"], 128)
    return {"out": torch.matmul(a, w.T).to(DTYPES[s["case"]["dtype"]])}


def _plain_experts(s):
    c, offsets = s["case"], s["offsets"].long()
    i = torch.arange(s["out"].shape[0], device="cuda")
    expert = torch.searchsorted(offsets[1:].contiguous(), i, right=True)
    here = expert < c["experts"]
    expert = expert.clamp(max=c["experts"] - 1)
    a = _values(s["a"], s["a_scales"], 1)
    if s["rows"] is not None:
        a = a[s["rows"].clamp(min=0).long()]
    # each expert's rows in a part of their own, as long as the longest
    at = expert * s["longest"] + i - offsets[expert]
    put = torch.where(here, at, c["experts"] * s["longest"])
    parts = torch.zeros((c["experts"] * s["longest"] + 1, c["k"]), device="cuda").index_copy_(0, put[here], a[here])
    w = _values(s["w"], s["w_scales"], 128)
    out = torch.bmm(parts[:-1].unflatten(0, (c["experts"], -1)), w.transpose(1, 2).contiguous()).flatten(0, 1)
    s["out"][here] = out[at[here]].to(s["out"].dtype)
    return {"out": s["out"]}


def _taken(rows, places):
    """The rows [T][top][width] of every pair in 32 bits, zero for a pair that has none."""
    return torch.where((places >= 0)[..., None], rows[places.clamp(min=0).long()].float(), 0.0)


def _plain_dispatch(s):
    offsets, tokens, places = _sorted(s["ids"], s["case"]["experts"])
    s["rows"].copy_(torch.where((tokens >= 0)[:, None], s["x"][tokens.clamp(min=0).long()], s["rows"]))
    out = {"offsets": offsets, "tokens": tokens, "places": places, "rows": s["rows"]}
    if s["case"]["back"]:
        out["grad_x"] = _taken(s["grad"], places).sum(1).to(s["x"].dtype)
    return out


def _plain_combine(s):
    y = _taken(s["y"], s["places"])
    out = {"out": (y * s["weights"][..., None]).sum(1).to(s["y"].dtype)}
    if s["case"]["back"]:
        grad = s["grad"].float()
        out["grad_weights"] = (y * grad[:, None]).sum(-1)
        here = s["places"] >= 0
        s["rows"][s["places"][here].long()] = (grad[:, None] * s["weights"][..., None])[here].to(s["rows"].dtype)
        out["grad_y"] = s["rows"]
    return out


# ------------------------------------------------------------------------------------- the definitions in 64 bits

def _e4m3(x):
    """The nearest E4M3 value, ties to even, at most 448: a grid of 8 steps to the octave, of 2^-9 below 2^-6."""
    a = x.abs()
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    return torch.copysign((torch.round(a / step) * step).clamp(max=448.0), x)


def _number(codes):
    """Four exponent bits, three of mantissa."""
    b = codes.contiguous().view(torch.uint8)
    table = torch.tensor([(1 - 2 * (i >> 7)) * ((i & 7) / 512 if (i >> 3) & 15 == 0 else 2.0 ** (((i >> 3) & 15) - 7) * (1 + (i & 7) / 8))
                          for i in range(256)], dtype=torch.float64, device=b.device)
    return table[b.int()]


def _scaled(codes, scales, tall):
    """codes [N][K] times the scales of their blocks, block column by block column."""
    x = _number(codes)
    for j in range(scales.shape[1]):
        column = scales[:, j].double()
        x[:, 128 * j:128 * j + 128] *= (column.repeat_interleave(tall)[:x.shape[0]] if tall > 1 else column)[:, None]
    return x


def _exact_quantize(c, s):
    x = s["x"].double()
    if c["form"] == "gated":
        gate, up = x[:, :c["cols"]], x[:, c["cols"]:]
        x = gate * torch.sigmoid(gate) * up
    stack = x if x.dim() == 3 else x[None]
    tall = 128 if c["form"] == "weight" else 1
    codes = torch.empty_like(stack)
    scales = torch.empty((stack.shape[0], -(-c["rows"] // tall), _blocks(c["cols"])), dtype=torch.float64, device="cuda")
    for j in range(scales.shape[2]):
        part = stack[..., 128 * j:128 * j + 128]
        top = part.abs().amax(-1)
        if tall > 1:
            top = torch.nn.functional.pad(top, (0, -top.shape[1] % tall)).unflatten(1, (-1, tall)).amax(-1)
        scales[..., j] = top.clamp(min=2.0 ** -100) / 448.0
        by = scales[..., j].repeat_interleave(tall, 1)[:, :c["rows"]] if tall > 1 else scales[..., j]
        codes[..., 128 * j:128 * j + 128] = _e4m3(part / by[..., None])
    return {"codes": codes.reshape(x.shape), "scales": scales if x.dim() == 3 else scales[0]}


def _exact_experts(c, s):
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    ends = s["offsets"].tolist()
    for e in range(c["experts"]):
        lo, hi = ends[e], ends[e + 1]
        if lo == hi:
            continue
        pick = slice(lo, hi) if s["rows"] is None else s["rows"][lo:hi].long()
        codes = s["a"].view(torch.uint8)[pick]
        out[lo:hi] = _scaled(codes, s["a_scales"][pick], 1) @ _scaled(s["w"][e], s["w_scales"][e], 128).T
    return {"out": out}


def exact(case, seed):
    """Outputs from the definitions, in 64 bits. Places, offsets and copied rows have no such value."""
    c, s = case, prepare(case, seed)
    if c["op"] == "quantize":
        return _exact_quantize(c, s)
    if c["op"] == "product":
        return {"out": _scaled(s["a"], s["a_scales"], 1) @ _scaled(s["w"], s["w_scales"], 128).T}
    if c["op"] == "experts":
        return _exact_experts(c, s)
    if c["op"] == "dispatch":
        if not c["back"]:
            return None
        places = _sorted(s["ids"], c["experts"])[2]
        grad = torch.zeros((c["tokens"], c["width"]), dtype=torch.float64, device="cuda")
        for j in range(c["top"]):
            has = places[:, j] >= 0
            grad[has] += s["grad"][places[has, j].long()].double()
        return {"offsets": None, "tokens": None, "places": None, "rows": None, "grad_x": grad}
    out = torch.zeros((c["tokens"], c["width"]), dtype=torch.float64, device="cuda")
    grad_y = torch.zeros(s["y"].shape, dtype=torch.float64, device="cuda")
    grad_w = torch.zeros(s["weights"].shape, dtype=torch.float64, device="cuda")
    for j in range(c["top"]):
        has = s["places"][:, j] >= 0
        at, weight = s["places"][has, j].long(), s["weights"][has, j].double()[:, None]
        out[has] += weight * s["y"][at].double()
        if c["back"]:
            grad_y[at] = weight * s["grad"][has].double()
            grad_w[has, j] = (s["grad"][has].double() * s["y"][at].double()).sum(1)
    return {"out": out, "grad_y": grad_y, "grad_weights": grad_w} if c["back"] else {"out": out}
