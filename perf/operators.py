"""What the key/value cache's operators are timed and compared on.

The cache holds keys and values in NVFP4 (E2M1 codes, one E4M3 scale for 16 consecutive values of a head, one FP32
global scale per head and side) in pages of `page` tokens. Three operators work on it:

* append:    rotary positions (one to three axes) for queries and keys, then quantization of keys and values into
             the slots of their tokens; the slots are read back as the values that they now stand for;
* attention: softmax(q k^T / sqrt(D)) v over the pages of each sequence, for single tokens, drafted tokens under a
             tree mask, and prefill chunks (causal, with or without a window);
* pages:     fork (share whole pages, copy the one that is partly filled), resize (free or take pages as sequences
             shrink and grow) and compact (move the live pages to the front of the pool, renumber the tables).

Head counts follow the linear layers of the 27B-class model that the library's GEMM workloads use: 6144 = (40 + 2 * 4)
* 128 columns of QKV and 5120 = 40 * 128 of the output projection, over 64 layers. The other sizes are generic.

A page of one layer holds, for each KV head: key codes [page][D/2] (element 2j in the low nibble of byte j), key scales
[page][D/16], value codes in groups of four tokens and eight elements [page/4][D/8][4 tokens][4 bytes], and value scales
[D/16][page].
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
MAX_POS = 16384          # rows of the rotary table


# ------------------------------------------------------------------------------------------------------ the cases

def _append(name, tokens, q_heads=40, kv_heads=4, head_dim=128, rot=128, axes=1, interleaved=False, page=64,
            dtype="bf16", pad=0):
    return dict(name=name, op="append", tokens=tokens, q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim, rot=rot,
                axes=axes, interleaved=interleaved, page=page, dtype=dtype, pad=pad)


def _attention(name, batch, min_len, max_len, min_q=1, max_q=1, q_heads=40, kv_heads=4, head_dim=128, page=64,
               dtype="bf16", window=0, tree=False, pick=1):
    return dict(name=name, op="attention", batch=batch, min_len=min_len, max_len=max_len, min_q=min_q, max_q=max_q,
                q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim, page=page, dtype=dtype, window=window,
                tree=tree, pick=pick)


def _pages(name, op, pool, batch, max_len, layers=64, children=0, page=64, kv_heads=4, head_dim=128, pick=1):
    return dict(name=name, op=op, pool=pool, batch=batch, max_len=max_len, layers=layers, children=children, page=page,
                kv_heads=kv_heads, head_dim=head_dim, pick=pick)


def listed():
    return [
        # one decode step of a full batch: 61 sequences and 3 padding rows of a captured graph
        _append("append_decode_64", 64, pad=3),
        # a prefill chunk of text and image tokens: three axes (time, height, width), keys read out of the QKV product
        _append("append_prefill_8192", 8192, axes=3),
        # the smallest call: one token for one user with a short history, where latency is all
        _attention("decode_1_short", 1, 731, 731, page=16),
        # an ordinary decode step: 64 sequences of very different lengths, one of them empty
        _attention("decode_64_ragged", 64, 0, 8192, pick=2),
        # one user deep in a long document: the only parallelism is along the keys
        _attention("decode_1_long", 1, 262139, 262139, page=256),
        # checking drafted tokens: 3 to 8 of them for each of 32 sequences, in a tree
        _attention("draft_tree_32", 32, 200, 4096, min_q=3, max_q=8, page=32, tree=True, pick=3),
        # prefill chunks on top of cached history: the largest case, bound by arithmetic
        _attention("prefill_4x2048", 4, 2048, 8192, min_q=1501, max_q=2048, pick=4),
        # a small windowed layer in half precision, chunks and single tokens in one ragged batch
        _attention("window_f16", 3, 100, 3000, min_q=1, max_q=777, q_heads=14, kv_heads=2, head_dim=64, page=16,
                   dtype="f16", window=512, pick=5),
        # four samples from one prompt: little to copy, latency counts
        _pages("fork_4", "fork", 256, 2, 1000, children=4, page=16),
        # 64 beams taken from 8 sequences, all layers
        _pages("fork_64", "fork", 320, 8, 1500, children=64, pick=2),
        # sequences end, roll back rejected drafts and grow: bookkeeping over a large pool, no page is moved
        _pages("resize_256", "resize", 65536, 256, 16384, pick=3),
        # the pool is packed before part of it is handed back: 40 % of the pages are alive and scattered
        _pages("compact_3000", "compact", 3000, 48, 512, page=16, pick=4),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    heads = [(40, 4), (32, 8), (14, 2), (28, 4), (8, 8), (16, 1)]
    page = rng.choice([16, 32, 64, 128, 256])
    kind = rng.choice(["append", "attention", "attention", "attention", "pages"])
    if kind == "append":
        hq, hkv = rng.choice(heads)
        d = rng.choice([64, 80, 96, 128, 192, 256])
        c = _append("", _log_int(rng, 1, 4096), hq, hkv, d, rng.choice([d, d // 2]), rng.randint(1, 3),
                    rng.random() < 0.3, page, rng.choice(["bf16", "f16"]), rng.randint(0, 2))
        c["pad"] = min(c["pad"], c["tokens"] - 1)
    elif kind == "attention":
        hq, hkv = rng.choice(heads)
        d = rng.choice([64, 64, 80, 96, 128, 128, 192, 256])
        form = rng.choice(["decode", "decode", "tree", "prefill"])
        top = _log_int(rng, 1, 32768)
        batch, low, min_q, max_q, window = _log_int(rng, 1, 128), rng.choice([0, 1, (top + 1) // 2]), 1, 1, 0
        if form == "tree":
            min_q, max_q = 1, rng.randint(2, 16)
        elif form == "prefill":
            batch, max_q = _log_int(rng, 1, 8), _log_int(rng, 9, 2048)
            min_q = rng.choice([1, (max_q + 1) // 2])
        if form != "tree" and rng.random() < 0.25:
            window = _log_int(rng, 16, 4096)
        c = _attention("", batch, low, top, min_q, max_q, hq, hkv, d, page, rng.choice(["bf16", "f16"]), window,
                       form == "tree", rng.randrange(1 << 20))
        # no dearer than the largest listed case: the padded keys and scores of the plain form count too
        while c["batch"] * c["max_len"] * hkv * d > 1 << 27 or c["batch"] * c["max_q"] * hq * c["max_len"] > 1 << 31:
            c["batch"], c["max_len"] = max(1, c["batch"] * 2 // 3), max(1, c["max_len"] * 3 // 4)
        c["min_len"] = min(c["min_len"], c["max_len"])
    else:
        op = rng.choice(["fork", "resize", "compact"])
        batch = _log_int(rng, 1, 128)
        top = _log_int(rng, 1, 2048)
        if op == "resize":
            top *= rng.choice([1, 8])
        need = batch * -(-top // page)
        pool = need + need // 2 + rng.randint(1, 64)
        children = _log_int(rng, 1, 64) if op == "fork" else 0
        c = _pages("", op, pool + children, batch, top, rng.choice([1, 4, 16, 64]), children, page,
                   rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 256]), rng.randrange(1 << 20))
        while op != "resize" and c["layers"] * c["pool"] * _page_bytes(c) > 2_000_000_000:
            if c["layers"] > 1:
                c["layers"] //= 2
            else:
                c["batch"] = max(1, c["batch"] // 2)
                c["pool"] = c["pool"] // 2 + c["children"] + c["batch"] * -(-top // page)
                if c["batch"] == 1:
                    break
    del c["name"]
    return c


def _page_bytes(c):
    return c["kv_heads"] * c["page"] * (c["head_dim"] // 16) * 18


def _lengths(c):
    """(cached tokens, new queries) of each sequence: part of the case, not of the seed."""
    r = random.Random(c["pick"])
    lens, counts = [], []
    for b in range(c["batch"]):
        n = r.randint(c.get("min_q", 1), c.get("max_q", 1))
        low = max(1, c.get("min_len", 1))
        lens.append(min(c["max_len"], max(low, _log_int(r, low, max(low, c["max_len"])))))
        counts.append(n)
    if c["batch"] > 1:
        lens[0] = c["max_len"]
        lens[-1] = c.get("min_len", 1)
        counts[0] = c.get("max_q", 1)
    # a sequence shorter than its queries: the first of them have no key to see
    return lens, counts


def _pairs(c):
    """(query, key) pairs that a causal (windowed) pass attends, per query head; a tree mask leaves about half of the
    new keys."""
    total, w = 0, c["window"]
    lens, counts = _lengths(c)
    for n, q in zip(lens, counts):
        first, last = n - q + 1, n                       # keys that the first and the last query see
        for lo, hi in ((max(1, first), last),):
            if w and hi > w:
                total += (hi - max(lo, w + 1) + 1) * w
                hi = min(hi, w)
            if hi >= lo:
                total += (lo + hi) * (hi - lo + 1) // 2
    return total


def work(case):
    c = case
    if c["op"] == "append":
        d, t = c["head_dim"], c["tokens"]
        rows = t * c["head_dim"] * 2
        table = min(t, MAX_POS) * c["rot"] * 4
        moved = rows * (2 * c["q_heads"] + 2 * c["kv_heads"]) + table          # q in and out, k and v in
        cached = 2 * t * c["kv_heads"] * d * 9 // 16
        return {"bytes": moved + 2 * cached + 2 * rows * c["kv_heads"], "flops": 3 * t * c["rot"] * (c["q_heads"] + c["kv_heads"])}
    if c["op"] == "attention":
        lens, counts = _lengths(c)
        seen = sum(min(n, c["window"] + q) if c["window"] else n for n, q in zip(lens, counts))
        rows = sum(counts) * c["q_heads"]
        return {"bytes": seen * c["kv_heads"] * c["head_dim"] * 9 // 8 + rows * (4 * c["head_dim"] + 4),
                "flops": 4 * c["head_dim"] * c["q_heads"] * _pairs(c)}
    lens, _ = _lengths(c)
    tables = 4 * sum(-(-n // c["page"]) for n in lens)
    if c["op"] == "resize":
        return {"bytes": 8 * c["pool"] + 2 * tables + 8 * c["batch"], "flops": 0}
    if c["op"] == "fork":
        moved = sum(1 for p in _parents(c) if lens[p] % c["page"])
        new = 8 * sum(-(-lens[p] // c["page"]) for p in _parents(c))
        return {"bytes": 2 * moved * c["layers"] * _page_bytes(c) + 8 * c["pool"] + new, "flops": 0}
    live = sum(-(-n // c["page"]) for n in lens)
    moved = live * (c["pool"] - live) // c["pool"]         # live pages past the first `live`, as they lie on average
    return {"bytes": 2 * moved * c["layers"] * _page_bytes(c) + 8 * c["pool"] + 2 * tables, "flops": 0}


def _parents(c):
    r = random.Random(c["pick"] + 1)
    return [r.randrange(c["batch"]) for _ in range(c["children"])]


# ----------------------------------------------------------------------------------------------------- the inputs

def _heads(pages, c):
    """Views of a pool [pages][bytes]: key codes and scales [pages][heads][page][...], value codes
    [pages][heads][page/4][4][D/8][4], value scales [pages][heads][page][D/16]."""
    p, d, h = c["page"], c["head_dim"], c["kv_heads"]
    x = pages[:, :_page_bytes(c)].unflatten(1, (h, p * d * 9 // 8))
    cuts = [0, p * d // 2, p * d * 9 // 16, p * d * 17 // 16, p * d * 9 // 8]
    k, ks, v, vs = (x[:, :, a:b] for a, b in zip(cuts, cuts[1:]))
    return [k.unflatten(2, (p, d // 2)), ks.unflatten(2, (p, d // 16)),
            v.unflatten(2, (p // 4, d // 8, 4, 4)).transpose(3, 4), vs.unflatten(2, (d // 16, p)).transpose(2, 3)]


def _tokens(v_codes, page, at):
    """The value codes [T][heads][D/2] of tokens by page and place."""
    return v_codes[page, :, at // 4, at % 4].flatten(2)


def _quantize(x, g):
    """[..][D] in 32 bits under the global scale g (a number per row, broadcast) -> packed codes, scale bytes."""
    y = x.unflatten(-1, (-1, 16))
    top = y.abs().amax(-1)
    byte = ((top / 6.0) * g).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = byte.float()
    r = torch.where(s != 0, g / torch.where(s != 0, s, 1.0), 0.0)
    v = (y * r[..., None]).abs()
    step = torch.where(v < 2.0, 0.5, torch.where(v < 4.0, 1.0, 2.0))
    v = (torch.round(v / step) * step).clamp(max=6.0)
    code = torch.where(v < 2.0, 2.0 * v, torch.where(v < 4.0, v + 2.0, 4.0 + v / 2.0))
    code = torch.where(s[..., None].isnan(), 0.0, code).to(torch.uint8)
    code = torch.where(s[..., None] != 0, code | (torch.signbit(y).to(torch.uint8) << 3), 0).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), byte.view(torch.uint8)


def _values(codes, scales):
    """Codes times block scales, in 32 bits: [..][D/2], [..][D/16] -> [..][D]."""
    lut = torch.tensor(E2M1, device=codes.device)
    v = torch.stack([lut[(codes & 15).int()], lut[(codes >> 4).int()]], -1).flatten(-2)
    return (v.unflatten(-1, (-1, 16)) * scales.view(torch.float8_e4m3fn).float()[..., None]).flatten(-2)


def _key_like(shape, gen):
    """Keys as layers make them: a few strong channels, the same ones at every position."""
    x = torch.randn(shape, generator=gen, device="cuda")
    strong = 1.0 + 5.0 * (torch.rand(shape[1:], generator=gen, device="cuda") < 0.04).float()
    return x * strong


def _tables(c, lens, gen, ids):
    """Page tables [batch][width]: pages in no order, -1 past each sequence's end."""
    width = max(1, -(-max(c["max_len"], 1) // c["page"])) + 3
    cols = torch.arange(width, device="cuda")
    need = (lens + c["page"] - 1) // c["page"]
    use = cols[None, :] < need[:, None]
    at = torch.cumsum(use.flatten().long(), 0).reshape(use.shape) - 1
    return torch.where(use, ids[at.clamp(min=0)], -1).int()


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if c["op"] == "append":
        return _prepare_append(c, gen)
    if c["op"] == "attention":
        return _prepare_attention(c, gen)
    return _prepare_pages(c, gen)


def _prepare_append(c, gen):
    t, d, hq, hkv, p = c["tokens"], c["head_dim"], c["q_heads"], c["kv_heads"], c["page"]
    dtype = DTYPES[c["dtype"]]
    qkv = torch.randn((t, (hq + 2 * hkv) * d), generator=gen, device="cuda")
    qkv[:, hq * d:(hq + hkv) * d] = _key_like((t, hkv * d), gen)
    qkv = qkv.to(dtype)
    q, k, v = (x.unflatten(1, (-1, d)) for x in qkv.split([hq * d, hkv * d, hkv * d], 1))
    # a long prompt fills pages in order; a decode step writes one token to each of many pages
    fresh = t > 128
    n_pages = -(-t // p) + 2 if fresh else 2 * t
    order = torch.randperm(n_pages, generator=gen, device="cuda")
    i = torch.arange(t, device="cuda")
    if fresh:
        slots = order[(i + 5) // p] * p + (i + 5) % p
    else:
        slots = order[i] * p + torch.randint(0, p, (t,), generator=gen, device="cuda")
    if c["pad"]:
        slots[t - c["pad"]:] = -1
    # calibrated on other data: a few blocks reach past the largest scale and saturate
    k_g = 2688.0 / (24.0 + 4.0 * torch.rand(hkv, generator=gen, device="cuda"))
    v_g = 2688.0 / (4.0 + torch.rand(hkv, generator=gen, device="cuda"))
    half = c["rot"] // 2
    freq = 1e6 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / max(1, half))
    angle = torch.arange(MAX_POS, device="cuda", dtype=torch.float64)[:, None] * freq
    if fresh:
        pos = i[None, :].repeat(c["axes"], 1)
        image = (i // 97) % 2 == 1                          # runs of image patches between runs of text
        for a in range(1, c["axes"]):
            pos[a] = torch.where(image, i - i % 97 + (i % 97) // (1 if a == 2 else 10), i)
    else:
        pos = torch.randint(0, MAX_POS, (1, t), generator=gen, device="cuda").repeat(c["axes"], 1)
    axis_of = None
    if c["axes"] > 1:                                       # the first quarter of the pairs turns with time
        axis_of = (torch.arange(half, device="cuda") * 4 // max(1, half)).clamp(max=c["axes"] - 1).to(torch.uint8)
    pages = torch.full((n_pages, _page_bytes(c)), 0, dtype=torch.uint8, device="cuda")
    s = dict(case=c, q=q, k=k, v=v, slots=slots, k_g=k_g, v_g=v_g, cos=torch.cos(angle).float(),
             sin=torch.sin(angle).float(), positions=pos.int().contiguous(), axis_of=axis_of, pages=pages,
             q_out=torch.empty((t, hq, d), dtype=dtype, device="cuda"))
    if own:
        s["cache"] = _cache(s)
    return s


def _cache(s):
    import nvfp4_block_scaled_amd as nv
    c = s["case"]
    return nv.KVCache(s["pages"], c["page"], c["kv_heads"], c["head_dim"], s["k_g"], s["v_g"])


def _prepare_attention(c, gen):
    lens, counts = _lengths(c)
    d, hkv, p = c["head_dim"], c["kv_heads"], c["page"]
    n = torch.tensor(lens, device="cuda")
    used = sum(-(-x // p) for x in lens)
    n_pages = used + 2 + used // 8
    ids = torch.randperm(n_pages, generator=gen, device="cuda")
    table = _tables(c, n, gen, ids)
    # pages that nobody owns, and slots past a sequence's end, hold what was there before: any byte, NaN scales too
    pages = torch.randint(0, 256, (n_pages, _page_bytes(c)), generator=gen, device="cuda", dtype=torch.uint8)
    k_g = 2688.0 / (28.0 + 4.0 * torch.rand(hkv, generator=gen, device="cuda"))
    v_g = 2688.0 / (5.0 + torch.rand(hkv, generator=gen, device="cuda"))
    sections = _heads(pages, c)
    owned = table[table >= 0].long()
    filled = torch.zeros((n_pages, p), dtype=torch.bool, device="cuda")
    cols = torch.arange(table.shape[1], device="cuda")
    left = (n[:, None] - cols * p)[table >= 0]
    filled[owned] = torch.arange(p, device="cuda") < left[:, None]
    for lo in range(0, n_pages, 4096):
        hi = min(n_pages, lo + 4096)
        keep = filled[lo:hi, None, :, None]
        for side, g in ((0, k_g), (2, v_g)):
            x = torch.randn((hi - lo, hkv, p, d), generator=gen, device="cuda")
            if side == 0:
                x *= 1.0 + 5.0 * ((torch.arange(hkv * d, device="cuda").reshape(hkv, 1, d) * 7919) % 97 < 4).float()
            codes, scales = _quantize(x, g.reshape(hkv, 1, 1))
            kept = keep
            if side == 2:                                       # four tokens to a group
                codes, kept = codes.unflatten(2, (p // 4, 4)).unflatten(4, (d // 8, 4)), keep.unflatten(2, (p // 4, 4))[..., None]
            sections[side][lo:hi] = torch.where(kept, codes, sections[side][lo:hi])
            sections[side + 1][lo:hi] = torch.where(keep, scales, sections[side + 1][lo:hi])
    t, most = sum(counts), max(counts)
    q = (torch.randn((t, c["q_heads"], d), generator=gen, device="cuda") * 0.7).to(DTYPES[c["dtype"]])
    start = torch.tensor([0] + counts, device="cuda").cumsum(0).int()
    mask = None
    if c["tree"]:                     # each drafted token sees itself, its parent and the parent's ancestors
        parent = (torch.rand((t,), generator=gen, device="cuda") * torch.arange(t, device="cuda")).long()
        mask = torch.zeros((t, most), dtype=torch.bool, device="cuda")
        row = torch.arange(t, device="cuda") - torch.repeat_interleave(start[:-1].long(), torch.tensor(counts, device="cuda"))
        first = torch.arange(t, device="cuda") - row
        parent = torch.where(row > 0, first + parent % row.clamp(min=1), first)
        at = torch.arange(t, device="cuda")
        for _ in range(most):
            mask[torch.arange(t, device="cuda"), at - first] = True
            at = parent[at]
    s = dict(case=c, q=q, table=table, lens=n.int(), start=start, mask=mask, pages=pages, k_g=k_g, v_g=v_g, most=most,
             counts=counts, one=c["min_q"] == c["max_q"] == 1, scale=d ** -0.5,
             out=torch.empty((t, c["q_heads"], d), dtype=q.dtype, device="cuda"))
    if own:
        import nvfp4_block_scaled_amd as nv
        s["cache"] = _cache(s)
        s["ws"] = nv.nvfp4_kv_attention_workspace(t, c["q_heads"], s["cache"], c["batch"], table.shape[1], most)
    return s


def _prepare_pages(c, gen):
    lens, _ = _lengths(c)
    n = torch.tensor(lens, device="cuda")
    ids = torch.randperm(c["pool"], generator=gen, device="cuda")
    table = _tables(c, n, gen, ids)
    refs = torch.zeros(c["pool"], dtype=torch.int32, device="cuda")
    refs[table[table >= 0].long()] = 1
    if c["batch"] > 2:                # two sequences share what the shorter one has of whole pages
        whole = (n[1:3] // c["page"]).min()
        cols = torch.arange(table.shape[1], device="cuda")
        old = table[2].clone()
        shared = (cols < whole) & (old >= 0)
        refs[old[shared].long()] -= 1
        table[2] = torch.where(shared, table[1], old)
        refs[table[2][shared].long()] += 1
    s = dict(case=c, table=table, refs=refs, lens=n.int())
    if c["op"] == "resize":           # a quarter ends, a quarter gives back drafted tokens, the rest grows
        b = torch.arange(c["batch"], device="cuda")
        step = torch.randint(1, 2 * c["page"], (c["batch"],), generator=gen, device="cuda")
        room = (table.shape[1] * c["page"])
        new = torch.where(b % 4 == 3, 0, torch.where(b % 4 == 1, (n - step).clamp(min=0), (n + step).clamp(max=room)))
        s["new_lens"] = new.int()
        return s
    size = c["layers"] * c["pool"] * _page_bytes(c)
    s["pages"] = torch.randint(-2 ** 31, 2 ** 31 - 1, (size // 4,), generator=gen, device="cuda",
                               dtype=torch.int32).view(torch.uint8).reshape(c["layers"], c["pool"], _page_bytes(c))
    if c["op"] == "fork":
        s["parents"] = torch.tensor(_parents(c), device="cuda").int()
    return s


# ------------------------------------------------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return _own(op, state)
    return {"append": _plain_append, "attention": _plain_attention, "fork": _plain_fork, "resize": _plain_resize,
            "compact": _plain_compact}[op](state)


def _own(op, s):
    import nvfp4_block_scaled_amd as nv
    c = s["case"]
    if op == "append":
        q = nv.nvfp4_kv_append(s["cache"], s["k"], s["v"], s["slots"], q=s["q"], cos=s["cos"], sin=s["sin"],
                               positions=s["positions"], axis_of=s["axis_of"], interleaved=c["interleaved"],
                               q_out=s["q_out"])
        k, v = nv.nvfp4_kv_read(s["cache"], s["slots"], s["k"].dtype)
        return {"q": q, "k": k, "v": v}
    if op == "attention":
        out, lse = nv.nvfp4_kv_attention(s["q"], s["cache"], s["table"], s["lens"], None if s["one"] else s["start"],
                                         s["most"], scale=s["scale"], window=c["window"], mask=s["mask"], out=s["out"],
                                         return_lse=True, ws=s["ws"])
        return {"out": out, "lse": lse}
    if op == "fork":
        table, refs, short = nv.nvfp4_kv_fork(s["pages"], s["table"], s["lens"], s["refs"], s["parents"], c["page"])
        return {"table": table, "refs": refs, "short": short, "pages": s["pages"].view(torch.int32)}
    if op == "resize":
        table, refs, short = nv.nvfp4_kv_resize(s["table"], s["lens"], s["new_lens"], s["refs"], c["page"])
        return {"table": table, "refs": refs, "short": short}
    table, refs, live = nv.nvfp4_kv_compact(s["pages"], s["table"], s["refs"])
    return {"table": table, "refs": refs, "live": live, "pages": s["pages"].view(torch.int32)}


def _rotate(x, s):
    """Rotary positions in 32 bits: x [T][heads][D]; the first `rot` values of a head turn in pairs."""
    c = s["case"]
    half = c["rot"] // 2
    axis = s["axis_of"].long() if s["axis_of"] is not None else torch.zeros(half, dtype=torch.long, device=x.device)
    at = s["positions"].long()[axis].T                                     # [T][half]: the position of each pair
    cos, sin = s["cos"].gather(0, at)[:, None], s["sin"].gather(0, at)[:, None]
    x = x.float()
    turn, rest = x[..., :c["rot"]], x[..., c["rot"]:]
    if c["interleaved"]:
        a, b = turn[..., 0::2], turn[..., 1::2]
        return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2), rest], -1)
    a, b = turn[..., :half], turn[..., half:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin, rest], -1)


def _plain_append(s):
    c = s["case"]
    p, hkv = c["page"], c["kv_heads"]
    s["q_out"].copy_(_rotate(s["q"], s))
    k_codes, k_scales, v_codes, v_scales = _heads(s["pages"], c)
    fits = (s["slots"] >= 0) & (s["slots"] < s["pages"].shape[0] * p)
    page, at = s["slots"][fits] // p, s["slots"][fits] % p
    g_k, g_v = s["k_g"].reshape(hkv, 1), s["v_g"].reshape(hkv, 1)
    k_codes[page, :, at], k_scales[page, :, at] = _quantize(_rotate(s["k"], s)[fits], g_k)
    codes, v_scales[page, :, at] = _quantize(s["v"][fits].float(), g_v)
    v_codes[page, :, at // 4, at % 4] = codes.unflatten(2, (-1, 4))
    page, at = s["slots"].clamp(min=0) // p, s["slots"].clamp(min=0) % p
    k = _values(k_codes[page, :, at], k_scales[page, :, at]) / g_k
    v = _values(_tokens(v_codes, page, at), v_scales[page, :, at]) / g_v
    keep = fits[:, None, None]
    return {"q": s["q_out"], "k": torch.where(keep, k, 0.0).to(s["k"].dtype), "v": torch.where(keep, v, 0.0).to(s["k"].dtype)}


def _plain_attention(s):
    c = s["case"]
    p, d, hq, hkv, b, most = c["page"], c["head_dim"], c["q_heads"], c["kv_heads"], c["batch"], s["most"]
    width = max(1, -(-c["max_len"] // p))
    held = [x[s["table"][:, :width].long().clamp(min=0)].transpose(1, 2) for x in _heads(s["pages"], c)]
    held[2] = held[2].flatten(5).flatten(3, 4)                             # value codes token by token again
    held = [x.flatten(4).flatten(2, 3) for x in held]
    g_k, g_v = s["k_g"].reshape(hkv, 1, 1), s["v_g"].reshape(hkv, 1, 1)
    k = _values(held[0], held[1]) / g_k                                    # [batch][kv head][key][D]
    v = _values(held[2], held[3]) / g_v
    key = torch.arange(width * p, device=k.device)
    lens, start = s["lens"].long(), s["start"].long()
    v = torch.where((key < lens[:, None])[:, None, :, None], v, 0.0)       # what lies past the end may be NaN
    count = start[1:] - start[:-1]
    i = torch.arange(most, device=k.device)
    rows = (start[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)           # [batch][query], padded to the longest
    q = s["q"][rows].float().unflatten(2, (hkv, hq // hkv)).permute(0, 2, 1, 3, 4).flatten(2, 3)
    at = lens[:, None] - count[:, None] + i                                # the query's own position
    see = (key[None, None, :] <= at[:, :, None]) & (key < lens[:, None, None])
    if c["window"]:
        see &= key[None, None, :] > at[:, :, None] - c["window"]
    if s["mask"] is not None:
        new = key[None, :] - (lens - count)[:, None]                       # which new token a key is, < 0: an old one
        m = s["mask"][rows].gather(2, new.clamp(0, most - 1)[:, None, :].expand(-1, most, -1))
        see = (key < lens[:, None, None]) & ((new < 0)[:, None, :] | m)
    see = see.repeat_interleave(hq // hkv, 1)[:, None]
    x = torch.where(see, torch.matmul(q, k.transpose(2, 3)) * s["scale"], -math.inf)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    x = torch.exp(x - top)
    total = x.sum(-1, keepdim=True)
    out = torch.matmul(x, v) / torch.where(total == 0, 1.0, total)
    lse = (top + torch.log(total))[..., 0]
    seq = torch.repeat_interleave(torch.arange(b, device=k.device), count, output_size=s["q"].shape[0])
    row = torch.arange(s["q"].shape[0], device=k.device) - start[seq]
    out = out.unflatten(2, (most, hq // hkv)).permute(0, 2, 1, 3, 4).flatten(2, 3)[seq, row]
    lse = lse.unflatten(2, (most, hq // hkv)).permute(0, 2, 1, 3).flatten(2, 3)[seq, row]
    return {"out": out.to(s["q"].dtype), "lse": lse}


def _free_pages(refs, most):
    """The first free pages in ascending order (at least `most` entries), and how many there are."""
    order = torch.argsort((refs > 0).int(), stable=True)[:max(1, most)]
    return order.int(), (refs <= 0).sum()


def _plain_fork(s):
    c = s["case"]
    p, parents = c["page"], s["parents"].long()
    n = s["lens"].long()[parents]
    whole, part = n // p, n % p > 0
    free, count = _free_pages(s["refs"], len(parents))
    rank = torch.cumsum(part.long(), 0) - 1
    served = ~part | (rank < count)
    new = free[rank.clamp(0, free.shape[0] - 1)]
    cols = torch.arange(s["table"].shape[1], device=n.device)
    old = s["table"][parents]
    shared = (cols < whole[:, None]) & served[:, None]
    last = (cols == whole[:, None]) & (part & served)[:, None]
    table = torch.where(shared, old, torch.where(last, new[:, None], -1))
    refs = s["refs"].clone()
    refs.scatter_add_(0, old.clamp(min=0).long().flatten(), shared.int().flatten())
    refs[table[last].long()] = 1
    s["pages"][:, table[last].long()] = s["pages"][:, old[last].long()]
    return {"table": table, "refs": refs, "short": (~served).sum().int().reshape(1), "pages": s["pages"].view(torch.int32)}


def _plain_resize(s):
    p = s["case"]["page"]
    was, now = (s["lens"].long() + p - 1) // p, (s["new_lens"].long() + p - 1) // p
    cols = torch.arange(s["table"].shape[1], device=was.device)
    drop = (cols >= now[:, None]) & (cols < was[:, None])
    grow = (cols >= was[:, None]) & (cols < now[:, None])
    refs = s["refs"].clone()
    refs.scatter_add_(0, s["table"].clamp(min=0).long().flatten(), -drop.int().flatten())
    free, count = _free_pages(refs, grow.numel())
    rank = (torch.cumsum(grow.flatten().long(), 0) - 1).reshape(grow.shape)
    take = grow & (rank < count)
    new = free[rank.clamp(0, free.shape[0] - 1)]
    table = torch.where(take, new, torch.where(drop | grow, -1, s["table"]))
    refs[table[take].long()] = 1
    return {"table": table, "refs": refs, "short": (grow & ~take).sum().int().reshape(1)}


def _plain_compact(s):
    refs, table = s["refs"], s["table"]
    live = refs > 0
    count = live.sum()
    ids = torch.arange(refs.shape[0], device=refs.device)
    src = ids[live & (ids >= count)]
    dst = ids[~live & (ids < count)]
    to = ids.clone()
    to[src] = dst
    s["pages"][:, dst] = s["pages"][:, src]
    new = torch.where(ids < count, refs, 0)
    new[dst] = refs[src]
    moved = to[table.clamp(min=0).long()].int()
    return {"table": torch.where(table >= 0, moved, table), "refs": new, "live": count.int().reshape(1),
            "pages": s["pages"].view(torch.int32)}


# ------------------------------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    """Outputs from the definitions, in 64 bits, one sequence (or all tokens of an append) at a time. Tables, counts
    and copied pages are whole numbers and have no such value."""
    if case["op"] == "append":
        return _exact_append(case, prepare(case, seed))
    if case["op"] == "attention":
        return _exact_attention(case, prepare(case, seed))
    return None


def _e4m3(x):
    """The nearest E4M3 value of x >= 0, ties to even, at most 448: a grid of 8 steps to the octave, of 2^-9 below 2^-6."""
    step = torch.exp2(torch.floor(torch.log2(x.clamp(min=2.0 ** -6))) - 3)
    return (torch.round(x / step) * step).clamp(max=448.0)


def _e2m1(x):
    """The nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 to |x|, ties to the even code, with x's sign."""
    a = x.abs()
    step = torch.exp2(torch.floor(torch.log2(a.clamp(1.0, 4.0))) - 1)
    return torch.copysign((torch.round(a / step) * step).clamp(max=6.0), x)


def _held(x, g):
    """What a cache holds of x [..][D] under the global scale g: code * scale / g, block by block of 16."""
    y = x.reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    s = _e4m3(y.abs().amax(-1, keepdim=True) / 6 * g[..., None])
    return torch.where(s > 0, _e2m1(y * g[..., None] / s.clamp(min=2.0 ** -10)) * s / g[..., None], 0.0).reshape(x.shape)


def _exact_append(c, s):
    half = c["rot"] // 2

    def turned(x):
        x = x.double()
        out = x.clone()
        for j in range(half):
            axis = 0 if s["axis_of"] is None else int(s["axis_of"][j])
            at = s["positions"][axis].long()
            cos, sin = s["cos"][at, j].double()[:, None], s["sin"][at, j].double()[:, None]
            a, b = (2 * j, 2 * j + 1) if c["interleaved"] else (j, j + half)
            out[..., a] = x[..., a] * cos - x[..., b] * sin
            out[..., b] = x[..., b] * cos + x[..., a] * sin
        return out

    keep = (s["slots"] >= 0)[:, None, None]
    return {"q": turned(s["q"]), "k": torch.where(keep, _held(turned(s["k"]), s["k_g"].double()[:, None]), 0.0),
            "v": torch.where(keep, _held(s["v"].double(), s["v_g"].double()[:, None]), 0.0)}


def _exact_attention(c, s):
    d, p, hq, hkv = c["head_dim"], c["page"], c["q_heads"], c["kv_heads"]
    size, group = p * d * 9 // 8, hq // hkv

    def number(codes, scales):
        """E2M1: sign, two exponent bits, one of mantissa; E4M3: sign, four, three."""
        n = torch.stack([codes & 15, codes >> 4], -1).flatten(1).long()
        e, m = (n >> 1) & 3, (n & 1).double()
        v = torch.where(e == 0, m / 2, torch.exp2(e.double() - 1) * (1 + m / 2)) * (1 - 2 * (n >> 3))
        b = scales.long()
        e, m = (b >> 3) & 15, (b & 7).double()
        f = torch.where(e == 0, m / 512, torch.exp2(e.double() - 7) * (1 + m / 8)) * (1 - 2 * (b >> 7))
        return v * f.repeat_interleave(16, 1)

    out = torch.zeros((s["q"].shape[0], hq, d), dtype=torch.float64, device="cuda")
    lse = torch.full((s["q"].shape[0], hq), -math.inf, dtype=torch.float64, device="cuda")
    row = 0
    for b, (n, count) in enumerate(zip(_lengths(c)[0], s["counts"])):
        rows = slice(row, row + count)
        row += count
        if n == 0:
            continue
        raw = s["pages"][s["table"][b, :-(-n // p)].long(), :hkv * size].reshape(-1, hkv, size)
        key = torch.arange(n, device="cuda")
        own_pos = n - count + torch.arange(count, device="cuda")[:, None]
        see = key <= own_pos
        if c["window"]:
            see = see & (own_pos - key < c["window"])
        if s["mask"] is not None:
            new = min(n, count)
            see = torch.ones((count, n), dtype=torch.bool, device="cuda")
            see[:, n - new:] = s["mask"][rows, count - new:count]
        for h in range(hkv):
            x = raw[:, h]
            codes, scales = x[:, :p * d // 2].reshape(-1, d // 2), x[:, p * d // 2:p * d * 9 // 16].reshape(-1, d // 16)
            k = number(codes[:n], scales[:n]) / s["k_g"][h].double()
            codes = x[:, p * d * 9 // 16:p * d * 17 // 16].reshape(-1, d // 8, 4, 4).permute(0, 2, 1, 3).reshape(-1, d // 2)
            scales = x[:, p * d * 17 // 16:].reshape(-1, d // 16, p).permute(0, 2, 1).reshape(-1, d // 16)
            v = number(codes[:n], scales[:n]) / s["v_g"][h].double()
            for j in range(h * group, (h + 1) * group):
                z = (s["q"][rows, j].double() @ k.T) * s["scale"]
                z = torch.where(see, z, -math.inf)
                total = torch.logsumexp(z, 1)
                weight = torch.where(see, torch.exp(z - torch.where(total.isinf(), 0.0, total)[:, None]), 0.0)
                out[rows, j] = weight @ v
                lse[rows, j] = total
    return {"out": out, "lse": lse}
