"""FP8 products and the experts' operators where other tests do not look: gates far from zero, tensors of a call over one another."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_amd as nv
from oracle import fp8

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def rng(seed):
    return np.random.default_rng(seed)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
def test_gates_far_from_zero(kind):
    """A gate masked with a large negative value takes no part, however large the factor; one a little below -87, whose e^g
    FP32 does not hold, does where the factor brings the product back. A row has one gate, alone in a block (with factors up
    to u) and beside ordinary values in the next, for each u. e^g is off by an ulp of 2^t and half of one of its correction,
    two products by half each: 2.5 ulps, under 2^-21 of the value; the scale by that and its own half step, and a code's value
    by half a step of E4M3 (2^-4 of the value, at least 2^-10 of a scale) and that."""
    r = rng(7)
    dtype = TYPES[kind]
    low = torch.finfo(dtype).min
    gates = [-86.5, -87.0, -87.5, -88.0, -88.7, -89.0, -95.0, -103.0, -104.0, -110.0, -150.0, -1e3, -1e4, low / 2, low, 86.5, 88.0, 200.0]
    if kind != "f16":
        gates += [-170.0, -179.0, -181.0, -1e10, -1e30]
    us = [1.0, -3.0, 300.0] + ([6e4] if kind == "f16" else [1e10, -1e30, 1e35, 3e38])
    M, K = len(gates), 256 * len(us)
    g, u = r.standard_normal((M, K)) * 4, r.standard_normal((M, K)) * 1e-3
    for b, top in enumerate(us):
        for i, gate in enumerate(gates):
            v = top if gate < 0 else np.sign(top) * min(abs(top), 300.0)          # g u stays in range
            g[i, 256 * b:256 * b + 128] = gate
            u[i, 256 * b:256 * b + 128] = v * r.uniform(0.1, 1.0, 128)
            g[i, 256 * b + 128 + 5 * b], u[i, 256 * b + 128 + 5 * b] = gate, v
    x = torch.from_numpy(np.concatenate([g, u], 1)).to(dtype)
    codes, scales = nv.nvfp4_fp8_quantize(x.cuda(), gated=True)
    want = fp8.silu_mul(x.double().numpy())
    top = np.abs(want).reshape(M, -1, 128).max(2)
    assert top[gates.index(low)].max() < 1.0 and (kind == "f16" or top.max() > 100.0)
    s = np.maximum(top, 2.0 ** -100) / 448.0
    got_s = scales.cpu().numpy().astype(np.float64)
    assert (np.abs(got_s - s) <= (2.0 ** -21 + 2.0 ** -24) * s).all()
    wide_s = fp8.spread(got_s, 1, want.shape)
    got = fp8.values(codes.view(torch.uint8).cpu().numpy()) * wide_s
    tol = np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10 * wide_s) * (1 + 2.0 ** -18) + 2.0 ** -20 * np.abs(want)
    assert (np.abs(got - want) <= tol).all()


@pytest.mark.gpu
@pytest.mark.parametrize("g,u", [(-np.inf, 0.0), (-np.inf, 1.0), (np.inf, 1.0), (np.nan, 1.0), (-1e4, np.inf), (-1e4, np.nan), (-100.0, -np.inf),
                                 (200.0, np.nan)])
def test_gates_far_from_zero_keep_nan_and_infinity(g, u):
    """An infinity or a NaN of either half makes its block's scale and codes NaN, and no other's."""
    x = torch.ones((3, 2 * 384))
    x[1, 130], x[1, 384 + 130] = g, u
    codes, scales = nv.nvfp4_fp8_quantize(x.cuda(), gated=True)
    assert scales.isnan().cpu().tolist() == [[False] * 3, [False, True, False], [False] * 3]
    assert int(codes.float().isnan().sum()) == 128 and bool(codes.float()[1, 128:256].isnan().all())


class Room:
    """Tensors at chosen bytes of one buffer."""

    def __init__(self, size):
        self.bytes = torch.zeros(size, dtype=torch.uint8, device="cuda")

    def at(self, first, shape, dtype=torch.float32):
        n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
        return self.bytes[first:first + n].view(dtype).view(shape)


def refused(call):
    with pytest.raises(ValueError, match="overlaps"):
        call()


@pytest.mark.gpu
def test_rows_over_places_or_weights_are_refused():
    """A workgroup would read places that another one's rows have replaced."""
    room = Room(1 << 16)
    places, weights = room.at(1024, (4, 2), torch.int32), room.at(2048, (4, 2))          # 32 bytes each
    x, y = torch.ones((4, 8), device="cuda"), torch.ones((8, 8), device="cuda")
    places.copy_(torch.arange(8, device="cuda").view(4, 2))
    for first in (1056, 2048, 1024 - 256):                                               # behind, over the weights, before
        nv.nvfp4_moe_gather(x, places, out=room.at(first, (8, 8)))
    nv.nvfp4_moe_combine(y, places, out=room.at(2048, (4, 8)))
    nv.nvfp4_moe_combine(y, places, weights, out=room.at(2080, (4, 8)))
    nv.nvfp4_moe_combine_backward(x, y, places, weights, grad_y=room.at(2080, (8, 8)))
    torch.cuda.synchronize()
    assert places.flatten().tolist() == list(range(8))
    for first in (1052, 1024, 1024 - 252):
        refused(lambda: nv.nvfp4_moe_gather(x, places, out=room.at(first, (8, 8))))
        refused(lambda: nv.nvfp4_moe_gather_backward(y, places, out=room.at(min(first + 128, 1052), (4, 8))))
        refused(lambda: nv.nvfp4_moe_combine_backward(x, y, places, weights, grad_y=room.at(first, (8, 8))))
    for first in (2076, 2048, 2048 - 124):
        refused(lambda: nv.nvfp4_moe_combine(y, places, weights, out=room.at(first, (4, 8))))
        refused(lambda: nv.nvfp4_moe_combine_backward(x, y, places, weights, grad_y=room.at(first, (8, 8))))


@pytest.mark.gpu
def test_codes_over_scales_are_refused():
    room = Room(1 << 16)
    x = torch.ones((4, 256), device="cuda")
    codes = room.at(1024, (4, 256), torch.float8_e4m3fn)
    nv.nvfp4_fp8_quantize(x, codes=codes, scales=room.at(2048, (4, 2)))
    nv.nvfp4_fp8_quantize_weight(x, codes=codes, scales=room.at(1016, (1, 2)))
    for first in (2044, 1024, 1024 - 28):
        refused(lambda: nv.nvfp4_fp8_quantize(x, codes=codes, scales=room.at(first, (4, 2))))
    refused(lambda: nv.nvfp4_fp8_quantize_weight(x, codes=codes, scales=room.at(1020, (1, 2))))


@pytest.mark.gpu
def test_workspaces_over_other_tensors_are_refused():
    """As far as the call uses them; what lies behind that in a larger one is no matter."""
    M, N, K = 4, 260, 4112
    need = nv.lib().nvfp4_fp8_gemm_workspace_bytes(M, N, K)
    assert need > 0
    room = Room(need + (1 << 23))
    sizes = [((M, K), torch.float8_e4m3fn), ((M, fp8.blocks(K)), torch.float32), ((N, K), torch.float8_e4m3fn),
             ((fp8.blocks(N), fp8.blocks(K)), torch.float32), ((M, N), torch.bfloat16)]
    behind, first = [], -(-need // 256) * 256
    for shape, dtype in sizes:
        behind.append(room.at(first, shape, dtype))
        first += -(-int(np.prod(shape)) * 4 // 256) * 256
    ws = room.bytes
    nv.nvfp4_fp8_gemm(*behind[:4], out=behind[4], ws=ws)
    for i in range(5):
        t = list(behind)
        t[i] = room.at((need - 1) // 256 * 256, *sizes[i])
        refused(lambda: nv.nvfp4_fp8_gemm(*t[:4], out=t[4], ws=ws))
    need = nv.lib().nvfp4_moe_sort_workspace_bytes(3000, 4, 64)
    assert need > 0
    ids = room.at(need, (3000, 4), torch.int32)
    nv.nvfp4_moe_sort(ids, 64, ws=ws)
    refused(lambda: nv.nvfp4_moe_sort(room.at(need - 16, (3000, 4), torch.int32), 64, ws=ws))
    torch.cuda.synchronize()


def test_columns_of_one_buffer_lie_apart():
    """Rows of one stride whose columns differ share no bytes, though their spans do."""
    from nvfp4_block_scaled_amd.fp8 import _apart
    room = torch.zeros((12, 24))
    for out, other in ((room[:8, :8], room[:4, 8:24]), (room[:4, 8:24], room[2:10, :8]), (room[3:, 20:], room[:, 4:20]), (room[2:3, 4:8], room[:, 8:12])):
        _apart(out, "out", other)
        _apart(other, "out", out)
    half = room.half()
    _apart(half[:, :8], "out", half[:, 8:])
    mixed = room.view(torch.uint8)[:, 40:].view(torch.bfloat16)                  # other types, the same bytes between rows
    _apart(room[:, :10], "out", mixed)
    for out, other in ((room[:8, :9], room[:4, 8:]), (room[:4, 7:], room[2:10, :8]), (room[:2], room[1:, 4:8]), (room[:11, :11], mixed),
                       (room[:8, :8], room.view(24, 12)[:, 8:]), (room[:, :8], room.view(-1)[8:24]), (room.T[:8], room[:, 8:])):
        refused(lambda: _apart(out, "out", other))
        refused(lambda: _apart(other, "out", out))


@pytest.mark.gpu
def test_rows_between_columns_of_one_buffer():
    T, top, width = 9, 3, 40
    g = torch.Generator("cuda").manual_seed(1)
    places = torch.randperm(T * top, generator=g, device="cuda").int().view(T, top)
    room = torch.full((T * top, 3 * width + 2), 9.0, dtype=torch.bfloat16, device="cuda")
    x, rows, back = room[:T, :width], room[:, width + 1:2 * width + 1], room[:T, 2 * width + 2:]
    x.copy_(torch.randint(-4, 5, (T, width), generator=g, device="cuda"))
    kept = x.clone()
    nv.nvfp4_moe_gather(x, places, out=rows)
    nv.nvfp4_moe_combine(rows, places, out=back)
    assert torch.equal(rows[places.flatten().long()], kept.repeat_interleave(top, 0)) and torch.equal(back, top * kept) and torch.equal(x, kept)
    _, weights = nv.nvfp4_moe_combine_backward(kept, rows, places, torch.ones((T, top), device="cuda"), grad_y=room[:, :width])
    assert torch.equal(room[:, :width], rows) and torch.equal(weights, (kept.float() ** 2).sum(1, keepdim=True).expand(T, top))
    assert bool((room[:, width] == 9.0).all()) and bool((room[:, 2 * width + 1] == 9.0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(300, 700, 128), (64, 3000, 5120), (1013, 1030, 4112), (2000, 2100, 1040), (5000, 4000, 528)])
def test_how_exact_products_are(M, N, K):
    """The matrix core's sums are off by 1.3e-5 of a result in the mean square on gaussian rows, whatever K (blocks' errors and
    results grow alike); twice that is allowed here. It is a sixteenth of FP16's rounding and still seen: an output is e + d
    rounded, d what the sums are off, so the mean of (out - e)^2 is that of d^2 and of the rounding's square, and the latter is
    that of (round(e) - e)^2 but for chance. Only the outputs that d carries over a tie differ there, 2 |d| / step or some
    3 % of them (under 10 %), each by some 1e-8 of the result's square: over 210000 outputs a hundredth of what is allowed."""
    r = np.random.default_rng(K)
    x = torch.from_numpy(r.standard_normal((M, K)).astype(np.float32)).cuda()
    y = torch.from_numpy(r.standard_normal((N, K)).astype(np.float32) * np.float32(K ** -0.5)).cuda()
    a, sa = nv.nvfp4_fp8_quantize(x)
    w, sw = nv.nvfp4_fp8_quantize_weight(y)
    number = torch.from_numpy(fp8.values(np.arange(256).astype(np.uint8))).cuda()
    wide = lambda s: s.double().repeat_interleave(128, 1)[:, :K]      # noqa: E731
    want = (number[a.view(torch.uint8).int()] * wide(sa)) @ (number[w.view(torch.uint8).int()] * wide(sw).repeat_interleave(128, 0)[:N]).T
    got = nv.nvfp4_fp8_gemm(a, sa, w, sw, out_dtype="f16").double()
    off = float(((got - want) ** 2 - (want.half().double() - want) ** 2).mean() / (want ** 2).mean())
    assert off <= (2 * 1.3e-5) ** 2, off
    assert float((got != want.half().double()).double().mean()) < 0.1


def test_transposed_codes_and_scales_are_those_of_the_transposed_weight():
    """Blocks of 128 x 128 are the same ones either way, whole or cut."""
    w = np.random.default_rng(3).standard_normal((272, 400)).astype(np.float32)
    (c, s), (ct, st) = fp8.quantize(w, 128), fp8.quantize(np.ascontiguousarray(w.T), 128)
    np.testing.assert_array_equal(c.T, ct)
    np.testing.assert_array_equal(s.T, st)


@pytest.mark.gpu
@pytest.mark.parametrize("T,top,experts,N,K", [(5, 2, 3, 48, 272), (300, 3, 6, 272, 400), (1500, 2, 4, 528, 144)])
def test_gradient_of_the_input_of_products_by_expert(T, top, experts, N, K):
    """Of sum(c combine(products(x))) to x, through the public calls alone: combine's gradient, quantized, by the transposed
    weights, summed over each token's rows. In FP8 the rows' gradients are within half a step of E4M3 (2^-4 of the value, at
    least 2^-10 of a scale), their products as exact as any, each rounded to BF16, and so is the sum."""
    r = np.random.default_rng(T)
    w, sw = nv.nvfp4_fp8_quantize_weight(torch.from_numpy(r.standard_normal((experts, N, K)).astype(np.float32) * np.float32(K ** -0.5)).cuda())
    ids = torch.from_numpy(np.argsort(r.random((T, experts)), 1)[:, :top].astype(np.int32)).cuda()
    ids[::4, 0] = -1
    offsets, tokens, places = nv.nvfp4_moe_sort(ids, experts)
    weights = torch.from_numpy(r.random((T, top)).astype(np.float32)).cuda()
    x, c = (torch.from_numpy(r.standard_normal(n).astype(np.float32)).to(torch.bfloat16).cuda() for n in ((T, K), (T, N)))
    a, sa = nv.nvfp4_fp8_quantize(x)
    y = torch.zeros((T * top, N), dtype=torch.bfloat16, device="cuda")
    nv.nvfp4_fp8_gemm_grouped(a, sa, w, sw, offsets, rows=tokens, out=y)

    wt, swt = w.view(torch.uint8).transpose(1, 2).contiguous(), sw.transpose(1, 2).contiguous()
    grad_y, _ = nv.nvfp4_moe_combine_backward(c, y, places, weights, grad_y=torch.zeros_like(y))
    g, sg = nv.nvfp4_fp8_quantize(grad_y)
    rows = torch.zeros((T * top, K), dtype=torch.bfloat16, device="cuda")
    nv.nvfp4_fp8_gemm_grouped(g, sg, wt, swt, offsets, out=rows)
    got = nv.nvfp4_moe_gather_backward(rows, places).double().cpu().numpy()

    held = np.stack([fp8.values(c) * fp8.spread(s.astype(np.float64), 128, c.shape) for c, s in zip(w.view(torch.uint8).cpu().numpy(), sw.cpu().numpy())])
    ids, c, weights, sg, places = (t.double().cpu().numpy() for t in (ids, c, weights, sg, places))
    want, tol, total = np.zeros((T, K)), np.zeros((T, K)), np.zeros((T, K))
    wide = fp8.spread(sg, 1, (T * top, N))
    for t in range(T):
        for j in range(top):
            e = int(ids[t, j])
            if e < 0:
                continue
            grad = weights[t, j] * c[t]
            part, size = grad @ held[e], np.abs(grad) @ np.abs(held[e])
            off = np.maximum(2.0 ** -4 * np.abs(grad), 2.0 ** -10 * wide[int(places[t, j])]) + 2.0 ** -8 * np.abs(grad)      # and BF16 before
            inner = off @ np.abs(held[e]) * 1.01 + (7 * 2.0 ** -13 + (N / 8 + 3 * fp8.blocks(N)) * 2.0 ** -24) * size * 1.1
            want[t] += part
            tol[t] += inner + 2.0 ** -8 * (np.abs(part) + inner)
            total[t] += np.abs(part) + inner
    assert (np.abs(got - want) <= tol + 2.0 ** -8 * (np.abs(want) + tol) + 2.0 ** -20 * total + 1e-30).all()
    # in the mean square FP8 alone: an error of up to 2^-4 of a value either way is 2^-4 / sqrt(3), 0.036, at most
    assert np.sqrt(((got - want) ** 2).mean() / (want ** 2).mean()) < 0.05

    def loss(v):      # in float64, from x's values
        out = np.zeros((T, N))
        for t in range(T):
            for j in range(top):
                if ids[t, j] >= 0:
                    out[t] += weights[t, j] * (held[int(ids[t, j])] @ v[t])
        return (out * c).sum()
    v, h = x.double().cpu().numpy(), 1e-3
    for t, k in ((0, 0), (T - 1, K - 1), (T // 2, 130)):
        step = np.zeros_like(v)
        step[t, k] = h                                                            # linear in x: exact but for rounding
        assert abs((loss(v + step) - loss(v - step)) / (2 * h) - got[t, k]) <= tol[t, k] + 2.0 ** -7 * total[t, k] + 1e-6
