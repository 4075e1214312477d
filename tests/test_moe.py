"""Tokens to experts and back against the oracle's pair-by-pair loops, and a layer of experts as a whole."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_amd as nv
from oracle import fp8, moe

TYPES = {"bf16": (torch.bfloat16, 2.0 ** -8), "f16": (torch.float16, 2.0 ** -11), "f32": (torch.float32, 2.0 ** -24)}


def rng(seed):
    return np.random.default_rng(seed)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def ids_of(r, T, top, experts, how):
    if how == "distinct":
        order = np.argsort(r.random((T, experts)), 1)[:, :top] if T else np.zeros((0, top), int)
        return order.astype(np.int64)
    if how == "same":                                              # every choice is one expert
        return np.full((T, top), r.integers(experts), np.int64)
    if how == "none":
        return np.full((T, top), -1, np.int64)
    ids = r.integers(0, experts, (T, top))                         # an expert may come twice for a token
    return np.where(r.random((T, top)) < 0.3, r.choice([-1, experts, -7, 2 ** 31 - 1], (T, top)), ids)


def test_oracle_sort_by_hand():
    offsets, tokens, places = moe.sort(np.array([[2, 0], [0, -1], [2, 2]]), 3)
    assert offsets.tolist() == [0, 2, 2, 5] and tokens.tolist() == [0, 1, 0, 2, 2, -1]
    assert places.tolist() == [[2, 0], [1, -1], [3, 4]]


@pytest.mark.gpu
@pytest.mark.parametrize("how", ["distinct", "same", "none", "mixed"])
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("T,top,experts", [(0, 2, 4), (1, 1, 1), (1, 8, 64), (17, 8, 60), (64, 3, 5), (513, 8, 257), (1000, 8, 896), (33, 2, 897),
                                           (2000, 8, 1024), (1025, 8, 64), (4096, 10, 384)])
def test_sort(T, top, experts, wide, how):
    r = rng(T + experts)
    ids = ids_of(r, T, top, experts, how)
    want = moe.sort(ids, experts)
    for got, w in zip(nv.nvfp4_moe_sort(dev(ids if wide else ids.astype(np.int32)), experts), want):
        assert got.dtype == torch.int32
        np.testing.assert_array_equal(got.cpu().numpy(), w)


@pytest.mark.gpu
def test_sort_of_wide_ids_and_dirty_workspace():
    """Ids past 32 bits stand for no expert; the workspace may hold any bytes, and so may the outputs before."""
    r = rng(2)
    ids = r.integers(0, 64, (3000, 4)).astype(np.int64)
    ids[::7, 1] += 1 << 32
    want = moe.sort(ids, 64)
    for fill in (0, 0xFF):
        ws = torch.full((nv.lib().nvfp4_moe_sort_workspace_bytes(3000, 4, 64),), fill, dtype=torch.uint8, device="cuda")
        assert ws.numel() > 0
        for got, w in zip(nv.nvfp4_moe_sort(dev(ids), 64, ws=ws), want):
            np.testing.assert_array_equal(got.cpu().numpy(), w)


def tensors(r, shape, kind, pad=0):
    """A matrix of `kind`, as columns of a wider one with pad, on the device and in float64."""
    x = torch.from_numpy(r.standard_normal(shape).astype(np.float32)).to(TYPES[kind][0])
    wide = torch.full((shape[0], shape[1] + pad), 3e4, dtype=x.dtype)
    wide[:, :shape[1]] = x
    return wide.cuda()[:, :shape[1]], x.double().numpy()


SHAPES = [(0, 2, 4, 8, 0), (1, 1, 1, 1, 0), (1, 8, 64, 64, 0), (17, 8, 60, 200, 3), (64, 3, 5, 2051, 1), (40, 11, 30, 4100, 8), (300, 2, 8, 37, 0)]


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("how", ["distinct", "mixed", "none"])
@pytest.mark.parametrize("T,top,experts,width,pad", SHAPES)
def test_gather(T, top, experts, width, pad, how, kind):
    r = rng(T + width)
    _, _, places = moe.sort(ids_of(r, T, top, experts, how), experts)
    x, xs = tensors(r, (T, width), kind, pad)
    out = torch.full((T * top, width + pad), 9.0, dtype=x.dtype, device="cuda")
    nv.nvfp4_moe_gather(x, dev(places), out=out[:, :width])
    np.testing.assert_array_equal(out[:, :width].double().cpu().numpy(), moe.gather(xs, places, np.full((T * top, width), 9.0)))
    assert bool((out[:, width:] == 9.0).all())


def combine_tolerance(want, size, kind, top):
    """top products and as many sums in FP32, half a step each, and half a step of the output: of FP16, whose steps below
    2^-14 are all 2^-24, at least 2^-25."""
    inner = 2 * top * 2.0 ** -24 * size
    return np.maximum(TYPES[kind][1] * (np.abs(want) + inner), 2.0 ** -25 if kind == "f16" else 0.0) + inner + 1e-30


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("how", ["distinct", "mixed", "none"])
@pytest.mark.parametrize("T,top,experts,width,pad", SHAPES)
def test_combine_and_its_gradients(T, top, experts, width, pad, how, kind):
    r = rng(T + width + 1)
    _, _, places = moe.sort(ids_of(r, T, top, experts, how), experts)
    y, ys = tensors(r, (T * top, width), kind, pad)
    w = r.random((T, top)).astype(np.float32) - np.float32(0.2)
    at, wd = dev(places), dev(w)
    for weights, wt in ((w, wd), (None, None)):
        want, size = moe.combine(ys, places, weights)
        out = torch.full((T, width + pad), 9.0, dtype=y.dtype, device="cuda")
        nv.nvfp4_moe_combine(y, at, wt, out=out[:, :width])
        assert (np.abs(out[:, :width].double().cpu().numpy() - want) <= combine_tolerance(want, size, kind, top)).all()
        assert bool((out[:, width:] == 9.0).all())
    assert torch.equal(nv.nvfp4_moe_gather_backward(y, at), out[:, :width])
    g, gs = tensors(r, (T, width), kind, pad)
    grad_y = torch.full((T * top, width + pad), 9.0, dtype=y.dtype, device="cuda")
    _, grad_w = nv.nvfp4_moe_combine_backward(g, y, at, wd, grad_y=grad_y[:, :width])
    want_y, want_w, size = moe.combine_backward(gs, ys, places, w, np.full((T * top, width), 9.0))
    # one product in FP32, rounded to the output's type
    tol = (TYPES[kind][1] + 2.0 ** -23) * np.abs(want_y) + (2.0 ** -25 if kind == "f16" else 1e-30)
    assert (np.abs(grad_y[:, :width].double().cpu().numpy() - want_y) <= tol).all()
    assert bool((grad_y[:, width:] == 9.0).all())
    # products and sums of `width` terms in any order
    assert (np.abs(grad_w.double().cpu().numpy() - want_w) <= width * 2.0 ** -24 * size + 1e-30).all()


@pytest.mark.gpu
def test_gradients_against_differences():
    """FP32 rows: the loss sum(combine(gather(x) * s) * c) by its own small steps in float64 and by the gradients."""
    r = rng(9)
    T, top, experts, width = 7, 3, 5, 33
    ids = ids_of(r, T, top, experts, "mixed")
    _, _, places = moe.sort(ids, experts)
    x, c = r.standard_normal((T, width)), r.standard_normal((T, width))
    w, s = r.random((T, top)), r.standard_normal(T * top)[:, None]

    def loss(x, w):
        rows = moe.gather(x, places, np.zeros((T * top, width))) * s
        return (moe.combine(rows, places, w)[0] * c).sum()
    f32 = lambda v: dev(v.astype(np.float32))                      # noqa: E731
    at = dev(places)
    out = torch.zeros((T * top, width), device="cuda")
    rows = nv.nvfp4_moe_gather(f32(x), at, out=out) * f32(s)
    grad_rows = torch.zeros_like(rows)
    _, grad_w = nv.nvfp4_moe_combine_backward(f32(c), rows, at, f32(w), grad_y=grad_rows)
    grad_x = nv.nvfp4_moe_gather_backward(grad_rows * f32(s), at)
    h = 1e-3                                                       # the loss is linear in each: differences are exact but for rounding
    for _ in range(20):
        t, i, j = r.integers(T), r.integers(width), r.integers(top)
        dx, dw = np.zeros_like(x), np.zeros_like(w)
        dx[t, i], dw[t, j] = h, h
        assert abs((loss(x + dx, w) - loss(x - dx, w)) / (2 * h) - float(grad_x[t, i])) < 1e-4
        assert abs((loss(x, w + dw) - loss(x, w - dw)) / (2 * h) - float(grad_w[t, j])) < 1e-3


@pytest.mark.gpu
def test_places_out_of_range_stand_for_no_row():
    x, y = torch.ones((2, 40), device="cuda"), torch.ones((4, 40), device="cuda")
    at = torch.tensor([[4, 1], [-2 ** 31, 2 ** 31 - 1]], dtype=torch.int32, device="cuda")
    out = torch.zeros((4, 40), device="cuda")
    nv.nvfp4_moe_gather(x, at, out=out)
    assert out.sum(1).tolist() == [0.0, 40.0, 0.0, 0.0]
    w = torch.full((2, 2), 2.0, device="cuda")
    assert nv.nvfp4_moe_combine(y, at, w)[:, 0].tolist() == [2.0, 0.0]
    grad_y, grad_w = nv.nvfp4_moe_combine_backward(x, y, at, w, grad_y=out.zero_())
    assert grad_w.tolist() == [[0.0, 40.0], [0.0, 0.0]] and grad_y.sum(1).tolist() == [0.0, 80.0, 0.0, 0.0]


@pytest.mark.gpu
@pytest.mark.parametrize("T,hidden,between,experts,top", [(1, 256, 128, 8, 2), (50, 272, 144, 16, 4), (700, 256, 384, 6, 2)])
def test_a_layer_of_experts(T, hidden, between, experts, top):
    """Sort, quantize, gate and up by expert with the tokens' rows taken through the index, silu(gate) up, down, combine: each
    step against float64 from what the one before it gave."""
    r = rng(T)
    x = torch.from_numpy(r.standard_normal((T, hidden)).astype(np.float32)).to(torch.bfloat16).cuda()
    up = nv.nvfp4_fp8_quantize_weight(torch.from_numpy(r.standard_normal((experts, 2 * between, hidden)).astype(np.float32) * 0.06).cuda())
    down = nv.nvfp4_fp8_quantize_weight(torch.from_numpy(r.standard_normal((experts, hidden, between)).astype(np.float32) * 0.06).cuda())
    ids = ids_of(r, T, top, experts, "distinct")
    ids[::5, 0] = -1
    weights = dev(r.random((T, top)).astype(np.float32))
    offsets, tokens, places = nv.nvfp4_moe_sort(dev(ids), experts)
    a, sa = nv.nvfp4_fp8_quantize(x)
    h = torch.zeros((T * top, 2 * between), dtype=torch.bfloat16, device="cuda")
    nv.nvfp4_fp8_gemm_grouped(a, sa, up[0], up[1], offsets, rows=tokens, out=h)
    b, sb = nv.nvfp4_fp8_quantize(h, gated=True)
    y = torch.zeros((T * top, hidden), dtype=torch.bfloat16, device="cuda")
    nv.nvfp4_fp8_gemm_grouped(b, sb, down[0], down[1], offsets, out=y)
    out = nv.nvfp4_moe_combine(y, places, weights)

    def host(t):
        return t.view(torch.uint8).cpu().numpy() if t.dtype == torch.float8_e4m3fn else t.cpu().numpy()
    ends, index = host(offsets), host(tokens)
    for got, (m, s), (w, sw), rows, K in ((h, (a, sa), up, index, hidden), (y, (b, sb), down, None, between)):
        want, size, hit = fp8.grouped(host(m), host(s), host(w), host(sw), ends, rows, np.zeros(got.shape))
        assert hit.sum() == ends[-1]
        inner = (7 * 2.0 ** -13 + (K / 8 + 3 * fp8.blocks(K)) * 2.0 ** -24) * size
        assert (np.abs(got.double().cpu().numpy() - want) <= 2.0 ** -8 * (np.abs(want) + inner) + inner).all()
    want, size = moe.combine(y.double().cpu().numpy(), host(places), weights.cpu().numpy())
    assert (np.abs(out.double().cpu().numpy() - want) <= combine_tolerance(want, size, "bf16", top)).all()
