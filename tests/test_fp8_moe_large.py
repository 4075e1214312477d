"""Calls of the FP8 and the experts' operators whose workgroups have more than 2^32 threads together, which is more than one
launch takes in a row: many narrow rows, thin weights, very wide experts. Results are those of smaller calls, or plain copies."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_amd as nv
from oracle import fp8

pytestmark = pytest.mark.gpu


def same(a, b):
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_of_many_tokens(dtype):
    T, width = (1 << 24) + 5, 3
    g = torch.Generator("cuda").manual_seed(4)
    places = torch.randperm(T, generator=g, device="cuda").int()[:, None]
    x = torch.randint(-8, 9, (T, width), generator=g, device="cuda").to(dtype)
    weights = torch.exp2(torch.randint(-1, 2, (T, 1), generator=g, device="cuda").float())
    at = places[:, 0].long()
    rows = nv.nvfp4_moe_gather(x, places)
    assert torch.equal(rows[at], x)
    assert torch.equal(nv.nvfp4_moe_combine(rows, places, weights), x * weights.to(dtype))
    assert torch.equal(nv.nvfp4_moe_gather_backward(rows, places), x)
    grad = torch.randint(-8, 9, (T, width), generator=g, device="cuda").to(dtype)
    grad_y, grad_w = nv.nvfp4_moe_combine_backward(grad, rows, places, weights)
    assert torch.equal(grad_y[at], grad * weights.to(dtype))
    assert torch.equal(grad_w[:, 0], (grad * x).float().sum(1) if dtype == torch.float32 else (grad.float() * x.float()).sum(1))


def test_quantize_many_narrow_rows():
    rows = (1 << 29) + 40
    x = torch.empty((rows, 16), dtype=torch.bfloat16, device="cuda").normal_()
    codes, scales = nv.nvfp4_fp8_quantize(x)
    for at in range(0, rows, 1 << 26):
        c, s = nv.nvfp4_fp8_quantize(x[at:at + (1 << 26)])
        assert same(codes[at:at + (1 << 26)], c) and torch.equal(scales[at:at + (1 << 26)], s)


def test_quantize_many_thin_weights():
    """Of one row each: a block of a weight is one of a row then."""
    w = torch.empty((1 << 20, 1, 2064), dtype=torch.bfloat16, device="cuda").normal_()
    codes, scales = nv.nvfp4_fp8_quantize_weight(w)
    c, s = nv.nvfp4_fp8_quantize(w[:, 0])
    assert same(codes[:, 0], c) and torch.equal(scales[:, 0], s)


def test_products_with_very_wide_experts():
    """1024 experts of 2^21 and some rows, one block of K; the last expert has the rows."""
    r = np.random.default_rng(6)
    E, N, K, M = 1024, (1 << 21) + 32, 16, 3
    table = np.array([0xC0, 0xB8, 0xB0, 0x00, 0x30, 0x38, 0x40], np.uint8)
    a, last = r.choice(table, (M, K)), r.choice(table, (N, K))
    w = torch.zeros((E, N, K), dtype=torch.uint8, device="cuda")
    w[-1] = torch.from_numpy(last).cuda()
    sw = torch.ones((E, fp8.blocks(N), 1), device="cuda")
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[-1] = M
    got = nv.nvfp4_fp8_gemm_grouped(torch.from_numpy(a).cuda(), torch.ones((M, 1), device="cuda"), w, sw, offsets)
    want = torch.from_numpy(fp8.values(a) @ fp8.values(last).T).float().to(torch.bfloat16)      # exact: 16 products in quarters of at most 4
    assert torch.equal(got.cpu(), want)
