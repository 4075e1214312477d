"""FP8 products at sizes that together reach every tile, K in parts, several tiles to a workgroup, long rows and the kernel
for what the tiles do not take; calls at once, captured ones and workspaces of any content.

Values are small integers and scales powers of two, so every sum is exact: codes of at most 2, products in quarters of at
most 4, scales' products 2^-2 .. 2^2; K = 17408 of them stay below 2^19 in units of 2^-4, within the 24 bits of FP32."""
import numpy as np
import pytest
import torch

import nvfp4_block_scaled_amd as nv
from oracle import fp8

pytestmark = pytest.mark.gpu


def rng(seed):
    return np.random.default_rng(seed)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def codes_dev(a):
    return dev(a).view(torch.float8_e4m3fn)


def small_integers(r, shape):
    table = np.array([0xC0, 0xB8, 0xB0, 0x00, 0x30, 0x38, 0x40, 0x00], np.uint8)
    return table[r.integers(0, 8, shape, np.uint8)]


def powers(r, shape):
    return np.exp2(r.integers(-1, 2, shape)).astype(np.float32)


def product_case(r, M, N, K):
    return small_integers(r, (M, K)), powers(r, (M, fp8.blocks(K))), small_integers(r, (N, K)), powers(r, (fp8.blocks(N), fp8.blocks(K)))


def on_device(a, sa, w, sw):
    return codes_dev(a), dev(sa), codes_dev(w), dev(sw)


def bf16(x):
    return torch.from_numpy(x).float().to(torch.bfloat16)


@pytest.mark.parametrize("M,N,K", [
    (3, 70, 400), (65, 130, 512), (4, 16, 2464),                      # 64 x 64 tiles; four blocks and a part of one; in parts
    (130, 300, 8336), (61, 2064, 8336), (700, 130, 9008),             # parts of unlike length
    (4, 16, 144), (4, 16, 272), (1410, 5381, 272),                    # 64 x 128: two and three blocks; more tiles than places
    (69, 2400, 11552), (67, 6096, 5264),                              # 128 x 128 in parts
    (6856, 528, 272), (1594, 9567, 272), (2060, 2100, 1040),          # and whole, one tile or two to a workgroup
    (7318, 1058, 272), (2851, 8475, 272), (4100, 4100, 656),          # 256 x 256
    (1, 5120, 17408), (5, 300, 128), (70, 40, 112),                   # one row; one block of K
])
def test_every_shape_of_tiles(M, N, K):
    case = product_case(rng(M + N + K), M, N, K)
    want = bf16(fp8.product(*case)[0])
    on = on_device(*case)
    out = torch.full((M + 1, N + 1), 9.0, dtype=torch.bfloat16, device="cuda")
    got = nv.nvfp4_fp8_gemm(*on, out=out[:M, :N])
    assert torch.equal(got.cpu(), want)
    assert bool((out[M] == 9.0).all()) and bool((out[:, N] == 9.0).all())
    ws = nv.nvfp4_fp8_gemm_workspace(M, N, K)
    if ws is not None:                                                # of any content, and with room behind it
        wide = torch.full((ws.numel() + 256,), 0xFF, dtype=torch.uint8, device="cuda")
        assert torch.equal(nv.nvfp4_fp8_gemm(*on, ws=wide[:ws.numel()]).cpu(), want)
        assert bool((wide[ws.numel():] == 0xFF).all())


def grouped_want(a, sa, w, sw, offsets, rows, M):
    """Of each expert all its rows at once; rows without one: 9."""
    want = np.full((M, w.shape[1]), 9.0)
    for e in range(len(offsets) - 1):
        at = np.arange(offsets[e], offsets[e + 1])
        src = at if rows is None else rows[at]
        at, src = at[(src >= 0) & (src < len(a))], src[(src >= 0) & (src < len(a))]
        if len(at):
            want[at] = fp8.product(a[src], sa[src], w[e], sw[e])[0]
    return bf16(want)


@pytest.mark.parametrize("indexed", [False, True])
@pytest.mark.parametrize("rows,N,K,experts", [
    (342, 75, 400, 187), (182, 139, 528, 160),                        # 32 x 128 tiles, one or more to a workgroup
    (4, 16, 400, 3), (187, 278, 400, 119), (70, 300, 1040, 5),        # 64 x 64
    (6, 18, 272, 2), (224, 258, 272, 231), (700, 520, 144, 6),        # 64 x 128
    (1015, 7107, 272, 5), (2305, 2696, 272, 23), (1500, 1300, 784, 4),  # 256 x 256
    (90, 200, 128, 9), (40, 70, 8336, 5),                             # one block of K; 66 of them
])
def test_every_shape_of_tiles_by_expert(rows, N, K, experts, indexed):
    r = rng(rows + N + K + indexed)
    M = rows + 3
    tokens = max(1, rows // 2) if indexed else M
    offsets = np.concatenate([[0], np.cumsum(r.multinomial(rows, r.dirichlet(np.full(experts, 1.0))))]).astype(np.int32)
    a, sa = small_integers(r, (tokens, K)), powers(r, (tokens, fp8.blocks(K)))
    w, sw = small_integers(r, (experts, N, K)), powers(r, (experts, fp8.blocks(N), fp8.blocks(K)))
    index = r.integers(0, tokens, M).astype(np.int32) if indexed else None
    if indexed:
        index[[0, rows - 1]] = [tokens, -1]
    out = torch.full((M + 1, N + 1), 9.0, dtype=torch.bfloat16, device="cuda")
    got = nv.nvfp4_fp8_gemm_grouped(*on_device(a, sa, w, sw), dev(offsets), rows=dev(index) if indexed else None, out=out[:M, :N])
    assert torch.equal(got.cpu(), grouped_want(a, sa, w, sw, offsets, index, M))
    assert bool((out[M] == 9.0).all()) and bool((out[:, N] == 9.0).all())


def test_many_experts_with_long_rows():
    """More tiles than the device holds, 66 blocks each. One weight under scales of 2^(e % 3) for expert e."""
    r = rng(11)
    E, M, N, K = 130, 400, 280, 8336
    a, sa, w, sw = product_case(r, M, N, K)
    offsets = np.concatenate([[0], np.cumsum(r.multinomial(M, np.full(E, 1 / E)))]).astype(np.int32)
    scale = np.exp2(np.arange(E) % 3)
    want = fp8.product(a, sa, w, sw)[0] * scale[np.repeat(np.arange(E), np.diff(offsets))][:, None]
    many = codes_dev(w).view(torch.uint8).expand(E, -1, -1).contiguous().view(torch.float8_e4m3fn)
    got = nv.nvfp4_fp8_gemm_grouped(codes_dev(a), dev(sa), many, dev((sw * scale[:, None, None]).astype(np.float32)), dev(offsets))
    assert torch.equal(got.cpu(), bf16(want))


def test_rows_longer_than_the_tiles_reach():
    """K just past 2^23. Sums of 2^23 products in quarters of at most 4, signs and zeros at random: below 2^24 quarters."""
    r = rng(12)
    M, N, K = 2, 5, (1 << 23) + 144
    a, w = small_integers(r, (M, K)), small_integers(r, (N, K))
    sa, sw = np.ones((M, fp8.blocks(K)), np.float32), np.ones((1, fp8.blocks(K)), np.float32)
    got = nv.nvfp4_fp8_gemm(*on_device(a, sa, w, sw))
    assert torch.equal(got.cpu(), bf16(fp8.values(a) @ fp8.values(w).T))


def test_tokens_past_four_gigabytes():
    """Indexed rows of a matrix that 32-bit offsets do not reach: the first, the last and one between."""
    r = rng(13)
    K, N = 4112, 130
    tokens = (1 << 32) // K + 9
    a = torch.zeros((tokens, K), dtype=torch.uint8, device="cuda")
    sa = torch.ones((tokens, fp8.blocks(K)), dtype=torch.float32, device="cuda")
    index = np.array([tokens - 1, 0, tokens // 2, tokens - 1, 5], np.int32)
    rows = small_integers(r, (5, K))
    rows[3], rows[4] = rows[0], 0
    a[dev(index[:3]).long()] = dev(rows[:3])
    w, sw = small_integers(r, (2, N, K)), powers(r, (2, 2, fp8.blocks(K)))
    offsets = np.array([0, 3, 5], np.int32)
    got = nv.nvfp4_fp8_gemm_grouped(a.view(torch.float8_e4m3fn), sa, codes_dev(w), dev(sw), dev(offsets), rows=dev(index))
    assert torch.equal(got.cpu(), grouped_want(rows, np.ones((5, fp8.blocks(K))), w, sw, offsets, None, 5))


def test_two_calls_at_once():
    """On two streams, in parts of K, without a workspace of the caller: each has its own."""
    cases = [product_case(rng(20 + i), 40, 260, 4112) for i in range(2)]
    on = [on_device(*c) for c in cases]
    want = [bf16(fp8.product(*c)[0]) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(nv.nvfp4_fp8_gemm(*on[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(g.cpu(), want[i]) for g in got[i])


@pytest.mark.parametrize("M,N,K", [(40, 260, 4112), (300, 700, 272), (2100, 4200, 400)])
def test_captured_products_replayed_between_others(M, N, K):
    case = product_case(rng(M), M, N, K)
    other = product_case(rng(M + 1), M, N, K)
    a, sa, w, sw = on_device(*case)
    ws = nv.nvfp4_fp8_gemm_workspace(M, N, K)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        nv.nvfp4_fp8_gemm(a, sa, w, sw, ws=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = nv.nvfp4_fp8_gemm(a, sa, w, sw, ws=ws)
    for c in (case, other, case):
        a.view(torch.uint8).copy_(dev(c[0]))
        sa.copy_(dev(c[1]))
        w.view(torch.uint8).copy_(dev(c[2]))
        sw.copy_(dev(c[3]))
        graph.replay()
        eager = nv.nvfp4_fp8_gemm(a, sa, w, sw)
        torch.cuda.synchronize()
        want = bf16(fp8.product(*c)[0])
        assert torch.equal(got.cpu(), want) and torch.equal(eager.cpu(), want)


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float16, torch.float32])
def test_quantizers_of_inputs_past_the_caches(kind):
    """Over 64 MB in all: rows of a wider matrix, gated rows and a weight give what parts of them, each under 64 MB, do."""
    g = torch.Generator("cuda").manual_seed(3)
    x = torch.randn((4400, 8 * 1040 + 8), generator=g, device="cuda").to(kind)[:, :8 * 1040]
    for gated in (False, True):
        codes, scales = nv.nvfp4_fp8_quantize(x, gated=gated)
        for at in range(0, 4400, 400):
            c, s = nv.nvfp4_fp8_quantize(x[at:at + 400], gated=gated)
            assert torch.equal(codes[at:at + 400].view(torch.uint8), c.view(torch.uint8)) and torch.equal(scales[at:at + 400], s)
    codes, scales = nv.nvfp4_fp8_quantize_weight(x)
    for at in range(0, 4400, 384):
        c, s = nv.nvfp4_fp8_quantize_weight(x[at:at + 384])
        assert torch.equal(codes[at:at + 384].view(torch.uint8), c.view(torch.uint8)) and torch.equal(scales[at // 128:at // 128 + 3], s)


def test_outputs_over_inputs_are_refused():
    """Every output that the caller gives, over every input; behind the input's last byte it may begin."""
    room = torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")

    def at(first, shape, dtype):
        n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
        return room[first:first + n].view(dtype).view(shape)
    f8, f4, b2 = torch.float8_e4m3fn, torch.float32, torch.bfloat16
    x, codes, scales = at(0, (4, 256), b2), at(2048, (4, 256), f8), at(4096, (4, 2), f4)
    nv.nvfp4_fp8_quantize(x, codes=codes, scales=scales)
    for bad in (dict(codes=at(2032, (4, 256), f8)), dict(scales=at(2044, (4, 2), f4)), dict(codes=at(0, (4, 256), torch.uint8))):
        with pytest.raises(ValueError):
            nv.nvfp4_fp8_quantize(x, **bad)
    w, sw = at(8192, (16, 256), f8), at(16384, (1, 2), f4)
    nv.nvfp4_fp8_quantize_weight(x, codes=codes, scales=at(4096, (1, 2), f4))
    with pytest.raises(ValueError):
        nv.nvfp4_fp8_quantize_weight(x, codes=at(1024, (4, 256), f8))
    offsets, rows = at(20480, (2,), torch.int32), at(20496, (4,), torch.int32)
    out = at(2048 - 128, (4, 16), b2)
    nv.nvfp4_fp8_gemm(codes, scales, w, sw, out=out)
    nv.nvfp4_fp8_gemm_grouped(codes, scales, w[None], sw[None], offsets, rows=rows, out=out)
    for first in (2048 - 126, 2048 + 1022, 4096 + 30, 8192 + 4094, 16384 + 6):
        with pytest.raises(ValueError):
            nv.nvfp4_fp8_gemm(codes, scales, w, sw, out=at(first, (4, 16), b2))
    for first in (2048, 20480 + 6, 20496 + 14):
        with pytest.raises(ValueError):
            nv.nvfp4_fp8_gemm_grouped(codes, scales, w[None], sw[None], offsets, rows=rows, out=at(first, (4, 16), b2))
    torch.cuda.synchronize()


@pytest.mark.parametrize("rows,K", [(33, 128), (70, 256), (41, 3968), (35, 4096), (9, 4112), (1, 16400), (1000, 16), (3, 100000)])
def test_quantized_rows_across_workgroups(rows, K):
    """Rows of 1, 2, 31, 32, 33 and many blocks, 32 blocks to a workgroup; zeros of both signs keep theirs."""
    x = rng(K).standard_normal((rows, K)).astype(np.float32)
    x[:, ::7] = 0.0
    x[:, 3::11] = -0.0
    x[rows // 2, K // 2:] = -0.0
    codes, scales = nv.nvfp4_fp8_quantize(dev(x))
    want_c, want_s = fp8.quantize(x)
    np.testing.assert_array_equal(scales.cpu().numpy(), want_s)
    np.testing.assert_array_equal(codes.view(torch.uint8).cpu().numpy(), want_c)
