"""FP8 products in every tile shape over few and many blocks of K: each case says which shape it is for, and a query of the
library's choice confirms it for a device of 256 CUs.

Values are small integers under scales that are powers of two: codes of at most 2 in halves, scales of 1/2, 1 and 2, so
every product is a multiple of 2^-4 of at most 16, and 8448 of them stay below 2^24 such units: any order of summing is exact."""
import ctypes

import numpy as np
import pytest
import torch

import nvfp4_block_scaled_amd as nv
from oracle import fp8

CUS = 256
KINDS = {"bf16": torch.bfloat16, "f16": torch.float16}
# blocks of K: 592 4 and a part, 640 5, 1136 8 and a part, 1152 9, 8336 65 and a part, 8448 66 (row scales are read four at a time, column scales 64)
DENSE = [((64, 64), 45, 9270, 8336), ((64, 64), 127, 8789, 8336), ((64, 128), 905, 8327, 1136), ((64, 128), 770, 9386, 8336),
         ((128, 128), 6406, 2358, 592), ((128, 128), 9392, 1553, 1152), ((128, 128), 9293, 1548, 8336),
         ((256, 256), 5510, 4447, 592), ((256, 256), 5510, 4447, 640), ((256, 256), 8840, 2708, 1136), ((256, 256), 8840, 2708, 1152),
         ((256, 256), 6669, 3620, 8336), ((256, 256), 6669, 3620, 8448)]
GROUPED = [((32, 128), 1933, 106, 8336, 130), ((32, 128), 228, 3675, 8336, 3), ((32, 128), 1272, 579, 8448, 20),
           ((64, 64), 684, 33, 8336, 20), ((64, 64), 70, 300, 1136, 5), ((64, 128), 551, 194, 8336, 130), ((64, 128), 8106, 195, 8336, 3),
           ((64, 128), 7347, 129, 8448, 130), ((256, 256), 7612, 932, 592, 20), ((256, 256), 9383, 776, 640, 3),
           ((256, 256), 8829, 795, 1136, 20), ((256, 256), 8277, 919, 8336, 3), ((256, 256), 9252, 782, 8448, 20),
           ((256, 256), 2359, 2718, 592, 20)]


def plan(M, N, K, experts=0):
    """(rows, columns, parts of K) of the tiles that a product takes; zeros: the kernel for what tiles do not take."""
    f = nv.lib().nvfp4_fp8_gemm_plan
    f.argtypes, f.restype = [ctypes.c_int64] * 3 + [ctypes.c_int32] * 2, ctypes.c_int32
    v = f(M, N, K, experts, CUS)
    return v >> 20, v >> 8 & 0xFFF, v & 0xFF


def test_cases_take_the_shapes_that_they_are_for():
    for shape, M, N, K in DENSE:
        assert plan(M, N, K) == shape + (1,), (M, N, K)
    for shape, M, N, K, experts in GROUPED:
        assert plan(M, N, K, experts) == shape + (1,), (M, N, K, experts)
    assert plan(5, 300, 128) == plan(1, 1, (1 << 23) + 16) == plan(90, 200, 112, 9) == (0, 0, 0)
    assert plan(1, 5120, 17408)[:2] == (64, 64) and plan(1, 5120, 17408)[2] > 1
    assert plan(69, 2400, 11552)[:2] == (128, 128) and plan(69, 2400, 11552)[2] > 1


def matrix(g, rows, K, tall):
    """(codes [*rows][K], scales)"""
    table = torch.tensor([0xC0, 0xB8, 0xB0, 0x00, 0x30, 0x38, 0x40, 0x00], dtype=torch.uint8, device="cuda")
    codes = table[torch.randint(0, 8, (*rows, K), generator=g, device="cuda")]
    n = rows[-1]
    scales = torch.exp2(torch.randint(-1, 2, (*rows[:-1], fp8.blocks(n) if tall else n, fp8.blocks(K)), generator=g, device="cuda").float())
    return codes, scales


def stands_for(codes, scales, tall):
    number = torch.from_numpy(fp8.values(np.arange(256).astype(np.uint8))).cuda()
    s = scales.double().repeat_interleave(128, -1)[..., :codes.shape[-1]]
    return number[codes.int()] * (s.repeat_interleave(128, -2)[..., :codes.shape[-2], :] if tall else s)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape,M,N,K", DENSE)
def test_long_products_in_every_shape(shape, M, N, K, kind):
    g = torch.Generator("cuda").manual_seed(M + K)
    (a, sa), (w, sw) = matrix(g, (M,), K, False), matrix(g, (N,), K, True)
    want = (stands_for(a, sa, False) @ stands_for(w, sw, True).T).float().to(KINDS[kind])
    room = torch.full((M + 1, N + 1), 9.0, dtype=KINDS[kind], device="cuda")
    got = nv.nvfp4_fp8_gemm(a, sa, w, sw, out_dtype=kind, out=room[:M, :N])
    assert torch.equal(got, want)
    assert bool((room[M] == 9.0).all()) and bool((room[:, N] == 9.0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("indexed", [False, True])
@pytest.mark.parametrize("shape,M,N,K,experts", GROUPED)
def test_long_products_by_expert_in_every_shape(shape, M, N, K, experts, indexed, kind):
    g = torch.Generator("cuda").manual_seed(M + K + indexed)
    tokens = M // 2 if indexed else M
    (a, sa), (w, sw) = matrix(g, (tokens,), K, False), matrix(g, (experts, N), K, True)
    r = np.random.default_rng(M)
    ends = np.concatenate([[0], np.cumsum(r.multinomial(M - 2, r.dirichlet(np.full(experts, 2.0))))]).astype(np.int32)     # two rows of no expert
    rows = torch.randint(0, tokens, (M,), generator=g, device="cuda").int() if indexed else None
    room = torch.full((M + 1, N + 1), 9.0, dtype=KINDS[kind], device="cuda")
    got = nv.nvfp4_fp8_gemm_grouped(a, sa, w, sw, torch.from_numpy(ends).cuda(), rows=rows, out_dtype=kind, out=room[:M, :N])
    x = stands_for(a, sa, False)
    for e in range(experts):
        lo, hi = int(ends[e]), int(ends[e + 1])
        mine = x[rows[lo:hi].long()] if indexed else x[lo:hi]
        assert torch.equal(got[lo:hi], (mine @ stands_for(w[e], sw[e], True).T).float().to(KINDS[kind])), e
    assert bool((room[ends[-1]:] == 9.0).all()) and bool((room[:, N] == 9.0).all())
