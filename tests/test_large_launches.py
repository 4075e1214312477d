"""Calls with 2^32 threads and more, which the runtime drops the rest of along one dimension: a weight of 2^36 values is prepared
whole, an activation of 2^37 is tiled whole, and W4A16 products of so many columns that their launch does not run whole are refused."""
import pytest
import torch

import nvfp4_block_scaled_amd as nv

pytestmark = pytest.mark.gpu


def test_prepare_weight_of_many_blocks():
    """Equal to what its parts give: tiles of 32 rows lie one behind the other, codes first."""
    N, K, part = (1 << 20) + 32, 1 << 16, 1 << 17
    codes = torch.empty((N, K // 2), dtype=torch.uint8, device="cuda").random_()
    scales = torch.empty((N, K // 16), dtype=torch.uint8, device="cuda").random_(0, 127)
    whole, bad = nv.nvfp4_prepare_weight(codes, scales)
    assert int(bad) == 0
    for at in range(0, N, part):
        n = min(part, N - at)
        want, _ = nv.nvfp4_prepare_weight(codes[at:at + n], scales[at:at + n])
        assert torch.equal(whole[at * (K // 2):(at + n) * (K // 2)], want[:n * (K // 2)])
        first = N * (K // 2) + at * (K // 16)
        assert torch.equal(whole[first:first + n * (K // 16)], want[n * (K // 2):])


def test_tile_activation_of_many_units():
    """As the weight above; tiles of codes, then those of scales."""
    M, K, part = (1 << 20) + 32, 1 << 17, 1 << 16
    codes = torch.empty((M, K // 2), dtype=torch.uint8, device="cuda").random_()
    scales = torch.empty((M, K // 16), dtype=torch.uint8, device="cuda").random_()
    whole = nv.nvfp4_tile_activation(codes, scales)
    for at in range(0, M, part):
        n = min(part, M - at)
        want = nv.nvfp4_tile_activation(codes[at:at + n], scales[at:at + n])
        assert torch.equal(whole[at * (K // 2):(at + n) * (K // 2)], want[:n * (K // 2)])
        first = M * (K // 2) + at * (K // 16)
        assert torch.equal(whole[first:first + n * (K // 16)], want[n * (K // 2):])


def many_columns(N, K=64):
    """A prepared weight whose groups of 32 rows are all alike."""
    codes = torch.randint(0, 256, (32, K // 2), dtype=torch.uint8, device="cuda")
    scales = torch.randint(0x30, 0x40, (32, K // 16), dtype=torch.uint8, device="cuda")
    one, _ = nv.nvfp4_prepare_weight(codes, scales)
    return torch.cat([one[:16 * K].repeat(N // 32), one[16 * K:].repeat(N // 32)]), one


@pytest.mark.parametrize("M,N", [(1, (1 << 28) + 256), (8, (1 << 28) + 288)])
def test_w4a16_of_too_many_columns_is_refused(M, N):
    w, _ = many_columns(N)
    with pytest.raises(ValueError):
        nv.nvfp4_gemm_w4a16(torch.zeros((M, 64), dtype=torch.bfloat16, device="cuda"), w, N, 64, 1.0)


@pytest.mark.parametrize("M,N", [(1, 1 << 27), (8, (1 << 28) + 256)])
def test_w4a16_of_many_columns(M, N):
    torch.manual_seed(1)
    w, one = many_columns(N)
    x = torch.randn((M, 64), device="cuda").to(torch.bfloat16)
    y = nv.nvfp4_gemm_w4a16(x, w, N, 64, 1.0)
    small = nv.nvfp4_gemm_w4a16(x, one, 32, 64, 1.0)
    assert torch.equal(y.view(M, N // 32, 32), y[:, None, :32].expand(M, N // 32, 32))
    assert bool(((y[:, :32] - small).abs() <= 2.0 ** -7 * small.abs() + 1e-3).all())
