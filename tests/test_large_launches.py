"""Calls with 2^32 threads and more, which the runtime drops the rest of along one dimension: a weight of 2^36 values is prepared
whole."""
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
