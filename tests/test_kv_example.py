"""The example's attention block against a dense float64 computation from what the cache holds."""
import math
import os
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


def test_block_matches_dense_attention_through_fork_and_compact():
    import kv_decode
    import nvfp4_block_scaled_amd as nv
    b = kv_decode.Block(hidden=512, q_heads=4, kv_heads=2, head_dim=64, page=16, pool=64, batch=6, width=12, max_pos=256)
    gen = torch.Generator(device="cuda").manual_seed(3)

    def x(n):
        return torch.randn((n, 512), generator=gen, device="cuda").to(torch.bfloat16)

    def check(q, o, counts):
        """Each query's output from the values that nvfp4_kv_read gives for its sequence."""
        row = 0
        for s, n in enumerate(counts):
            total = int(b.lens[s])
            t = torch.arange(total, device="cuda")
            slots = b.table[s, t // 16].long() * 16 + t % 16
            k, v = (a.double() for a in nv.nvfp4_kv_read(b.cache, slots, torch.float32))
            for i in range(n):
                seen = total - n + i + 1
                for h in range(4):
                    p = torch.softmax(k[:seen, h // 2] @ q[row, h].double() / math.sqrt(64), 0)
                    want = p @ v[:seen, h // 2]
                    # BF16 output (2^-8), FP16 probabilities (2^-11), read-back rounded to FP32
                    tol = 2.0 ** -8 * want.abs() + 2.0 ** -10 * (p @ v[:seen, h // 2].abs()) + 1e-6
                    assert bool(((o[row, h].double() - want).abs() <= tol).all()), (s, i, h)
                row += 1

    lens = [40, 7, 16, 0, 0, 0]
    counts = torch.tensor(lens, dtype=torch.int32, device="cuda")
    y, q, o, short = b.forward(x(sum(lens)), counts, kv_decode.offsets(counts), max(lens))
    assert int(short) == 0 and y.shape == (63, 512) and bool(y.isfinite().all())
    check(q, o, lens)
    assert int(b.fork(torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda"), torch.arange(3, 6, device="cuda"))) == 0
    one = torch.ones(6, dtype=torch.int32, device="cuda")
    for step in range(20):
        _, q, o, short = b.forward(x(6), one, kv_decode.offsets(one), 1)
        if step in (0, 9, 19):
            check(q, o, [1] * 6)
    assert int(short) == 0
    b.resize((b.lens * torch.tensor([0, 1, 1, 1, 0, 1], device="cuda")).int())
    live = int(b.compact())
    assert live == int((b.refs > 0).sum()) and bool((b.refs[:live] > 0).all())
    counts = torch.tensor([0, 1, 1, 1, 0, 1], dtype=torch.int32, device="cuda")
    _, q, o, _ = b.forward(x(4), counts, kv_decode.offsets(counts), 1)
    check(q, o, counts.tolist())


def test_example_runs():
    import kv_decode
    b = kv_decode.main(["--prompts", "2", "--tokens", "100", "--samples", "2", "--steps", "3"])
    assert bool((b.lens[::2] > 0).all()) and not bool(b.lens[1::2].any())
