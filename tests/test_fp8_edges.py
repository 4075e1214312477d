"""FP8 in blocks where earlier tests did not look: gates far from zero."""
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
