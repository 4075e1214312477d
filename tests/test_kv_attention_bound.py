"""Attention over long sequences against float64 within a bound that a few lost values would break.

For a row that sees n keys with weights p_j (sum 1), an output element differs from sum_j p_j v_j by at most
* each p_j rounded to FP16, 2^-11 of itself and independent of the others: no more than 2^-11 sum p_j |v_j|, and by
  Hoeffding's inequality 8 * 2^-11 sqrt(sum p_j^2 v_j^2) with a chance of 3e-14 to pass it;
* 2^-25 for each p_j that is subnormal in FP16, where the largest is at least 2^6: 2^-31 |v| each, and only those below
  2^-19 of the row's largest;
* scores, FP32 over D products and the softmax's factor: delta, twice (weights and their sum);
* FP32 sums of at most 512 terms one after the other (a wave's share of a piece, the waves, the pieces): 2^-15;
* the output's own rounding.
"""
import math

import numpy as np
import pytest
import torch

import nvfp4_block_scaled_amd as nv
import synth
from oracle import kv
from test_kv_cache import dev, make_cache


def reference(q, k, v, scale, see, lost=()):
    """q [rows][D] against k, v [n][D] float64 where see [rows][n]: (out, lse, bound on out before its rounding, bound
    on lse). lost: keys whose values count as zero, though their weights stay in the sum."""
    n, D = k.shape
    t = np.where(see, scale * (q @ k.T), -np.inf)
    top = t.max(1, keepdims=True)
    p = np.exp(t - top)
    total = p.sum(1, keepdims=True)
    small = (p < 2.0 ** -19) & see
    p = p / total
    kept = v.copy()
    kept[list(lost)] = 0.0
    mass = p @ np.abs(v)
    big = scale * np.where(see, np.abs(q) @ np.abs(k).T, 0.0).max(1, keepdims=True)
    delta = 2.0 ** -20 + (D + 8) * 2.0 ** -23 * big
    rounding = np.minimum(2.0 ** -11 * mass, 8 * 2.0 ** -11 * np.sqrt((p * p) @ (v * v)))
    bound = rounding + small.sum(1, keepdims=True) * 2.0 ** -31 * np.abs(v).max() + (2 * delta + 2.0 ** -15) * mass
    lse = (top + np.log(total))[:, 0]
    return p @ kept, lse, bound, delta[:, 0] + 2.0 ** -15 + 2.0 ** -21 * (np.abs(lse) + 16)


def worst(got, want, bound, dtype):
    """The largest error over its bound, the output's rounding included."""
    u, least = (2.0 ** -8, 0.0) if dtype == "bf16" else (2.0 ** -11, 2.0 ** -25)
    err, tol = np.abs(got - want), bound * (1 + u) + u * np.abs(want) + least
    return float(np.divide(err, tol, out=np.zeros_like(err), where=err != 0).max())     # (no error where none may be: 0)


def case(seed, lens, counts, hq, hkv, D, P, dtype):
    """Inputs, and per (sequence, KV head) what reference() takes: the rows are the sequence's queries and the heads of
    its group, each seeing the keys up to its own."""
    r = synth.rng(seed)
    pages, table, k_g, v_g = make_cache(r, lens, P, hkv, D)
    qt = torch.from_numpy((r.standard_normal((sum(counts), hq, D)) * 0.05).astype(np.float32)).to(
        torch.bfloat16 if dtype == "bf16" else torch.float16)
    q = qt.double().numpy()
    k, v = kv.exact_values(pages, P, hkv, D, k_g, v_g)
    G, row, parts = hq // hkv, 0, []
    for b, (n, m) in enumerate(zip(lens, counts)):
        slots = (table[b, :-(-n // P), None].astype(np.int64) * P + np.arange(P)).reshape(-1)[:n]
        see = np.repeat(np.arange(n) <= np.arange(n - m, n)[:, None], G, axis=0)
        for h in range(hkv):
            parts.append((slice(row, row + m), slice(h * G, h * G + G), q[row:row + m, h * G:h * G + G].reshape(m * G, D),
                          k[slots, h], v[slots, h], see))
        row += m
    return pages, table, k_g, v_g, qt, parts


SIZES = [(128, 256, 20011), (64, 16, 5000), (256, 64, 6001), (96, 32, 9001)]
FORMS = [("one token", [1], 4, 1), ("one token beside short ones", [1, 1, 1], 4, 2), ("drafts", [5, 4], 4, 2),
         ("a chunk", [40, 33], 4, 2)]


def lengths(n, counts):
    return [n, 130, 77][:len(counts)] if len(counts) != 2 else [n, 77]


@pytest.mark.gpu
@pytest.mark.parametrize("D,P,n", SIZES)
@pytest.mark.parametrize("name,counts,hq,hkv", FORMS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_split_sequences_within_the_bound(D, P, n, name, counts, hq, hkv, dtype):
    lens = lengths(n, counts)
    pages, table, k_g, v_g, qt, parts = case(D + n, lens, counts, hq, hkv, D, P, dtype)
    cache = nv.KVCache(dev(pages), P, hkv, D, dev(k_g), dev(v_g))
    start = dev(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)) if max(counts) > 1 else None
    out, lse = nv.nvfp4_kv_attention(qt.cuda(), cache, dev(table), dev(np.array(lens, np.int32)), start, max(counts),
                                     return_lse=True)
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for rows, heads, q, k, v, see in parts:
        want, w_lse, bound, l_bound = reference(q, k, v, 1 / math.sqrt(D), see)
        assert worst(out[rows, heads].reshape(want.shape), want, bound, dtype) <= 1.0
        assert (np.abs(lse[rows, heads].reshape(-1) - w_lse) <= l_bound).all()


@pytest.mark.gpu
@pytest.mark.parametrize("extra", [0, 1, 40, 2000])
@pytest.mark.parametrize("counts", [[1, 1, 1], [9, 1, 30]])
def test_tables_wider_than_their_sequences(extra, counts):
    """A captured step's table has room for the longest context it may meet; the unused columns hold any id."""
    D, P, lens = 128, 16, [300, 1, 77]
    pages, table, k_g, v_g, qt, parts = case(5, lens, counts, 8, 2, D, P, "bf16")
    table = np.concatenate([table, synth.rng(extra).integers(-5, 99, (3, extra)).astype(np.int32)], 1)
    cache = nv.KVCache(dev(pages), P, 2, D, dev(k_g), dev(v_g))
    start = dev(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)) if max(counts) > 1 else None
    out, lse = nv.nvfp4_kv_attention(qt.cuda(), cache, dev(table), dev(np.array(lens, np.int32)), start, max(counts),
                                     return_lse=True)
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    for rows, heads, q, k, v, see in parts:
        want, w_lse, bound, l_bound = reference(q, k, v, 1 / math.sqrt(D), see)
        assert worst(out[rows, heads].reshape(want.shape), want, bound, "bf16") <= 1.0
        assert (np.abs(lse[rows, heads].reshape(-1) - w_lse) <= l_bound).all()


@pytest.mark.parametrize("D,P,n", SIZES)
@pytest.mark.parametrize("name,counts,hq,hkv", FORMS)
def test_the_bound_sees_sixteen_lost_keys(D, P, n, name, counts, hq, hkv):
    """The values of one group of 16 keys lost, anywhere in the long sequence, break it; FP16 weights do not."""
    lens = lengths(n, counts)
    parts = case(D + n, lens, counts, hq, hkv, D, P, "bf16")[-1]
    for _, _, q, k, v, see in parts[:hkv]:
        want, _, bound, _ = reference(q, k, v, 1 / math.sqrt(D), see)
        for first in (0, 16, 128, n // 32 * 16, n - max(counts) - 16):
            less = reference(q, k, v, 1 / math.sqrt(D), see, range(first, first + 16))[0]
            assert worst(less, want, bound, "bf16") > 1.0, first
        t = np.where(see, q @ k.T / math.sqrt(D), -np.inf)
        p = np.exp(t - t.max(1, keepdims=True))
        near = (p * 64).astype(np.float16).astype(np.float64) / 64 @ v / p.sum(1, keepdims=True)
        assert worst(near, want, bound, "bf16") <= 1.0
