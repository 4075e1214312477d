"""GPU parity of the key/value cache (nvfp4_kv_*) against the CPU oracle (oracle/kv.py).

Cache bytes, read-back values, tables and counts must match bit for bit. Attention outputs lie
inside a bound derived from the kernel's roundings: FP16 probabilities (unit roundoff 2^-11), scores
summed in FP32, FP16 values below 2^-24 after a factor of at least 2^6 on the largest, and the output
type's own rounding.
"""
import math

import numpy as np
import pytest
import torch

import nvfp4_block_scaled_amd as nv
import synth
from oracle import formats, kv

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _init():
    nv.init()


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def rounded(x, dtype):
    """float array -> (device tensor of dtype, the float32 values it holds)."""
    t = torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(TYPES[dtype])
    return t.cuda(), t.float().numpy()


def bits(t):
    return t.contiguous().view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()]).cpu().numpy()


# ------------------------------------------------------------------- append

def rope_inputs(r, rot, axes, T, max_pos=257):
    half = rot // 2
    ang = np.outer(np.arange(max_pos), 10000.0 ** (-np.arange(half) / max(1, half)))
    cos, sin = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)
    pos = r.integers(0, max_pos, (axes, T)).astype(np.int32)
    axis_of = r.integers(0, axes, half).astype(np.uint8) if axes > 1 else None
    return cos, sin, pos, axis_of


APPEND = [
    # T, Hq, Hkv, D, rot, axes, interleaved, page, dtype
    (1, 10, 1, 128, 128, 1, False, 16, "bf16"),
    (37, 40, 4, 128, 128, 3, False, 64, "bf16"),
    (130, 6, 2, 64, 64, 2, True, 32, "f16"),
    (19, 4, 4, 80, 40, 1, False, 16, "bf16"),        # pairs that no 16-byte access holds
    (19, 4, 2, 80, 80, 2, True, 16, "f16"),
    (21, 3, 3, 96, 48, 3, False, 128, "f16"),
    (9, 2, 1, 16, 16, 1, False, 256, "bf16"),
    (11, 2, 1, 16, 2, 1, True, 16, "bf16"),
    (33, 5, 5, 256, 256, 1, False, 16, "bf16"),
    (17, 9, 9, 192, 64, 3, True, 32, "bf16"),
    (65, 0, 3, 112, 0, 1, False, 64, "f16"),          # no queries, no rotation
    (300, 17, 1, 144, 36, 4, False, 16, "f16"),
]


@pytest.mark.parametrize("T,hq,hkv,D,rot,axes,inter,P,dtype", APPEND)
def test_append_and_read_bit_exact(T, hq, hkv, D, rot, axes, inter, P, dtype):
    r = synth.rng(T * 1000 + D)
    n_pages = -(-T // P) + 3
    size = nv.nvfp4_kv_page_bytes(P, hkv, D)
    assert size == kv.page_bytes(P, hkv, D)
    # q, k, v as columns of one product, as a fused projection gives them
    x = r.standard_normal((T, (hq + 2 * hkv) * D)) * np.exp(r.uniform(-3, 3, (T, 1)))
    x[:, hq * D: hq * D + 16] = 0.0                    # a zero block
    x[0, hq * D + 16:hq * D + 32] *= 1e4 if dtype == "bf16" else 1e2     # past the largest scale
    x[T // 2, -16:] = 1e-30 if dtype == "bf16" else 1e-7                 # a scale that rounds to zero
    xt, xf = rounded(x, dtype)
    cut = [hq * D, (hq + hkv) * D]
    view = lambda t, a, b: t[:, a:b].unflatten(1, (-1, D))     # noqa: E731
    q = view(xt, 0, cut[0]) if hq else None
    k, v = view(xt, cut[0], cut[1]), view(xt, cut[1], x.shape[1])
    kf, vf = (a.reshape(T, hkv, D) for a in (xf[:, cut[0]:cut[1]], xf[:, cut[1]:]))
    slots = r.permutation(n_pages * P)[:T].astype(np.int64)
    if T > 4:
        slots[2], slots[T - 1], slots[1] = -1, n_pages * P, -(1 << 40)
    k_g, v_g = (np.exp(r.uniform(3, 7, hkv)).astype(np.float32) for _ in range(2))
    kw = {}
    if rot:
        cos, sin, pos, axis_of = rope_inputs(r, rot, axes, T)
        kw = dict(cos=dev(cos), sin=dev(sin), positions=dev(pos) if axes > 1 else dev(pos[0]),
                  axis_of=None if axis_of is None else dev(axis_of), interleaved=inter)
        kf = kv.rotate(kf, cos, sin, pos, axis_of, inter)
    before = r.integers(0, 256, (n_pages, size + 48)).astype(np.uint8)
    pages = dev(before)[:, :size]                      # rows 48 bytes apart from each other
    cache = nv.KVCache(pages, P, hkv, D, dev(k_g), dev(v_g))
    got_q = nv.nvfp4_kv_append(cache, k, v, dev(slots), q=q, **kw)
    want = kv.append(before[:, :size], P, kf, vf, slots, k_g, v_g)
    np.testing.assert_array_equal(pages.cpu().numpy(), want)
    if hq:
        qf = xf[:, :cut[0]].reshape(T, hq, D)
        if rot:
            qf = kv.rotate(qf, cos, sin, pos, axis_of, inter)
        np.testing.assert_array_equal(bits(got_q), bits(torch.from_numpy(qf).to(TYPES[dtype])))
        assert nv.nvfp4_kv_append(cache, k, v, dev(slots), q=q, q_out=q, **kw) is q      # in place
        assert torch.equal(q, got_q)
    # read back: three types, slots outside the pool give zeros
    wk, wv = kv.held(want, P, hkv, D, k_g, v_g)
    inside = (slots >= 0) & (slots < n_pages * P)
    at = np.where(inside, slots, 0)
    for dt in (torch.float32, torch.bfloat16, torch.float16):
        got = nv.nvfp4_kv_read(cache, dev(slots), dt)
        for g, w in zip(got, (wk, wv)):
            w = np.where(inside[:, None, None], w[at], np.float32(0))
            ok = ~np.isnan(w)                           # (garbage in other slots may be NaN)
            wt = torch.from_numpy(w).to(dt).float().numpy()
            np.testing.assert_array_equal(g.float().cpu().numpy()[ok], wt[ok])
            assert np.isnan(g.float().cpu().numpy()[~ok]).all()


def test_append_special_values():
    """NaN marks its block, an infinity saturates it; a position outside the table gives NaN."""
    P, D = 16, 32
    x = np.ones((3, 1, D), np.float32)
    x[0, 0, 5] = np.nan
    x[1, 0, 20] = -np.inf
    xt, xf = rounded(x, "bf16")
    pages = torch.zeros((1, nv.nvfp4_kv_page_bytes(P, 1, D)), dtype=torch.uint8, device="cuda")
    cache = nv.KVCache(pages, P, 1, D)
    slots = np.arange(3, dtype=np.int64)
    nv.nvfp4_kv_append(cache, xt, xt, dev(slots))
    one = np.ones(1, np.float32)
    want = kv.append(np.zeros(pages.shape, np.uint8), P, xf, xf, slots, one, one)
    np.testing.assert_array_equal(pages.cpu().numpy(), want)
    k, v = nv.nvfp4_kv_read(cache, dev(slots), torch.float32)
    for a in (k, v):
        a = a.cpu().numpy()
        assert np.isnan(a[0, 0, :16]).all() and not np.isnan(a[0, 0, 16:]).any()
        assert a[1, 0, 20] == -2688.0 and np.isfinite(a[1]).all()
    cos = torch.ones((4, D // 2), device="cuda")
    q = nv.nvfp4_kv_append(cache, xt, xt, dev(slots), q=xt[1:].new_ones((3, 2, D)), cos=cos, sin=cos * 0,
                           positions=dev(np.array([3, 4, -1], np.int32)))
    assert torch.equal(q.isnan().any(2).any(1).cpu(), torch.tensor([False, True, True]))
    k, v = nv.nvfp4_kv_read(cache, dev(slots), torch.float32)
    assert k[1:].isnan().all() and not v[2].isnan().any()


def test_append_nothing():
    pages = torch.zeros((1, nv.nvfp4_kv_page_bytes(16, 2, 64)), dtype=torch.uint8, device="cuda")
    cache = nv.KVCache(pages, 16, 2, 64)
    e = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    s = torch.empty(0, dtype=torch.int64, device="cuda")
    q = nv.nvfp4_kv_append(cache, e, e, s, q=torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda"))
    assert q.shape == (0, 4, 64)
    k, v = nv.nvfp4_kv_read(cache, s)
    assert k.shape == v.shape == (0, 2, 64)


# ---------------------------------------------------------------- attention

def make_cache(r, lens, P, hkv, D, extra_cols=1, garbage=True, spread=1.0):
    """Pages in no order with random contents; every byte that no token owns is random (NaN scales too)."""
    need = [-(-int(n) // P) for n in lens]
    total = sum(need)
    n_pages = total + 3
    size = kv.page_bytes(P, hkv, D)
    pages = r.integers(0, 256, (n_pages, size)).astype(np.uint8) if garbage else np.zeros((n_pages, size), np.uint8)
    ids = r.permutation(n_pages)
    table = np.full((len(lens), max(need + [0]) + extra_cols), -1, np.int32)
    at, slots = 0, []
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
        t = np.arange(int(lens[b]))
        slots.append(table[b, t // P].astype(np.int64) * P + t % P)
    slots = np.concatenate(slots) if slots else np.zeros(0, np.int64)
    k_g, v_g = (np.exp(r.uniform(3, 6, hkv)).astype(np.float32) for _ in range(2))
    # contents through the byte format: random codes and ordinary scales
    kc, ks, vc, vs = kv._sections(pages, P, hkv, D)
    T = slots.size
    codes = r.integers(0, 256, (2, T, hkv, D // 2)).astype(np.uint8)
    scales = formats.round_e4m3_byte((2.0 ** r.uniform(1, 7, (2, T, hkv, D // 16)) * spread))
    p, o = slots // P, slots % P
    kc[p, :, o], ks[p, :, o] = codes[0], scales[0]
    vc[p, :, o // 4, :, o % 4, :] = codes[1].reshape(T, hkv, D // 8, 4)
    vs[p, :, :, o] = scales[1]
    return pages, table, k_g, v_g


def check(got, lse, ref, dtype, D, what=""):
    out, rlse, mass, big, vmax = ref
    g = got.float().cpu().numpy().astype(np.float64)
    u = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -11
    n = 1 << 20
    delta = 2.0 ** -20 + (D + 8) * 2.0 ** -23 * big
    tol = (1 + u) * ((2.0 ** -11 + 2 * delta[..., None]) * mass + n * 2.0 ** -31 * vmax[..., None])
    tol = tol + u * np.abs(out) + (2.0 ** -24 if dtype == "f16" else 0.0)
    assert np.array_equal(np.isnan(g), np.isnan(out)), what
    err = np.where(np.isnan(out), 0.0, np.abs(g - out))
    assert np.all(err <= np.where(np.isnan(out), 1.0, tol)), (what, float((err - tol)[~np.isnan(out)].max()))
    if lse is not None:
        l = lse.cpu().numpy().astype(np.float64)
        assert np.array_equal(np.isnan(l), np.isnan(rlse)) and np.array_equal(l == -np.inf, rlse == -np.inf), what
        fine = np.isfinite(rlse)
        ltol = delta + 2.0 ** -21 * (np.abs(rlse) + 16)
        assert np.all(np.abs(l - rlse)[fine] <= ltol[fine]), (what, np.abs(l - rlse)[fine].max())


def attend(seed, lens, counts, hq, hkv, D, P, dtype="bf16", q_start=True, causal=True, window=0, mask=None, max_q=None,
           qscale=0.05, edit=None, pad=0):
    r = synth.rng(seed)
    lens = np.asarray(lens, np.int32)
    pages, table, k_g, v_g = make_cache(r, lens, P, hkv, D)
    if edit:
        edit(pages, table)
    T = int(np.sum(counts))
    qt, qf = rounded(r.standard_normal((T, hq, D + pad)) * qscale, dtype)
    start = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    cache = nv.KVCache(dev(pages), P, hkv, D, dev(k_g), dev(v_g))
    scale = 1.0 / math.sqrt(D)
    args = dict(q_start=dev(start) if q_start else None, max_q=max_q or max(list(counts) + [1]), causal=causal,
                window=window, mask=None if mask is None else dev(mask), return_lse=True)
    got, lse = nv.nvfp4_kv_attention(qt[..., :D], cache, dev(table), dev(lens), **args)
    k, v = kv.exact_values(pages, P, hkv, D, k_g, v_g)
    ref = kv.attention(qf[..., :D].astype(np.float64), k, v, P, table, lens, start if q_start else None, scale, causal,
                       window, mask)
    check(got, lse, ref, dtype, D, (seed, hq, hkv, D, P, dtype))
    again, lse2 = nv.nvfp4_kv_attention(qt[..., :D], cache, dev(table), dev(lens), **args)
    assert torch.equal(bits_t(got), bits_t(again)) and torch.equal(bits_t(lse), bits_t(lse2))
    return got, lse


def bits_t(t):
    return t.view({2: torch.int16, 4: torch.int32}[t.element_size()])


EDGE_LENS = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 130, 255, 257, 500]


@pytest.mark.parametrize("hq,hkv,D,P,dtype", [
    (10, 1, 128, 16, "bf16"), (8, 2, 64, 32, "f16"), (5, 5, 256, 64, "bf16"), (16, 1, 128, 128, "f16"),
    (3, 1, 80, 16, "bf16"), (6, 2, 96, 256, "bf16"), (2, 2, 16, 16, "f16"), (4, 2, 48, 32, "bf16"),
    (8, 4, 192, 16, "f16"), (24, 1, 112, 64, "bf16"), (40, 1, 128, 32, "bf16"), (96, 2, 160, 16, "bf16"),
    (20, 1, 240, 32, "f16")])
def test_decode(hq, hkv, D, P, dtype):
    attend(hq * 100 + D, EDGE_LENS, [1] * len(EDGE_LENS), hq, hkv, D, P, dtype, q_start=False)


@pytest.mark.parametrize("hq,hkv,D,P,dtype", [(10, 1, 128, 16, "bf16"), (4, 2, 64, 64, "f16"), (2, 1, 256, 32, "bf16"),
                                             (3, 3, 80, 16, "f16"), (40, 2, 128, 32, "bf16"), (1, 1, 192, 16, "bf16")])
@pytest.mark.parametrize("form", ["causal", "window", "full"])
def test_chunks(hq, hkv, D, P, dtype, form):
    """Several queries a sequence, sequences shorter than their queries (rows that see no key), none at all."""
    lens = [0, 1, 5, 40, 129, 200, 333, 64]
    counts = [1, 1, 9, 33, 3, 65, 0, 64]
    attend(D + hq, lens, counts, hq, hkv, D, P, dtype, causal=form != "full", window=37 if form == "window" else 0)


@pytest.mark.parametrize("hq,hkv,D,P", [(10, 1, 128, 64), (4, 4, 64, 16), (2, 1, 256, 128)])
def test_long_chunk(hq, hkv, D, P):
    attend(7, [700, 900], [300, 260], hq, hkv, D, P)
    attend(8, [700, 900], [300, 260], hq, hkv, D, P, window=200, dtype="f16")


@pytest.mark.parametrize("hq,hkv,D,P,dtype", [(10, 1, 128, 32, "bf16"), (4, 2, 64, 16, "f16"), (2, 1, 256, 64, "bf16"),
                                             (40, 4, 128, 16, "bf16")])
def test_tree_mask(hq, hkv, D, P, dtype):
    r = synth.rng(3)
    lens, counts = [3, 50, 200, 8, 0, 31, 1000], [3, 7, 16, 8, 2, 1, 5]     # history of no key, and a row with no key
    mask = (r.random((sum(counts), 18)) < 0.5).astype(np.uint8)
    mask[0] = 0
    attend(11, lens, counts, hq, hkv, D, P, dtype, mask=mask)


@pytest.mark.parametrize("D,P,n", [(128, 256, 20011), (64, 16, 5000), (256, 64, 6001)])
def test_split_and_join(D, P, n):
    """One sequence split over many workgroups, alone and beside short ones."""
    attend(21, [n], [1], 4, 1, D, P, q_start=False)
    attend(22, [3, n, 0, 130], [1] * 4, 4, 2, D, P, q_start=False, dtype="f16")
    attend(23, [n, 77], [5, 4], 4, 2, D, P)


@pytest.mark.parametrize("batch", [64, 65, 129, 300, 1030])
def test_many_sequences(batch):
    """More sequences than a wave has lanes: single tokens, several queries (some sequences have none), and a few long ones."""
    r = synth.rng(batch)
    lens = r.integers(0, 40, batch)
    lens[[1, batch // 2, batch - 1]] = 1500, 0, 2100
    attend(1000 + batch, lens, [1] * batch, 4, 2, 64, 16, q_start=False)
    attend(2000 + batch, lens, r.integers(0, 4, batch), 10, 1, 64, 32, dtype="f16")
    attend(3000 + batch, lens, r.integers(0, 3, batch), 36, 2, 64, 16)
    attend(4000 + batch, np.minimum(lens, 60), r.integers(0, 2, batch), 4, 2, 128, 16)


def test_query_shapes():
    """Strided and misaligned queries, a query of zeros, one with an infinity, and very small and large ones."""
    attend(31, [40, 77], [1, 1], 6, 2, 64, 16, q_start=False, pad=3)
    attend(32, [40, 77], [1, 1], 6, 2, 64, 16, q_start=False, pad=8)
    attend(33, [40, 77], [1, 1], 6, 2, 64, 16, q_start=False, qscale=1e-30)
    attend(34, [40, 77], [1, 1], 6, 2, 64, 16, q_start=False, qscale=30.0)
    pages = torch.full((2, nv.nvfp4_kv_page_bytes(16, 1, 64)), 0x22, dtype=torch.uint8, device="cuda")
    cache = nv.KVCache(pages, 16, 1, 64)
    table, lens = dev(np.array([[1, 0]], np.int32)), dev(np.array([30], np.int32))
    q = torch.zeros((1, 2, 64), dtype=torch.bfloat16, device="cuda")
    q[0, 1, 3] = math.inf
    out, lse = nv.nvfp4_kv_attention(q, cache, table, lens, return_lse=True)
    assert not out[0, 0].isnan().any() and out[0, 1].isnan().all() and lse[0, 1].isnan()
    assert abs(lse[0, 0].item() - math.log(30)) < 1e-6


def test_masked_nan_stays_out():
    """NaN keys and values of later tokens, of tokens before the window and of an unseen branch reach no
    row that does not see them, and every row that does."""
    P, hkv, D = 16, 1, 64
    n, new = 150, 40

    def poison(at):
        def edit(pages, table):
            kc, ks, vc, vs = kv._sections(pages, P, hkv, D)
            page, o = int(table[0, at // P]), at % P
            vs[page, 0, 2, o] = 0x7F
        return edit

    def poison_key(at):
        def edit(pages, table):
            kc, ks, vc, vs = kv._sections(pages, P, hkv, D)
            ks[int(table[0, at // P]), 0, at % P, 1] = 0xFF
        return edit
    for at in (115, 130, 149):
        out, _ = attend(41, [n], [new], 4, hkv, D, P, edit=poison(at))
        seen = np.arange(n - new, n) >= at
        bad = out.isnan().cpu().numpy()
        assert bad[seen][:, :, 32:48].all() and not bad[~seen].any() and not bad[:, :, :32].any()
        attend(42, [n], [new], 4, hkv, D, P, edit=poison_key(at))
    for at in (20, 100):
        out, _ = attend(43, [n], [new], 4, hkv, D, P, edit=poison(at), window=30)
        seen = np.arange(n - new, n) < at + 30
        assert np.array_equal(out.isnan().any(2).any(1).cpu().numpy(), seen)
    mask = np.tril(np.ones((8, 8), np.uint8))
    mask[:, 3] = 0
    mask[3, 3] = 1
    out, _ = attend(44, [n], [8], 4, hkv, D, P, edit=poison(n - 8 + 3), mask=mask)
    assert np.array_equal(out.isnan().any(2).any(1).cpu().numpy(), np.arange(8) == 3)


def test_page_ids_outside_the_pool_are_masked():
    def edit(pages, table):
        table[0, 1] = -7
        table[1, 0] = 10 ** 6
    attend(51, [60, 10, 33], [1, 1, 1], 4, 2, 64, 16, q_start=False, edit=edit)
    attend(52, [60, 10, 33], [9, 2, 20], 4, 2, 64, 16, edit=edit)


def test_lengths_out_of_range_are_clamped():
    r = synth.rng(5)
    pages, table, k_g, v_g = make_cache(r, [64, 64], 16, 1, 64, extra_cols=0)
    cache = nv.KVCache(dev(pages), 16, 1, 64, dev(k_g), dev(v_g))
    q, _ = rounded(r.standard_normal((2, 2, 64)), "bf16")
    a = nv.nvfp4_kv_attention(q, cache, dev(table), dev(np.array([64, 0], np.int32)))
    b = nv.nvfp4_kv_attention(q, cache, dev(table), dev(np.array([1 << 30, -5], np.int32)))
    assert torch.equal(a, b) and not a[1].any()


def test_offsets_past_32_bits():
    """Pages more than 4 GiB apart: append, read, attention and copies reach them."""
    P, hkv, D = 16, 1, 64
    size = nv.nvfp4_kv_page_bytes(P, hkv, D)
    stride = (1 << 31) + 16 * size // 16 * 16
    whole = torch.empty(2 * stride + stride // 2, dtype=torch.uint8, device="cuda")
    pages = whole.as_strided((3, size), (stride, 1))
    pages.zero_()
    r = synth.rng(6)
    cache = nv.KVCache(pages, P, hkv, D)
    kt, kf = rounded(r.standard_normal((20, 1, D)), "bf16")
    slots = np.concatenate([2 * P + np.arange(16), np.arange(4)]).astype(np.int64)
    nv.nvfp4_kv_append(cache, kt, kt, dev(slots))
    one = np.ones(1, np.float32)
    want = kv.append(np.zeros((3, size), np.uint8), P, kf, kf, slots, one, one)
    np.testing.assert_array_equal(pages.cpu().numpy(), want)
    qt, qf = rounded(r.standard_normal((1, 4, D)), "bf16")
    table, lens = np.array([[2, 0]], np.int32), np.array([20], np.int32)
    got, lse = nv.nvfp4_kv_attention(qt, cache, dev(table), dev(lens), return_lse=True)
    k, v = kv.exact_values(want, P, hkv, D, one, one)
    check(got, lse, kv.attention(qf.astype(np.float64), k, v, P, table, lens, None, 1 / 8), "bf16", D)
    nv.nvfp4_kv_copy_pages(pages, dev(np.array([2], np.int32)), dev(np.array([1], np.int32)))
    assert torch.equal(pages[1], pages[2])


def test_other_stream_and_graph():
    """A stream of its own, and a captured step replayed with other lengths and queries."""
    r = synth.rng(9)
    lens = np.array([700, 1, 333], np.int32)
    pages, table, k_g, v_g = make_cache(r, [800, 800, 800], 16, 2, 128)
    cache = nv.KVCache(dev(pages), 16, 2, 128, dev(k_g), dev(v_g))
    tb, ln = dev(table), dev(lens)
    qs = [rounded(r.standard_normal((3, 8, 128)) * 0.1, "bf16")[0] for _ in range(3)]
    ws = nv.nvfp4_kv_attention_workspace(3, 8, cache, 3, table.shape[1])
    eager = []
    for i, q in enumerate(qs):
        eager.append(nv.nvfp4_kv_attention(q, cache, tb, (ln + i).contiguous(), ws=ws).clone())
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        other = nv.nvfp4_kv_attention(qs[0], cache, tb, ln)
    s.synchronize()
    assert torch.equal(other, eager[0])
    q, out, n = qs[0].clone(), torch.empty_like(qs[0]), ln.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nv.nvfp4_kv_attention(q, cache, tb, n, out=out, ws=ws)
    for i in (0, 1, 2, 1, 0):
        q.copy_(qs[i])
        n.copy_(ln + i)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager[i]), i


@pytest.mark.parametrize("hq,counts", [(8, [1, 1, 1]), (8, [20, 1, 3])])
def test_workspace_needs_no_initialisation(hq, counts):
    """Any bytes in the workspace, and one workspace for calls of several sizes in turn."""
    r = synth.rng(19)
    lens = np.array([9000, 40, 2500], np.int32)
    pages, table, k_g, v_g = make_cache(r, lens, 32, 1, 128)
    cache = nv.KVCache(dev(pages), 32, 1, 128, dev(k_g), dev(v_g))
    tb, ln = dev(table), dev(lens)
    T = sum(counts)
    q = rounded(r.standard_normal((T, hq, 128)) * 0.1, "bf16")[0]
    start = dev(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32))
    ws = nv.nvfp4_kv_attention_workspace(T, hq, cache, 3, table.shape[1], max(counts))
    assert ws is not None
    want = nv.nvfp4_kv_attention(q, cache, tb, ln, start, max(counts))
    for fill in (0, 0xFF, 0x7F, None, None):
        if fill is None:
            ws.copy_(torch.randint(0, 256, ws.shape, dtype=torch.uint8, device="cuda"))
        else:
            ws.fill_(fill)
        for n in (ln, ln // 3, ln):
            got = nv.nvfp4_kv_attention(q, cache, tb, n, start, max(counts), ws=ws)
            assert n is not ln or torch.equal(got, want)


# -------------------------------------------------------------------- pages

def page_state(r, n_pages, batch, width, P, fill=0.6):
    lens = np.array([int(r.integers(0, width * P + 1)) for _ in range(batch)], np.int32)
    lens[0] = 0 if batch > 2 else lens[0]
    if batch > 1:
        lens[1] = (lens[1] // P) * P                       # a whole number of pages
    need = -(-lens // P)
    while need.sum() > n_pages * fill:
        b = int(np.argmax(need))
        lens[b] //= 2
        need = -(-lens // P)
    ids = r.permutation(n_pages)
    table, refs, at = np.full((batch, width), -1, np.int32), np.zeros(n_pages, np.int32), 0
    for b in range(batch):
        table[b, :need[b]] = ids[at:at + need[b]]
        at += need[b]
    refs[ids[:at]] = 1
    refs[ids[at:at + 2]] = -3                              # below zero counts as free
    return table, lens, refs


POOLS = [(1, 1, 1, 16), (7, 3, 4, 16), (64, 5, 20, 32), (5000, 40, 100, 16), (40000, 300, 70, 64)]


@pytest.mark.parametrize("n_pages,batch,width,P", POOLS)
@pytest.mark.parametrize("in_place", [False, True])
def test_fork(n_pages, batch, width, P, in_place):
    r = synth.rng(n_pages + batch)
    table, lens, refs = page_state(r, n_pages, batch, width, P)
    parents = r.integers(0, batch, max(1, min(2 * batch, 1500))).astype(np.int32)
    if len(parents) > 5:
        parents[1], parents[4] = -1, batch
        lens[parents[0]] = width * P + 1 if n_pages == 64 else lens[parents[0]]
    layers, size = 3, 208
    pool = r.integers(0, 256, (layers, n_pages, size)).astype(np.uint8)
    pages, refs_d = dev(pool), dev(refs)
    child, new, short = nv.nvfp4_kv_fork(pages, dev(table), dev(lens), refs_d, dev(parents), P,
                                         out_refs=refs_d if in_place else None)
    w_child, w_refs, w_short, copies = kv.fork(P, table, lens, refs, parents)
    np.testing.assert_array_equal(child.cpu().numpy(), w_child)
    np.testing.assert_array_equal(new.cpu().numpy(), w_refs)
    assert int(short) == w_short
    if not in_place:
        np.testing.assert_array_equal(refs_d.cpu().numpy(), refs)
    for a, b in copies:
        pool[:, b] = pool[:, a]
    np.testing.assert_array_equal(pages.cpu().numpy(), pool)


@pytest.mark.parametrize("n_pages,batch,width,P", POOLS)
@pytest.mark.parametrize("in_place", [False, True])
def test_resize(n_pages, batch, width, P, in_place):
    r = synth.rng(n_pages * 3 + batch)
    table, lens, refs = page_state(r, n_pages, batch, width, P)
    if batch > 2:                                          # shared pages
        w = min(lens[1], lens[2]) // P
        refs[table[2, :w]] -= 1
        table[2, :w] = table[1, :w]
        refs[table[2, :w]] += 1
    new_lens = r.integers(0, width * P + 1, batch).astype(np.int32)
    new_lens[::4] = 0
    new_lens[1::4] = lens[1::4]
    if batch > 4:
        new_lens[3] = -9                                   # taken as 0
    t, f = dev(table), dev(refs)
    got, new, short = nv.nvfp4_kv_resize(t, dev(lens), dev(new_lens), f, P, out_table=t if in_place else None,
                                         out_refs=f if in_place else None)
    w_table, w_refs, w_short = kv.resize(P, table, lens, new_lens, refs)
    np.testing.assert_array_equal(got.cpu().numpy(), w_table)
    np.testing.assert_array_equal(new.cpu().numpy(), w_refs)
    assert int(short) == w_short


@pytest.mark.parametrize("n_pages,batch,width,P", POOLS)
@pytest.mark.parametrize("in_place", [False, True])
def test_compact(n_pages, batch, width, P, in_place):
    r = synth.rng(n_pages * 7 + batch)
    table, lens, refs = page_state(r, n_pages, batch, width, P)
    table[r.random(table.shape) < 0.05] = -1
    layers, size = 2, 4240
    if n_pages * layers * size > 1 << 28:
        size = 48
    pool = r.integers(0, 256, (layers, n_pages, size)).astype(np.uint8)
    big = torch.zeros((layers, n_pages, size + 16), dtype=torch.uint8, device="cuda")
    pages = big[:, :, :size]
    pages.copy_(dev(pool))
    t, f = dev(table), dev(refs)
    got, new, live = nv.nvfp4_kv_compact(pages, t, f, out_table=t if in_place else None, out_refs=f if in_place else None)
    w_table, w_refs, w_live, moves = kv.compact(table, refs)
    np.testing.assert_array_equal(got.cpu().numpy(), w_table)
    np.testing.assert_array_equal(new.cpu().numpy(), w_refs)
    assert int(live) == w_live
    for a, b in moves:
        pool[:, b] = pool[:, a]
    np.testing.assert_array_equal(pages.cpu().numpy(), pool)


def test_compact_full_and_empty_pools():
    pages = torch.zeros((5, 16), dtype=torch.uint8, device="cuda")
    table = dev(np.array([[4, 0, -1]], np.int32))
    for refs in (np.ones(5, np.int32), np.zeros(5, np.int32)):
        t, f, live = nv.nvfp4_kv_compact(pages, table, dev(refs))
        assert torch.equal(t, table) and int(live) == refs.sum() and np.array_equal(f.cpu().numpy(), refs)


def test_copy_pages():
    r = synth.rng(1)
    pool = r.integers(0, 256, (4, 50, 1040)).astype(np.uint8)
    pages = dev(pool)
    ids = r.permutation(50).astype(np.int32)
    src, dst = ids[:20].copy(), ids[20:40].copy()
    src[3], dst[5], src[7] = -1, 50, 10 ** 9               # skipped
    nv.nvfp4_kv_copy_pages(pages, dev(src), dev(dst))
    for a, b in zip(src, dst):
        if 0 <= a < 50 and 0 <= b < 50:
            pool[:, b] = pool[:, a]
    np.testing.assert_array_equal(pages.cpu().numpy(), pool)
    nv.nvfp4_kv_copy_pages(pages, dev(src[:0]), dev(dst[:0]))


# ----------------------------------------------------------------- refusals

def _small():
    pages = torch.zeros((4, nv.nvfp4_kv_page_bytes(16, 2, 64)), dtype=torch.uint8, device="cuda")
    return nv.KVCache(pages, 16, 2, 64), pages


def test_refuses_bad_arguments():
    cache, pages = _small()
    x = torch.zeros((3, 2, 64), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((3, 4, 64), dtype=torch.bfloat16, device="cuda")
    slots = torch.zeros(3, dtype=torch.int64, device="cuda")
    table = torch.zeros((3, 2), dtype=torch.int32, device="cuda")
    lens = torch.zeros(3, dtype=torch.int32, device="cuda")
    cs = torch.zeros((4, 32), device="cuda")
    pos = torch.zeros(3, dtype=torch.int32, device="cuda")
    bad_value = [
        lambda: nv.KVCache(pages, 24, 2, 64), lambda: nv.KVCache(pages, 16, 2, 72), lambda: nv.KVCache(pages, 16, 3, 64),
        lambda: nv.KVCache(pages[:, ::2], 16, 1, 64), lambda: nv.KVCache(pages, 16, 2, 64, torch.ones(1, device="cuda")),
        lambda: nv.nvfp4_kv_append(cache, x[:, :1], x, slots), lambda: nv.nvfp4_kv_append(cache, x, x[:2], slots),
        lambda: nv.nvfp4_kv_append(cache, x, x, slots[:2]), lambda: nv.nvfp4_kv_append(cache, x, x, slots, q_out=q),
        lambda: nv.nvfp4_kv_append(cache, x, x, slots, cos=cs), lambda: nv.nvfp4_kv_append(cache, x, x, slots, positions=pos),
        lambda: nv.nvfp4_kv_append(cache, x, x, slots, cos=torch.zeros((4, 33), device="cuda"),
                                   sin=torch.zeros((4, 33), device="cuda"), positions=pos),
        lambda: nv.nvfp4_kv_append(cache, x, x, slots, cos=cs, sin=cs, positions=pos[:2]),
        lambda: nv.nvfp4_kv_append(cache, x, x, slots, q=q, q_out=torch.empty((3, 4, 72), dtype=q.dtype, device="cuda")[:, :, 1:65]),
        lambda: nv.nvfp4_kv_append(cache, x, x, slots, q=q, q_out=torch.empty((1, 4, 64), dtype=q.dtype, device="cuda").expand(3, -1, -1)),
        lambda: nv.nvfp4_kv_attention(q[:2], cache, table, lens), lambda: nv.nvfp4_kv_attention(q[:, :3], cache, table, lens),
        lambda: nv.nvfp4_kv_attention(q, cache, table, lens[:2]), lambda: nv.nvfp4_kv_attention(q, cache, table, lens, scale=0.0),
        lambda: nv.nvfp4_kv_attention(q, cache, table, lens, scale=math.inf),
        lambda: nv.nvfp4_kv_attention(q, cache, table, lens, window=-1),
        lambda: nv.nvfp4_kv_attention(q, cache, table, lens, causal=False, window=4),
        lambda: nv.nvfp4_kv_attention(q, cache, table, lens, window=4, mask=torch.ones((3, 1), dtype=torch.bool, device="cuda")),
        lambda: nv.nvfp4_kv_attention(q, cache, table, lens, q_start=lens, max_q=3),
        lambda: nv.nvfp4_kv_attention(q, cache, torch.zeros((3, 200), dtype=torch.int32, device="cuda"), lens,
                                      ws=torch.empty(16, dtype=torch.uint8, device="cuda")),
        lambda: nv.nvfp4_kv_fork(pages, table, lens, lens, lens, 16),           # counts of another pool
        lambda: nv.nvfp4_kv_fork(pages, table, lens, torch.zeros(4, dtype=torch.int32, device="cuda"), lens, 24),
        lambda: nv.nvfp4_kv_resize(table, lens, lens[:2], lens, 16),
        lambda: nv.nvfp4_kv_compact(pages[:, :40], table, torch.zeros(4, dtype=torch.int32, device="cuda")),
        lambda: nv.nvfp4_kv_copy_pages(pages, lens, lens[:2]),
    ]
    for i, f in enumerate(bad_value):
        with pytest.raises(ValueError):
            f()
            pytest.fail(f"case {i} was taken")
    bad_type = [
        lambda: nv.KVCache(pages.view(torch.int8), 16, 2, 64), lambda: nv.KVCache(pages.cpu(), 16, 2, 64),
        lambda: nv.nvfp4_kv_append(None, x, x, slots), lambda: nv.nvfp4_kv_append(cache, x.float(), x, slots),
        lambda: nv.nvfp4_kv_append(cache, x, x.half(), slots), lambda: nv.nvfp4_kv_append(cache, x, x, slots.int()),
        lambda: nv.nvfp4_kv_append(cache, x.cpu(), x, slots), lambda: nv.nvfp4_kv_read(cache, slots, torch.float64),
        lambda: nv.nvfp4_kv_attention(q.float(), cache, table, lens), lambda: nv.nvfp4_kv_attention(q, cache, table.long(), lens),
        lambda: nv.nvfp4_kv_attention(q, cache, table, lens.cpu()),
        lambda: nv.nvfp4_kv_attention(q, cache, table, lens, mask=torch.ones((3, 1), device="cuda")),
        lambda: nv.nvfp4_kv_copy_pages(pages, lens.long(), lens),
    ]
    for i, f in enumerate(bad_type):
        with pytest.raises(TypeError):
            f()
            pytest.fail(f"case {i} was taken")
