"""Edges of the key/value cache's operators: full pools, page ids without a page, very long windows, and arguments
that only just do or do not fit."""
import ctypes
import math

import numpy as np
import pytest
import torch

import nvfp4_block_scaled_amd as nv
import synth
from oracle import kv
from test_kv_cache import attend, dev


@pytest.mark.gpu
@pytest.mark.parametrize("fill", [0, 0xFF])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("n_pages", [16383, 16384, 16385, 32768])
def test_compact_of_full_pools(n_pages, in_place, fill):
    """No free page, or one, around the 16384 counts that one workgroup scans; any bytes in the workspace."""
    r = synth.rng(n_pages)
    pool = r.integers(0, 256, (2, n_pages, 16)).astype(np.uint8)
    table = r.permutation(n_pages).astype(np.int32).reshape(1, -1)
    ws = torch.empty(nv.lib().nvfp4_kv_pages_workspace_bytes(n_pages, 1), dtype=torch.uint8, device="cuda")
    for free in (None, 0, n_pages // 2, n_pages - 1):
        refs = r.integers(1, 5, n_pages).astype(np.int32)
        if free is not None:
            refs[free] = 0
        pages, t, f = dev(pool), dev(table), dev(refs)
        ws.fill_(fill)
        got, new, live = nv.nvfp4_kv_compact(pages, t, f, out_table=t if in_place else None,
                                             out_refs=f if in_place else None, ws=ws)
        w_table, w_refs, w_live, moves = kv.compact(table, refs)
        np.testing.assert_array_equal(got.cpu().numpy(), w_table)
        np.testing.assert_array_equal(new.cpu().numpy(), w_refs)
        assert int(live) == w_live
        want = pool.copy()
        for a, b in moves:
            want[:, b] = want[:, a]
        np.testing.assert_array_equal(pages.cpu().numpy(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("hq,hkv,D,P,dtype", [(4, 2, 64, 16, "bf16"), (40, 2, 128, 64, "f16"), (4, 1, 256, 32, "bf16"),
                                             (6, 2, 96, 16, "f16")])
@pytest.mark.parametrize("cols", [[0], [1], [2, 3], [5, 7]])
def test_nan_of_the_first_page_stays_out_of_ids_outside_the_pool(hq, hkv, D, P, dtype, cols):
    """Ids without a page well inside a sequence; the page that is read in their place holds NaN in every value scale.
    Few and many rows, in one piece and split."""
    def edit(pages, table):
        for col, bad in zip(cols, (-7, pages.shape[0])):
            a = int(table[0, col])
            pages[[0, a]] = pages[[a, 0]]                  # nobody else owns the first page
            table[table == 0] = a
            table[0, col] = bad
        kv._sections(pages, P, hkv, D)[3][0] = 0x7F
    for i, (lens, counts) in enumerate([([600], [1]), ([600], [40]), ([5000, 600], [40, 9])]):
        attend(61 + i, lens, counts, hq, hkv, D, P, dtype, edit=edit)
        attend(61 + i, lens, counts, hq, hkv, D, P, dtype, causal=False, edit=edit)


FAKE, ODD = 0x10000, 0x10001            # never dereferenced: every call below is refused before a launch
B = ctypes.byref


def _descriptor(**kw):
    a = dict(pages=FAKE, num_pages=8, page_stride=16 * 2 * 64 * 9 // 8, page_size=16, kv_heads=2, head_dim=64, reserved=0,
             k_g=None, v_g=None)
    a.update(kw)
    return nv._Cache(*a.values())


@pytest.mark.parametrize("total,heads", [(3, 4), (40, 4), (1, 2)])
def test_workspace_query_takes_any_max_q_that_the_call_takes(total, heads):
    """A caller may pass a fixed max_q: past total_q it asks for what the call asks for, and never for less."""
    L, c, mask = nv.lib(), _descriptor(), nv._Mask(0.1, 1, 0, None, 0)
    rows = nv._Rows(FAKE, 128, 64)
    want = L.nvfp4_kv_attention_workspace_bytes(B(c), total, heads, 3, 100, total)
    assert want > 0
    for max_q in (total, total + 1, total + 2, total + 3, 1000, 0x7FFFFFFF):
        need = L.nvfp4_kv_attention_workspace_bytes(B(c), total, heads, 3, 100, max_q)
        assert need == want, max_q

        def call(ws, n):
            return L.nvfp4_kv_attention(B(c), rows, 1, total, heads, FAKE, 100, 100, FAKE, FAKE, 3, max_q, B(mask), rows, None,
                                        ws, n, None)
        assert call(FAKE, need - 1) == nv.ERR_WORKSPACE and call(ODD, need) == nv.ERR_ALIGN      # (enough, but misaligned)
    assert L.nvfp4_kv_attention_workspace_bytes(B(c), total, heads, 3, 100, 0) == 0
    assert L.nvfp4_kv_attention_workspace_bytes(B(c), total, heads, 3, 100, 1 << 31) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("heads", [1, 40])
def test_window_past_2_to_the_30(heads):
    """A billion keys (one page, named over and over) behind a first page whose scores would outweigh them all: windows
    that leave just that page out, and one that takes it in. Sums of equal terms: nothing to round but the output.
    (1 is held as 6 times the E4M3 number next to 1 / 6, 0.171875.)"""
    P, D, n = 256, 16, (1 << 30) + 1024
    pages = torch.zeros((2, nv.nvfp4_kv_page_bytes(P, 1, D)), dtype=torch.uint8, device="cuda")
    cache = nv.KVCache(pages, P, 1, D)
    x = torch.full((P, 1, D), 6.0, dtype=torch.bfloat16, device="cuda")
    at = torch.arange(P, device="cuda")
    nv.nvfp4_kv_append(cache, x, x, at)
    nv.nvfp4_kv_append(cache, x * 0, x / 6, at + P)
    table = torch.ones((1, n // P), dtype=torch.int32, device="cuda")
    table[0, 0] = 0
    q = torch.full((1, heads, D), 4.0, dtype=torch.bfloat16, device="cuda")
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    one = 6.0 * 0.171875
    for window, value, lse in ((n - P, one, math.log(n - P)), (1 << 29, one, math.log(1 << 29)), (n, 6.0, 96 + math.log(P)),
                               (1 << 40, 6.0, 96 + math.log(P))):
        out, got = nv.nvfp4_kv_attention(q, cache, table, lens, window=window, return_lse=True)
        assert bool((out == value).all()), window
        assert bool(((got - lse).abs() <= 2.0 ** -20 * lse).all()), window


@pytest.mark.gpu
def test_window_as_long_as_the_table():
    for window in (1, 95, 96, 97, 1 << 31, 1 << 62):
        attend(71, [96, 50, 1], [1, 1, 1], 4, 2, 64, 16, q_start=False, window=window)
        attend(72, [96, 50, 1], [30, 9, 1], 4, 2, 64, 16, window=window)


def test_resize_refuses_tables_whose_entries_pass_31_bits():
    """The entries that sequences take are added up in 32 bits."""
    def call(batch, width, ws):
        need = nv.lib().nvfp4_kv_pages_workspace_bytes(8, batch)
        return nv.lib().nvfp4_kv_resize(8, 1, FAKE, width, width, batch, FAKE, FAKE, FAKE, FAKE, width, FAKE, FAKE, ws, need,
                                        None)
    for batch, width in ((1 << 24, 128), (2, 1 << 30), (3, 0x7FFFFFFF // 3 + 1)):
        assert call(batch, width, FAKE) == nv.ERR_SHAPE
    for batch, width in ((1 << 24, 127), (1, 0x7FFFFFFF), (3, 0x7FFFFFFF // 3)):
        assert call(batch, width, ODD) == nv.ERR_ALIGN             # taken, up to the misaligned workspace


def test_fork_refuses_children_inside_the_table():
    """Children's rows that share an entry with the table that is read (another child may still read it)."""
    pool = nv._Pool(FAKE, 1, 0, 8, 64, 48)
    need = nv.lib().nvfp4_kv_pages_workspace_bytes(8, 3)

    def call(at, children, ts=10, cs=10, batch=4, width=4):
        """table at FAKE, children `at` entries behind it."""
        return nv.lib().nvfp4_kv_fork(B(pool), 16, FAKE, ts, width, batch, FAKE, FAKE, FAKE, children, FAKE + 4 * at, cs, FAKE, FAKE,
                                      FAKE, need, None)
    for at, children in ((0, 3), (0, 1), (1, 3), (3, 3), (7, 3), (9, 3), (20, 3), (30, 1), (33, 1), (-20, 3), (-23, 3)):
        assert call(at, children) == nv.ERR_VALUE, (at, children)
    assert call(3, 1, batch=1) == nv.ERR_VALUE and call(8, 3, cs=12) == nv.ERR_VALUE


@pytest.mark.gpu
@pytest.mark.parametrize("at,children", [(34, 3), (4, 3), (6, 3), (5, 1), (24, 1), (-24, 3), (-26, 3), (-60, 3)])
def test_fork_takes_children_beside_the_table(at, children):
    """Before it, behind it, and in other columns of the same rows; table rows of 4 in 10."""
    P, width = 16, 4
    whole = torch.full((140,), -9, dtype=torch.int32, device="cuda")
    table, child = whole[70:].as_strided((4, width), (10, 1)), whole[70 + at:].as_strided((children, width), (10, 1))
    table.copy_(dev(np.array([[5, 0, 2, -1], [7, -1, -1, -1], [-1] * 4, [-1] * 4], np.int32)))
    lens, refs = np.array([40, 16, 0, 0], np.int32), np.array([1, 0, 1, 0, 0, 1, 0, 1], np.int32)
    parents = np.array([1, 0, 2], np.int32)[:children]
    before = whole.cpu().numpy()
    w_child, w_refs, w_short, _ = kv.fork(P, table.cpu().numpy(), lens, refs, parents)
    pages = torch.zeros((8, 48), dtype=torch.uint8, device="cuda")
    got, new, short = nv.nvfp4_kv_fork(pages, table, dev(lens), dev(refs), dev(parents), P, out_table=child)
    assert got is child and int(short) == w_short == 0
    np.testing.assert_array_equal(new.cpu().numpy(), w_refs)
    for c in range(children):
        before[70 + at + 10 * c:70 + at + 10 * c + width] = w_child[c]
    np.testing.assert_array_equal(whole.cpu().numpy(), before)


@pytest.mark.gpu
def test_fork_refuses_rows_of_its_table():
    table = torch.zeros((4, 3), dtype=torch.int32, device="cuda")
    lens, refs = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.ones(8, dtype=torch.int32, device="cuda")
    pages = torch.zeros((8, 48), dtype=torch.uint8, device="cuda")
    for out in (table, table[2:], table[:2]):
        parents = torch.zeros(out.shape[0], dtype=torch.int32, device="cuda")
        with pytest.raises(ValueError):
            nv.nvfp4_kv_fork(pages, table, lens, refs, parents, 16, out_table=out)


@pytest.mark.gpu
def test_inputs_the_kernels_cannot_read_are_copied_once():
    """A last dimension that is strided, rows at odd strides, a misaligned base: one new tensor of the same values."""
    cache = nv.KVCache(torch.zeros((1, nv.nvfp4_kv_page_bytes(16, 2, 64)), dtype=torch.uint8, device="cuda"), 16, 2, 64)
    slots, lens = torch.arange(3, device="cuda"), torch.full((3,), 3, dtype=torch.int32, device="cuda")
    table = torch.zeros((3, 1), dtype=torch.int32, device="cuda")
    good = torch.randn((3, 2, 64), device="cuda").to(torch.bfloat16)
    strided, odd, shifted = (torch.empty(n, dtype=torch.bfloat16, device="cuda") for n in (768, 390, 385))
    strided, odd, shifted = strided.view(3, 2, 128)[:, :, ::2], odd.view(3, 2, 65)[:, :, :64], shifted[1:].view(3, 2, 64)
    out = torch.empty_like(good)
    count = lambda: torch.cuda.memory_stats()["allocation.all.allocated"]     # noqa: E731

    def made(x):
        before = count()
        nv.nvfp4_kv_append(cache, x, x, slots)
        between = count()
        nv.nvfp4_kv_attention(x, cache, table, lens, out=out)
        return between - before, count() - between
    assert made(good) == (0, 0)
    want = out.clone()
    for x in (strided, odd, shifted):
        x.copy_(good)
        assert made(x) == (2, 1)                            # k and v; q
        assert torch.equal(out, want)


@pytest.mark.gpu
@pytest.mark.parametrize("batch,T,n", [(6, 40, 600), (1030, 8192, 1 << 20), (1100, 700, 1 << 20)])
@pytest.mark.parametrize("heads", [2, 16])
def test_sequences_that_overlap_in_q_start_stay_in_bounds(batch, T, n, heads):
    """q_start has to ascend. Where it does not, sums over sequences pass 32 bits in the second size; what is written
    is not defined then, but nothing outside the outputs and the workspace is, and the next call is right."""
    P, D = 256, 16
    pages = torch.zeros((2, nv.nvfp4_kv_page_bytes(P, 1, D)), dtype=torch.uint8, device="cuda")
    cache = nv.KVCache(pages, P, 1, D)
    table = torch.ones((batch, -(-n // P)), dtype=torch.int32, device="cuda")
    lens = torch.full((batch,), n, dtype=torch.int32, device="cuda")
    start = torch.zeros(batch + 1, dtype=torch.int32, device="cuda")
    start[1::2] = T
    q = torch.ones((T, heads, D), dtype=torch.bfloat16, device="cuda")
    room = 1 << 16
    out, lse = torch.full((T * heads * D + 2 * room,), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((T * heads + 2 * room,), 7.0, device="cuda")
    size = nv.nvfp4_kv_attention_workspace(T, heads, cache, batch, table.shape[1], T).numel()
    ws = torch.full((size + 2 * room,), 7, dtype=torch.uint8, device="cuda")
    args = dict(out=out[room:-room].view(T, heads, D), lse=lse[room:-room].view(T, heads), ws=ws[room:-room])
    nv.nvfp4_kv_attention(q, cache, table, lens, start, T, **args)
    torch.cuda.synchronize()
    for t in (out, lse, ws):
        assert bool((t[:room] == 7).all()) and bool((t[-room:] == 7).all())
    start = torch.full((batch + 1,), T, dtype=torch.int32, device="cuda")
    start[0] = 0
    nv.nvfp4_kv_attention(q, cache, table, lens, start, T, causal=False, **args)
    assert not args["out"].any() and bool(((args["lse"] - math.log(n)).abs() < 1e-5).all())
