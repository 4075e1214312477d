"""Edges of the key/value cache's operators: full pools, page ids without a page, very long windows, and arguments
that only just do or do not fit."""
import ctypes

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
