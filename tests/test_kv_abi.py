"""Host-only checks of the nvfp4_kv_* entry points: sizes, and bad arguments refused before any launch."""
import ctypes
import math

import pytest

import nvfp4_block_scaled_amd as nv

FAKE, ODD = 0x10000, 0x10001            # never dereferenced
B = ctypes.byref


def cache(**kw):
    a = dict(pages=FAKE, num_pages=8, page_stride=16 * 2 * 64 * 9 // 8, page_size=16, kv_heads=2, head_dim=64, reserved=0,
             k_g=None, v_g=None)
    a.update(kw)
    return nv._Cache(*a.values())


def rows(base=FAKE, t=128, h=64):
    return nv._Rows(base, t, h)


def test_page_bytes():
    f = nv.lib().nvfp4_kv_page_bytes
    assert f(64, 4, 128) == 4 * 64 * 128 * 9 // 8
    for bad in ((24, 4, 128), (8, 4, 128), (512, 4, 128), (0, 4, 128), (64, 0, 128), (64, 4, 120), (64, 4, 272), (64, 4, 0)):
        assert f(*bad) == 0


@pytest.mark.parametrize("change,status", [
    (dict(page_size=24), nv.ERR_SHAPE), (dict(kv_heads=0), nv.ERR_SHAPE), (dict(head_dim=40), nv.ERR_SHAPE),
    (dict(num_pages=0), nv.ERR_SHAPE), (dict(num_pages=1 << 31), nv.ERR_SHAPE), (dict(page_stride=16), nv.ERR_SHAPE),
    (dict(pages=None), nv.ERR_NULL), (dict(pages=ODD), nv.ERR_ALIGN), (dict(page_stride=2312), nv.ERR_ALIGN),
    (dict(k_g=ODD), nv.ERR_ALIGN), (dict(page_stride=1 << 62), nv.ERR_SHAPE)])
def test_cache_descriptor(change, status):
    L = nv.lib()
    c = cache(**change)
    assert L.nvfp4_kv_read(B(c), FAKE, 3, 0, rows(), rows(), None) == status
    assert L.nvfp4_kv_append(B(c), rows(), rows(), rows(None), rows(None), 1, 3, 0, FAKE, None, None) == status
    assert L.nvfp4_kv_attention_workspace_bytes(B(c), 3, 4, 3, 100, 1) == 0


def test_append_argument_checks():
    L = nv.lib()

    def call(c=None, k=None, v=None, q=None, qo=None, dtype=1, tokens=3, heads=4, slots=FAKE, **rope):
        r = dict(cos=FAKE, sin=FAKE, positions=FAKE, axis_of=None, max_pos=9, position_stride=3, rot_dim=64, axes=1,
                 interleaved=0, reserved=0)
        r.update(rope)
        return L.nvfp4_kv_append(B(c or cache()), k or rows(), v or rows(), q or rows(), qo or rows(), dtype, tokens, heads,
                                 slots, B(nv._Rope(*r.values())), None)
    assert call(tokens=0) == nv.OK
    assert call(dtype=0) == nv.ERR_DTYPE and call(dtype=3) == nv.ERR_DTYPE
    assert call(tokens=-1) == nv.ERR_SHAPE and call(heads=0) == nv.ERR_SHAPE
    assert call(rot_dim=63) == nv.ERR_SHAPE and call(rot_dim=66) == nv.ERR_SHAPE and call(rot_dim=-2) == nv.ERR_SHAPE
    assert call(max_pos=0) == nv.ERR_SHAPE and call(axes=0) == nv.ERR_SHAPE and call(axes=256) == nv.ERR_SHAPE
    assert call(axes=2, position_stride=2) == nv.ERR_SHAPE
    assert call(interleaved=2) == nv.ERR_VALUE
    assert call(k=rows(None)) == nv.ERR_NULL and call(slots=None) == nv.ERR_NULL and call(qo=rows(None)) == nv.ERR_NULL
    assert call(cos=None) == nv.ERR_NULL and call(positions=None) == nv.ERR_NULL
    for bad in (rows(ODD), rows(FAKE, 129, 64), rows(FAKE, 128, 63)):
        assert call(k=bad) == nv.ERR_ALIGN and call(v=bad) == nv.ERR_ALIGN and call(q=bad) == nv.ERR_ALIGN
        assert call(qo=bad) == nv.ERR_ALIGN
    assert call(slots=0x10004) == nv.ERR_ALIGN and call(sin=ODD) == nv.ERR_ALIGN
    assert L.nvfp4_kv_append(None, rows(), rows(), rows(), rows(), 1, 3, 4, FAKE, None, None) == nv.ERR_NULL


def test_read_argument_checks():
    L = nv.lib()
    f = lambda **k: L.nvfp4_kv_read(B(cache()), *{**dict(s=FAKE, t=3, d=0, k=rows(), v=rows()), **k}.values(), None)  # noqa: E731
    assert f(t=0) == nv.OK and f(t=-1) == nv.ERR_SHAPE and f(d=3) == nv.ERR_DTYPE and f(s=None) == nv.ERR_NULL
    assert f(v=rows(None)) == nv.ERR_NULL and f(k=rows(ODD)) == nv.ERR_ALIGN and f(s=0x10004) == nv.ERR_ALIGN
    assert f(t=1 << 60) == nv.ERR_SHAPE


def test_attention_argument_checks():
    L = nv.lib()
    base = dict(c=None, q=None, dtype=1, total=3, heads=4, table=FAKE, ts=100, mp=100, lens=FAKE, qs=None, batch=3, max_q=1,
                mask=None, out=None, lse=None, ws=None, n=0)
    mk = dict(scale=0.1, causal=1, window=0, mask=None, mask_stride=0)

    def call(m={}, **kw):
        a = {**base, **kw}
        return L.nvfp4_kv_attention(B(a["c"] or cache()), a["q"] or rows(), a["dtype"], a["total"], a["heads"], a["table"],
                                    a["ts"], a["mp"], a["lens"], a["qs"], a["batch"], a["max_q"],
                                    B(nv._Mask(*{**mk, **m}.values())), a["out"] or rows(), a["lse"], a["ws"], a["n"], None)
    need = L.nvfp4_kv_attention_workspace_bytes(B(cache()), 3, 4, 3, 100, 1)
    assert need > 0 and L.nvfp4_kv_attention_workspace_bytes(B(cache()), 3, 4, 3, 4, 1) == 0     # 64 keys: nothing to join
    assert L.nvfp4_kv_attention_workspace_bytes(B(cache()), 3, 3, 3, 100, 1) == 0
    assert call(dtype=0) == nv.ERR_DTYPE
    assert call(heads=3) == nv.ERR_SHAPE and call(total=-1) == nv.ERR_SHAPE and call(batch=-1) == nv.ERR_SHAPE
    assert call(ts=99) == nv.ERR_SHAPE and call(mp=-1) == nv.ERR_SHAPE and call(max_q=0) == nv.ERR_SHAPE
    assert call(total=4) == nv.ERR_SHAPE                                    # one query per sequence
    assert call(total=1 << 40, qs=FAKE) == nv.ERR_SHAPE and call(mp=1 << 30) == nv.ERR_SHAPE
    assert call(mp=(0x7FFFFFFF >> 4) - 63, ts=1 << 40) == nv.ERR_SHAPE
    for s in (0.0, -1.0, math.inf, math.nan):
        assert call(dict(scale=s)) == nv.ERR_VALUE
    assert call(dict(causal=2)) == nv.ERR_VALUE and call(dict(window=-1)) == nv.ERR_VALUE
    assert call(dict(window=4, causal=0)) == nv.ERR_VALUE
    assert call(dict(window=4, mask=FAKE, mask_stride=9)) == nv.ERR_VALUE
    assert call(dict(mask=FAKE, mask_stride=0)) == nv.ERR_SHAPE
    assert call(total=0, batch=0) == nv.OK
    assert call(q=rows(None)) == nv.ERR_NULL and call(out=rows(None)) == nv.ERR_NULL and call(lens=None) == nv.ERR_NULL
    assert call(table=None) == nv.ERR_NULL
    assert call(q=rows(ODD)) == nv.ERR_ALIGN and call(out=rows(FAKE, 100, 64)) == nv.ERR_ALIGN
    assert call(lens=ODD) == nv.ERR_ALIGN and call(lse=ODD) == nv.ERR_ALIGN
    assert call() == nv.ERR_WORKSPACE and call(ws=FAKE, n=need - 1) == nv.ERR_WORKSPACE
    assert call(ws=ODD, n=need) == nv.ERR_ALIGN


def test_page_operation_checks():
    L = nv.lib()
    good = dict(base=FAKE, layers=2, layer_stride=1 << 20, num_pages=8, page_stride=64, page_bytes=48)
    pool = lambda **k: B(nv._Pool(*{**good, **k}.values()))       # noqa: E731
    need = L.nvfp4_kv_pages_workspace_bytes(8, 3)
    assert need > 0 and L.nvfp4_kv_pages_workspace_bytes(0, 3) == 0 and L.nvfp4_kv_pages_workspace_bytes(8, -1) == 0

    def copy(p=None, src=FAKE, dst=FAKE, n=3):
        return L.nvfp4_kv_copy_pages(p or pool(), src, dst, n, None)

    def fork(p=None, ps=16, t=FAKE, ts=4, w=4, b=3, lens=FAKE, refs=FAKE, par=FAKE, n=3, out=FAKE, os=4, ro=FAKE, sh=FAKE,
             ws=FAKE, nws=need):
        return L.nvfp4_kv_fork(p or pool(), ps, t, ts, w, b, lens, refs, par, n, out, os, ro, sh, ws, nws, None)

    def resize(n=8, ps=16, t=FAKE, ts=4, w=4, b=3, lens=FAKE, new=FAKE, refs=FAKE, out=FAKE, os=4, ro=FAKE, sh=FAKE, ws=FAKE,
               nws=need):
        return L.nvfp4_kv_resize(n, ps, t, ts, w, b, lens, new, refs, out, os, ro, sh, ws, nws, None)

    def compact(p=None, t=FAKE, ts=4, w=4, b=3, refs=FAKE, out=FAKE, os=4, ro=FAKE, live=FAKE, ws=FAKE, nws=need):
        return L.nvfp4_kv_compact(p or pool(), t, ts, w, b, refs, out, os, ro, live, ws, nws, None)
    bad = [(dict(layers=0), nv.ERR_SHAPE), (dict(num_pages=0), nv.ERR_SHAPE), (dict(page_stride=32), nv.ERR_SHAPE),
           (dict(page_bytes=8), nv.ERR_SHAPE), (dict(layer_stride=-16), nv.ERR_SHAPE), (dict(base=None), nv.ERR_NULL),
           (dict(base=ODD), nv.ERR_ALIGN), (dict(page_bytes=40), nv.ERR_ALIGN), (dict(layer_stride=8), nv.ERR_ALIGN)]
    for change, status in bad:
        for f in (copy, fork, compact):
            assert f(pool(**change)) == status, (f, change)
    assert copy(n=0) == nv.OK and copy(n=-1) == nv.ERR_SHAPE and copy(src=None) == nv.ERR_NULL and copy(dst=ODD) == nv.ERR_ALIGN
    assert fork(ps=24) == nv.ERR_SHAPE and resize(ps=0) == nv.ERR_SHAPE and resize(n=0) == nv.ERR_SHAPE
    for f in (fork, resize, compact):
        assert f(ts=3) == nv.ERR_SHAPE and f(w=0) == nv.ERR_SHAPE and f(b=0) == nv.ERR_SHAPE and f(os=3) == nv.ERR_SHAPE
        assert f(w=1 << 32, ts=1 << 32, os=1 << 32) == nv.ERR_SHAPE
        assert f(t=None) == nv.ERR_NULL and f(refs=None) == nv.ERR_NULL and f(ro=None) == nv.ERR_NULL
        assert f(t=ODD) == nv.ERR_ALIGN and f(refs=ODD) == nv.ERR_ALIGN and f(out=ODD) == nv.ERR_ALIGN
        assert f(ws=None) == nv.ERR_WORKSPACE and f(nws=need - 1) == nv.ERR_WORKSPACE and f(ws=ODD) == nv.ERR_ALIGN
    assert fork(n=-1) == nv.ERR_SHAPE and fork(par=None) == nv.ERR_NULL and fork(sh=None) == nv.ERR_NULL
    assert resize(new=None) == nv.ERR_NULL and compact(live=None) == nv.ERR_NULL
    assert resize(os=8) == nv.ERR_SHAPE                    # in place, but with other rows


def test_binding_rejects_host_tensors():
    import torch
    with pytest.raises(TypeError):
        nv.KVCache(torch.zeros((1, 16 * 64 * 9 // 8), dtype=torch.uint8), 16, 1, 64)
    with pytest.raises(TypeError):
        nv.nvfp4_kv_copy_pages(torch.zeros((2, 16), dtype=torch.uint8), torch.zeros(1, dtype=torch.int32),
                               torch.zeros(1, dtype=torch.int32))
