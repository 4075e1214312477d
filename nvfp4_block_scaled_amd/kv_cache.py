"""Key/value cache in NVFP4: the Python entry points over the C ABI's nvfp4_kv_* (include/nvfp4.h).

  cache = KVCache(pages, page_size, kv_heads, head_dim, k_g, v_g)       # uint8 pages [num_pages][>= page bytes]
  q = nvfp4_kv_append(cache, k, v, slots, q=q, cos=cos, sin=sin, positions=positions)
  out = nvfp4_kv_attention(q, cache, table, lens)                       # one query per sequence
  table, refs, short = nvfp4_kv_resize(table, lens, new_lens, refs, page_size)

Marshalling and checks only, like the rest of the package. Everything is enqueued on the current
stream and nothing synchronises. A length, a slot, a position or a page id lies in device memory
and is checked there: what the C header says of one that is out of range holds.
"""
import ctypes
import math

import torch

from . import (_Cache, _check, _dev, _f32_dev, _Mask, _on_device, _Pool, _ptr, _Rope, _Rows, _stream, _workspace_arg,
               lib)

_DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_HALF = (torch.bfloat16, torch.float16)


def nvfp4_kv_page_bytes(page_size, kv_heads, head_dim):
    """Bytes of one page of one layer (0: not a geometry that the cache takes)."""
    return int(lib().nvfp4_kv_page_bytes(page_size, kv_heads, head_dim))


class KVCache:
    """One layer's pages and what they are: uint8 device tensor [num_pages][bytes] with contiguous
    rows of at least nvfp4_kv_page_bytes(...) bytes, and the global scales of keys and values
    (contiguous float32 [kv_heads], finite and > 0, or None: 1)."""

    def __init__(self, pages, page_size, kv_heads, head_dim, k_g=None, v_g=None):
        need = nvfp4_kv_page_bytes(page_size, kv_heads, head_dim)
        if need == 0:
            raise ValueError("page_size must be 16, 32, 64, 128 or 256, head_dim a multiple of 16 up to 256, "
                             "kv_heads 1 .. 65535")
        _on_device(pages, "pages")
        if pages.dtype != torch.uint8:
            raise TypeError("pages must be uint8")
        if pages.dim() != 2 or pages.shape[0] < 1 or pages.shape[1] < need or pages.stride(1) != 1:
            raise ValueError(f"pages must be [num_pages][>={need}] with contiguous rows")
        if pages.shape[0] > 1 and pages.stride(0) < need:
            raise ValueError("pages overlap")
        if (k_g is not None and k_g.dim() != 1) or (v_g is not None and v_g.dim() != 1):
            raise ValueError("k_g and v_g must be [kv_heads]")
        self.pages = pages
        self.page_size, self.kv_heads, self.head_dim = page_size, kv_heads, head_dim
        self.k_g = _f32_dev(k_g, "k_g", kv_heads)
        self.v_g = _f32_dev(v_g, "v_g", kv_heads)
        stride = pages.stride(0) if pages.shape[0] > 1 else (need + 15) // 16 * 16
        self._c = _Cache(pages.data_ptr(), pages.shape[0], stride, page_size, kv_heads, head_dim, 0,
                         None if k_g is None else k_g.data_ptr(), None if v_g is None else v_g.data_ptr())

    @property
    def num_pages(self):
        return self.pages.shape[0]

    def _arg(self):
        _on_device(self.pages, "cache")
        return ctypes.byref(self._c)


def _cache(cache):
    if not isinstance(cache, KVCache):
        raise TypeError("cache must be a KVCache")
    return cache


def _rows(t, name, tokens, heads, dim, dtypes, copy=False):
    """(tensor kept alive, nvfp4_rows) of a [tokens][heads][dim] tensor. The kernels read 16 bytes at
    a time: a misaligned or strided input is copied once (copy), an output refused."""
    _on_device(t, name)
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be one of {[str(d) for d in dtypes]}, got {t.dtype}")
    if t.dim() != 3 or tuple(t.shape) != (tokens, heads, dim):
        raise ValueError(f"{name} must be [{tokens}][{heads}][{dim}], got {tuple(t.shape)}")
    ts = t.stride(0) if tokens > 1 else heads * dim
    hs = t.stride(1) if heads > 1 else dim
    if t.numel() and (t.stride(2) != 1 or t.data_ptr() % 16 or ts % 8 or hs % 8):
        if not copy:
            raise ValueError(f"{name} needs a contiguous last dimension, a 16-byte aligned base and strides of "
                             "tokens and heads that are multiples of 8")
        t = t.contiguous().clone()
        ts, hs = heads * dim, dim
    return t, _Rows(t.data_ptr(), ts, hs)


def _disjoint_rows(t, name):
    """An output's rows must not overlap (a broadcast view would be written by many threads)."""
    tokens, heads, dim = t.shape
    ts, hs = (abs(s) if n > 1 else None for s, n in ((t.stride(0), tokens), (t.stride(1), heads)))
    small, n_small, large = (hs, heads, ts) if ts is None or (hs is not None and hs <= ts) else (ts, tokens, hs)
    if (small is not None and small < dim) or (large is not None and large < (dim if small is None else small * n_small)):
        raise ValueError(f"{name} has rows that overlap")


def _ints(t, name, dtype, shape):
    _dev(t, name)
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    return t


def _table(t, name, rows=None, width=None):
    """A page table [rows][width], int32, contiguous rows that do not overlap: (rows, width, row stride)."""
    _on_device(t, name)
    if t.dtype != torch.int32:
        raise TypeError(f"{name} must be int32")
    if t.dim() != 2 or (rows is not None and t.shape[0] != rows) or (width is not None and t.shape[1] != width):
        raise ValueError(f"{name} must be [{'batch' if rows is None else rows}][{'width' if width is None else width}], "
                         f"got {tuple(t.shape)}")
    if (t.shape[1] > 1 and t.stride(1) != 1) or (t.shape[0] > 1 and t.stride(0) < t.shape[1]):
        raise ValueError(f"{name} needs contiguous rows")
    return t.shape[0], t.shape[1], t.stride(0) if t.shape[0] > 1 else t.shape[1]


def nvfp4_kv_append(cache, k, v, slots, q=None, cos=None, sin=None, positions=None, axis_of=None, interleaved=False,
                    q_out=None):
    """Turns q and k to their positions, quantizes k and v [T][kv_heads][head_dim] into their slots
    (int64 [T], page * page_size + place; one outside the pool, like -1, writes nothing), and returns
    the turned queries (q_out, or a new tensor; q itself may be q_out; None without q).

    cos, sin: float32 [max_pos][rot / 2] (None: no rotation); positions: int32 [T] or [axes][T];
    axis_of: uint8 [rot / 2], the axis whose position turns each pair (None: the first); interleaved:
    pairs (2j, 2j + 1) instead of (j, j + rot / 2)."""
    c = _cache(cache)
    if not isinstance(k, torch.Tensor) or k.dim() != 3:
        raise TypeError("k must be a [T][kv_heads][head_dim] tensor")
    T = k.shape[0]
    k, ks = _rows(k, "k", T, c.kv_heads, c.head_dim, _HALF, copy=True)
    v, vs = _rows(v, "v", T, c.kv_heads, c.head_dim, (k.dtype,), copy=True)
    slots = _ints(slots, "slots", torch.int64, (T,))
    qs, os_, heads = _Rows(), _Rows(), 0
    if q is not None:
        heads = q.shape[1] if isinstance(q, torch.Tensor) and q.dim() == 3 else 0
        src, qs = _rows(q, "q", T, heads, c.head_dim, (k.dtype,), copy=True)
        if heads < 1:
            raise ValueError("q has no heads")
        q_out = torch.empty((T, heads, c.head_dim), dtype=k.dtype, device=k.device) if q_out is None else q_out
        q_out, os_ = _rows(q_out, "q_out", T, heads, c.head_dim, (k.dtype,))
        _disjoint_rows(q_out, "q_out")
    elif q_out is not None:
        raise ValueError("q_out without q")
    rope = None
    if cos is not None or sin is not None:
        if cos is None or sin is None or positions is None:
            raise ValueError("cos, sin and positions go together")
        cos, sin = _f32_dev(cos, "cos"), _f32_dev(sin, "sin")
        if cos.dim() != 2 or cos.shape != sin.shape:
            raise ValueError("cos and sin must be [max_pos][rot / 2]")
        _dev(positions, "positions")
        if positions.dtype != torch.int32:
            raise TypeError("positions must be int32")
        if positions.dim() not in (1, 2) or positions.shape[-1] != T:
            raise ValueError("positions must be [T] or [axes][T]")
        axes = positions.shape[0] if positions.dim() == 2 else 1
        if axis_of is not None:
            _ints(axis_of, "axis_of", torch.uint8, (cos.shape[1],))
        rope = _Rope(cos.data_ptr(), sin.data_ptr(), positions.data_ptr(),
                     None if axis_of is None else axis_of.data_ptr(), cos.shape[0], T, 2 * cos.shape[1], axes,
                     int(bool(interleaved)), 0)
    elif positions is not None or axis_of is not None:
        raise ValueError("positions without cos and sin")
    _check(lib().nvfp4_kv_append(c._arg(), ks, vs, qs, os_, _DTYPES[k.dtype], T, heads, _ptr(slots),
                                 None if rope is None else ctypes.byref(rope), _stream()))
    return q_out


def nvfp4_kv_read(cache, slots, dtype=torch.bfloat16, k=None, v=None):
    """What slots (int64 [T]) hold, as (k, v) [T][kv_heads][head_dim] of `dtype` (float32, bfloat16 or
    float16); zeros for a slot outside the pool."""
    c = _cache(cache)
    if dtype not in _DTYPES:
        raise TypeError("dtype must be float32, bfloat16 or float16")
    T = slots.shape[0] if isinstance(slots, torch.Tensor) and slots.dim() == 1 else -1
    slots = _ints(slots, "slots", torch.int64, (T,))
    shape = (T, c.kv_heads, c.head_dim)
    k = torch.empty(shape, dtype=dtype, device=slots.device) if k is None else k
    v = torch.empty(shape, dtype=dtype, device=slots.device) if v is None else v
    k, ks = _rows(k, "k", *shape, (dtype,))
    v, vs = _rows(v, "v", *shape, (dtype,))
    _disjoint_rows(k, "k")
    _disjoint_rows(v, "v")
    _check(lib().nvfp4_kv_read(c._arg(), _ptr(slots), T, _DTYPES[dtype], ks, vs, _stream()))
    return k, v


def _attention_need(c, total_q, q_heads, batch, max_pages, max_q):
    return int(lib().nvfp4_kv_attention_workspace_bytes(c._arg(), total_q, q_heads, batch, max_pages, max_q))


def nvfp4_kv_attention_workspace(total_q, q_heads, cache, batch, max_pages, max_q=1):
    """A workspace for nvfp4_kv_attention calls of these sizes (None when they need none)."""
    n = _attention_need(_cache(cache), total_q, q_heads, batch, max_pages, min(max_q, max(1, total_q)))
    return torch.empty(n, dtype=torch.uint8, device=cache.pages.device) if n else None


def nvfp4_kv_attention(q, cache, table, lens, q_start=None, max_q=None, scale=None, causal=True, window=0, mask=None,
                       out=None, lse=None, return_lse=False, ws=None):
    """Attention of queries q [total_q][q_heads][head_dim] over the pages of each sequence.

    table: int32 [batch][max_pages]; lens: int32 [batch], tokens in the cache with the new ones;
    q_start: int32 [batch + 1] row offsets (None: one query per sequence) with max_q at least the
    longest sequence's queries (None: total_q). scale: 1 / sqrt(head_dim) by default. window > 0:
    each query sees the last `window` keys up to its own. mask: bool or uint8 [total_q][>= max_q], which
    of the sequence's new tokens a query sees (drafted trees; replaces causal). Returns out, or (out,
    lse) with lse float32 [total_q][q_heads]. A query that sees no key gets zeros and -inf."""
    c = _cache(cache)
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise TypeError("q must be a [total_q][q_heads][head_dim] tensor")
    total, heads = q.shape[0], q.shape[1]
    q, qs = _rows(q, "q", total, heads, c.head_dim, _HALF, copy=True)
    batch, width, stride = _table(table, "table")
    lens = _ints(lens, "lens", torch.int32, (batch,))
    if q_start is None:
        if total != batch:
            raise ValueError("without q_start there is one query per sequence")
        max_q = 1
    else:
        q_start = _ints(q_start, "q_start", torch.int32, (batch + 1,))
        max_q = max(1, total) if max_q is None else int(max_q)
        if max_q < 1:
            raise ValueError("max_q must be >= 1")
    max_q = min(max_q, max(1, total))
    mask_stride = 0
    if mask is not None:
        _on_device(mask, "mask")
        if mask.dtype not in (torch.bool, torch.uint8):
            raise TypeError("mask must be bool or uint8")
        if mask.dim() != 2 or mask.shape[0] != total or mask.shape[1] < max_q:
            raise ValueError(f"mask must be [{total}][>={max_q}]")
        if mask.shape[1] > 1 and mask.stride(1) != 1:
            raise ValueError("mask needs contiguous rows")
        mask_stride = max(mask.stride(0), max_q) if total > 1 else max_q
        if total > 1 and mask.stride(0) < max_q:
            raise ValueError("mask rows overlap")
    if out is None:
        out = torch.empty((total, heads, c.head_dim), dtype=q.dtype, device=q.device)
    out, os_ = _rows(out, "out", total, heads, c.head_dim, (q.dtype,))
    _disjoint_rows(out, "out")
    if lse is not None:
        _f32_dev(lse, "lse")
        if tuple(lse.shape) != (total, heads):
            raise ValueError(f"lse must be [{total}][{heads}]")
    elif return_lse:
        lse = torch.empty((total, heads), dtype=torch.float32, device=q.device)
    need = _attention_need(c, total, heads, batch, width, max_q)
    if ws is None and need > 0:
        ws = torch.empty(need, dtype=torch.uint8, device=q.device)
    wsp, nws = _workspace_arg(ws, need)
    m = _Mask(1.0 / math.sqrt(c.head_dim) if scale is None else scale, int(bool(causal)), int(window),
              None if mask is None else mask.data_ptr(), mask_stride)
    _check(lib().nvfp4_kv_attention(c._arg(), qs, _DTYPES[q.dtype], total, heads, _ptr(table), stride, width, _ptr(lens),
                                    _ptr(q_start), batch, max_q, ctypes.byref(m), os_, _ptr(lse), wsp, nws, _stream()))
    return (out, lse) if return_lse or lse is not None else out


def _pool(pages, page_bytes=None):
    """nvfp4_kv_pool of uint8 pages [num_pages][bytes] or [layers][num_pages][bytes]."""
    _on_device(pages, "pages")
    if pages.dtype != torch.uint8:
        raise TypeError("pages must be uint8")
    if pages.dim() not in (2, 3) or pages.stride(-1) != 1 or pages.numel() == 0:
        raise ValueError("pages must be [num_pages][bytes] or [layers][num_pages][bytes] with contiguous pages")
    n, size = pages.shape[-2], pages.shape[-1]
    layers = pages.shape[0] if pages.dim() == 3 else 1
    stride = pages.stride(-2) if n > 1 else (size + 15) // 16 * 16
    layer_stride = pages.stride(0) if layers > 1 else 0
    page_bytes = size if page_bytes is None else page_bytes
    if page_bytes < 1 or page_bytes > size:
        raise ValueError(f"page_bytes must be 1 .. {size}")
    if stride < size or (layers > 1 and layer_stride < (n - 1) * stride + size):
        raise ValueError("pages overlap")
    return n, ctypes.byref(_Pool(pages.data_ptr(), layers, layer_stride, n, stride, page_bytes))


def _pages_ws(ws, num_pages, batch, device):
    need = int(lib().nvfp4_kv_pages_workspace_bytes(num_pages, batch))
    if ws is None:
        ws = torch.empty(max(need, 16), dtype=torch.uint8, device=device)
    return _workspace_arg(ws, need)


def _one_int(t, name, device):
    return torch.empty(1, dtype=torch.int32, device=device) if t is None else _ints(t, name, torch.int32, (1,))


def nvfp4_kv_copy_pages(pages, src, dst):
    """Copies page src[i] to page dst[i] (int32 [n]) in every layer of pages ([num_pages][bytes] or
    [layers][num_pages][bytes], uint8). No page is both a source and a destination."""
    n, pool = _pool(pages)
    count = src.shape[0] if isinstance(src, torch.Tensor) and src.dim() == 1 else -1
    src = _ints(src, "src", torch.int32, (count,))
    dst = _ints(dst, "dst", torch.int32, (count,))
    _check(lib().nvfp4_kv_copy_pages(pool, _ptr(src), _ptr(dst), count, _stream()))


def nvfp4_kv_fork(pages, table, lens, refs, parents, page_size, out_table=None, out_refs=None, short=None, ws=None):
    """Forks sequences parents (int32 [children]): whole pages are shared, the partly filled one is copied
    to the lowest free page in all layers. Returns (child_table [children][width], refs, short int32 [1]:
    children that could not be served, whose rows are -1). out_refs may be refs."""
    n, pool = _pool(pages)
    batch, width, stride = _table(table, "table")
    lens = _ints(lens, "lens", torch.int32, (batch,))
    refs = _ints(refs, "refs", torch.int32, (n,))
    children = parents.shape[0] if isinstance(parents, torch.Tensor) and parents.dim() == 1 else -1
    parents = _ints(parents, "parents", torch.int32, (children,))
    out_table = torch.empty((children, width), dtype=torch.int32, device=refs.device) if out_table is None else out_table
    _, _, out_stride = _table(out_table, "out_table", children, width)
    out_refs = torch.empty_like(refs) if out_refs is None else _ints(out_refs, "out_refs", torch.int32, (n,))
    short = _one_int(short, "short", refs.device)
    wsp, nws = _pages_ws(ws, n, children, refs.device)
    _check(lib().nvfp4_kv_fork(pool, page_size, _ptr(table), stride, width, batch, _ptr(lens), _ptr(refs), _ptr(parents),
                               children, _ptr(out_table), out_stride, _ptr(out_refs), _ptr(short), wsp, nws, _stream()))
    return out_table, out_refs, short


def nvfp4_kv_resize(table, lens, new_lens, refs, page_size, out_table=None, out_refs=None, short=None, ws=None):
    """Gives back and takes pages as sequences go from lens to new_lens tokens (0 ends one). Returns
    (table, refs, short int32 [1]: entries that found no page). out_table and out_refs may be the inputs."""
    batch, width, stride = _table(table, "table")
    lens = _ints(lens, "lens", torch.int32, (batch,))
    new_lens = _ints(new_lens, "new_lens", torch.int32, (batch,))
    n = refs.shape[0] if isinstance(refs, torch.Tensor) and refs.dim() == 1 else -1
    refs = _ints(refs, "refs", torch.int32, (n,))
    out_table = torch.empty((batch, width), dtype=torch.int32, device=refs.device) if out_table is None else out_table
    _, _, out_stride = _table(out_table, "out_table", batch, width)
    out_refs = torch.empty_like(refs) if out_refs is None else _ints(out_refs, "out_refs", torch.int32, (n,))
    short = _one_int(short, "short", refs.device)
    wsp, nws = _pages_ws(ws, n, batch, refs.device)
    _check(lib().nvfp4_kv_resize(n, page_size, _ptr(table), stride, width, batch, _ptr(lens), _ptr(new_lens), _ptr(refs),
                                 _ptr(out_table), out_stride, _ptr(out_refs), _ptr(short), wsp, nws, _stream()))
    return out_table, out_refs, short


def nvfp4_kv_compact(pages, table, refs, out_table=None, out_refs=None, live=None, ws=None):
    """Packs a pool: live pages (refs > 0) past the first n = their number move to the free ids below n, in
    all layers. Returns (table, refs, live int32 [1] = n). out_table and out_refs may be the inputs."""
    n, pool = _pool(pages)
    batch, width, stride = _table(table, "table")
    refs = _ints(refs, "refs", torch.int32, (n,))
    out_table = torch.empty((batch, width), dtype=torch.int32, device=refs.device) if out_table is None else out_table
    _, _, out_stride = _table(out_table, "out_table", batch, width)
    out_refs = torch.empty_like(refs) if out_refs is None else _ints(out_refs, "out_refs", torch.int32, (n,))
    live = _one_int(live, "live", refs.device)
    wsp, nws = _pages_ws(ws, n, batch, refs.device)
    _check(lib().nvfp4_kv_compact(pool, _ptr(table), stride, width, batch, _ptr(refs), _ptr(out_table), out_stride,
                                  _ptr(out_refs), _ptr(live), wsp, nws, _stream()))
    return out_table, out_refs, live
