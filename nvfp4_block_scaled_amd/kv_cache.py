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

from . import _Cache, _check, _Mask, _Pool, _Rope, _Rows, lib

_DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_HALF = (torch.bfloat16, torch.float16)


# A decode step calls these entry points once per layer, so what they cost on the host counts: the
# checks below ask each tensor for its device, type, shape and strides once.

def _device():
    """The current device's index (-2, which is no tensor's, without a GPU)."""
    try:
        return torch._C._cuda_getDevice()
    except (AttributeError, RuntimeError):
        return -2


def _stream(dev):
    return torch._C._cuda_getCurrentRawStream(dev)


def _at(t, name, dev):
    """t must be a tensor on the current device (a host pointer handed to a kernel would fault the GPU)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    at = t.get_device()
    if at != dev:
        if at < 0 or not t.is_cuda:
            raise TypeError(f"{name} must be a CUDA (HIP) tensor")
        raise ValueError(f"{name} is on {t.device}, not on the current device cuda:{dev}")


def _flat(t, name, dev, dtype, shape):
    """A contiguous tensor of this type and shape; returns its address."""
    _at(t, name, dev)
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def nvfp4_kv_page_bytes(page_size, kv_heads, head_dim):
    """Bytes of one page of one layer (0: not a geometry that the cache takes)."""
    return int(lib().nvfp4_kv_page_bytes(page_size, kv_heads, head_dim))


class KVCache:
    """One layer's pages and what they are: uint8 device tensor [num_pages][bytes] with contiguous
    rows of at least nvfp4_kv_page_bytes(...) bytes, and the global scales of keys and values
    (contiguous float32 [kv_heads], finite and > 0, or None: 1)."""

    def __init__(self, pages, page_size, kv_heads, head_dim, k_g=None, v_g=None):
        dev = _device()
        need = nvfp4_kv_page_bytes(page_size, kv_heads, head_dim)
        if need == 0:
            raise ValueError("page_size must be 16, 32, 64, 128 or 256, head_dim a multiple of 16 up to 256, "
                             "kv_heads 1 .. 65535")
        _at(pages, "pages", dev)
        if pages.dtype != torch.uint8:
            raise TypeError("pages must be uint8")
        if pages.dim() != 2 or pages.shape[0] < 1 or pages.shape[1] < need or pages.stride(1) != 1:
            raise ValueError(f"pages must be [num_pages][>={need}] with contiguous rows")
        if pages.shape[0] > 1 and pages.stride(0) < need:
            raise ValueError("pages overlap")
        for g, name in ((k_g, "k_g"), (v_g, "v_g")):
            if g is not None:
                _flat(g, name, dev, torch.float32, (kv_heads,))
        self.pages, self.k_g, self.v_g = pages, k_g, v_g
        self.page_size, self.kv_heads, self.head_dim = page_size, kv_heads, head_dim
        self.device = dev
        stride = pages.stride(0) if pages.shape[0] > 1 else (need + 15) // 16 * 16
        self._c = _Cache(pages.data_ptr(), pages.shape[0], stride, page_size, kv_heads, head_dim, 0,
                         None if k_g is None else k_g.data_ptr(), None if v_g is None else v_g.data_ptr())
        self._ref = ctypes.byref(self._c)

    @property
    def num_pages(self):
        return self.pages.shape[0]


def _cache(cache, dev):
    if not isinstance(cache, KVCache):
        raise TypeError("cache must be a KVCache")
    if cache.device != dev:
        raise ValueError(f"cache is on cuda:{cache.device}, not on the current device cuda:{dev}")
    return cache


def _rows(t, name, dev, tokens, heads, dim, dtypes, output=False):
    """(tensor kept alive, nvfp4_rows) of a [tokens][heads][dim] tensor. The kernels read 16 bytes at a
    time: a misaligned or strided input is copied once, an output of that kind refused, and so is an
    output with rows that overlap (a broadcast view would be written by many threads)."""
    _at(t, name, dev)
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be one of {[str(d) for d in dtypes]}, got {t.dtype}")
    if t.shape != (tokens, heads, dim):
        raise ValueError(f"{name} must be [{tokens}][{heads}][{dim}], got {list(t.shape)}")
    ts, hs, ds = t.stride()
    if tokens <= 1:
        ts = heads * dim
    if heads <= 1:
        hs = dim
    at = t.data_ptr()
    if (ds != 1 or at % 16 or ts % 8 or hs % 8) and t.numel():
        if output:
            raise ValueError(f"{name} needs a contiguous last dimension, a 16-byte aligned base and strides of "
                             "tokens and heads that are multiples of 8")
        t = t.clone(memory_format=torch.contiguous_format)
        ts, hs, at = heads * dim, dim, t.data_ptr()
    if output and not ((hs >= dim and ts >= heads * hs) or (ts >= dim and hs >= tokens * ts)
                       or (tokens <= 1 and hs >= dim) or (heads <= 1 and ts >= dim)):
        raise ValueError(f"{name} has rows that overlap")
    return t, _Rows(at, ts, hs)


def _table(t, name, dev, rows=None, width=None):
    """A page table [rows][width], int32, contiguous rows that do not overlap: (address, rows, width, row stride)."""
    _at(t, name, dev)
    if t.dtype != torch.int32:
        raise TypeError(f"{name} must be int32")
    if t.dim() != 2 or (rows is not None and t.shape != (rows, width)):
        raise ValueError(f"{name} must be [{'batch' if rows is None else rows}][{'width' if width is None else width}], "
                         f"got {list(t.shape)}")
    n, w = t.shape
    stride, one = t.stride()
    if (w > 1 and one != 1) or (n > 1 and stride < w):
        raise ValueError(f"{name} needs contiguous rows")
    return t.data_ptr(), n, w, stride if n > 1 else w


def _length(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a CUDA (HIP) tensor")
    if t.dim() != 1:
        raise ValueError(f"{name} must have one dimension")
    return t.shape[0]


def _bytes(ws, need, dev):
    """(address, bytes) of a caller's workspace, or of a new one (kept alive by the caller's reference)."""
    if ws is None:
        if need == 0:
            return None, None, 0
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        return ws, ws.data_ptr(), need
    _at(ws, "ws", dev)
    if not ws.is_contiguous():
        raise ValueError("ws must be contiguous")
    have = ws.numel() * ws.element_size()
    if have < need:
        raise ValueError(f"ws holds {have} bytes, {need} are needed")
    return ws, ws.data_ptr(), have


def nvfp4_kv_append(cache, k, v, slots, q=None, cos=None, sin=None, positions=None, axis_of=None, interleaved=False,
                    q_out=None):
    """Turns q and k to their positions, quantizes k and v [T][kv_heads][head_dim] into their slots
    (int64 [T], page * page_size + place; one outside the pool, like -1, writes nothing), and returns
    the turned queries (q_out, or a new tensor; q itself may be q_out; None without q).

    cos, sin: float32 [max_pos][rot / 2] (None: no rotation); positions: int32 [T] or [axes][T];
    axis_of: uint8 [rot / 2], the axis whose position turns each pair (None: the first); interleaved:
    pairs (2j, 2j + 1) instead of (j, j + rot / 2)."""
    dev = _device()
    c = _cache(cache, dev)
    if not isinstance(k, torch.Tensor) or k.dim() != 3:
        raise TypeError("k must be a [T][kv_heads][head_dim] tensor")
    T, D = k.shape[0], c.head_dim
    k, ks = _rows(k, "k", dev, T, c.kv_heads, D, _HALF)
    kind = (k.dtype,)
    v, vs = _rows(v, "v", dev, T, c.kv_heads, D, kind)
    slots_at = _flat(slots, "slots", dev, torch.int64, (T,))
    qs = os_ = _Rows()
    heads = 0
    if q is not None:
        heads = q.shape[1] if isinstance(q, torch.Tensor) and q.dim() == 3 else 0
        q, qs = _rows(q, "q", dev, T, heads, D, kind)
        if heads < 1:
            raise ValueError("q has no heads")
        if q_out is None:
            q_out = torch.empty((T, heads, D), dtype=k.dtype, device=k.device)
        q_out, os_ = _rows(q_out, "q_out", dev, T, heads, D, kind, output=True)
    elif q_out is not None:
        raise ValueError("q_out without q")
    rope = None
    if cos is not None or sin is not None:
        if cos is None or sin is None or positions is None:
            raise ValueError("cos, sin and positions go together")
        if not isinstance(cos, torch.Tensor) or not isinstance(positions, torch.Tensor):
            raise TypeError("cos and positions must be CUDA (HIP) tensors")
        if cos.dim() != 2:
            raise ValueError("cos and sin must be [max_pos][rot / 2]")
        axes = positions.shape[0] if positions.dim() == 2 else 1
        rope = ctypes.byref(_Rope(
            _flat(cos, "cos", dev, torch.float32, cos.shape), _flat(sin, "sin", dev, torch.float32, cos.shape),
            _flat(positions, "positions", dev, torch.int32, (axes, T) if positions.dim() == 2 else (T,)),
            None if axis_of is None else _flat(axis_of, "axis_of", dev, torch.uint8, (cos.shape[1],)), cos.shape[0], T,
            2 * cos.shape[1], axes, 1 if interleaved else 0, 0))
    elif positions is not None or axis_of is not None:
        raise ValueError("positions without cos and sin")
    _check(lib().nvfp4_kv_append(c._ref, ks, vs, qs, os_, _DTYPES[k.dtype], T, heads, slots_at, rope, _stream(dev)))
    return q_out


def nvfp4_kv_read(cache, slots, dtype=torch.bfloat16, k=None, v=None):
    """What slots (int64 [T]) hold, as (k, v) [T][kv_heads][head_dim] of `dtype` (float32, bfloat16 or
    float16); zeros for a slot outside the pool."""
    dev = _device()
    c = _cache(cache, dev)
    if dtype not in _DTYPES:
        raise TypeError("dtype must be float32, bfloat16 or float16")
    T = _length(slots, "slots")
    slots_at = _flat(slots, "slots", dev, torch.int64, (T,))
    shape = (T, c.kv_heads, c.head_dim)
    if k is None and v is None:
        k, v = torch.empty((2,) + shape, dtype=dtype, device=slots.device).unbind(0)
    else:
        k = torch.empty(shape, dtype=dtype, device=slots.device) if k is None else k
        v = torch.empty(shape, dtype=dtype, device=slots.device) if v is None else v
    k, ks = _rows(k, "k", dev, *shape, (dtype,), output=True)
    v, vs = _rows(v, "v", dev, *shape, (dtype,), output=True)
    _check(lib().nvfp4_kv_read(c._ref, slots_at, T, _DTYPES[dtype], ks, vs, _stream(dev)))
    return k, v


def nvfp4_kv_attention_workspace(total_q, q_heads, cache, batch, max_pages, max_q=1):
    """A workspace for nvfp4_kv_attention calls of these sizes (None when they need none)."""
    c = _cache(cache, _device())
    n = lib().nvfp4_kv_attention_workspace_bytes(c._ref, total_q, q_heads, batch, max_pages, min(max_q, max(1, total_q)))
    return torch.empty(n, dtype=torch.uint8, device=cache.pages.device) if n else None


def nvfp4_kv_attention(q, cache, table, lens, q_start=None, max_q=None, scale=None, causal=True, window=0, mask=None,
                       out=None, lse=None, return_lse=False, ws=None):
    """Attention of queries q [total_q][q_heads][head_dim] over the pages of each sequence.

    table: int32 [batch][max_pages]; lens: int32 [batch], tokens in the cache with the new ones;
    q_start: int32 [batch + 1] row offsets (None: one query per sequence) with max_q at least the
    longest sequence's queries (None: total_q). scale: 1 / sqrt(head_dim) by default. window > 0:
    each query sees the last `window` keys up to its own. mask: bool or uint8 [total_q][>= max_q], which
    of the sequence's new tokens a query sees (drafted trees; replaces causal). Returns out, or (out,
    lse) with lse float32 [total_q][q_heads]. A query that sees no key gets zeros and -inf; a row past the
    last sequence's is left as it was. How far sequences are split follows the table's width, not lens."""
    dev = _device()
    c = _cache(cache, dev)
    if not isinstance(q, torch.Tensor) or q.dim() != 3:
        raise TypeError("q must be a [total_q][q_heads][head_dim] tensor")
    total, heads, D = q.shape[0], q.shape[1], c.head_dim
    q, qs = _rows(q, "q", dev, total, heads, D, _HALF)
    table_at, batch, width, stride = _table(table, "table", dev)
    lens_at = _flat(lens, "lens", dev, torch.int32, (batch,))
    if q_start is None:
        if total != batch:
            raise ValueError("without q_start there is one query per sequence")
        start_at, max_q = None, 1
    else:
        start_at = _flat(q_start, "q_start", dev, torch.int32, (batch + 1,))
        max_q = total if max_q is None else int(max_q)
        if max_q < 1 and total > 0:
            raise ValueError("max_q must be >= 1")
        max_q = max(1, min(max_q, total))
    mask_at, mask_stride = None, 0
    if mask is not None:
        _at(mask, "mask", dev)
        if mask.dtype not in (torch.bool, torch.uint8):
            raise TypeError("mask must be bool or uint8")
        if mask.dim() != 2 or mask.shape[0] != total or mask.shape[1] < max_q:
            raise ValueError(f"mask must be [{total}][>={max_q}]")
        mask_stride, one = mask.stride()
        if (mask.shape[1] > 1 and one != 1) or (total > 1 and mask_stride < max_q):
            raise ValueError("mask needs contiguous rows")
        mask_at, mask_stride = mask.data_ptr(), max(mask_stride, max_q)
    if out is None:
        out = torch.empty((total, heads, D), dtype=q.dtype, device=q.device)
    out, os_ = _rows(out, "out", dev, total, heads, D, (q.dtype,), output=True)
    if lse is None:
        if return_lse:
            lse = torch.empty((total, heads), dtype=torch.float32, device=q.device)
            lse_at = lse.data_ptr()
        else:
            lse_at = None
    else:
        lse_at = _flat(lse, "lse", dev, torch.float32, (total, heads))
    L = lib()
    # (the call itself compares a caller's workspace with what it needs)
    need = 0 if ws is not None else L.nvfp4_kv_attention_workspace_bytes(c._ref, total, heads, batch, width, max_q)
    ws, ws_at, ws_bytes = _bytes(ws, need, dev)
    m = _Mask(1.0 / math.sqrt(D) if scale is None else scale, 1 if causal else 0, window, mask_at, mask_stride)
    _check(L.nvfp4_kv_attention(c._ref, qs, _DTYPES[q.dtype], total, heads, table_at, stride, width, lens_at, start_at,
                                batch, max_q, ctypes.byref(m), os_, lse_at, ws_at, ws_bytes, _stream(dev)))
    return (out, lse) if lse is not None else out


def _pool(pages, dev):
    """(number of pages, nvfp4_kv_pool) of uint8 pages [num_pages][bytes] or [layers][num_pages][bytes]."""
    _at(pages, "pages", dev)
    if pages.dtype != torch.uint8:
        raise TypeError("pages must be uint8")
    if pages.dim() not in (2, 3) or pages.numel() == 0 or pages.stride(-1) != 1:
        raise ValueError("pages must be [num_pages][bytes] or [layers][num_pages][bytes] with contiguous pages")
    n, size = pages.shape[-2:]
    layers = pages.shape[0] if pages.dim() == 3 else 1
    stride = pages.stride(-2) if n > 1 else (size + 15) // 16 * 16
    layer_stride = pages.stride(0) if layers > 1 else 0
    if stride < size or (layers > 1 and layer_stride < (n - 1) * stride + size):
        raise ValueError("pages overlap")
    return n, ctypes.byref(_Pool(pages.data_ptr(), layers, layer_stride, n, stride, size))


def _outputs(out_table, out_refs, one, rows, width, refs, n, dev):
    """Output table, counts and single int32 of a page operation, allocated where not given, and their addresses."""
    if out_table is None:
        out_table = torch.empty((rows, width), dtype=torch.int32, device=refs.device)
    table_at, _, _, stride = _table(out_table, "out_table", dev, rows, width)
    if out_refs is None:
        out_refs = torch.empty_like(refs)
    refs_at = _flat(out_refs, "out_refs", dev, torch.int32, (n,))
    if one is None:
        one = torch.empty(1, dtype=torch.int32, device=refs.device)
    return out_table, table_at, stride, out_refs, refs_at, one, _flat(one, "short or live", dev, torch.int32, (1,))


def _pages_ws(L, ws, n, batch, dev):
    return _bytes(ws, 0 if ws is not None else L.nvfp4_kv_pages_workspace_bytes(n, batch), dev)


def nvfp4_kv_copy_pages(pages, src, dst):
    """Copies page src[i] to page dst[i] (int32 [n]) in every layer of pages ([num_pages][bytes] or
    [layers][num_pages][bytes], uint8). No page is both a source and a destination."""
    dev = _device()
    n, pool = _pool(pages, dev)
    count = _length(src, "src")
    src_at = _flat(src, "src", dev, torch.int32, (count,))
    dst_at = _flat(dst, "dst", dev, torch.int32, (count,))
    _check(lib().nvfp4_kv_copy_pages(pool, src_at, dst_at, count, _stream(dev)))


def nvfp4_kv_fork(pages, table, lens, refs, parents, page_size, out_table=None, out_refs=None, short=None, ws=None):
    """Forks sequences parents (int32 [children]): whole pages are shared, the partly filled one is copied
    to the lowest free page in all layers. Returns (child_table [children][width], refs, short int32 [1]:
    children that could not be served, whose rows are -1). out_refs may be refs; out_table lies apart from
    table (rows of the same table are refused, other columns of a wider one are not)."""
    dev = _device()
    n, pool = _pool(pages, dev)
    table_at, batch, width, stride = _table(table, "table", dev)
    lens_at = _flat(lens, "lens", dev, torch.int32, (batch,))
    refs_at = _flat(refs, "refs", dev, torch.int32, (n,))
    children = _length(parents, "parents")
    parents_at = _flat(parents, "parents", dev, torch.int32, (children,))
    out_table, ot_at, ot_stride, out_refs, or_at, short, short_at = _outputs(out_table, out_refs, short, children, width,
                                                                             refs, n, dev)
    L = lib()
    ws, ws_at, ws_bytes = _pages_ws(L, ws, n, children, dev)
    _check(L.nvfp4_kv_fork(pool, page_size, table_at, stride, width, batch, lens_at, refs_at, parents_at, children, ot_at,
                           ot_stride, or_at, short_at, ws_at, ws_bytes, _stream(dev)))
    return out_table, out_refs, short


def nvfp4_kv_resize(table, lens, new_lens, refs, page_size, out_table=None, out_refs=None, short=None, ws=None):
    """Gives back and takes pages as sequences go from lens to new_lens tokens (0 ends one). Returns
    (table, refs, short int32 [1]: entries that found no page). out_table and out_refs may be the inputs."""
    dev = _device()
    table_at, batch, width, stride = _table(table, "table", dev)
    lens_at = _flat(lens, "lens", dev, torch.int32, (batch,))
    new_at = _flat(new_lens, "new_lens", dev, torch.int32, (batch,))
    n = _length(refs, "refs")
    refs_at = _flat(refs, "refs", dev, torch.int32, (n,))
    out_table, ot_at, ot_stride, out_refs, or_at, short, short_at = _outputs(out_table, out_refs, short, batch, width,
                                                                             refs, n, dev)
    L = lib()
    ws, ws_at, ws_bytes = _pages_ws(L, ws, n, batch, dev)
    _check(L.nvfp4_kv_resize(n, page_size, table_at, stride, width, batch, lens_at, new_at, refs_at, ot_at, ot_stride,
                             or_at, short_at, ws_at, ws_bytes, _stream(dev)))
    return out_table, out_refs, short


def nvfp4_kv_compact(pages, table, refs, out_table=None, out_refs=None, live=None, ws=None):
    """Packs a pool: live pages (refs > 0) past the first n = their number move to the free ids below n, in
    all layers. Returns (table, refs, live int32 [1] = n). out_table and out_refs may be the inputs."""
    dev = _device()
    n, pool = _pool(pages, dev)
    table_at, batch, width, stride = _table(table, "table", dev)
    refs_at = _flat(refs, "refs", dev, torch.int32, (n,))
    out_table, ot_at, ot_stride, out_refs, or_at, live, live_at = _outputs(out_table, out_refs, live, batch, width, refs, n,
                                                                           dev)
    L = lib()
    ws, ws_at, ws_bytes = _pages_ws(L, ws, n, batch, dev)
    _check(L.nvfp4_kv_compact(pool, table_at, stride, width, batch, refs_at, ot_at, ot_stride, or_at, live_at, ws_at,
                              ws_bytes, _stream(dev)))
    return out_table, out_refs, live
