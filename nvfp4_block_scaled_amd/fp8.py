"""FP8 products with block scales: the Python entry points over the C ABI's nvfp4_fp8_* (include/nvfp4.h).

  a, a_scales = nvfp4_fp8_quantize(x)                       # E4M3 codes, a scale per 128 values of a row
  w, w_scales = nvfp4_fp8_quantize_weight(weight)           # a scale per 128 x 128 values
  y = nvfp4_fp8_gemm(a, a_scales, w, w_scales)
  y = nvfp4_fp8_gemm_grouped(a, a_scales, w, w_scales, offsets, rows=tokens)      # w [experts][N][K]

Marshalling and checks only. Everything is enqueued on the current stream and nothing synchronises.
Codes are float8_e4m3fn (or uint8) tensors. Offsets and row numbers lie in device memory and are
checked there: what the C header says of one that is out of range holds.
"""
import torch

from . import _check, lib
from .kv_cache import _at, _bytes, _device, _DTYPES, _flat, _stream

_CODES = (torch.float8_e4m3fn, torch.uint8)
_OUT = {"bf16": torch.bfloat16, "f16": torch.float16}


def _blocks(n):
    return -(-n // 128)


def _floats(t, name, dev):
    """t must be a float32, bfloat16 or float16 tensor on the current device; returns its dtype's code."""
    _at(t, name, dev)
    if t.dtype not in _DTYPES:
        raise TypeError(f"{name} must be float32, bfloat16 or float16, got {t.dtype}")
    return _DTYPES[t.dtype]


def _matrix(t, name):
    """A [rows][cols] input with contiguous rows that do not overlap (copied once if it has none):
    (tensor kept alive, row stride)."""
    rows, cols = t.shape
    if t.is_contiguous():
        return t, cols
    if (cols > 1 and t.stride(1) != 1) or (rows > 1 and t.stride(0) < cols):
        t = t.clone(memory_format=torch.contiguous_format)
    return t, t.stride(0) if rows > 1 else cols


def _rows_out(out, name, dev, rows, cols, dtype):
    """A caller's [rows][cols] output with contiguous rows that do not overlap: its row stride."""
    _at(out, name, dev)
    if out.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}")
    if out.shape != (rows, cols):
        raise ValueError(f"{name} must be [{rows}][{cols}], got {list(out.shape)}")
    if out.numel() and ((cols > 1 and out.stride(1) != 1) or (rows > 1 and out.stride(0) < cols)):
        raise ValueError(f"{name} needs contiguous rows that do not overlap")
    return out.stride(0) if rows > 1 else cols


def _span(t):
    """Bytes from a tensor's first element to its last."""
    if t.is_contiguous():
        return t.nbytes
    if t.numel() == 0:
        return 0
    return (sum((n - 1) * st for n, st in zip(t.shape, t.stride())) + 1) * t.element_size()


def _meet(lo, hi, t):
    """Whether the bytes lo .. hi - 1 and those from t's first element to its last have some in common."""
    return t.data_ptr() < hi and lo < t.data_ptr() + _span(t)


def _side_by_side(a, b):
    """Whether two matrices of one row stride lie in different columns of it."""
    if a.dim() != 2 or b.dim() != 2 or a.stride(1) != 1 or b.stride(1) != 1:
        return False
    row = a.stride(0) * a.element_size()
    if row < 1 or row != b.stride(0) * b.element_size():
        return False
    first = (b.data_ptr() - a.data_ptr()) % row
    return a.shape[1] * a.element_size() <= first <= row - b.shape[1] * b.element_size()


def _apart(out, name, *others):
    """What is written must not share bytes with what else the call reads or writes (of tensors that are not matrices
    in columns of one buffer: all from the first element to the last)."""
    lo, hi = out.data_ptr(), out.data_ptr() + _span(out)
    for t in others:
        if _meet(lo, hi, t) and not _side_by_side(out, t):
            raise ValueError(f"{name} overlaps another tensor of the call")


def _work(ws, need, dev, *others):
    """kv_cache's _bytes for a workspace, whose first `need` bytes must not share storage with the call's other tensors."""
    given = ws is not None
    ws, at, have = _bytes(ws, need, dev)
    if given and need and any(_meet(at, at + need, t) for t in others):
        raise ValueError("ws overlaps another tensor of the call")
    return ws, at, have


def _code_out(t, name, dev, shape, like):
    if t is None:
        t = like.new_empty(shape, dtype=torch.float8_e4m3fn)
        return t, t.data_ptr()
    as_bytes = isinstance(t, torch.Tensor) and t.dtype == torch.uint8
    at = _flat(t, name, dev, torch.uint8 if as_bytes else torch.float8_e4m3fn, shape)
    _apart(t, name, like)
    return t, at


def _scale_out(t, name, dev, shape, like, codes):
    if t is None:
        t = like.new_empty(shape, dtype=torch.float32)
        return t, t.data_ptr()
    at = _flat(t, name, dev, torch.float32, shape)
    _apart(t, name, like, codes)
    return t, at


def nvfp4_fp8_quantize(x, gated=False, codes=None, scales=None):
    """Rows [M][K] in float32, bfloat16 or float16 -> (codes float8_e4m3fn [M][K], scales float32
    [M][ceil(K/128)]). gated: x is [M][2K], a gate beside a factor, and silu(gate) * factor is
    quantized. K % 16 == 0."""
    dev = _device()
    kind = _floats(x, "x", dev)
    if x.dim() != 2:
        raise ValueError("x must be [rows][columns]")
    M, K = x.shape
    if gated:
        if K % 2:
            raise ValueError("x must hold a gate and a factor of equal width")
        K //= 2
    if K < 1 or K % 16:
        raise ValueError("K % 16 == 0 is required")
    x, ld = _matrix(x, "x")
    codes, codes_at = _code_out(codes, "codes", dev, (M, K), x)
    scales, scales_at = _scale_out(scales, "scales", dev, (M, _blocks(K)), x, codes)
    _check(lib().nvfp4_fp8_quantize(x.data_ptr(), kind, M, K, ld, 1 if gated else 0, codes_at, scales_at, _stream(dev)))
    return codes, scales


def nvfp4_fp8_quantize_weight(w, codes=None, scales=None):
    """A weight [N][K], or a stack [experts][N][K], in float32, bfloat16 or float16 -> (codes of the same
    shape, scales float32 [..][ceil(N/128)][ceil(K/128)]). K % 16 == 0."""
    dev = _device()
    kind = _floats(w, "w", dev)
    if w.dim() not in (2, 3):
        raise ValueError("w must be [N][K] or [experts][N][K]")
    N, K = w.shape[-2:]
    E = w.shape[0] if w.dim() == 3 else 1
    if N < 1 or K < 1 or K % 16:
        raise ValueError("N >= 1 and K % 16 == 0 are required")
    es, ld, one = w.stride() if w.dim() == 3 else (0,) + w.stride()
    if (K > 1 and one != 1) or (N > 1 and ld < K) or (E > 1 and es < 0):
        w = w.clone(memory_format=torch.contiguous_format)
        ld, es = K, N * K
    ld = ld if N > 1 else K
    es = es if E > 1 else 0
    lead = tuple(w.shape[:-2])
    codes, codes_at = _code_out(codes, "codes", dev, lead + (N, K), w)
    scales, scales_at = _scale_out(scales, "scales", dev, lead + (_blocks(N), _blocks(K)), w, codes)
    _check(lib().nvfp4_fp8_quantize_weight(w.data_ptr(), kind, E, N, K, ld, es, codes_at, scales_at, _stream(dev)))
    return codes, scales


def _fp8(codes, scales, name, dev, dims, tall):
    """Checks an FP8 matrix or stack; returns the addresses of its codes and scales."""
    _at(codes, name, dev)
    if codes.dtype not in _CODES:
        raise TypeError(f"{name} must be float8_e4m3fn (or uint8), got {codes.dtype}")
    if codes.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions")
    if not codes.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    N, K = codes.shape[-2:]
    if K < 1 or K % 16:
        raise ValueError(f"{name} needs K % 16 == 0")
    shape = tuple(codes.shape[:-2]) + (_blocks(N) if tall else N, _blocks(K))
    return codes.data_ptr(), _flat(scales, name + "_scales", dev, torch.float32, shape)


def _out(out, out_dtype, dev, M, N, *inputs):
    if out_dtype not in _OUT:
        raise TypeError("out_dtype must be 'bf16' or 'f16'")
    dtype = _OUT[out_dtype]
    if out is None:
        return inputs[0].new_empty((M, N), dtype=dtype), N, _DTYPES[dtype]
    ld = _rows_out(out, "out", dev, M, N, dtype)
    _apart(out, "out", *inputs)
    return out, ld, _DTYPES[dtype]


def nvfp4_fp8_gemm_workspace(M, N, K):
    """A workspace for nvfp4_fp8_gemm calls of these sizes on the current device (None when they need none)."""
    n = lib().nvfp4_fp8_gemm_workspace_bytes(M, N, K)
    return torch.empty(n, dtype=torch.uint8, device="cuda") if n else None


def nvfp4_fp8_gemm(a, a_scales, w, w_scales, out_dtype="bf16", out=None, ws=None):
    """out [M][N] = a w^T of an FP8 activation [M][K] and weight [N][K] (nvfp4_fp8_quantize and
    nvfp4_fp8_quantize_weight give both), as out_dtype 'bf16' or 'f16'. ws: nvfp4_fp8_gemm_workspace's
    (None: allocated when needed)."""
    dev = _device()
    a_at, as_at = _fp8(a, a_scales, "a", dev, 2, False)
    w_at, ws_at = _fp8(w, w_scales, "w", dev, 2, True)
    M, K = a.shape
    N = w.shape[0]
    if w.shape[1] != K:
        raise ValueError(f"a has {K} columns, w {w.shape[1]}")
    if N < 1:
        raise ValueError("w has no rows")
    out, ld, kind = _out(out, out_dtype, dev, M, N, a, a_scales, w, w_scales)
    ws, wsp, nws = _work(ws, lib().nvfp4_fp8_gemm_workspace_bytes(M, N, K), dev, out, a, a_scales, w, w_scales)
    _check(lib().nvfp4_fp8_gemm(a_at, as_at, w_at, ws_at, M, N, K, out.data_ptr(), kind, ld, wsp, nws, _stream(dev)))
    return out


def nvfp4_fp8_gemm_grouped(a, a_scales, w, w_scales, offsets, rows=None, out_dtype="bf16", out=None):
    """Products of rows sorted by expert with each expert's weight, w [experts][N][K]: rows offsets[e] ..
    offsets[e+1] - 1 of out (int32 [experts + 1], nvfp4_moe_sort's) with w[e].

    rows: int32 [M], the row of a that each row of out multiplies (nvfp4_moe_sort's tokens; then a holds
    one row per token); None: a's rows are sorted already. Rows of out that no expert has are left as
    they were (undefined in a new out)."""
    dev = _device()
    a_at, as_at = _fp8(a, a_scales, "a", dev, 2, False)
    w_at, ws_at = _fp8(w, w_scales, "w", dev, 3, True)
    K, (E, N) = a.shape[1], w.shape[:2]
    if w.shape[2] != K:
        raise ValueError(f"a has {K} columns, w {w.shape[2]}")
    if not 1 <= E <= 1024 or N < 1:
        raise ValueError("w must hold 1 .. 1024 experts of at least one row")
    offsets_at = _flat(offsets, "offsets", dev, torch.int32, (E + 1,))
    rows_at, M = None, a.shape[0]
    if rows is not None:
        if not isinstance(rows, torch.Tensor) or rows.dim() != 1:
            raise TypeError("rows must be a CUDA (HIP) tensor of one dimension")
        M = rows.shape[0]
        rows_at = _flat(rows, "rows", dev, torch.int32, (M,))
    out, ld, kind = _out(out, out_dtype, dev, M, N, a, a_scales, w, w_scales, offsets, *(() if rows is None else (rows,)))
    _check(lib().nvfp4_fp8_gemm_grouped(a_at, as_at, a.shape[0], rows_at, w_at, ws_at, E, offsets_at, M, N, K,
                                        out.data_ptr(), kind, ld, _stream(dev)))
    return out
