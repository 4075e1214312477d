"""Tokens to experts and back: the Python entry points over the C ABI's nvfp4_moe_* (include/nvfp4.h).

  offsets, tokens, places = nvfp4_moe_sort(ids, experts)          # ids [T][top]
  rows = nvfp4_moe_gather(x, places)                              # [T * top][width], by expert
  out = nvfp4_moe_combine(y, places, weights)                     # [T][width]

and their gradients. Marshalling and checks only; everything is enqueued on the current stream and
nothing synchronises. Ids and places lie in device memory and are checked there: one that is out of
range stands for no row.
"""
import torch

from . import _check, lib
from .fp8 import _apart, _floats, _matrix, _rows_out, _work
from .kv_cache import _at, _device, _flat, _stream

_IDS = {torch.int32: 4, torch.int64: 8}


def nvfp4_moe_sort(ids, experts, ws=None):
    """Sorts (token, choice) pairs by expert: ids [T][top], int32 or int64, in 0 .. experts - 1 (any other,
    like -1, takes no part). Returns (offsets int32 [experts + 1], tokens int32 [T * top], the token of each
    sorted pair and -1 behind the last, places int32 [T][top], each pair's place or -1)."""
    dev = _device()
    _at(ids, "ids", dev)
    if ids.dtype not in _IDS:
        raise TypeError("ids must be int32 or int64")
    if ids.dim() != 2 or ids.shape[1] < 1:
        raise ValueError("ids must be [tokens][top]")
    if not 1 <= experts <= 1024:
        raise ValueError("experts must be 1 .. 1024")
    ids = ids.contiguous()
    T, top = ids.shape
    offsets = ids.new_empty(experts + 1, dtype=torch.int32)
    tokens = ids.new_empty(T * top, dtype=torch.int32)
    places = ids.new_empty((T, top), dtype=torch.int32)
    ws, wsp, nws = _work(ws, lib().nvfp4_moe_sort_workspace_bytes(T, top, experts), dev, ids)
    _check(lib().nvfp4_moe_sort(ids.data_ptr(), _IDS[ids.dtype], T, top, experts, offsets.data_ptr(), tokens.data_ptr(),
                                places.data_ptr(), wsp, nws, _stream(dev)))
    return offsets, tokens, places


def _places(places, dev):
    """(address, tokens, top)"""
    shape = places.shape if isinstance(places, torch.Tensor) else ()
    if len(shape) != 2 or shape[1] < 1:
        raise TypeError("places must be a CUDA (HIP) tensor [tokens][top]")
    return _flat(places, "places", dev, torch.int32, shape), shape[0], shape[1]


def _input(t, name, dev, rows):
    """(tensor kept alive, its dtype's code, row stride, columns)"""
    kind = _floats(t, name, dev)
    shape = t.shape
    if len(shape) != 2 or shape[0] != rows or shape[1] < 1:
        raise ValueError(f"{name} must be [{rows}][>= 1], got {list(shape)}")
    t, ld = _matrix(t, name)
    return t, kind, ld, shape[1]


def _output(out, name, dev, rows, width, like, *inputs):
    if out is None:
        return like.new_empty((rows, width)), width
    ld = _rows_out(out, name, dev, rows, width, like.dtype)
    _apart(out, name, *inputs)
    return out, ld


def nvfp4_moe_gather(x, places, out=None):
    """The tokens' rows x [T][width] (float32, bfloat16 or float16) in the order of their experts: row
    places[t][j] of out [T * top][width] is x[t]. Rows that no place names are left as they were
    (undefined in a new out)."""
    dev = _device()
    at, T, top = _places(places, dev)
    x, kind, ldx, width = _input(x, "x", dev, T)
    out, ldo = _output(out, "out", dev, T * top, width, x, x, places)
    _check(lib().nvfp4_moe_gather(x.data_ptr(), kind, ldx, at, T, top, width, out.data_ptr(), ldo, _stream(dev)))
    return out


def _weights(weights, dev, T, top):
    return _flat(weights, "weights", dev, torch.float32, (T, top))


def nvfp4_moe_combine(y, places, weights=None, out=None):
    """The sorted rows y [T * top][width] back to their tokens: out[t] = sum_j weights[t][j] y[places[t][j]]
    (weights float32 [T][top]; None: ones), summed in FP32 in the order of j and rounded once."""
    dev = _device()
    at, T, top = _places(places, dev)
    y, kind, ldy, width = _input(y, "y", dev, T * top)
    w_at = None if weights is None else _weights(weights, dev, T, top)
    out, ldo = _output(out, "out", dev, T, width, y, y, places, *(() if weights is None else (weights,)))
    _check(lib().nvfp4_moe_combine(y.data_ptr(), kind, ldy, at, w_at, T, top, width, out.data_ptr(), ldo, _stream(dev)))
    return out


def nvfp4_moe_gather_backward(grad, places, out=None):
    """The gradient of nvfp4_moe_gather's x from that of its rows, grad [T * top][width]: each token's rows added."""
    return nvfp4_moe_combine(grad, places, None, out)


def nvfp4_moe_combine_backward(grad, y, places, weights, grad_y=None):
    """The gradients of nvfp4_moe_combine's y and weights from its out's, grad [T][width]: (grad_y
    [T * top][width] with row places[t][j] = weights[t][j] grad[t], grad_weights float32 [T][top]). Rows
    of grad_y that no place names are left as they were (undefined in a new grad_y)."""
    dev = _device()
    at, T, top = _places(places, dev)
    y, kind, ldy, width = _input(y, "y", dev, T * top)
    grad, other, ldg, columns = _input(grad, "grad", dev, T)
    if other != kind:
        raise TypeError("grad and y must have one type")
    if columns != width:
        raise ValueError(f"grad has {columns} columns, y {width}")
    w_at = _weights(weights, dev, T, top)
    grad_y, ldo = _output(grad_y, "grad_y", dev, T * top, width, y, y, grad, places, weights)
    grad_weights = y.new_empty((T, top), dtype=torch.float32)
    _check(lib().nvfp4_moe_combine_backward(grad.data_ptr(), ldg, y.data_ptr(), ldy, kind, at, w_at, T, top, width,
                                            grad_y.data_ptr(), ldo, grad_weights.data_ptr(), _stream(dev)))
    return grad_y, grad_weights
