"""Tokens to experts and back, pair by pair, in float64."""
import numpy as np


def sort(ids, experts):
    """(offsets, tokens, places) of (token, choice) pairs by expert, then by number."""
    T, top = ids.shape
    lists = [[] for _ in range(experts)]
    for t in range(T):
        for j in range(top):
            if 0 <= ids[t, j] < experts:
                lists[ids[t, j]].append((t, j))
    offsets = np.zeros(experts + 1, np.int32)
    tokens = np.full(T * top, -1, np.int32)
    places = np.full((T, top), -1, np.int32)
    at = 0
    for e, pairs in enumerate(lists):
        for t, j in pairs:
            tokens[at], places[t, j] = t, at
            at += 1
        offsets[e + 1] = at
    return offsets, tokens, places


def _pairs(places):
    rows = places.size
    for t in range(places.shape[0]):
        for j in range(places.shape[1]):
            if 0 <= places[t, j] < rows:
                yield t, j, places[t, j]


def gather(x, places, out):
    out = np.array(out)
    for t, _, p in _pairs(places):
        out[p] = x[t]
    return out


def combine(y, places, weights=None):
    """(out, the same of absolute values) in float64."""
    out = np.zeros((places.shape[0], y.shape[1]))
    size = np.zeros_like(out)
    for t, j, p in _pairs(places):
        v = y[p].astype(np.float64) * (1.0 if weights is None else float(weights[t, j]))
        out[t] += v
        size[t] += np.abs(v)
    return out, size


def combine_backward(grad, y, places, weights, grad_y):
    """(grad_y, grad_weights, the latter of absolute values) in float64."""
    grad_y = np.array(grad_y, np.float64)
    grad_w = np.zeros(places.shape)
    size = np.zeros(places.shape)
    for t, j, p in _pairs(places):
        g, v = grad[t].astype(np.float64), y[p].astype(np.float64)
        grad_y[p] = float(weights[t, j]) * g
        grad_w[t, j] = g @ v
        size[t, j] = np.abs(g) @ np.abs(v)
    return grad_y, grad_w, size
