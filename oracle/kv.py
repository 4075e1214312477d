"""Key/value cache in NVFP4: page layout, append with rotary positions, attention, page management.

Test infrastructure (see the package docstring). Plain numpy and loops, written from the definitions:

* a page holds for each head: key codes [P][D/2], key scales [P][D/16], value codes [P/4][D/8][4][4]
  (token group, octet, token, byte), value scales [D/16][P];
* rotary: a' = a cos - b sin, b' = b cos + a sin, each operation rounded to FP32;
* a block of 16 is quantized by the steps of quantize.py under its head's global scale, with NaN blocks
  marked by scale byte 0x7F;
* attention in float64;
* pages: reference counts, lowest free id first.
"""
import numpy as np

from . import formats, quantize


def page_bytes(P, heads, D):
    return heads * P * D * 9 // 8


def rotate(x, cos, sin, positions, axis_of, interleaved):
    """x [T][H][D] float32; cos, sin [max_pos][half]; positions [axes][T]; axis_of [half] or None."""
    T, H, D = x.shape
    half = cos.shape[1]
    out = x.astype(np.float32).copy()
    for j in range(half):
        pos = positions[0 if axis_of is None else axis_of[j]]
        inside = (pos >= 0) & (pos < cos.shape[0])
        at = np.where(inside, pos, 0)
        c = np.where(inside, cos[at, j], np.float32(np.nan)).astype(np.float32)[:, None]
        s = np.where(inside, sin[at, j], np.float32(np.nan)).astype(np.float32)[:, None]
        ia, ib = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
        a, b = x[:, :, ia].astype(np.float32), x[:, :, ib].astype(np.float32)
        with np.errstate(invalid="ignore", over="ignore"):
            out[:, :, ia] = a * c - b * s
            out[:, :, ib] = b * c + a * s
    return out


def quantize_row(x, g):
    """[D] float32 under g -> (codes [D/2], scales [D/16])."""
    bad = np.isnan(x).reshape(-1, 16).any(1)
    clean = np.where(np.repeat(bad, 16), np.float32(0), x)
    codes, scales = quantize.quantize_f32_rows_with_g(clean[None], g)
    codes, scales = codes[0].copy(), scales[0].copy()
    scales[bad] = 0x7F
    return codes, scales


def _sections(pages, P, heads, D):
    """Views [pages][heads] of the four parts."""
    x = pages[:, :page_bytes(P, heads, D)].reshape(pages.shape[0], heads, P * D * 9 // 8)
    n = pages.shape[0]
    a, b, c = P * D // 2, P * D * 9 // 16, P * D * 17 // 16
    return (x[:, :, :a].reshape(n, heads, P, D // 2), x[:, :, a:b].reshape(n, heads, P, D // 16),
            x[:, :, b:c].reshape(n, heads, P // 4, D // 8, 4, 4), x[:, :, c:].reshape(n, heads, D // 16, P))


def append(pages, P, k, v, slots, k_g, v_g):
    """Writes FP32 (already turned) k and v [T][heads][D] into a copy of pages [n][page bytes]."""
    pages = np.ascontiguousarray(pages).copy()
    T, heads, D = k.shape
    kc, ks, vc, vs = _sections(pages, P, heads, D)
    for t in range(T):
        page, at = int(slots[t]) // P, int(slots[t]) % P
        if slots[t] < 0 or page >= pages.shape[0]:
            continue
        for h in range(heads):
            kc[page, h, at], ks[page, h, at] = quantize_row(k[t, h], k_g[h])
            codes, scales = quantize_row(v[t, h], v_g[h])
            vc[page, h, at // 4, :, at % 4, :] = codes.reshape(D // 8, 4)
            vs[page, h, :, at] = scales
    return pages


def held(pages, P, heads, D, k_g, v_g):
    """The FP32 values fl32(code * scale / g) of every slot: k, v [pages * P][heads][D]."""
    kc, ks, vc, vs = _sections(pages, P, heads, D)
    n = pages.shape[0]
    vcodes = vc.transpose(0, 1, 2, 4, 3, 5).reshape(n, heads, P, D // 2)
    vscales = vs.transpose(0, 1, 3, 2)
    out = []
    for codes, scales, g in ((kc, ks, k_g), (vcodes, vscales, v_g)):
        x = formats.decode_e2m1(formats.unpack_nibbles(codes)).reshape(n, heads, P, D // 16, 16)
        x = x * formats.decode_e4m3(scales)[..., None]
        x = x.astype(np.float32) / np.asarray(g, np.float32).reshape(1, heads, 1, 1, 1)
        out.append(x.reshape(n, heads, P, D).transpose(0, 2, 1, 3).reshape(n * P, heads, D))
    return out


def exact_values(pages, P, heads, D, k_g, v_g):
    """The same in float64, code * scale / g without rounding."""
    ones = np.ones(heads, np.float32)
    k, v = held(pages, P, heads, D, ones, ones)
    return (k.astype(np.float64) / np.asarray(k_g, np.float64).reshape(1, heads, 1),
            v.astype(np.float64) / np.asarray(v_g, np.float64).reshape(1, heads, 1))


def attention(q, k, v, P, table, lens, q_start, scale, causal=True, window=0, mask=None, num_pages=None):
    """float64 attention of q [T][Hq][D] over k, v [slots][heads][D]. Returns (out, lse, weight sums
    sum_j p_j |v_j|, largest scale * sum |q k|, largest |v| seen) per row, for error bounds."""
    T, hq, D = q.shape
    heads = k.shape[1]
    G = hq // heads
    num_pages = k.shape[0] // P if num_pages is None else num_pages
    out, lse = np.zeros((T, hq, D)), np.full((T, hq), -np.inf)
    mass, big, vmax = np.zeros((T, hq, D)), np.zeros((T, hq)), np.zeros((T, hq))
    for b in range(len(lens)):
        n = int(np.clip(lens[b], 0, table.shape[1] * P))
        q0, q1 = (b, b + 1) if q_start is None else (int(q_start[b]), int(q_start[b + 1]))
        ids = table[b, :-(-n // P)].astype(np.int64)
        inside = np.repeat((ids >= 0) & (ids < num_pages), P)[:n]
        slots = (np.where((ids >= 0) & (ids < num_pages), ids, 0)[:, None] * P + np.arange(P)).reshape(-1)[:n]
        for i in range(q1 - q0):
            pos = n - (q1 - q0) + i
            j = np.arange(n)
            see = inside.copy()
            if mask is not None:
                new = j - (n - (q1 - q0))
                see &= (new < 0) | (mask[q0 + i][np.clip(new, 0, mask.shape[1] - 1)] != 0)
            elif causal:
                see &= j <= pos
                if window:
                    see &= j > pos - window
            at = slots[see]
            if at.size == 0:
                continue
            for h in range(hq):
                kk, vv = k[at, h // G], v[at, h // G]
                x = q[q0 + i, h]
                with np.errstate(invalid="ignore", over="ignore"):
                    s = scale * (kk @ x)
                    m = s.max()
                    p = np.exp(s - m)
                    total = p.sum()
                    out[q0 + i, h] = (p @ vv) / total
                    lse[q0 + i, h] = m + np.log(total)
                    mass[q0 + i, h] = (p @ np.abs(vv)) / total
                    big[q0 + i, h] = scale * (np.abs(kk) @ np.abs(x)).max()
                    vmax[q0 + i, h] = np.nanmax(np.abs(vv))       # (a NaN value's row is NaN in that block only)
    return out, lse, mass, big, vmax


def fork(P, table, lens, refs, parents):
    """(child table, refs, short, [(src, dst)] pages to copy)."""
    refs, n_pages, width = refs.copy(), refs.shape[0], table.shape[1]
    child = np.full((len(parents), width), -1, np.int32)
    free = [i for i in range(n_pages) if refs[i] <= 0]
    short, copies = 0, []
    for c, p in enumerate(parents):
        if p < 0 or p >= table.shape[0] or lens[p] < 0 or lens[p] > width * P:
            short += 1
            continue
        whole, part = divmod(int(lens[p]), P)
        if part:
            src = int(table[p, whole])
            if src < 0 or src >= n_pages or not free:
                short += 1
                continue
            dst = free.pop(0)
            copies.append((src, dst))
            refs[dst] = 1
            child[c, whole] = dst
        for i in range(whole):
            e = int(table[p, i])
            child[c, i] = e
            if 0 <= e < n_pages:
                refs[e] += 1
    return child, refs, short, copies


def resize(P, table, lens, new_lens, refs):
    table, refs = table.copy(), refs.copy()
    width = table.shape[1]
    count = lambda n: -(-int(np.clip(n, 0, width * P)) // P)      # noqa: E731
    for b in range(table.shape[0]):
        for i in range(count(new_lens[b]), count(lens[b])):
            e = int(table[b, i])
            if 0 <= e < refs.shape[0]:
                refs[e] -= 1
            table[b, i] = -1
    free = [i for i in range(refs.shape[0]) if refs[i] <= 0]
    short = 0
    for b in range(table.shape[0]):
        for i in range(count(lens[b]), count(new_lens[b])):
            if free:
                page = free.pop(0)
                refs[page] = 1
                table[b, i] = page
            else:
                table[b, i] = -1
                short += 1
    return table, refs, short


def compact(table, refs):
    """(table, refs, live, [(src, dst)])."""
    n = refs.shape[0]
    live = int((refs > 0).sum())
    movers = [i for i in range(live, n) if refs[i] > 0]
    holes = [i for i in range(live) if refs[i] <= 0]
    to = dict(zip(movers, holes))
    new = np.where(np.arange(n) < live, refs, 0).astype(np.int32)
    for a, b in to.items():
        new[b] = refs[a]
    return np.vectorize(lambda e: to.get(int(e), int(e)), otypes=[np.int32])(table), new, live, list(to.items())
