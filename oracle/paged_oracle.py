"""Float64 forms of the paged cache's operators (numpy): quantised rows, and
softmax attention of a sequence's last rows over its rows.  Shares no code with
the GPU path."""
import math

import numpy as np


def quantise(x):
    """(values y, bytes b) of rows [..., 64]: y on the e4m3 grid with x ~ y * 2^(b - 127), b the least of 1 .. 246 at
    which a row's largest finite magnitude is at most 448 * 2^(b - 127), past which magnitudes are 448; infinite and NaN
    elements are NaN.  Element by element, from the grid's definition."""
    x = np.asarray(x, dtype=np.float64)
    rows = x.reshape(-1, x.shape[-1])
    val, code = np.empty_like(rows), np.empty(len(rows), dtype=np.uint8)
    for r, row in enumerate(rows):
        fin = np.isfinite(row)
        top = float(np.max(np.abs(row[fin]))) if fin.any() else 0.0
        b = 1
        while b < 246 and top > math.ldexp(448.0, b - 127):
            b += 1
        code[r] = b
        for i, v in enumerate(row):
            if not fin[i]:
                val[r, i] = np.nan
                continue
            y = max(-448.0, min(448.0, v * 2.0 ** (127 - b)))
            exp = max(math.frexp(y)[1] - 1, -6) if y else -6
            step = 2.0 ** (exp - 3)
            val[r, i] = round(y / step) * step          # (Python's round: halves to even)
    return val.reshape(x.shape), code.reshape(x.shape[:-1])


def scale_of(code):
    code = np.asarray(code).astype(np.int64)
    return np.where(code == 255, np.nan, 2.0 ** (code - 127.0))


def rows_of(pages, table, length):
    """A sequence's rows [length, H, 64] out of pages [P, H, R, 64] (float64, scaled already)."""
    R = pages.shape[2]
    if length == 0:
        return np.zeros((0,) + (pages.shape[1], pages.shape[3]))
    used = [pages[table[i]].transpose(1, 0, 2) for i in range(-(-length // R))]
    return np.concatenate(used)[:length]


def attend(q, K, V, scale):
    """Rows q [n, Hq, 64], the last n of a sequence with rows K, V [L, H, 64]: (out, lse, mass, size).  `mass`: the
    weights' mean of |v| (what a relative error of the weights is multiplied by); `size`: the largest sum of
    |products| in a row's scores (what a rounding of a product is a part of)."""
    n, Hq = q.shape[:2]
    L, H = K.shape[:2]
    out, mass = np.zeros((n, Hq, 64)), np.zeros((n, Hq, 64))
    lse, size = np.full((n, Hq), -np.inf), np.zeros((n, Hq))
    for i in range(n):
        seen = L - n + i + 1
        if seen <= 0:
            continue
        for h in range(Hq):
            k, v = K[:seen, h // (Hq // H)], V[:seen, h // (Hq // H)]
            x = (k @ q[i, h]) * scale
            m = x.max()
            w = np.exp(x - m)
            lse[i, h] = m + np.log(w.sum())
            w /= w.sum()
            out[i, h] = w @ v
            mass[i, h] = w @ np.abs(v)
            size[i, h] = (np.abs(k) @ np.abs(q[i, h])).max() * scale
    return out, lse, mass, size
