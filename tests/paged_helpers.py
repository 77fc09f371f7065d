"""Caches, packed rows and bounds that the paged-cache tests share."""
import numpy as np
import torch

from oracle import paged_oracle as po

BF16, E4M3 = torch.bfloat16, torch.float8_e4m3fn
U32, U16 = 2.0 ** -24, 2.0 ** -8       # half a step, relative


def f64(t):
    return t.detach().to(torch.float32).double().cpu().numpy()


def i32(a, dev):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(dev)


def make_pages(P, H, R, dtype, dev, layout="plain", fill=0x7F):
    """(k_pages, v_pages, k_scale, v_scale) full of the byte `fill` (0x7f: NaN in e4m3, 3.4e38 in bf16; 0xff: NaN in both).
    layout: "plain", "interleaved" (K and V of a page side by side), "rows" (heads inside of a page's rows)."""
    esz = 1 if dtype == E4M3 else 2
    both = torch.full((2 * P * H * R * 64 * esz,), fill, dtype=torch.uint8, device=dev).view(dtype)
    if layout == "plain":
        k, v = both.view(2, P, H, R, 64)
    elif layout == "interleaved":
        x = both.view(P, 2, H, R, 64)
        k, v = x[:, 0], x[:, 1]
    else:
        k, v = both.view(2, P, R, H, 64).transpose(2, 3)
    if dtype == BF16:
        return k, v, None, None
    if layout == "interleaved":
        s = torch.full((P, 2, H, R), 255, dtype=torch.uint8, device=dev)
        return k, v, s[:, 0], s[:, 1]
    return (k, v) + tuple(torch.full((P, H, R), 255, dtype=torch.uint8, device=dev) for _ in range(2))


def make_table(lens, R, spare, seed, width=None):
    """Distinct pages in no order for sequences of these lengths: (table, pages in the pool).  Entries that are not
    needed name no page."""
    used = [-(-n // R) for n in lens]
    P = sum(used) + spare
    order = np.random.default_rng(seed).permutation(P)
    table = np.full((len(lens), max(max(used, default=0), 1) if width is None else width), -7, dtype=np.int32)
    at = 0
    for s, n in enumerate(used):
        table[s, :n] = order[at:at + n]
        at += n
    return table, max(P, 1)


def values(pages, scale):
    """Float64 [P, H, R, 64] of what pages stand for."""
    x = f64(pages)
    return x if scale is None else x * po.scale_of(scale.cpu().numpy())[..., None]


def check_attention(q, got, lse, cache, table, lens, cu, scale, weight_error, max_rows=None):
    """Every row against the float64 form.  Bounds: a score is off by at most 66 roundings of its products' sizes
    (64 products and sums, the scale) and 2^-23 of itself where it is multiplied for a power of two; a weight by twice
    that (its own and the sum's), 2^-21 of exponentials and what the weights are rounded to (`weight_error` of a
    sequence's packed rows); the sum of weights by a rounding for each of its terms.  Then o's own rounding."""
    k, v, ks, vs = cache
    K, V = values(k, ks), values(v, vs)
    qn, o, z = f64(q), f64(got), None if lse is None else f64(lse)
    for s, L in enumerate(lens):
        b, e = int(cu[s]), int(cu[s + 1])
        if e == b or (max_rows is not None and e - b > max_rows):
            continue
        ref, rl, mass, size = po.attend(qn[b:e], po.rows_of(K, table[s], L), po.rows_of(V, table[s], L), scale)
        top = np.where(np.isfinite(rl), np.abs(rl), 0) + size
        ds = 66 * U32 * size + 2.0 ** -23 * top
        dw = 2 * ds + 2.0 ** -21 + L * U32
        tol = 1.01 * U16 * np.abs(ref) + (weight_error(e - b) + dw + (L + 64) * U32)[..., None] * mass + 1e-37
        bad = ~(np.abs(o[b:e] - ref) <= tol)
        assert not bad.any(), (s, L, e - b, np.argwhere(bad)[:3], np.max(np.abs(o[b:e] - ref) / np.maximum(tol, 1e-300)))
        if z is not None:
            fin = np.isfinite(rl)
            assert np.array_equal(z[b:e][~fin], rl[~fin])
            dz = ds[fin] + 2.0 ** -21 + L * U32 + 2 * U32 * np.abs(rl[fin])
            assert np.all(np.abs(z[b:e][fin] - rl[fin]) <= dz)
