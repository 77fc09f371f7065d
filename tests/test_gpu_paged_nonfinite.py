"""Attention over the paged cache with NaN and infinities in queries, keys and values, and numbers next to them."""
import numpy as np
import pytest
import torch

from oracle import paged_oracle as po
from paged_helpers import BF16, E4M3, check_attention, f64, values
from test_gpu_paged_attention import _run, _setup, weights

pytestmark = pytest.mark.gpu


def _check_nan_rows(q, c, table, lens, cu, dev, bad):
    """Row heads of `bad` [rows, heads] are NaN and so is their log; the others are what they are without."""
    out, lse = _run(q, c, table, lens, cu, dev)
    o, z = f64(out), f64(lse)
    assert np.isnan(o[bad]).all() and np.isnan(z[bad]).all()
    assert np.isfinite(o[~bad]).all() and np.isfinite(z[~bad]).all()
    return out, lse


@pytest.mark.parametrize("width", [None, 200])     # whole items; items over several CTAs
@pytest.mark.parametrize("cache", [BF16, E4M3])
@pytest.mark.parametrize("rows,G", [(1, 1), (4, 2), (40, 1), (40, 3), (300, 1), (300, 2)])
def test_nan_queries_of_a_prompt(cuda_device, rows, G, cache, width):
    """Rows of a prompt whose query holds a NaN: every score is NaN, and there are blocks with nothing else."""
    lens = [rows, rows + 300]
    q, c, table, cu = _setup(lens, [rows, rows], G, 2, 16, cache, cuda_device, seed=31, width=width)
    clean, clean_lse = _run(q, c, table, lens, cu, cuda_device)
    bad = torch.zeros(q.shape[:2], dtype=torch.bool, device=cuda_device)
    for at in (0, 5, 126, 130):
        if at < rows:
            bad[at, at % q.shape[1]] = bad[rows + at, 0] = True
    q = q.clone()
    q[..., 7] = torch.where(bad, torch.nan, q[..., 7].float()).to(BF16)
    out, lse = _check_nan_rows(q, c, table, lens, cu, cuda_device, bad.cpu().numpy())
    assert torch.equal(out[~bad], clean[~bad]) and torch.equal(lse[~bad], clean_lse[~bad])


@pytest.mark.parametrize("width", [None, 200])
@pytest.mark.parametrize("cache", [BF16, E4M3])
@pytest.mark.parametrize("rows,G", [(3, 2), (40, 1), (300, 1), (300, 3)])
def test_nan_keys_that_a_row_sees(cuda_device, rows, G, cache, width):
    """A NaN key in row 0 of a prompt is all that its row 0 sees; 130 of them are all that a sequence's first block has."""
    lens = [rows, 400]
    q, c, table, cu = _setup(lens, [rows, rows], G, 2, 16, cache, cuda_device, seed=32, width=width)
    flat = (lambda x: x.view(torch.uint8)) if cache == E4M3 else (lambda x: x)   # (indexing e4m3 goes by its bytes)
    nan = 0x7F if cache == E4M3 else float("nan")
    flat(c[0])[int(table[0, 0]), 0, 0, 3] = nan
    for i in range(9):
        flat(c[0])[int(table[1, i]), 1, :(16 if i < 8 else 2), 60] = nan
    heads = np.arange(2 * G) // G
    bad = np.zeros((2 * rows, 2 * G), dtype=bool)
    bad[:rows, heads == 0] = True
    bad[rows:, heads == 1] = True
    _check_nan_rows(q, c, table, lens, cu, cuda_device, bad)


@pytest.mark.parametrize("width", [None, 200])
@pytest.mark.parametrize("cache", [BF16, E4M3])
@pytest.mark.parametrize("rows", [40, 300])
def test_nothing_but_scores_of_minus_infinity(cuda_device, rows, cache, width):
    """Keys of -infinity under queries of ones (in e4m3 pages: scores that the scale takes there): nothing is seen."""
    lens = [rows]
    q, c, table, cu = _setup(lens, [rows], 1, 1, 16, cache, cuda_device, seed=33, width=width)
    if cache == BF16:
        c[0][torch.from_numpy(table[0, :-(-rows // 16)]).long()] = float("-inf")
    else:
        c[0].view(torch.uint8).fill_(0xB8)        # -1
        c[2].fill_(127)
    out, lse = _run(torch.ones_like(q), c, table, lens, cu, cuda_device, scale=1e38)
    assert not f64(out).any() and np.all(f64(lse) == -np.inf)


def _values_at(c, table, s, row, head, dims, what):
    """Write `what` into elements of one cached row of V."""
    R = c[1].shape[2]
    c[1][int(table[s, row // R]), head, row % R, dims] = what


@pytest.mark.parametrize("width", [None, 200])
def test_whole_items_behind_those_that_are_done_over(cuda_device, width):
    """Several hundred short chunks, so that a CTA has many items one behind the other; every fifth sequence has infinities
    and NaN in V, in rows that all of its packed rows see, some, or one.  They change the elements that see them, and no
    bit beside."""
    S, G, H = 700, 2, 2
    rng = np.random.default_rng(34)
    lens = [int(x) for x in rng.integers(40, 70, S)]
    rows = [int(x) for x in rng.integers(9, 36, S)]
    q, c, table, cu = _setup(lens, rows, G, H, 16, BF16, cuda_device, seed=34, width=width)
    clean, clean_lse = _run(q, c, table, lens, cu, cuda_device)
    size = torch.nan_to_num(c[1].float(), nan=0.0).abs().max().item()
    want = {}
    for s in range(0, S, 5):
        for h in range(H):
            at = [0, int(lens[s] - rows[s] + 3 + h), lens[s] - 1]           # seen by all rows, from the fourth on, by the last
            for row, dim, what in zip(at, (1, 17, 63), (float("inf"), float("nan"), float("-inf"))):
                _values_at(c, table, s, row, h, dim, what)
                want[s, h, dim] = row, what
    out, lse = _run(q, c, table, lens, cu, cuda_device)
    o, ref = f64(out), f64(clean)
    assert torch.equal(lse, clean_lse)
    for s in range(S):
        b, e = int(cu[s]), int(cu[s + 1])
        if s % 5:
            assert torch.equal(out[b:e], clean[b:e])
            continue
        first = lens[s] - rows[s]
        same = np.ones((e - b, G * H, 64), dtype=bool)
        for (t, h, dim), (row, what) in want.items():
            if t == s:
                sees = np.arange(e - b) + first >= row
                got = o[b:e, h * G:(h + 1) * G, dim][sees]
                assert np.isnan(got).all() if np.isnan(what) else np.all(got == what)
                same[:, h * G:(h + 1) * G, dim] = False
                # (who does not see it: the same weights, rounded to bf16 or not, and o's own rounding, twice)
                got, old = (x[b:e, h * G:(h + 1) * G, dim][~sees] for x in (o, ref))
                assert np.all(np.abs(got - old) <= 2 * 2.0 ** -8 * (size + np.abs(old)))
        assert np.array_equal(o[b:e][same], ref[b:e][same])


@pytest.mark.parametrize("width", [None, 200])
@pytest.mark.parametrize("cache", [BF16, E4M3])
@pytest.mark.parametrize("S", [40, 300, 700])
def test_tokens_and_chunks_that_see_nan(cuda_device, S, cache, width):
    """Single tokens, drafted ones, chunks and empty sequences side by side, some of which see a NaN in one element of V, and
    some of whose rows do not see one in their last row."""
    G, H = 2, 2
    rng = np.random.default_rng(39)
    lens = [int(x) for x in rng.integers(40, 400, S)]
    rows = [int(x) for x in rng.choice([0, 1, 4, 8, 20, 35], S)]
    q, c, table, cu = _setup(lens, rows, G, H, 16, cache, cuda_device, seed=39, width=width)
    clean, clean_lse = _run(q, c, table, lens, cu, cuda_device)
    bits = c[1].view(torch.uint8) if cache == E4M3 else c[1]
    nan = 0x7F if cache == E4M3 else float("nan")
    for s in range(0, S, 3):
        bits[int(table[s, 1]), 1, 5, 33] = nan
        last = lens[s] - 1
        bits[int(table[s, last // 16]), 0, last % 16, 50] = nan
    out, lse = _run(q, c, table, lens, cu, cuda_device)
    assert torch.equal(lse, clean_lse)
    for s in range(S):
        b, e = int(cu[s]), int(cu[s + 1])
        x, y = out[b:e], clean[b:e]
        if s % 3 == 0 and e > b:
            sees = max(0, 21 - (lens[s] - rows[s]))             # packed rows from this one on see row 21
            assert torch.isnan(x[sees:, G:, 33]).all() and torch.isnan(x[-1, :G, 50]).all()
            assert torch.isfinite(x[:sees, G:, 33].float()).all()
            same = torch.ones(x.shape, dtype=torch.bool, device=cuda_device)
            same[:, G:, 33] = same[:, :G, 50] = False
            x, y = x[same], y[same]
            assert torch.isfinite(out[b:e - 1, :G, 50].float()).all()
        assert torch.equal(x, y)
    keep = np.concatenate([np.arange(cu[s], cu[s + 1] - 1) for s in range(S) if rows[s] > 0])     # no row's last, key head 0
    ref_cu = np.concatenate([[0], np.cumsum([max(r - 1, 0) for r in rows])])
    one = tuple(None if x is None else x[:, :1] for x in c)
    check_attention(q[keep][:, :G], out[keep][:, :G], None, one, table, [n - (r > 0) for n, r in zip(lens, rows)], ref_cu, 0.125,
                    lambda n: weights(G, cache)(n + 1))


@pytest.mark.parametrize("width", [None, 200])
def test_nan_scores_beside_values_that_are_not_finite(cuda_device, width):
    """Row heads whose scores are NaN are NaN in every element, next to others, of the same and of other items of a CTA, that
    see an infinity in one."""
    S, G, H = 500, 2, 2
    lens, rows = [60] * S, [30] * S
    q, c, table, cu = _setup(lens, rows, G, H, 16, BF16, cuda_device, seed=38, width=width)
    q = q.clone()
    q.view(S, 30, G * H, 64)[:, 7, 1, 2] = float("nan")
    c[1][torch.from_numpy(table[::3, 0].copy()).long(), :, 4, 40] = float("inf")
    out, lse = _run(q, c, table, lens, cu, cuda_device)
    o, z = f64(out).reshape(S, 30, G * H, 64), f64(lse).reshape(S, 30, G * H)
    nan = np.zeros((S, 30, G * H), dtype=bool)
    nan[:, 7, 1] = True
    assert np.isnan(o[nan]).all() and np.array_equal(np.isnan(z), nan) and np.isfinite(z[~nan]).all()
    assert np.all(o[::3, ..., 40][~nan[::3]] == np.inf)
    o[::3, ..., 40] = 0
    assert np.isfinite(o[~nan]).all()


@pytest.mark.parametrize("width", [None, 200])
@pytest.mark.parametrize("cache", [BF16, E4M3])
@pytest.mark.parametrize("rows,G", [(1, 1), (5, 3), (40, 2), (300, 1)])
def test_small_weights_of_infinities_and_nan(cuda_device, rows, G, cache, width):
    """Values whose weight is no fp32 number: positive all the same, so that an infinity stays one and a NaN one; and what
    a score of -infinity hides (a NaN in V too) is not seen."""
    lens, H = [rows + 310], 2
    q, c, table, cu = _setup(lens, [rows], G, H, 16, cache, cuda_device, seed=35, width=width)
    q = torch.ones_like(q)
    low, hidden, hi = [3, 150, 305], 200, 290              # before and behind the row with the greatest score
    R, flat = 16, (lambda x: x.view(torch.uint8)) if cache == E4M3 else (lambda x: x)
    one = (lambda x: {-50.0: 0xE4, 40.0: 0x62}[x]) if cache == E4M3 else float      # (e4m3: -48 and 40)
    at = lambda row: (int(table[0, row // R]), slice(None), row % R)  # noqa: E731
    for row in low:
        flat(c[0])[at(row)] = one(-50.0)
    flat(c[0])[at(hi)] = one(40.0)
    if cache == E4M3:
        for x in (c[2], c[3]):
            x[torch.from_numpy(table[0, :-(-lens[0] // R)]).long()] = 127
    clean, clean_lse = _run(q, c, table, lens, cu, cuda_device)
    assert np.isfinite(f64(clean)).all()
    nan, inf = (0x7F, 0x7F) if cache == E4M3 else (float("nan"), float("inf"))
    for dim, row, what in ((0, low[0], inf), (9, low[1], inf), (18, low[2], inf), (27, low[0], nan), (36, low[2], nan)):
        flat(c[1])[at(row)][..., dim] = what
    if cache == BF16:
        c[1][at(low[1])][..., 18] = float("-inf")          # with the other sign in row low[2]: NaN
        c[0][at(hidden)] = float("-inf")
        c[1][at(hidden)] = float("nan")
        c[1][at(hidden)] = 0
        _, clean_lse = _run(q, c, table, lens, cu, cuda_device)
        c[1][at(hidden)] = float("nan")
    out, lse = _run(q, c, table, lens, cu, cuda_device)
    o = f64(out)
    special = [0, 9, 18, 27, 36]
    if cache == BF16:
        assert np.all(o[..., [0, 9]] == np.inf) and np.isnan(o[..., [18, 27, 36]]).all()
    else:
        assert np.isnan(o[..., special]).all()
    rest = np.delete(o, special, -1)
    assert np.isfinite(rest).all() and np.isfinite(f64(lse)).all()
    assert torch.equal(lse, clean_lse)


@pytest.mark.parametrize("width", [None, 700])
@pytest.mark.parametrize("cache", [BF16, E4M3])
@pytest.mark.parametrize("rows,G", [(1, 1), (4, 4), (40, 2), (300, 1)])
def test_values_whose_sums_pass_fp32(cuda_device, rows, G, cache, width):
    """Values of up to 3e38, of one sign and of both: the means are numbers, the sums of some hundred of them are not."""
    lens = [rows + 400, rows + 5]
    q, c, table, cu = _setup(lens, [rows, rows], G, 2, 16, cache, cuda_device, seed=36, width=width)
    flat = (lambda x: x.view(torch.uint8)) if cache == E4M3 else (lambda x: x)
    for s, L in enumerate(lens):
        pages = torch.from_numpy(table[s, :-(-L // 16)]).long()
        if cache == E4M3:
            c[3][pages] = 246
            flat(c[1])[pages] = 0x7E
            flat(c[1])[pages, :, ::3, 1::2] = 0xFE
        else:
            c[1][pages] = 3e38
            c[1][pages, :, ::3, 1::2] = -3e38
    out, lse = _run(q, c, table, lens, cu, cuda_device)
    assert np.isfinite(f64(out)).all()
    check_attention(q, out, lse, c, table, lens, cu, 0.125, weights(G, cache))


@pytest.mark.parametrize("cache", [BF16, E4M3])
def test_what_an_infinity_in_v_costs(cuda_device, cache):
    """Every row of a large chunk sees one (82,000 row heads, 20,000 rows): far from 0.38 us for each of them and cached row,
    one behind the other in a warp."""
    lens, rows, H = [21280], [1280], 64
    q, c, table, cu = _setup(lens, rows, 1, H, 256, cache, cuda_device, seed=37)
    clean, _ = _run(q, c, table, lens, cu, cuda_device)
    c[1].view(torch.uint8 if cache == E4M3 else BF16)[int(table[0, 77]), :, 200, 5] = 0x7F if cache == E4M3 else float("inf")
    ms = []
    for _ in range(3):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        out, _ = _run(q, c, table, lens, cu, cuda_device)
        b.record()
        torch.cuda.synchronize()
        ms.append(a.elapsed_time(b))
    same = torch.ones(64, dtype=torch.bool, device=cuda_device)
    same[5] = False
    assert torch.equal(out[..., same], clean[..., same]) and not torch.isfinite(out[..., 5].float()).any()
    assert min(ms) < 60, ms


@pytest.mark.parametrize("cache", [BF16, E4M3])
@pytest.mark.parametrize("rows", [1, 4, 8, 70])
@pytest.mark.parametrize("q_size,k_size,scale", [(1e-37, 1e37, 0.125), (2e-38, 4e37, 0.25), (1.0, 1e36, 1e-37), (1e-10, 3e37, 4e-28)])
def test_small_queries_and_scales(cuda_device, q_size, k_size, scale, rows, cache):
    """Queries, or a scale, next to the least fp32 numbers, and keys next to the greatest: scores of ordinary sizes."""
    lens = [400, 70]
    q, c, table, cu = _setup(lens, [rows, rows], 2, 2, 64, cache, cuda_device, seed=40, q_size=q_size, k_size=k_size)
    out, lse = _run(q, c, table, lens, cu, cuda_device, scale=scale)
    assert f64(lse).max() > 1 and f64(out).std() > 0.1
    check_attention(q, out, lse, c, table, lens, cu, scale, weights(2, cache))


def _by_definition(q, K, V, first, scale):
    """(o, log of the sum, tolerance of o) of rows q [n, heads, 64] of which row i sees K, V[:first + i + 1] (float64): NaN
    where a score is NaN or +infinity; elements of V that are not finite, with a score above -infinity, add up to o's."""
    n, Hq = q.shape[:2]
    o, z, tol = np.zeros((n, Hq, 64)), np.full((n, Hq), -np.inf), np.zeros((n, Hq, 64))
    for i in range(n):
        seen = first + i + 1
        for h in range(Hq):
            if seen <= 0:
                continue
            k, v = K[:seen, h // (Hq // K.shape[1])], V[:seen, h // (Hq // K.shape[1])]
            x = (k @ q[i, h]) * scale
            if np.isnan(x).any() or (x == np.inf).any():
                o[i, h] = z[i, h] = np.nan
                continue
            live = x > -np.inf
            if not live.any():
                continue
            x, v = x[live], v[live]
            w = np.exp(x - x.max())
            z[i, h] = x.max() + np.log(w.sum())
            w /= w.sum()
            fin = np.where(np.isfinite(v), v, 0.0)
            o[i, h] = w @ fin
            tol[i, h] = w @ np.abs(fin)
            special = np.where(np.isfinite(v), 0.0, v).sum(0)
            o[i, h] = np.where(special == 0, o[i, h], special)
    return o, z, tol


@pytest.mark.parametrize("seed", range(24))
def test_random_calls_with_numbers_that_are_not_finite(cuda_device, seed):
    dev, rng = cuda_device, np.random.default_rng(100 + seed)
    cache, R, H, G = [BF16, E4M3][seed % 2], int(rng.choice([16, 32, 64, 128])), int(rng.integers(1, 4)), int(rng.choice([1, 2, 3, 5, 8]))
    S = int(rng.integers(1, 9))
    lens = [int(x) for x in rng.choice([0, 1, 17, 60, 130, 300, 700], S)]
    rows = [int(x) for x in rng.choice([0, 1, 3, 7, 20, 70], S)]
    if sum(rows) == 0:
        rows[0] = 2
    width = None if seed % 3 else -(-max(lens + [1]) // R) + 60
    q, c, table, cu = _setup(lens, rows, G, H, R, cache, dev, seed=seed, width=width)
    bits = [x.view(torch.uint8) if cache == E4M3 else x for x in c[:2]]
    kinds = [0x7F] if cache == E4M3 else [float("nan"), float("inf"), float("-inf")]
    for x, share in ((0, 0.3), (1, 3.0)):                      # (elements a sequence, on average)
        for s in range(S):
            for _ in range(rng.poisson(share) if lens[s] else 0):
                row = int(rng.integers(lens[s]))
                bits[x][int(table[s, row // R]), int(rng.integers(H)), row % R, int(rng.integers(64))] = kinds[int(rng.integers(len(kinds)))]
    q = q.clone()
    for _ in range(int(rng.poisson(0.7))):
        q[int(rng.integers(len(q))), int(rng.integers(G * H)), int(rng.integers(64))] = float(rng.choice([np.nan, np.inf, -np.inf]))
    max_rows = max(rows) if seed % 4 == 1 else None
    out, lse = _run(q, c, table, lens, cu, dev, max_rows=max_rows)
    o, z, qn = f64(out), f64(lse), f64(q)
    with np.errstate(invalid="ignore", over="ignore"):
        K, V = (values(c[i], c[2 + i]) for i in range(2))
        for s in range(S):
            b, e = int(cu[s]), int(cu[s + 1])
            ref, rz, mass = _by_definition(qn[b:e], po.rows_of(K, table[s], lens[s]), po.rows_of(V, table[s], lens[s]), lens[s] - rows[s], 0.125)
            got, fin = o[b:e], np.isfinite(ref)
            assert np.array_equal(got[~fin], ref[~fin], equal_nan=True)
            # o's rounding, and weights rounded to bf16 at the most, scores and sums in fp32
            assert np.all(np.abs(got - ref)[fin] <= (1.01 * 2.0 ** -8 * np.abs(ref) + (2.0 ** -8 + 2.0 ** -12) * mass)[fin] + 1e-37)
            fz = np.isfinite(rz)
            assert np.array_equal(z[b:e][~fz], rz[~fz], equal_nan=True) and np.all(np.abs(z[b:e] - rz)[fz] < 1e-3)
