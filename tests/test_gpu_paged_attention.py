"""Softmax attention over the paged cache against the float64 form."""
import numpy as np
import pytest
import torch

from hybrid_linear_attention_packed_gb300 import (SpanLAError, kv_pages, packed_positions, rope_inv_freq, span_la_check,
                                                  span_la_kv_read, span_la_kv_write, span_la_qk_norm_rope,
                                                  span_la_softmax_branches_from_kv, span_la_softmax_paged,
                                                  span_la_softmax_pass)
from hybrid_linear_attention_packed_gb300 import spanla
from oracle import paged_oracle as po
from paged_helpers import BF16, E4M3, U16, check_attention, f64, i32, make_pages, make_table, values

pytestmark = pytest.mark.gpu

def weights(G, cache):
    """What the weights of n packed rows are rounded to, at most: more than 16 row heads to bf16; fewer to a sum of two
    bf16 numbers, or, over e4m3 pages, to fp16."""
    return lambda n: U16 if n * G > 16 else 2.0 ** -16 if cache == BF16 else 2.0 ** -11


def _setup(lens, rows, G, H, R, cache, dev, seed=0, layout="plain", v_size=1.0, q_size=1.0, width=None, k_size=1.0):
    """A cache whose rows of sequences hold numbers and all others NaN, and the queries."""
    g = torch.Generator(device=dev).manual_seed(seed)
    table, P = make_table(lens, R, 2, seed, width)
    c = make_pages(P, H, R, cache, dev, layout, fill=0xFF)
    cu = np.concatenate([[0], np.cumsum(lens)])
    T = int(cu[-1])
    k = torch.randn(T, H, 64, generator=g, device=dev) * k_size
    v = torch.randn(T, H, 64, generator=g, device=dev) * v_size
    v = v * torch.exp2(torch.randint(-4, 5, (T, H, 1), generator=g, device=dev).float())    # rows of different sizes
    if T:
        span_la_kv_write(k, v, c[0], c[1], i32(table, dev), i32(lens, dev), i32(cu, dev), c[2], c[3])
    n = int(sum(rows))
    q = (torch.randn(n, G * H, 64, generator=g, device=dev) * q_size).to(BF16)
    return q, c, table, np.concatenate([[0], np.cumsum(rows)])


def _run(q, c, table, lens, cu, dev, **kw):
    out = torch.full_like(q, float("nan"), memory_format=torch.contiguous_format)
    lse = torch.full(q.shape[:2], float("nan"), device=dev)
    span_la_softmax_paged(q, c[0], c[1], i32(table, dev), i32(lens, dev), i32(cu, dev), c[2], c[3], out=out, lse=lse, **kw)
    span_la_check()
    return out, lse


CASES = [
    # lens, rows, G, H, R
    ([1], [1], 1, 1, 16),
    ([1, 2, 15, 16, 17, 31, 32, 33], [1] * 8, 1, 3, 16),
    ([63, 64, 65, 127, 128, 129, 255, 257], [1] * 8, 4, 2, 32),
    ([700, 3, 1300], [1, 1, 1], 8, 2, 128),
    ([900, 40], [1, 1], 16, 1, 64),
    ([300, 77, 5], [4, 3, 2], 4, 2, 16),
    ([300, 77], [5, 16], 1, 5, 256),
    ([1000, 900], [2, 2], 3, 2, 64),
    ([257, 130], [17, 20], 1, 2, 32),
    ([129, 128, 127], [129, 128, 127], 1, 2, 64),
    ([400, 300, 1], [33, 300, 1], 2, 2, 16),
    ([513], [260], 3, 2, 128),
    ([700, 513], [100, 513], 5, 1, 32),
    ([300], [40], 32, 1, 64),
    ([260, 5], [9, 5], 128, 1, 16),
    ([900, 20, 450, 64, 1], [300, 1, 2, 64, 1], 1, 4, 64),
    ([2000], [1], 1, 16, 16),
    ([5000], [600], 1, 2, 256),
    ([700, 40, 520, 9], [260, 1, 270, 9], 8, 2, 16),     # (many row heads: e4m3 pages are expanded first)
    ([300, 33], [300, 20], 12, 1, 64),
]


@pytest.mark.parametrize("cache", [BF16, E4M3])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_attention(cuda_device, case, cache):
    lens, rows, G, H, R = CASES[case]
    q, c, table, cu = _setup(lens, rows, G, H, R, cache, cuda_device, seed=case)
    out, lse = _run(q, c, table, lens, cu, cuda_device)
    check_attention(q, out, lse, c, table, lens, cu, 0.125, weights(G, cache))


@pytest.mark.parametrize("cache", [BF16, E4M3])
@pytest.mark.parametrize("rows", [1, 4, 70])
@pytest.mark.parametrize("q_size,k_size", [(1e37, 1e-34), (1e35, 1e-35), (1e-35, 1e35)])
def test_queries_and_keys_of_far_sizes(cuda_device, q_size, k_size, rows, cache):
    lens = [400, 70]
    q, c, table, cu = _setup(lens, [rows, rows], 2, 2, 64, cache, cuda_device, seed=22, q_size=q_size, k_size=k_size)
    out, lse = _run(q, c, table, lens, cu, cuda_device)
    check_attention(q, out, lse, c, table, lens, cu, 0.125, weights(2, cache))


@pytest.mark.parametrize("cache", [BF16, E4M3])
@pytest.mark.parametrize("rows", [1, 2, 40])
@pytest.mark.parametrize("size", [1e-34, 1e-32, 1e-30, 1e35])
def test_small_and_large_values(cuda_device, size, rows, cache):
    """Values near the ends of the exponent's range: within one CTA, over several, and in chunks."""
    lens = [60, 9000]
    q, c, table, cu = _setup(lens, [rows, rows], 4, 1, 64, cache, cuda_device, seed=21, v_size=size)
    out, lse = _run(q, c, table, lens, cu, cuda_device)
    o = f64(out)
    assert np.abs(o).max() < 20 * size and np.abs(o[cu[0]:cu[1]]).max() > size / 100
    check_attention(q, out, lse, c, table, lens, cu, 0.125, weights(4, cache))


@pytest.mark.parametrize("cache", [BF16, E4M3])
@pytest.mark.parametrize("layout", ["interleaved", "rows"])
@pytest.mark.parametrize("rows", [[1, 1], [3, 90]])
def test_other_layouts_and_strided_queries(cuda_device, layout, cache, rows):
    lens = [333, 150]
    q, c, table, cu = _setup(lens, rows, 2, 3, 32, cache, cuda_device, seed=3, layout=layout)
    fused = torch.cat([q.reshape(len(q), -1), q.reshape(len(q), -1)[:, :128]], 1)
    strided = fused[:, :6 * 64].view(len(q), 6, 64)
    big = torch.full((2, 40), 1 << 30, dtype=torch.int32, device=cuda_device)         # a part of a wider table
    big[:, 5:5 + table.shape[1]] = i32(table, cuda_device)
    out, lse = _run(q, c, table, lens, cu, cuda_device)
    check_attention(q, out, lse, c, table, lens, cu, 0.125, weights(2, cache))
    again = span_la_softmax_paged(strided, c[0], c[1], big[:, 5:5 + table.shape[1]], i32(lens, cuda_device), i32(cu, cuda_device),
                                  c[2], c[3])
    span_la_check()
    assert torch.equal(again, out)


@pytest.mark.parametrize("cache", [BF16, E4M3])
@pytest.mark.parametrize("rows", [1, 4, 70])
@pytest.mark.parametrize("scale,q_size", [(1.0, 2.0), (0.01, 1.0), (0.3, 8.0), (1e-20, 1e18)])
def test_scales(cuda_device, rows, scale, q_size, cache):
    """Flat and peaked weights, large scores, queries of any size."""
    lens = [500, 70]
    q, c, table, cu = _setup(lens, [rows, rows], 2, 2, 64, cache, cuda_device, seed=7, q_size=q_size)
    out, lse = _run(q, c, table, lens, cu, cuda_device, scale=scale)
    check_attention(q, out, lse, c, table, lens, cu, scale, weights(2, cache))


@pytest.mark.parametrize("cache", [BF16, E4M3])
@pytest.mark.parametrize("rows", [1, 3, 40])
@pytest.mark.parametrize("big,small", [(2.0 ** 60, 2.0 ** -60), (2.0 ** 100, 1.0), (1.0, 2.0 ** -100)])
def test_values_of_far_sizes(cuda_device, rows, big, small, cache):
    """Rows of V whose sizes are far apart, the large ones with almost no weight or with most of it; rows of zeros."""
    lens = [200, 90]
    q, c, table, cu = _setup(lens, [rows, rows], 2, 2, 32, cache, cuda_device, seed=8)
    g = torch.Generator(device=cuda_device).manual_seed(1)
    T = sum(lens)
    k = torch.randn(T, 2, 64, generator=g, device=cuda_device)
    v = torch.randn(T, 2, 64, generator=g, device=cuda_device) * small
    v[7::31] *= big / small
    v[5::13] = 0
    k[7::62] = -4 * q[0, 0].float()          # hardly seen
    k[38::62] = 0.4 * q[0, 0].float()
    all_cu = np.concatenate([[0], np.cumsum(lens)])
    span_la_kv_write(k, v, c[0], c[1], i32(table, cuda_device), i32(lens, cuda_device), i32(all_cu, cuda_device), c[2], c[3])
    out, lse = _run(q, c, table, lens, cu, cuda_device, scale=1.0)
    check_attention(q, out, lse, c, table, lens, cu, 1.0, weights(2, cache))


@pytest.mark.parametrize("cache", [BF16, E4M3])
@pytest.mark.parametrize("rows,G", [(1, 1), (4, 2), (30, 4), (200, 1)])
def test_rows_that_see_nothing(cuda_device, rows, G, cache):
    """Sequences shorter than their packed rows, empty ones, sequences of no packed rows."""
    lens, n = [0, rows // 2, 40, 1, rows - 1, 300], [rows, rows, 0, rows, rows, rows]
    q, c, table, cu = _setup(lens, n, G, 2, 16, cache, cuda_device, seed=9)
    out, lse = _run(q, c, table, lens, cu, cuda_device)
    check_attention(q, out, lse, c, table, lens, cu, 0.125, weights(G, cache))
    assert (out[:rows] == 0).all() and torch.isneginf(lse[:rows]).all()


@pytest.mark.parametrize("what", [float("inf"), float("-inf"), float("nan"), 3.3e38])
@pytest.mark.parametrize("cache", [BF16, E4M3])
@pytest.mark.parametrize("rows,G", [(2, 1), (4, 4), (40, 2), (300, 1), (260, 8)])
def test_what_a_row_does_not_see_does_not_reach_it(cuda_device, rows, G, cache, what):
    """The last row of every sequence holds infinities or NaN: only the last packed row sees it."""
    lens = [rows + 5, 310, rows]
    q, c, table, cu = _setup(lens, [rows] * 3, G, 2, 32, cache, cuda_device, seed=11)
    before = [L - 1 for L in lens]
    clean, _ = _run(q, c, table, lens, cu, cuda_device)
    for x, dims in ((0, [3, 60]), (1, [0, 17, 63])):
        new = torch.randn(3, 2, 64, device=cuda_device)
        new[:, :, dims] = what
        pair = (new, torch.zeros_like(new)) if x == 0 else (torch.zeros_like(new), new)
        span_la_kv_write(pair[0], pair[1], c[0], c[1], i32(table, cuda_device), i32(lens, cuda_device), None, c[2], c[3])
        out, lse = _run(q, c, table, lens, cu, cuda_device)
        keep = np.concatenate([np.arange(cu[s], cu[s + 1] - 1) for s in range(3)])
        if x == 0:                                       # keys that are not seen change no bit
            assert torch.equal(out[keep], clean[keep])
        ref_cu = np.concatenate([[0], np.cumsum([rows - 1] * 3)])
        check_attention(q[keep], out[keep], lse[keep], c, table, before, ref_cu, 0.125, lambda n: weights(G, cache)(n + 1))
        seen = f64(out[cu[1] + rows - 1])
        if x == 1 and not (cache == E4M3 and np.isfinite(what)):
            finite = np.ones(64, dtype=bool)
            finite[dims] = False
            if not np.isfinite(what):
                assert not np.isfinite(seen[:, dims]).any()
            assert np.isfinite(seen[:, finite]).all()


def test_other_rows_of_the_call_are_left(cuda_device):
    """Packed rows of no sequence, and sequences of more rows than max_rows (reported)."""
    lens = [50, 60, 70]
    q, c, table, _ = _setup(lens, [10, 2, 2], 1, 2, 16, BF16, cuda_device)
    q = torch.cat([q, q])
    cu = [2, 12, 14, 16]
    out, _ = _run(q, c, table, lens, cu, cuda_device)
    check_attention(q, out, None, c, table, lens, cu, 0.125, weights(1, BF16))
    assert torch.isnan(out[:2]).all() and torch.isnan(out[16:]).all()
    out.fill_(float("nan"))
    span_la_softmax_paged(q, c[0], c[1], i32(table, cuda_device), i32(lens, cuda_device), i32(cu, cuda_device), max_rows=4, out=out)
    with pytest.raises(SpanLAError, match="out of range"):
        span_la_check()
    check_attention(q, out, None, c, table, lens, cu, 0.125, weights(1, BF16), max_rows=4)
    assert torch.isnan(out[2:12]).all()


@pytest.mark.parametrize("cache", [BF16, E4M3])
@pytest.mark.parametrize("rows,G", [(1, 2), (70, 2), (90, 24)])
def test_pages_out_of_range_are_not_seen_and_reported(cuda_device, rows, G, cache):
    lens = [100, 200, 300]
    q, c, table, cu = _setup(lens, [rows] * 3, G, 2, 16, cache, cuda_device, seed=5)
    bad = table.copy()
    bad[1, 2], bad[2, 0] = 1 << 30, -1
    lens_bad = np.array(lens)
    out = torch.full_like(q, float("nan"))
    span_la_softmax_paged(q, c[0], c[1], i32(bad, cuda_device), i32(lens_bad, cuda_device), i32(cu, cuda_device), c[2], c[3], out=out)
    with pytest.raises(SpanLAError, match="a page out of range"):
        span_la_check()
    check_attention(q[:rows], out[:rows], None, c, table, lens[:1], cu[:2], 0.125, weights(G, cache))
    assert torch.isfinite(out.float()).all()
    for s, gone in ((1, range(32, 48)), (2, range(16))):      # the others: as if those rows had scores of -infinity
        kv = [po.rows_of(values(c[x], c[2 + x]), table[s], lens[s]) for x in range(2)]
        keep = [j for j in range(lens[s]) if j not in gone]
        first = lens[s] - rows
        assert first > max(gone)
        ref, _, mass, _ = po.attend(f64(q[cu[s]:cu[s + 1]]), kv[0][keep], kv[1][keep], 0.125)
        tol = 1.01 * U16 * np.abs(ref) + (U16 + 2.0 ** -12) * mass
        assert np.all(np.abs(f64(out[cu[s]:cu[s + 1]]) - ref) <= tol)
    lens_bad[1] = -5
    out.fill_(float("nan"))
    span_la_softmax_paged(q, c[0], c[1], i32(table, cuda_device), i32(lens_bad, cuda_device), i32(cu, cuda_device), c[2], c[3], out=out)
    with pytest.raises(SpanLAError, match="offsets or length"):
        span_la_check()
    assert torch.isnan(out[rows:2 * rows]).all()
    keep = np.concatenate([np.arange(rows), np.arange(2 * rows, 3 * rows)])
    check_attention(q[keep], out[keep], None, c, table[[0, 2]], [100, 300], [0, rows, 2 * rows], 0.125, weights(G, cache))


@pytest.mark.parametrize("rows", [1, 4, 100])
def test_same_bits_again_and_on_another_stream(cuda_device, rows):
    lens = [1500, 30, 700, 64]
    q, c, table, cu = _setup(lens, [min(rows, n) for n in lens], 2, 4, 64, E4M3, cuda_device, seed=4)
    ref, lse = _run(q, c, table, lens, cu, cuda_device)
    args = [c[0], c[1], i32(table, cuda_device), i32(lens, cuda_device), i32(cu, cuda_device), c[2], c[3]]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(cuda_device) for _ in range(3)]
    outs = []
    for i in range(12):                                # calls in flight side by side
        s = streams[i % 3]
        o = torch.empty_like(q)
        span_la_softmax_paged(q, *args, out=o, stream=s)
        outs.append(o)
    torch.cuda.synchronize()
    span_la_check()
    assert all(torch.equal(o, ref) for o in outs)


def test_more_sequences_than_one_launch_takes(cuda_device):
    S = 2500
    rng = np.random.default_rng(0)
    lens = rng.integers(1, 40, S)
    q, c, table, cu = _setup(list(lens), [1] * S, 1, 1, 16, BF16, cuda_device, seed=6)
    out, lse = _run(q, c, table, lens, cu, cuda_device, max_rows=1)
    check_attention(q, out, lse, c, table, lens, cu, 0.125, weights(1, BF16))
    single = span_la_softmax_paged(q, c[0], c[1], i32(table, cuda_device), i32(lens, cuda_device))
    span_la_check()
    assert torch.equal(single, out)


def test_chunks_of_more_sequences_than_one_launch_takes(cuda_device):
    """Among single tokens, empty sequences and short ones."""
    S = 1100
    rng = np.random.default_rng(1)
    lens = rng.integers(0, 60, S)
    rows = np.minimum(rng.choice([0, 1, 3, 20, 35], S), lens)
    q, c, table, cu = _setup(list(lens), list(rows), 2, 1, 16, E4M3, cuda_device, seed=6)
    out, lse = _run(q, c, table, lens, cu, cuda_device)
    check_attention(q, out, lse, c, table, lens, cu, 0.125, weights(2, E4M3))


@pytest.mark.parametrize("rows", [2, 60])
def test_nothing_but_nan_and_infinities(cuda_device, rows):
    """Values that are all infinite, NaN, or of both signs of infinity: what the formula gives, row by row."""
    lens = [90, 70, 50, 40]
    q, c, table, cu = _setup(lens, [min(rows, n) for n in lens], 2, 2, 16, BF16, cuda_device, seed=12)
    c[1][torch.from_numpy(table[0, :6]).long()] = float("inf")
    c[1][torch.from_numpy(table[1, :5]).long()] = float("nan")
    c[1][int(table[2, 0]), :, 3] = float("inf")
    c[1][int(table[2, 0]), 0, 5, :7] = float("-inf")
    c[0][int(table[3, 0]), :, 2, 9] = float("nan")
    out, lse = _run(q, c, table, lens, cu, cuda_device)
    o = f64(out)
    assert np.all(o[cu[0]:cu[1]] == np.inf) and np.isnan(o[cu[1]:cu[2]]).all()
    for i, y in enumerate(o[cu[2]:cu[3]]):               # row 3 is +inf, row 5 of key head 0 -inf in seven elements
        seen = lens[2] - (cu[3] - cu[2]) + i + 1
        both, one = y[:2, :7], np.concatenate([y[:2, 7:].ravel(), y[2:].ravel()])
        assert np.isnan(both).all() if seen > 5 else np.all(both == np.inf) if seen > 3 else np.isfinite(both).all()
        assert np.all(one == np.inf) if seen > 3 else np.isfinite(one).all()
    for i, (y, z) in enumerate(zip(o[cu[3]:cu[4]], f64(lse)[cu[3]:cu[4]])):   # row 2's key is NaN
        hit = lens[3] - (cu[4] - cu[3]) + i + 1 > 2
        assert np.isnan(y).all() == hit and np.isnan(z).all() == hit and np.isfinite(y).all() != hit
    assert np.isfinite(f64(lse)[:cu[3]]).all()


@pytest.mark.parametrize("cache", [BF16, E4M3])
@pytest.mark.parametrize("rows", [1, 40])
def test_scores_past_fp32(cuda_device, rows, cache):
    """q . k of 64, -64 and 0 at a scale of 1e38: infinite scores of either sign, and weights of nothing else."""
    keys = [[1.0] * 90, [-1.0] * 300, [-1.0] * 128 + [0.0] * 200, [-1.0] * 150 + [1.0] * 60, [0.0] * 70]
    lens = [len(x) for x in keys]
    q, c, table, cu = _setup(lens, [rows] * 5, 1, 2, 16, cache, cuda_device, seed=14)
    at = np.concatenate([[0], np.cumsum(lens)])
    k = torch.tensor(np.concatenate(keys), device=cuda_device, dtype=torch.float32)[:, None, None].expand(-1, 2, 64).contiguous()
    v = torch.full_like(k, 3.0)
    span_la_kv_write(k, v, c[0], c[1], i32(table, cuda_device), i32(lens, cuda_device), i32(at, cuda_device), c[2], c[3])
    out, lse = _run(torch.ones_like(q), c, table, lens, cu, cuda_device, scale=1e38)
    o, z = f64(out), f64(lse)
    for s in (0, 3):
        assert np.isnan(o[cu[s]:cu[s + 1]]).all() and np.isnan(z[cu[s]:cu[s + 1]]).all()
    assert not o[cu[1]:cu[2]].any() and np.all(z[cu[1]:cu[2]] == -np.inf)
    for s, zero in ((2, 200), (4, 70)):
        n = zero - rows + 1 + np.arange(rows)                  # rows of score 0 that each sees
        assert np.all(o[cu[s]:cu[s + 1]] == 3.0)
        assert np.abs(z[cu[s]:cu[s + 1]] - np.log(n)[:, None]).max() < 1e-5


@pytest.mark.parametrize("cache", [BF16, E4M3])
@pytest.mark.parametrize("rows", [1, 30, 2100])
def test_a_table_of_no_pages(cuda_device, rows, cache):
    q, c, _, _ = _setup([5], [rows], 1, 1, 16, cache, cuda_device, seed=15)
    out, lse = _run(q, c, np.zeros((1, 0), np.int32), [0], [0, rows], cuda_device)
    assert not f64(out).any() and np.all(f64(lse) == -np.inf)


@pytest.mark.parametrize("cache", [BF16, E4M3])
@pytest.mark.parametrize("rows", [1, 40])
def test_sequences_that_share_pages(cuda_device, rows, cache):
    """Three sequences behind the same 96 rows, and one that is another's whole table."""
    q, c, table, cu = _setup([150, 300], [rows, rows], 2, 2, 32, cache, cuda_device, seed=16)
    shared = np.full((4, 10), -7, np.int32)
    shared[0, :5], shared[1, :10] = table[0, :5], table[1, :10]
    shared[2, :3], shared[2, 3:8] = table[0, :3], table[1, 3:8]        # 96 rows of one, then the other's
    shared[3, :10] = table[1, :10]
    lens, cu = [150, 300, 256, 290], np.arange(5) * rows
    q = torch.cat([q, q + 1])
    out, lse = _run(q, c, shared, lens, cu, cuda_device)
    check_attention(q, out, lse, c, shared, lens, cu, 0.125, weights(2, cache))


@pytest.mark.parametrize("cache", [BF16, E4M3])
@pytest.mark.parametrize("lens,rows,G,max_rows", [([3000, 200], [1, 2], 4, 2), ([900], [300], 2, 0), ([800, 500], [700, 1], 4, 0)])
def test_the_workspace_is_enough_and_any(cuda_device, cache, lens, rows, G, max_rows):
    """Calls without the extension module; with a workspace of just the bytes asked for, full of NaN, and what is behind it
    left as it was; and with the library's own."""
    dev = cuda_device
    q, c, table, cu = _setup(lens, rows, G, 2, 32, cache, dev, seed=17)
    ref, _ = _run(q, c, table, lens, cu, dev, max_rows=max_rows or None)
    t, n, r = i32(table, dev), i32(lens, dev), i32(cu, dev)
    cc, _ = spanla._kv_cache(c[0], c[1], t, n, r, c[2], c[3])
    lib = spanla._lib
    size = lib.span_la_softmax_paged_workspace(len(q), 2 * G, cc, max_rows)
    ws = torch.full((size + 4096,), 0xFF, dtype=torch.uint8, device=dev)
    for w in (ws.data_ptr(), None):
        out = torch.full_like(q, float("nan"))
        stream = torch.cuda.current_stream(dev).cuda_stream
        assert lib.span_la_softmax_paged(q.data_ptr(), q.stride(0), len(q), 2 * G, cc, max_rows, 0.0, out.data_ptr(), None, w, stream) == 0
        span_la_check()
        assert torch.equal(out, ref)
    assert (ws[size:] == 0xFF).all()


REFUSED = [
    ("attend", dict(page_table=lambda t: t.long()), "page_table"),
    ("attend", dict(page_table=lambda t: t.t()), "page_table|seq_len"),
    ("attend", dict(page_table=lambda t: t.cpu()), "page_table"),
    ("attend", dict(seq_len=lambda t: t[:1]), "seq_len"),
    ("attend", dict(row_cu=lambda t: t[:2]), "row_cu"),
    ("attend", dict(row_cu=lambda t: t.float()), "row_cu"),
    ("attend", dict(v_pages=lambda t: t[1:]), "share shape"),
    ("attend", dict(v_pages=lambda t: t.transpose(0, 1).contiguous().transpose(0, 1)), "strides"),
    ("attend", dict(k_pages=lambda t: t.float()), "share shape|dtype"),
    ("attend", dict(k_scale=lambda t: None), "k_scale"),
    ("attend", dict(v_scale=lambda t: t.float()), "v_scale"),
    ("attend", dict(q=lambda t: t.float()), "bf16"),
    ("attend", dict(q=lambda t: t[:, :3], out=lambda t: None, lse=lambda t: None), "multiple"),
    ("attend", dict(q=lambda t: t.cpu()), "q must"),
    ("attend", dict(out=lambda t: t[:1]), "out"),
    ("attend", dict(lse=lambda t: t.double()), "lse"),
    ("attend", dict(max_rows=lambda t: 0), "max_rows"),
    ("attend", dict(max_rows=lambda t: 1 << 32), "max_rows"),
    ("attend", dict(scale=lambda t: -1.0), "scale"),
    ("attend", dict(scale=lambda t: float("nan")), "scale"),
    ("write", dict(k=lambda t: t.half()), "dtype"),
    ("write", dict(v=lambda t: t.float()), "share"),
    ("write", dict(k=lambda t: t[:, :1], v=lambda t: t[:, :1]), r"\[T, 2, 64\]"),
    ("write", dict(row_cu=lambda t: None), "as many sequences"),
    ("read", dict(total_rows=lambda t: None), "total_rows"),
    ("read", dict(dtype=lambda t: torch.float16), "dtype"),
    ("read", dict(k_out=lambda t: t[:3]), "k_out"),
]


@pytest.mark.parametrize("case", range(len(REFUSED)))
def test_the_binding_names_what_is_wrong(cuda_device, case):
    op, change, what = REFUSED[case]
    lens, rows = [40, 20], [3, 2]
    q, c, table, cu = _setup(lens, rows, 2, 2, 16, E4M3, cuda_device, seed=19)
    cache = dict(k_pages=c[0], v_pages=c[1], page_table=i32(table, cuda_device), seq_len=i32(lens, cuda_device), row_cu=i32(cu, cuda_device),
                 k_scale=c[2], v_scale=c[3])
    k = torch.zeros(5, 2, 64, dtype=BF16, device=cuda_device)
    own = dict(attend=dict(q=q, max_rows=None, scale=0.0, out=torch.empty_like(q), lse=torch.empty(5, 4, device=cuda_device)),
               write=dict(k=k, v=k.clone()), read=dict(total_rows=5, dtype=BF16, k_out=None))[op]
    if "k_out" in change:
        own["k_out"] = k
    args = {**own, **cache}
    for name, f in change.items():
        args[name] = f(args[name])
    call = dict(attend=span_la_softmax_paged, write=span_la_kv_write, read=span_la_kv_read)[op]
    with pytest.raises((ValueError, SpanLAError), match=what):
        call(**args)
    span_la_check()


def test_the_same_without_the_extension_module(cuda_device, monkeypatch):
    dev, lens, rows = cuda_device, [100, 40], [30, 1]
    q, c, table, cu = _setup(lens, rows, 2, 2, 16, E4M3, dev, seed=18)
    args = (c[0], c[1], i32(table, dev), i32(lens, dev), i32(cu, dev))
    k, v = (torch.randn(31, 2, 64, device=dev) for _ in range(2))

    def step():
        span_la_kv_write(k, v, *args, c[2], c[3])
        back = span_la_kv_read(*args, 31, c[2], c[3])
        out = span_la_softmax_paged(q, *args, c[2], c[3])
        span_la_check()
        return (*back, out)

    ref = step()
    monkeypatch.setattr(spanla, "_fast", None)
    k, v = k.clone(), v.clone()
    assert all(torch.equal(a, b) for a, b in zip(step(), ref))


def test_captured_behind_another_stream(cuda_device):
    """Recorded where the rows come from a second stream, next to work on a third, and replayed; twice, so that two graphs
    are in flight."""
    dev, lens = cuda_device, [200, 33, 64]
    q, c, table, cu = _setup(lens, [3, 30, 1], 1, 2, 16, BF16, dev, seed=13)
    args = [c[0], c[1], i32(table, dev), i32(lens, dev), i32(cu, dev)]
    ref = span_la_softmax_paged(q, *args)
    src = q.clone()
    graphs, outs = [], []
    torch.cuda.synchronize()
    for _ in range(2):
        main, side = torch.cuda.Stream(dev), torch.cuda.Stream(dev)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=main):
            side.wait_stream(main)
            with torch.cuda.stream(side):
                x = src * 1.0
                k, v = span_la_kv_read(*args[:4], args[4], len(q))
            main.wait_stream(side)
            span_la_kv_write(k, v, *args)                       # (what is there already)
            o = span_la_softmax_paged(x, *args)
            o2 = o * 2
        graphs.append((g, main))
        outs.append((o, o2))
    for _ in range(3):
        for g, s in graphs:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    span_la_check()
    for o, o2 in outs:
        assert torch.equal(o, ref) and torch.equal(o2, ref * 2)


def test_generation_step_by_step_in_a_graph(cuda_device):
    """A prompt in chunks, then tokens: norm and rotation, cache write, attention, recorded once for the tokens and
    replayed with growing lengths.  Equals the softmax layer over whole sequences, to its own bound."""
    dev, H, R, S, prompt, steps = cuda_device, 4, 16, 3, 50, 20
    g = torch.Generator(device=dev).manual_seed(2)
    L = prompt + steps
    proj = torch.randn(S, L, 3 * H * 64, generator=g, device=dev).to(BF16)
    freq = rope_inv_freq(64)
    pos = torch.arange(L, device=dev, dtype=torch.int32)
    table, P = make_table([L] * S, R, 0, 3)
    c = make_pages(P, H, R, BF16, dev)
    dt = i32(table, dev)

    def layer(rows, where, lens, cu, max_rows):
        n = rows.shape[0]
        q, k, v = (rows[:, i * H * 64:(i + 1) * H * 64].view(n, H, 64) for i in range(3))
        q, k = span_la_qk_norm_rope(q, k, where, freq)
        span_la_kv_write(k, v, c[0], c[1], dt, lens, cu)
        return span_la_softmax_paged(q, c[0], c[1], dt, lens, cu, max_rows=max_rows)

    got = torch.empty(S, L, H, 64, dtype=BF16, device=dev)
    for a, b in ((0, 33), (33, prompt)):                # chunks
        cu = i32(np.arange(S + 1) * (b - a), dev)
        o = layer(proj[:, a:b].reshape(S * (b - a), -1), pos[a:b].repeat(S), i32([b] * S, dev), cu, b - a)
        got[:, a:b] = o.view(S, b - a, H, 64)
    rows, where, lens = proj[:, prompt].clone(), pos[prompt:prompt + 1].repeat(S), i32([prompt + 1] * S, dev)
    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        o = layer(rows, where, lens, None, None)
    for t in range(prompt, L):
        rows.copy_(proj[:, t]), where.fill_(t), lens.fill_(t + 1)
        graph.replay()
        got[:, t] = o
    torch.cuda.synchronize()
    span_la_check()
    flat = proj.reshape(S * L, -1)
    q, k, v = (flat[:, i * H * 64:(i + 1) * H * 64].view(S * L, H, 64) for i in range(3))
    vcu = (np.arange(S + 1) * L).astype(np.int32)
    q, k = span_la_qk_norm_rope(q, k, torch.from_numpy(packed_positions(vcu, None, None, S * L)).to(dev), freq)
    whole = span_la_softmax_pass(q, k, v.contiguous(), vcu, [], [])
    span_la_check()
    for s in range(S):
        ref, _, mass, _ = po.attend(f64(q[s * L:(s + 1) * L]), f64(k[s * L:(s + 1) * L]), f64(v[s * L:(s + 1) * L]), 0.125)
        tol = 1.01 * U16 * np.abs(ref) + (U16 + 2.0 ** -12) * mass       # as check_attention, its small terms in one
        assert np.all(np.abs(f64(got[s]) - ref) <= tol)
        assert np.all(np.abs(f64(got[s]) - f64(whole[s * L:(s + 1) * L])) <= 2 * tol)


@pytest.mark.parametrize("cache", [BF16, E4M3])
def test_branches_over_a_view_read_back(cuda_device, cache):
    """A view's keys and values kept in the cache, read back for the branches that are scored over it."""
    dev, H, view, blens = cuda_device, 3, 300, [20, 1, 64, 130]
    g = torch.Generator(device=dev).manual_seed(3)
    k, v = (torch.randn(view, H, 64, generator=g, device=dev).to(BF16) for _ in range(2))
    bcu = np.concatenate([[0], np.cumsum(blens)]).astype(np.int32)
    q, bk, bv = (torch.randn(int(bcu[-1]), H, 64, generator=g, device=dev).to(BF16) for _ in range(3))
    table, P = make_table([view], 64, 1, 0)
    c = make_pages(P, H, 64, cache, dev)
    args = [i32(table, dev), i32([view], dev), i32([0, view], dev)]
    span_la_kv_write(k, v, c[0], c[1], *args, c[2], c[3])
    vk, vv = span_la_kv_read(c[0], c[1], *args, view, c[2], c[3])
    if cache == BF16:
        assert torch.equal(vk, k) and torch.equal(vv, v)
    out = span_la_softmax_branches_from_kv(vk, vv, [0, view], q, bk, bv, bcu, [0] * 4)
    span_la_check()
    for b in range(4):
        rows = slice(int(bcu[b]), int(bcu[b + 1]))
        K, V = np.concatenate([f64(vk), f64(bk[rows])]), np.concatenate([f64(vv), f64(bv[rows])])
        ref, _, mass, _ = po.attend(f64(q[rows]), K, V, 0.125)
        assert np.all(np.abs(f64(out[rows]) - ref) <= 1.01 * U16 * np.abs(ref) + (U16 + 2.0 ** -12) * mass)
    # The same branches with their own rows in the cache, in pages of their own behind a copy of the view's last one.
    n = -(-(view + max(blens)) // 64)
    kp, vp, ks, vs = kv_pages(4 * n, H, 64, cache, dev)
    tb = i32(np.arange(4 * n).reshape(4, n), dev)
    lens = i32([view + b for b in blens], dev)
    full = [torch.cat([torch.cat([x, y[int(bcu[b]):int(bcu[b + 1])]]) for b in range(4)]) for x, y in ((k, bk), (v, bv))]
    span_la_kv_write(full[0], full[1], kp, vp, tb, lens, i32(np.concatenate([[0], np.cumsum([view + b for b in blens])]), dev), ks, vs)
    paged = span_la_softmax_paged(q, kp, vp, tb, lens, i32(bcu, dev), ks, vs)
    span_la_check()
    check_attention(q, paged, None, (kp, vp, ks, vs), tb.cpu().numpy(), [view + b for b in blens], bcu, 0.125, weights(1, cache))


def test_pages_past_two_to_the_32(cuda_device):
    P, H, R = 23000, 32, 128
    kp, vp, ks, vs = kv_pages(P, H, R, E4M3, cuda_device)
    lens = [257]
    table = np.array([[P - 1, 11, P - 2]])
    k, v = (torch.randn(257, H, 64, device=cuda_device) for _ in range(2))
    span_la_kv_write(k, v, kp, vp, i32(table, cuda_device), i32(lens, cuda_device), i32([0, 257], cuda_device), ks, vs)
    small = [torch.stack([x[int(p)] for p in table[0]]) for x in (kp.view(torch.uint8), vp.view(torch.uint8), ks, vs)]
    small = (small[0].view(E4M3), small[1].view(E4M3), small[2], small[3])
    for rows in (1, 40):
        q = torch.randn(rows, H, 64, device=cuda_device).to(BF16)
        out, lse = _run(q, (kp, vp, ks, vs), table, lens, [0, rows], cuda_device)
        check_attention(q, out, lse, small, np.arange(3)[None], lens, [0, rows], 0.125, weights(1, E4M3))
    del kp, vp, ks, vs
    torch.cuda.empty_cache()
