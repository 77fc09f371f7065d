"""Packed rows into the paged cache and back, bit for bit."""
import numpy as np
import pytest
import torch

from hybrid_linear_attention_packed_gb300 import SpanLAError, kv_pages, span_la_check, span_la_kv_read, span_la_kv_write
from oracle import paged_oracle as po
from paged_helpers import BF16, E4M3, f64, i32, make_pages, make_table, values

pytestmark = pytest.mark.gpu

LENS = ([1], [0, 5, 16, 17], [200, 1, 33, 64, 0, 129], [700])
ROWS = ([1], [0, 3, 16, 9], [200, 1, 2, 1, 0, 40], [700])


def _rows(T, H, dtype, dev, seed=0, fused=False):
    g = torch.Generator(device=dev).manual_seed(seed)
    size = torch.exp2(torch.randint(-30, 30, (T, H, 1), generator=g, device=dev).float())
    k, v = (torch.randn(T, H, 64, generator=g, device=dev) * size for _ in range(2))
    if not fused:
        return k.to(dtype), v.to(dtype)
    row = torch.cat([x.reshape(T, H * 64) for x in (v, k, v)], 1).to(dtype)      # parts of a projection's rows
    return row[:, H * 64:2 * H * 64].view(T, H, 64), row[:, 2 * H * 64:].view(T, H, 64)


def _bits(x):
    return x.contiguous().view(torch.uint8).cpu().numpy()


def _expected(k, v, cache, table, lens, cu):
    """The cache's bytes after the write, from its bytes before and the oracle."""
    vals = [f64(x) for x in (k, v)]
    pages = [f64(x) for x in cache[:2]]
    scales = [None if s is None else s.cpu().numpy().copy() for s in cache[2:]]
    R = cache[0].shape[2]
    for s, L in enumerate(lens):
        for i in range(cu[s], cu[s + 1]):
            pos = L - (cu[s + 1] - i)
            if pos < 0:
                continue
            for x in range(2):
                row = vals[x][i]
                if scales[x] is not None:
                    row, b = po.quantise(row)
                    scales[x][table[s, pos // R], :, pos % R] = b
                pages[x][table[s, pos // R], :, pos % R] = row
    return pages, scales


@pytest.mark.parametrize("layout", ["plain", "interleaved", "rows"])
@pytest.mark.parametrize("rows", [BF16, torch.float32])
@pytest.mark.parametrize("cache", [BF16, E4M3])
@pytest.mark.parametrize("case,H,R", [(0, 1, 16), (1, 3, 16), (2, 16, 32), (2, 5, 256), (3, 2, 64), (3, 1, 128)])
def test_write_and_read(cuda_device, case, H, R, cache, rows, layout):
    lens, n = LENS[case], ROWS[case]
    cu = np.concatenate([[0], np.cumsum(n)])
    T = int(cu[-1])
    table, P = make_table(lens, R, 2, seed=case)
    c = make_pages(P, H, R, cache, cuda_device, layout, fill=0)
    k, v = _rows(T, H, rows, cuda_device, case, fused=layout != "plain")
    want, scales = _expected(k, v, c, table, lens, cu)
    dt, dl, dc = i32(table, cuda_device), i32(lens, cuda_device), i32(cu, cuda_device)
    span_la_kv_write(k, v, c[0], c[1], dt, dl, dc, c[2], c[3])
    span_la_check()
    for x in range(2):
        if cache == E4M3:
            assert np.array_equal(c[2 + x].cpu().numpy(), scales[x])
            assert np.array_equal(f64(c[x]), want[x])                     # (pages of no row among them)
        else:
            want_bits = torch.from_numpy(want[x]).float().to(BF16)         # round to nearest even, once
            assert torch.equal(c[x].cpu(), want_bits)
    back = span_la_kv_read(c[0], c[1], dt, dl, dc, T, c[2], c[3], dtype=rows)
    span_la_check()
    for x in range(2):
        vals = values(c[x], c[2 + x])
        for s, L in enumerate(lens):
            ref = po.rows_of(vals, table[s], L)[L - n[s]:]
            assert np.array_equal(f64(back[x][cu[s]:cu[s + 1]]), ref)


@pytest.mark.parametrize("rows", [BF16, torch.float32])
def test_values_at_the_borders(cuda_device, rows):
    """Zeros, ties, 448 and just past it, subnormal rows, the largest numbers, infinities and NaN."""
    x = torch.zeros(16, 1, 64, device=cuda_device)
    x[1, 0, :5] = torch.tensor([448., 1.0625, 1.1875, 17., -19.])           # halfway between two values
    x[2, 0, :3] = torch.tensor([450., 1., 2.])
    x[3, 0, :3] = torch.tensor([2. ** -9, 2. ** -10, 448.])                 # e4m3's least, and half of it
    x[4, 0, :2] = torch.tensor([2. ** -130, 2. ** -133])
    x[5, 0, :2] = torch.tensor([3.38e38, -1.])
    x[6, 0, :4] = torch.tensor([float("inf"), 1., -2., float("nan")])
    x[7] = float("nan")
    x[8] = float("-inf")
    x[9, 0] = torch.linspace(-500, 500, 64)
    x[10, 0] = torch.linspace(-1, 1, 64) * 2. ** -126
    x[11] = 1.75 * 2. ** 20
    x[12] = 1.7578125 * 2. ** 20
    x[13, 0, 63] = -1e-30
    k, v = x.to(rows), (x * -3).to(rows)
    kp, vp, ks, vs = kv_pages(1, 1, 16, E4M3, cuda_device)
    one = [i32(a, cuda_device) for a in ([[0]], [16], [0, 16])]
    span_la_kv_write(k, v, kp, vp, *one, ks, vs)
    span_la_check()
    for src, pages, scale in ((k, kp, ks), (v, vp, vs)):
        y, b = po.quantise(f64(src)[:, 0])
        assert np.array_equal(scale.cpu().numpy()[0, 0], b)
        assert np.array_equal(f64(pages)[0, 0], y, equal_nan=True)
    back, _ = span_la_kv_read(kp, vp, *one, 16, ks, vs, dtype=torch.float32)
    assert np.array_equal(f64(back)[:, 0], values(kp, ks)[0, 0], equal_nan=True)
    ks[0, 0, 3], ks[0, 0, 5] = 255, 0                                      # NaN, and 2^-127
    back, _ = span_la_kv_read(kp, vp, *one, 16, ks, vs, dtype=torch.float32)
    assert torch.isnan(back[3]).all()
    assert np.array_equal(f64(back)[5, 0], f64(kp)[0, 0, 5] * 2.0 ** -127)


def test_rows_that_do_not_exist_are_left(cuda_device):
    """A sequence shorter than its packed rows, packed rows of no sequence, and one row of each sequence without row_cu."""
    lens, cu = [2, 0, 3], [1, 6, 8, 9]                 # rows 0 and 9 belong to none; 1..3 and 6, 7 do not exist
    table, P = make_table(lens, 16, 1, seed=1)
    k, v = _rows(10, 2, BF16, cuda_device)
    c = make_pages(P, 2, 16, BF16, cuda_device, fill=0)
    dt, dl, dc = i32(table, cuda_device), i32(lens, cuda_device), i32(cu, cuda_device)
    want, _ = _expected(k, v, c, table, lens, cu)
    span_la_kv_write(k, v, c[0], c[1], dt, dl, dc)
    span_la_check()
    assert np.array_equal(f64(c[0]), want[0]) and np.array_equal(f64(c[1]), want[1])
    outs = [torch.full((10, 2, 64), 7.0, dtype=BF16, device=cuda_device) for _ in range(2)]
    span_la_kv_read(c[0], c[1], dt, dl, dc, k_out=outs[0], v_out=outs[1])
    span_la_check()
    live = [4, 5, 8]
    for got, src in zip(outs, (k, v)):
        assert torch.equal(got[live], src[live])
        assert (got[[0, 1, 2, 3, 6, 7, 9]] == 7.0).all()
    c = make_pages(P, 2, 16, BF16, cuda_device, fill=0)
    span_la_kv_write(k[:3], v[:3], c[0], c[1], dt, dl)
    got = span_la_kv_read(c[0], c[1], dt, dl, None, k_out=outs[0][:3].clone(), v_out=outs[1][:3].clone())
    span_la_check()
    assert torch.equal(got[0][[0, 2]], k[[0, 2]]) and (got[0][1] == 7.0).all()


@pytest.mark.parametrize("what", ["page", "negative page", "length", "negative length", "offsets", "last offset"])
def test_metadata_out_of_range_is_skipped_and_reported(cuda_device, what):
    lens, cu = np.array([20, 20, 20]), np.array([0, 4, 8, 12])
    table, P = make_table(lens, 16, 1, seed=2)
    k, v = _rows(12, 2, BF16, cuda_device)
    bad_rows = range(4, 8)
    if what == "page":
        table[1, 1] = P
    elif what == "negative page":
        table[1, 1] = -1
    elif what == "length":
        lens[1] = 33
    elif what == "negative length":
        lens[1] = -1
    elif what == "offsets":
        cu[1], bad_rows = 9, range(0, 8)
    else:
        cu[3], bad_rows = 13, range(8, 12)
    c = make_pages(P, 2, 16, E4M3, cuda_device, fill=0)
    args = [i32(table, cuda_device), i32(lens, cuda_device), i32(cu, cuda_device)]
    span_la_kv_write(k, v, c[0], c[1], *args, c[2], c[3])
    with pytest.raises(SpanLAError, match="out of range"):
        span_la_check()
    span_la_check()                                    # reported once
    outs = [torch.full((12, 2, 64), 7.0, dtype=BF16, device=cuda_device) for _ in range(2)]
    span_la_kv_read(c[0], c[1], *args, None, c[2], c[3], k_out=outs[0], v_out=outs[1])
    with pytest.raises(SpanLAError, match="out of range"):
        span_la_check()
    good = [t for t in range(12) if t not in bad_rows]
    y, b = po.quantise(f64(k)[good])
    assert np.array_equal(f64(outs[0][good]), y * po.scale_of(b)[..., None])
    if what != "offsets":
        assert (outs[0][list(bad_rows)] == 7.0).all()


def test_pages_past_two_to_the_32(cuda_device):
    """The last pages of a pool of 6 GB (element and byte offsets past 2^32)."""
    P, H, R = 23000, 32, 128
    kp, vp, ks, vs = kv_pages(P, H, R, E4M3, cuda_device)
    assert kp.numel() > 2 ** 32
    k, v = _rows(130, H, BF16, cuda_device)
    args = [i32([[P - 1, 11, P - 2]], cuda_device), i32([257], cuda_device), i32([0, 130], cuda_device)]
    span_la_kv_write(k, v, kp, vp, *args, ks, vs)
    back = span_la_kv_read(kp, vp, *args, 130, ks, vs)
    span_la_check()
    y, b = po.quantise(f64(k))
    assert np.array_equal(f64(back[0]), y * po.scale_of(b)[..., None])
    del kp, vp, ks, vs
    torch.cuda.empty_cache()


def test_side_stream_and_graph(cuda_device):
    """Recorded once, replayed on other rows, lengths and pages."""
    lens = np.array([10, 31])
    table, P = make_table([64, 64], 16, 0, seed=5)
    c = make_pages(P, 3, 16, E4M3, cuda_device, fill=0)
    k, v = (x.clone() for x in _rows(2, 3, BF16, cuda_device))
    dt, dl = i32(table, cuda_device), i32(lens, cuda_device)
    side = torch.cuda.Stream(cuda_device)
    side.wait_stream(torch.cuda.current_stream(cuda_device))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        span_la_kv_write(k, v, c[0], c[1], dt, dl, None, c[2], c[3])
        back = span_la_kv_read(c[0], c[1], dt, dl, None, 2, c[2], c[3])
    for step in range(3):
        nk, nv = _rows(2, 3, BF16, cuda_device, seed=10 + step)
        k.copy_(nk), v.copy_(nv)
        g.replay()
        torch.cuda.synchronize()
        for x, got in ((nk, back[0]), (nv, back[1])):
            y, b = po.quantise(f64(x))
            assert np.array_equal(f64(got), y * po.scale_of(b)[..., None])
        dl.add_(1)
    span_la_check()
    with torch.cuda.stream(side):
        span_la_kv_write(k, v, c[0], c[1], dt, dl, None, c[2], c[3], stream=side)
    side.synchronize()
    span_la_check()
