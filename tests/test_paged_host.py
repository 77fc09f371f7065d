"""The paged cache's refusals (every problem that the host can see is reported
before any CUDA call) and its oracle (CPU)."""
import ctypes

import numpy as np
import pytest
import torch

from hybrid_linear_attention_packed_gb300 import build as spanla_build
from hybrid_linear_attention_packed_gb300 import spanla
from oracle import paged_oracle as po

FAKE = 1 << 20          # aligned addresses; never dereferenced on the host
K, V, KS, VS, TABLE, LEN, CU, Q, OUT, LSE = (FAKE << i for i in range(10))
INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def lib():
    return spanla.load_library(spanla_build.build())


def _cache(**kw):
    """5 pages of 2 heads and 16 rows, 3 sequences."""
    c = dict(k=K, v=V, k_scale=KS, v_scale=VS, page_stride=2048, head_stride=1024, row_stride=64, scale_page_stride=32,
             scale_head_stride=16, num_pages=5, page_rows=16, num_heads=2, dtype=2, num_seqs=3, table_width=4, table_stride=4,
             page_table=TABLE, seq_len=LEN, row_cu=CU)
    c.update(kw)
    return spanla.KvCache(**c)


def _detail(lib):
    return lib.span_la_last_error_detail().decode()


CACHE = [
    (dict(dtype=1), UNSUPPORTED, "cache dtype"),
    (dict(dtype=7), UNSUPPORTED, "cache dtype"),
    (dict(page_rows=8), UNSUPPORTED, "page_rows"),
    (dict(page_rows=48), UNSUPPORTED, "page_rows"),
    (dict(page_rows=512), UNSUPPORTED, "page_rows"),
    (dict(num_heads=0), INVALID, "num_heads"),
    (dict(num_heads=65536), INVALID, "num_heads"),
    (dict(num_pages=0), INVALID, "num_pages"),
    (dict(num_seqs=-1), INVALID, "num_seqs"),
    (dict(k=None), INVALID, "k and v pages"),
    (dict(v=V + 8), INVALID, "k and v pages"),
    (dict(k_scale=None), INVALID, "k_scale"),
    (dict(v_scale=VS + 4), INVALID, "k_scale"),
    (dict(page_stride=2048 + 8), INVALID, "strides"),
    (dict(head_stride=32), INVALID, "strides"),
    (dict(row_stride=1 << 50), INVALID, "strides"),
    (dict(page_stride=-2048), INVALID, "strides"),
    (dict(page_stride=1024), INVALID, "overlap"),
    (dict(head_stride=512), INVALID, "overlap"),
    (dict(row_stride=128), INVALID, "overlap"),
    (dict(scale_head_stride=8), INVALID, "scale strides"),
    (dict(scale_page_stride=16), INVALID, "overlap"),
    (dict(table_width=-1), INVALID, "table_width"),
    (dict(table_width=1 << 28, table_stride=1 << 28), INVALID, "table_width"),
    (dict(table_width=(1 << 26) + 1, table_stride=1 << 27), INVALID, "table_width"),
    (dict(table_stride=3), INVALID, "table_stride"),
    (dict(page_table=None), INVALID, "page_table"),
    (dict(seq_len=LEN + 2), INVALID, "seq_len"),
    (dict(row_cu=CU + 1), INVALID, "row_cu"),
    (dict(row_cu=None, num_seqs=4), INVALID, "as many sequences"),
]


@pytest.mark.parametrize("kw,status,what", CACHE)
def test_every_call_refuses_the_cache(lib, kw, status, what):
    c = _cache(**kw)
    for st in (lib.span_la_kv_write(Q, OUT, 128, 128, 3, 0, c, None), lib.span_la_kv_read(c, 3, 0, Q, OUT, None),
               lib.span_la_softmax_paged(Q, 256, 3, 4, c, 0, 0.0, OUT, LSE, None, None)):
        assert st == status and what in _detail(lib)


def test_no_cache(lib):
    assert lib.span_la_kv_read(None, 3, 0, Q, OUT, None) == INVALID


@pytest.mark.parametrize("kw,status,what", [
    (dict(dtype=2), UNSUPPORTED, "dtype"),
    (dict(rows=-1), INVALID, "rows"),
    (dict(k=None), INVALID, "k must be"),
    (dict(v=Q + 2), INVALID, "v must be"),
    (dict(ks=100), INVALID, "row stride"),
    (dict(vs=132), INVALID, "row stride"),
    (dict(vs=1 << 31), INVALID, "row stride"),
    (dict(k=K + 64), INVALID, "k pages overlaps k"),
    (dict(k=VS), INVALID, "v_scale overlaps k"),
    (dict(cache=dict(v=K)), INVALID, "k pages overlap v pages"),
    (dict(cache=dict(v=K + 9 * 1024)), INVALID, "k pages overlap v pages"),
    (dict(cache=dict(k_scale=VS)), INVALID, "k_scale overlaps v_scale"),
    (dict(cache=dict(k_scale=K + 16)), INVALID, "overlaps k_scale"),
    (dict(cache=dict(seq_len=V)), INVALID, "overlaps seq_len"),
    (dict(cache=dict(page_table=VS)), INVALID, "overlaps page_table"),
    (dict(cache=dict(page_stride=4096, v=K + 2048 - 16)), INVALID, "k pages overlap v pages"),
])
def test_write_refuses(lib, kw, status, what):
    a = dict(k=Q, v=OUT, ks=128, vs=128, rows=3, dtype=0, cache={})
    a.update(kw)
    st = lib.span_la_kv_write(a["k"], a["v"], a["ks"], a["vs"], a["rows"], a["dtype"], _cache(**a["cache"]), None)
    assert st == status and what in _detail(lib)


@pytest.mark.parametrize("kw,status,what", [
    (dict(dtype=2), UNSUPPORTED, "dtype"),
    (dict(k=None), INVALID, "k_out"),
    (dict(v=OUT + 4), INVALID, "v_out"),
    (dict(v=Q), INVALID, "k_out overlaps v_out"),
    (dict(k=K + 1024), INVALID, "k_out overlaps k pages"),
    (dict(v=CU), INVALID, "v_out overlaps row_cu"),
])
def test_read_refuses(lib, kw, status, what):
    a = dict(k=Q, v=OUT, dtype=0)
    a.update(kw)
    assert lib.span_la_kv_read(_cache(), 3, a["dtype"], a["k"], a["v"], None) == status and what in _detail(lib)


@pytest.mark.parametrize("kw,status,what", [
    (dict(heads=3), INVALID, "num_q_heads"),
    (dict(heads=0), INVALID, "num_q_heads"),
    (dict(heads=258), INVALID, "num_q_heads"),
    (dict(max_rows=-1), INVALID, "max_rows"),
    (dict(scale=-1.0), INVALID, "scale"),
    (dict(scale=float("inf")), INVALID, "scale"),
    (dict(scale=float("nan")), INVALID, "scale"),
    (dict(q=None), INVALID, "q must be"),
    (dict(stride=255), INVALID, "row stride"),
    (dict(out=None), INVALID, "out must be"),
    (dict(out=Q), INVALID, "out overlaps q"),
    (dict(out=K), INVALID, "out overlaps k pages"),
    (dict(lse=OUT + 4), INVALID, "out overlaps lse_out"),
    (dict(lse=LSE + 2), INVALID, "lse_out"),
    (dict(lse=LEN), INVALID, "lse_out overlaps seq_len"),
    (dict(ws=FAKE * 4096 + 8), INVALID, "workspace must be"),
    (dict(ws=OUT, max_rows=100, cache=dict(table_width=40, table_stride=40)), INVALID, "workspace overlaps"),
])
def test_attention_refuses(lib, kw, status, what):
    a = dict(q=Q, stride=256, heads=4, max_rows=0, scale=0.0, out=OUT, lse=LSE, ws=None, cache={})
    a.update(kw)
    st = lib.span_la_softmax_paged(a["q"], a["stride"], 3, a["heads"], _cache(**a["cache"]), a["max_rows"], a["scale"], a["out"], a["lse"], a["ws"],
                                   None)
    assert st == status and what in _detail(lib)


def test_nothing_to_do_needs_no_device(lib):
    c = _cache(num_seqs=0, page_table=None, seq_len=None, row_cu=None)
    assert lib.span_la_kv_write(None, None, 0, 0, 0, 0, c, None) == 0
    assert lib.span_la_kv_read(c, 0, 1, None, None, None) == 0
    assert lib.span_la_softmax_paged(None, 0, 0, 4, c, 0, 0.0, None, None, None, None) == 0
    c = _cache(num_seqs=0, row_cu=CU)             # rows of no sequence
    assert lib.span_la_softmax_paged(Q, 256, 3, 4, c, 0, 0.0, OUT, None, None, None) == 0


def test_workspace(lib):
    """Enough for any GPU, nothing where a call has nothing to do or is refused."""
    f = lib.span_la_softmax_paged_workspace
    big = _cache(table_width=4000, table_stride=4000)
    assert f(3, 4, big, 1) > 0 and f(3, 4, big, 100) > f(3, 4, big, 8)
    assert f(3, 4, big, 0) == f(3, 4, big, 3) and f(3, 4, _cache(), 1) == 0      # (one CTA needs none)
    assert f(3, 4, _cache(), 100) == 0 and f(3, 258, _cache(), 100) == 0          # (whole items; refused)
    assert f(0, 4, _cache(), 1) == 0 and f(3, 5, _cache(), 1) == 0 and f(3, 4, None, 1) == 0 and f(3, 4, _cache(num_seqs=0), 1) == 0


@pytest.mark.parametrize("kw,rows,heads,max_rows", [
    (dict(page_rows=48), 3, 4, 100), (dict(page_rows=0), 3, 4, 100), (dict(page_rows=1 << 20, table_width=1 << 20), 3, 4, 100),
    (dict(dtype=7), 3, 4, 100), (dict(dtype=1), 3, 4, 1), (dict(table_width=-1), 3, 4, 100), (dict(table_width=1 << 30), 3, 4, 100),
    (dict(num_pages=0), 3, 4, 100), (dict(num_heads=70000), 3, 70000, 100), (dict(num_seqs=-3), 3, 4, 100), (dict(row_cu=None), 4, 4, 0),
    (dict(num_heads=40000), 3, 80000, 100), (dict(), 1 << 31, 4, 0), (dict(), -1, 4, 0), (dict(), 3, 4, -1), (dict(), 3, 5, 100),
])
def test_workspace_of_what_a_call_refuses_is_nothing(lib, kw, rows, heads, max_rows):
    c = _cache(**{"table_width": 4000, "table_stride": 1 << 30, **kw})
    assert lib.span_la_softmax_paged(Q, heads * 64, rows, heads, c, max_rows, 0.0, OUT, None, None, None) in (INVALID, UNSUPPORTED)
    assert lib.span_la_softmax_paged_workspace(rows, heads, c, max_rows) == 0


def test_workspace_for_expanded_pages(lib):
    """Copies of e4m3 pages where some sequence has 2,048 row heads: the caller says so, or there are as many on average."""
    f = lib.span_la_softmax_paged_workspace
    wide = dict(num_seqs=256, table_width=64, table_stride=64)                    # 1,024 rows of 2 heads: 2 x 64 MiB of copies
    copies = 2 * 256 * 64 * 16 * 2 * 64 * 2
    single = _cache(**wide)                                                       # 256 single tokens of 8 heads a key head
    assert f(256, 16, single, 0) == f(256, 16, single, 255) < copies
    assert f(256, 16, single, 256) == f(256, 16, single, 255) + copies            # one sequence may have them all
    assert f(256 * 255, 16, single, 0) == f(256 * 255, 16, single, 255) < copies
    assert f(256 * 255 + 1, 16, single, 0) == f(256 * 255, 16, single, 256) > copies
    one = _cache(table_width=1000, table_stride=1000, num_seqs=1)
    assert f(1024, 4, one, 0) == f(1024, 4, one, 1024) > f(1023, 4, one, 0) + 2 * 16000 * 2 * 64 * 2 - 1


def test_layouts_that_interleave_are_taken(lib):
    """K and V of a page side by side, heads inside of rows: as far as the (missing) device, past every check."""
    if torch.cuda.is_available():
        pytest.skip("the addresses are not real")
    for kw in (dict(page_stride=4096, v=K + 2048), dict(head_stride=64, row_stride=128),
               dict(head_stride=64, row_stride=256, page_stride=4096, v=K + 128)):
        st = lib.span_la_kv_write(Q, OUT, 128, 128, 3, 0, _cache(**kw), None)
        assert st not in (0, INVALID), _detail(lib)


def test_tensors_must_be_on_the_device():
    """The binding names the argument (CPU tensors here)."""
    pages = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    t = torch.zeros(1, 4, dtype=torch.int32)
    with pytest.raises(ValueError, match="k_pages"):
        spanla._kv_cache(pages, pages, t, t[:, 0], None, None, None)


def test_struct_matches_the_header():
    assert ctypes.sizeof(spanla.KvCache) == 4 * 8 + 5 * 8 + 6 * 4 + 8 + 3 * 8


# ------------------------------------------------------------------ the oracle
def test_quantised_against_torch():
    g = torch.Generator().manual_seed(0)
    x = torch.randn(64, 64, generator=g) * torch.exp2(torch.randint(-40, 40, (64, 1), generator=g).float())
    y, b = po.quantise(x.numpy())
    back = (x.double() / torch.exp2(torch.from_numpy(b.astype(np.float64)) - 127)[:, None]).float().to(torch.float8_e4m3fn)
    assert np.array_equal(y, back.double().numpy())
    assert np.all(np.abs(y).max(-1) > 200) and np.all(np.abs(y).max(-1) <= 448)


def test_quantised_edges():
    x = np.zeros((6, 64))
    x[1, :2] = 448, 449                # one past the largest: the next power of two
    x[2, 0] = 448
    x[3, :4] = 1.0, 2.0 ** -20, -np.inf, np.nan
    x[4, 0] = 2.0 ** -140
    x[5, 0] = 3.3e38
    y, b = po.quantise(x)
    assert list(b) == [1, 128, 127, 127 - 8, 1, 246]
    assert y[1, 0] == 224 and y[2, 0] == 448 and y[3, 0] == 256
    assert y[3, 1] == 0 and np.isnan(y[3, 2]) and np.isnan(y[3, 3]) and y[4, 0] == 0 and y[5, 0] == 448


@pytest.mark.parametrize("n,L,Hq,H", [(1, 1, 2, 1), (5, 9, 4, 2), (6, 4, 3, 3)])
def test_attention_against_torch(n, L, Hq, H):
    g = torch.Generator().manual_seed(n)
    q, k, v = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((n, Hq, 64), (L, H, 64), (L, H, 64)))
    out, lse, mass, _ = po.attend(q.numpy(), k.numpy(), v.numpy(), 0.125)
    kk, vv = (x.repeat_interleave(Hq // H, 1).transpose(0, 1) for x in (k, v))
    seen = torch.arange(L)[None] <= (L - n + torch.arange(n))[:, None]
    x = (q.transpose(0, 1) @ kk.transpose(1, 2) * 0.125).masked_fill(~seen, -torch.inf)
    live = seen.any(-1).numpy()
    ref = (torch.softmax(x, -1) @ vv).transpose(0, 1).numpy()
    assert np.allclose(out[live], ref[live], atol=1e-12) and np.all(out[~live] == 0)
    assert np.allclose(lse[live], torch.logsumexp(x, -1).T.numpy()[live]) and np.all(np.isneginf(lse[~live]))
    assert np.all(np.abs(out) <= mass + 1e-12)
