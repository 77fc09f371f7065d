"""Attention over the paged cache with NaN and infinities in queries, keys and values."""
import numpy as np
import pytest
import torch

from paged_helpers import BF16, E4M3, f64
from test_gpu_paged_attention import _run, _setup

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
