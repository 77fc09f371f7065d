"""Decayed fp32 passes past 2^31 elements, and fp32 branches by cache key."""
import numpy as np
import pytest
import torch

from hybrid_linear_attention_packed_gb300 import (ViewStateCache, span_la_check, span_la_decay_branches_from_state,
                                                  span_la_decay_pass, workloads)
from oracle.decay_oracle import oracle_decay_pass

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24


def _f64(t):
    return t.detach().double().cpu().numpy()


def test_fp32_offsets_past_2_31_elements(cuda_device):
    """A view that crosses element 2^31 of every array, and a view and branches behind it.  Rows are compared within
    (2 n + 128) 2^-24 of the sum of absolute values over the n rows that a state remembers: with a = exp(-1/32) and
    less, a row 2,000 back counts e^-62."""
    H, rows = 16, 2_200_000
    if torch.cuda.get_device_properties(cuda_device).total_memory < 100 << 30:
        pytest.skip("needs 100 GB of device memory")
    g = torch.Generator(device=cuda_device).manual_seed(71)
    q, k, v = (torch.randn(rows, H, 64, generator=g, device=cuda_device) for _ in range(3))
    ld = np.float32([-(2.0 ** -(5 - h % 5)) for h in range(H)])
    vcu, bcu = [0, 50, rows - 400, rows - 100], [rows - 100, rows - 60, rows]
    out, state = span_la_decay_pass(q, k, v, torch.from_numpy(ld).to(cuda_device), vcu, bcu, [2, 1])
    span_la_check()
    m = 2000
    lo = rows - 400 - m                                  # the long view's last m rows, its states from zero before them
    x = [_f64(t[lo:]) for t in (q, k, v)]
    cu = np.array([0, m, m + 300], dtype=np.int32)
    bc = np.array([m + 300, m + 340, m + 400], dtype=np.int32)
    ref, ref_s = oracle_decay_pass(*x, ld, cu, bc, [1, 0])
    size, size_s = oracle_decay_pass(*(abs(t) for t in x), ld, cu, bc, [1, 0])
    tol = (2 * (m + 60) + 128) * U32
    got = _f64(out[lo:])
    live = slice(m - 64, None)                           # (the rows before remember less than they did)
    assert np.all(abs(got[live] - ref[live]) <= tol * size[live])
    assert np.all(abs(_f64(state[1:]) - ref_s) <= tol * size_s)
    across = (1 << 31) // (H * 64)                       # the row that holds element 2^31
    lo = across + 32 - m
    x = [_f64(t[lo:across + 32]) for t in (q, k, v)]
    ref, _ = oracle_decay_pass(*x, ld, [0, m], [], [])
    size, _ = oracle_decay_pass(*(abs(t) for t in x), ld, [0, m], [], [])
    assert np.all(abs(_f64(out[across - 32:across + 32]) - ref[-64:]) <= tol * size[-64:])


def test_fp32_branches_by_key(cuda_device):
    w = workloads.make_pass([300, 900], [30, 7, 200, 64], [0, 1, 1, 0], H=3, dtype="f32", seed=72)
    q, k, v = (x.to(cuda_device) for x in (w.q, w.k, w.v))
    ld = np.float32([-0.01, -0.5, 0.0])
    lds = torch.from_numpy(ld).to(cuda_device)
    _, states = span_la_decay_pass(q, k, v, lds, w.view_cu, None, None)
    keys = np.array([9, 2 ** 63 + 1], dtype=np.uint64)
    with ViewStateCache(3, 2) as cache:
        cache.put(keys, states)
        got = cache.branches(keys[w.branch_parent], q, k, v, w.branch_cu, log_decay=lds)
        ref = span_la_decay_branches_from_state(states, q, k, v, lds, w.branch_cu, w.branch_parent)
        span_la_check()
    lo = int(w.branch_cu[0])
    assert torch.equal(got[lo:], ref[lo:])
    x = [_f64(t) for t in (w.q, w.k, w.v)]
    want, _ = oracle_decay_pass(*x, ld, w.view_cu, w.branch_cu, w.branch_parent)
    size, _ = oracle_decay_pass(*(abs(t) for t in x), ld, w.view_cu, w.branch_cu, w.branch_parent)
    assert np.all(abs(_f64(got)[lo:] - want[lo:]) <= (2 * 1100 + 128) * U32 * size[lo:])
