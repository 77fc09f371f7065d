"""Refusals of the decayed passes, the single-token step and the q/k norm and
rotation: every problem is reported by the host before any CUDA call (CPU)."""
import ctypes

import numpy as np
import pytest
import torch

from hybrid_linear_attention_packed_gb300 import build as spanla_build
from hybrid_linear_attention_packed_gb300 import spanla

FAKE = 1 << 20   # an aligned non-NULL address; never dereferenced on the host
INVALID, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def lib():
    return spanla.load_library(spanla_build.build())


def _i32(a):
    a = np.ascontiguousarray(np.asarray(a, dtype=np.int32))
    return a, (a.ctypes.data if a.size else None)


OUT = FAKE * 16


def _pass(lib, vcu=(0, 50), bcu=(50, 60), par=(0,), T=100, H=2, D=64, dtype=0, q=FAKE, out=OUT, state=FAKE, ld=FAKE):
    (va, vp), (ba, bp), (pa, pp) = _i32(vcu), _i32(bcu), _i32(par)
    st = lib.span_la_decay_pass(q, q, q, spanla.Dims(T, H, D, dtype), ld, vp, max(len(va) - 1, 0), bp,
                                max(len(ba) - 1, 0), pp, out, state, None)
    return st, lib.span_la_last_error_detail().decode()


@pytest.mark.parametrize("kw,status,what", [
    (dict(vcu=(0, 50, 40)), INVALID, "non-decreasing"),
    (dict(vcu=(0, 101)), INVALID, "non-decreasing"),
    (dict(vcu=(-1, 10)), INVALID, "non-decreasing"),
    (dict(bcu=(40, 60)), INVALID, "overlap"),
    (dict(par=(1,)), INVALID, "branch_parent"),
    (dict(par=(-1,)), INVALID, "branch_parent"),
    (dict(D=128), UNSUPPORTED, "head_dim"),
    (dict(dtype=3), UNSUPPORTED, "dtype"),
    (dict(H=0), INVALID, "num_heads"),
    (dict(T=-1, vcu=(), bcu=(), par=()), INVALID, "total_rows"),
    (dict(q=None), INVALID, "non-NULL"),
    (dict(q=FAKE + 8), INVALID, "aligned"),
    (dict(out=None), INVALID, "non-NULL"),
    (dict(out=FAKE), INVALID, "out overlaps"),
    (dict(out=FAKE + 100 * 2 * 64 * 2 - 16), INVALID, "out overlaps"),
    (dict(state=None), INVALID, "view_state_out"),
    (dict(state=FAKE + 4), INVALID, "view_state_out"),
    (dict(ld=None), INVALID, "log_decay"),
    (dict(ld=FAKE + 2), INVALID, "log_decay"),
    (dict(H=65536), INVALID, "num_heads"),
])
def test_pass_refuses(lib, kw, status, what):
    st, detail = _pass(lib, **kw)
    assert st == status and what in detail


def test_nothing_to_do_needs_no_device(lib):
    assert _pass(lib, vcu=(), bcu=(), par=())[0] == 0
    _, bp = _i32([0, 0])
    _, pp = _i32([0])
    assert lib.span_la_decay_branches_from_state(FAKE, 1, None, None, None, spanla.Dims(0, 2, 64, 0), FAKE, bp, 1, pp,
                                                 None, None) == 0
    assert lib.span_la_decay_step(None, None, None, spanla.Dims(0, 2, 64, 0), None, None, 0, None, None, None) == 0


def _fork(lib, bcu=(0, 10), par=(0,), n=1, kept=FAKE, ld=FAKE, q=FAKE, out=OUT):
    (ba, bp), (pa, pp) = _i32(bcu), _i32(par)
    st = lib.span_la_decay_branches_from_state(kept, n, q, q, q, spanla.Dims(10, 2, 64, 0), ld, bp, len(ba) - 1, pp, out,
                                               None)
    return st, lib.span_la_last_error_detail().decode()


@pytest.mark.parametrize("kw,what", [
    (dict(bcu=(0, 11)), "non-decreasing"), (dict(par=(1,)), "branch_parent"), (dict(n=-1), "num_states"),
    (dict(kept=None), "cached_state"), (dict(kept=FAKE + 8), "cached_state"), (dict(ld=None), "log_decay"),
    (dict(q=None), "non-NULL"), (dict(out=FAKE + 64), "out overlaps"),
])
def test_fork_refuses(lib, kw, what):
    st, detail = _fork(lib, **kw)
    assert st == INVALID and what in detail


def _step(lib, n=3, H=2, D=64, dtype=0, q=FAKE, ld=FAKE, states=FAKE, num=8, index=(0, 5, 7), out=OUT):
    (ia, ip) = _i32(index if index is not None else [])
    st = lib.span_la_decay_step(q, q, q, spanla.Dims(n, H, D, dtype), ld, states, num, ip, out, None)
    return st, lib.span_la_last_error_detail().decode()


@pytest.mark.parametrize("kw,status,what", [
    (dict(index=(0, 5, 5)), INVALID, "twice"),
    (dict(index=(7, -1, 7)), INVALID, "twice"),
    (dict(index=(9000, 3, 9000), num=10000), INVALID, "twice"),
    (dict(index=(0, 8, 1)), INVALID, "state_index[1]"),
    (dict(index=(0, 1, -2)), INVALID, "state_index[2]"),
    (dict(index=None, num=2), INVALID, "as many states"),
    (dict(num=-1), INVALID, "num_states"),
    (dict(states=None), INVALID, "states"),
    (dict(states=FAKE + 4), INVALID, "states"),
    (dict(q=None), INVALID, "non-NULL"),
    (dict(out=FAKE + 2), INVALID, "aligned"),
    (dict(out=FAKE), INVALID, "out overlaps"),
    (dict(ld=FAKE + 1), INVALID, "log_decay"),
    (dict(D=32), UNSUPPORTED, "head_dim"),
    (dict(dtype=9), UNSUPPORTED, "dtype"),
    (dict(H=70000), INVALID, "num_heads"),
])
def test_step_refuses(lib, kw, status, what):
    st, detail = _step(lib, **kw)
    assert st == status and what in detail


def _side(in_=FAKE, out=FAKE * 16, weight=None, s_in=128, s_out=128, heads=2, per_head=0):
    return spanla.QkSide(in_, out, weight, s_in, s_out, heads, per_head)


def _rope(lib, q=None, k=None, rows=10, dtype=0, wdt=0, eps=1e-6, rotary=64, freq=True, pos=FAKE):
    f = np.ones(32) if freq is True else freq
    q = q or _side()
    k = k or _side(in_=FAKE * 64, out=FAKE * 128)
    st = lib.span_la_qk_norm_rope(q, k, rows, dtype, wdt, eps, f.ctypes.data if f is not None else None, rotary, 0, pos, None)
    return st, lib.span_la_last_error_detail().decode()


@pytest.mark.parametrize("kw,status,what", [
    (dict(dtype=2), UNSUPPORTED, "dtype"),
    (dict(wdt=2), UNSUPPORTED, "weight_dtype"),
    (dict(rows=-1), INVALID, "rows"),
    (dict(rotary=20), UNSUPPORTED, "rotary_dim"),
    (dict(rotary=80), UNSUPPORTED, "rotary_dim"),
    (dict(rotary=-16), UNSUPPORTED, "rotary_dim"),
    (dict(eps=-1.0), INVALID, "eps"),
    (dict(eps=float("nan")), INVALID, "eps"),
    (dict(freq=None), INVALID, "inv_freq"),
    (dict(freq=np.full(32, np.inf)), INVALID, "inv_freq[0]"),
    (dict(pos=None), INVALID, "positions"),
    (dict(pos=FAKE + 2), INVALID, "positions"),
    (dict(q=_side(in_=None)), INVALID, "q: in and out"),
    (dict(k=_side(out=FAKE + 8)), INVALID, "k: in and out"),
    (dict(q=_side(s_in=100)), INVALID, "row strides"),
    (dict(q=_side(s_out=132)), INVALID, "row strides"),
    (dict(q=_side(heads=-1)), INVALID, "num_heads"),
    (dict(q=_side(weight=FAKE + 1)), INVALID, "weight"),
    (dict(q=_side(out=FAKE + 256)), INVALID, "without being the same array"),
    (dict(q=_side(out=FAKE, s_out=256)), INVALID, "without being the same array"),
    (dict(q=_side(out=FAKE * 64)), INVALID, "q's out overlaps k's in"),
    (dict(k=_side(in_=FAKE * 64, out=FAKE * 16 + 128)), INVALID, "q's out overlaps k's out"),
])
def test_norm_rope_refuses(lib, kw, status, what):
    st, detail = _rope(lib, **kw)
    assert st == status and what in detail


def test_norm_rope_without_rows_or_heads_needs_no_device(lib):
    assert _rope(lib, rows=0)[0] == 0
    assert _rope(lib, q=_side(heads=0, in_=None, out=None), k=_side(heads=0, in_=None, out=None))[0] == 0


def test_binding_refuses_cpu_tensors_and_shapes(lib):
    x = torch.zeros(4, 2, 64)
    ld = torch.zeros(2)
    with pytest.raises(ValueError, match="CUDA"):
        spanla.span_la_decay_pass(x, x, x, ld, [0, 4], None, None)
    with pytest.raises(ValueError, match="CUDA"):
        spanla.span_la_decay_step(x, x, x, torch.zeros(4, 2, 64, 64), ld)
    with pytest.raises(ValueError, match="CUDA"):
        spanla.span_la_qk_norm_rope(x, x, torch.zeros(4, dtype=torch.int32), None)
    with pytest.raises(ValueError, match="dtype"):
        spanla.span_la_qk_norm_rope(x.half(), x.half(), torch.zeros(4, dtype=torch.int32), None)


def test_states_that_overlap_other_arguments(lib):
    st, detail = _pass(lib, state=OUT + 64)
    assert st == INVALID and "view_state_out overlaps out" in detail
    st, detail = _pass(lib, state=FAKE + 16)
    assert st == INVALID and "view_state_out overlaps q, k or v" in detail
    st, detail = _fork(lib, kept=OUT - 16)
    assert st == INVALID and "cached_state overlaps out" in detail
    st, detail = _step(lib, states=OUT)
    assert st == INVALID and "states overlaps out" in detail
    st, detail = _step(lib, states=FAKE)
    assert st == INVALID and "states overlaps q, k or v" in detail


@pytest.mark.parametrize("args", [
    ([0, 4], [4, 6], [1], 8), ([0, 4], [4, 6], [-1], 8), ([0, 4], [4, 6], [], 8), ([0, 4], None, [0], 8),
    ([0, 4], [4, 9], [0], 8), ([-1, 4], None, None, 8), ([0, 4, 3], None, None, 8), (None, [0, 2], [0], 8),
])
def test_packed_positions_refuses(args):
    with pytest.raises(ValueError):
        spanla.packed_positions(*args)


def test_packed_positions():
    pos = spanla.packed_positions([1, 4, 4], [4, 6, 6, 7], [0, 0, 1], 9)
    assert pos.dtype == np.int32 and pos.tolist() == [-1, 0, 1, 2, 3, 4, 0, -1, -1]
