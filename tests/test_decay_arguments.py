"""Arguments of the decayed calls and the q/k norm and rotation that have to be
refused on the host (CPU): outputs over the small arrays that a kernel reads
while it writes them, and offsets that do not fit 32 bits."""
import numpy as np
import pytest

from hybrid_linear_attention_packed_gb300 import build as spanla_build
from hybrid_linear_attention_packed_gb300 import spanla

INVALID = 1
A, OUT, STATES, SMALL = (1 << 20) * np.array([1, 16, 64, 256])   # addresses, never dereferenced on the host


@pytest.fixture(scope="module")
def lib():
    return spanla.load_library(spanla_build.build())


def _i32(a):
    a = np.ascontiguousarray(np.asarray(a, dtype=np.int32))
    return a, a.ctypes.data


def _detail(lib, st):
    assert st == INVALID
    return lib.span_la_last_error_detail().decode()


# [100][2][64] bf16: 25,600 bytes; states of two heads: 32,768 each
@pytest.mark.parametrize("ld", [OUT, OUT + 25_600 - 4, OUT - 4, STATES, STATES + 32_768 - 4])
def test_pass_refuses_log_decay_in_its_outputs(lib, ld):
    (v, vp), (b, bp), (p, pp) = _i32([0, 50]), _i32([50, 60]), _i32([0])
    st = lib.span_la_decay_pass(int(A), int(A), int(A), spanla.Dims(100, 2, 64, 0), int(ld), vp, 1, bp, 1, pp, int(OUT),
                                int(STATES), None)
    assert "log_decay" in _detail(lib, st)


@pytest.mark.parametrize("ld", [OUT, OUT + 25_600 - 4])
def test_fork_refuses_log_decay_in_its_output(lib, ld):
    (b, bp), (p, pp) = _i32([50, 60]), _i32([0])
    st = lib.span_la_decay_branches_from_state(int(STATES), 1, int(A), int(A), int(A), spanla.Dims(100, 2, 64, 0), int(ld), bp,
                                               1, pp, int(OUT), None)
    assert "log_decay" in _detail(lib, st)


@pytest.mark.parametrize("ld", [OUT, STATES, STATES + 8 * 32_768 - 8])
def test_step_refuses_log_decay_in_what_it_writes(lib, ld):
    st = lib.span_la_decay_step(int(A), int(A), int(A), spanla.Dims(3, 2, 64, 0), int(ld), int(STATES), 8, None, int(OUT), None)
    assert "log_decay" in _detail(lib, st)


# q out: ten rows of 256 bytes, 512 bytes apart; k out: ten rows of 128 bytes one behind the other
@pytest.mark.parametrize("weight,pos,what", [
    (SMALL, OUT, "positions"), (SMALL, OUT + 9 * 512 + 252, "positions"), (SMALL, STATES + 10 * 128 - 4, "positions"),
    (OUT + 512, SMALL, "weight"), (STATES, SMALL, "weight"),
])
def test_norm_rope_refuses_outputs_over_what_it_reads(lib, weight, pos, what):
    q = spanla.QkSide(int(A), int(OUT), int(weight), 128, 256, 2, 0)
    k = spanla.QkSide(int(4 * A), int(STATES), None, 64, 64, 1, 0)
    f = np.ones(32)
    st = lib.span_la_qk_norm_rope(q, k, 10, 0, 0, 1e-6, f.ctypes.data, 64, 0, int(pos), None)
    assert what in _detail(lib, st)


@pytest.mark.parametrize("bad", [[0, 2 ** 32], [0, 2 ** 31], [-2 ** 31 - 1, 4], np.array([0, 2 ** 32 + 4]),
                                 np.array([0, 2 ** 64 - 1], dtype=np.uint64), [0, 2 ** 70]])
def test_offsets_that_do_not_fit_32_bits_are_refused(lib, bad):
    """(Cut to 32 bits, 2^32 would be 0 and 2^32 + 4 would be 4.)"""
    with pytest.raises(ValueError, match="32 bits"):
        spanla.packed_positions(bad, None, None, 8)
    with pytest.raises(ValueError, match="32 bits"):
        spanla.plan_stats(bad, None, None, 1)


def test_offsets_that_fit_are_taken_as_before(lib):
    for cu in ([0, 4], np.array([0, 4], dtype=np.uint8), (0, 4), np.array([[0], [4]]), np.array([0.0, 4.0])):
        assert spanla.packed_positions(cu, None, None, 5).tolist() == [0, 1, 2, 3, -1]
    assert spanla._i32([]).size == 0 and spanla._i32([-2 ** 31, 2 ** 31 - 1]).tolist() == [-2 ** 31, 2 ** 31 - 1]


@pytest.mark.parametrize("cu", [[2 ** 31 - 1, -5], [3, 2 ** 31 - 1, -2 ** 31 + 1, 4]])
def test_offsets_whose_differences_wrap_are_refused(cu):
    with pytest.raises(ValueError, match="non-decreasing"):
        spanla.packed_positions(cu, None, None, 8)
