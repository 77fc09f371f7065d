"""The float64 forms the decayed kernels are compared with, against closed forms (CPU)."""
import numpy as np
import pytest

from hybrid_linear_attention_packed_gb300 import packed_positions, rope_inv_freq
from oracle import oracle_pass
from oracle.decay_oracle import oracle_decay_pass, oracle_decay_step, oracle_norm_rope


def _draw(T, H, seed):
    rng = np.random.default_rng(seed)
    return rng.standard_normal((3, T, H, 64))


def test_no_decay_is_the_undecayed_pass():
    q, k, v = _draw(60, 2, 0)
    vcu, bcu, par = [0, 20, 31], [31, 40, 60], [1, 0]
    out, st = oracle_decay_pass(q, k, v, [0.0, 0.0], vcu, bcu, par)
    ref, ref_st = oracle_pass(q, k, v, np.int32(vcu), np.int32(bcu), np.int32(par))
    assert np.allclose(out, ref, rtol=0, atol=1e-11) and np.allclose(st, ref_st, rtol=0, atol=1e-11)


@pytest.mark.parametrize("ld", [-1e-3, -0.7, -5.0, -np.inf])
def test_recurrence_is_the_unrolled_sum(ld):
    q, k, v = _draw(25, 1, 1)
    out, st = oracle_decay_pass(q, k, v, [ld], [0, 25], [], [])
    for t in range(25):
        o = sum(np.exp(ld * (t - j) if j < t else 0.0) * (q[t, 0] @ k[j, 0]) * v[j, 0] for j in range(t + 1))
        assert np.allclose(out[t, 0], o, rtol=0, atol=1e-12 * 64)
    w = np.exp(np.array([ld * (24 - j) if j < 24 else 0.0 for j in range(25)]))
    assert np.allclose(st[0, 0], (k[:, 0] * w[:, None]).T @ v[:, 0], rtol=0, atol=1e-11)


def test_steps_continue_a_pass_and_branches_continue_their_view():
    q, k, v = _draw(30, 3, 2)
    ld = np.array([-0.01, -1.0, 0.0])
    whole, final = oracle_decay_pass(q, k, v, ld, [0, 30], [], [])
    part, st = oracle_decay_pass(q, k, v, ld, [0, 18], [18, 30], [0])
    assert np.allclose(part, whole, rtol=0, atol=1e-12)
    S = st
    for t in range(18, 30):
        o, S = oracle_decay_step(q[t:t + 1], k[t:t + 1], v[t:t + 1], ld, S, [0])
        assert np.allclose(o[0], whole[t], rtol=0, atol=1e-12)
    assert np.allclose(S, final, rtol=0, atol=1e-12)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_norms_and_depends_on_distance(interleaved):
    rng = np.random.default_rng(3)
    x = rng.standard_normal((2, 1, 64))
    f = rope_inv_freq(32)
    at = lambda p0, p1: oracle_norm_rope(x, None, [p0, p1], f, 0.0, interleaved)  # noqa: E731
    a, b = at(5, 9), at(105, 109)
    assert np.allclose((a ** 2).mean(-1), 1.0) and np.isclose((a[0] * a[1]).sum(), (b[0] * b[1]).sum())
    assert np.allclose(at(0, 0)[..., 32:], a[..., 32:])   # past rotary_dim: norm only


def test_packed_positions():
    pos = packed_positions([1, 4, 6], [6, 8, 9], [1, 0], 11)
    assert pos.tolist() == [-1, 0, 1, 2, 0, 1, 2, 3, 3, -1, -1]
    assert packed_positions(None, None, None, 2).tolist() == [-1, -1]
