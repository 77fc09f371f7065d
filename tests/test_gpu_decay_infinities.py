"""Infinite states, values and keys through the decayed layer, by value and
sign against the float64 recurrence: S <- a S + k v^T and o = S^T q make an
infinity of an infinity, and a NaN only of 0 times one or of two of opposite
signs.  (Queries are positive here, and the infinities of a column have one
sign, so that the sums of the unrolled form and of the recurrence agree; no
factor a^n underflows.)"""
import numpy as np
import pytest
import torch

from hybrid_linear_attention_packed_gb300 import (span_la_check, span_la_decay_branches_from_state, span_la_decay_pass,
                                                  span_la_decay_step, workloads)
from oracle.decay_oracle import oracle_decay_pass, oracle_decay_step

pytestmark = pytest.mark.gpu

INF = float("inf")
DECAYS = np.float32([0.0, -0.004, -0.02, -0.05])


def _f64(t):
    return t.detach().double().cpu().numpy()


def _same_kinds(got, ref):
    for kind in (np.isposinf, np.isneginf, np.isnan):
        g, r = kind(got), kind(ref)
        assert np.array_equal(g, r), "%s: %d against %d elements, first at %s" % (
            kind.__name__, g.sum(), r.sum(), np.argwhere(g != r)[0])


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("ld", [None, 0.0, -0.004, -0.5, -0.9, -3.0, -INF])
def test_infinite_states_step_on(cuda_device, dtype, ld):
    H = 2
    g = torch.Generator(device=cuda_device).manual_seed(1)
    r = lambda *s: torch.randn(s, generator=g, device=cuda_device)  # noqa: E731
    q = (r(4, H, 64).abs() + 0.1).to(_dtype(dtype))
    k, v = r(4, H, 64).to(q.dtype), r(4, H, 64).to(q.dtype)
    states = r(4, H, 64, 64)
    states[0, 0, 3, 7] = INF
    states[1, 1, 5, :] = -INF
    states[2, 0, 9, 2], states[2, 1, 9, 2] = INF, float("nan")
    k[3, 0, 4] = INF                      # an infinite key: a row of the new state
    v[3, 1, 6] = -INF                     # an infinite value: a column, whose signs are the keys'
    k[3, 1] = k[3, 1].abs() + 0.1
    lds = None if ld is None else torch.full((H,), ld, device=cuda_device)
    S, ref_s = states.clone(), _f64(states)
    with np.errstate(invalid="ignore"):
        for _ in range(3):                # (the third token's state held an infinity from the second's)
            out = span_la_decay_step(q, k, v, S, lds)
            ref, ref_s = oracle_decay_step(_f64(q), _f64(k), _f64(v), np.full(H, 0.0 if ld is None else ld), ref_s, range(4))
            span_la_check()
            _same_kinds(_f64(S), ref_s)
            _same_kinds(_f64(out), ref)


LAYOUTS = {"heads": (4, [700, 130], [40, 300], [0, 1]), "one head over many SMs": (1, [3000], [200, 50], [0, 0])}


def _workload(layout, dtype, seed):
    H, views, branches, parent = LAYOUTS[layout]
    w = workloads.make_pass(views, branches, parent, H=H, dtype=dtype, seed=seed)
    w.q = w.q.abs() + 0.1
    return w, DECAYS[:H] if H > 1 else DECAYS[1:2]


def _compare(w, ld, dev):
    q, k, v = (x.to(dev) for x in (w.q, w.k, w.v))
    lds = torch.from_numpy(ld).to(dev)
    out, state = span_la_decay_pass(q, k, v, lds, w.view_cu, w.branch_cu, w.branch_parent)
    fork = span_la_decay_branches_from_state(state, q, k, v, lds, w.branch_cu, w.branch_parent)
    span_la_check()
    with np.errstate(invalid="ignore"):
        ref, ref_s = oracle_decay_pass(*(_f64(x) for x in (w.q, w.k, w.v)), ld, w.view_cu, w.branch_cu, w.branch_parent)
    _same_kinds(_f64(state), ref_s)
    _same_kinds(_f64(out), ref)
    lo = int(w.branch_cu[0])
    _same_kinds(_f64(fork)[lo:], ref[lo:])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", sorted(LAYOUTS))
def test_infinite_values_over_tiles_and_pieces(cuda_device, layout, dtype):
    w, ld = _workload(layout, dtype, 41)
    w.k = w.k.abs() + 0.1
    w.v[5, :, 3], w.v[5, :, 9] = INF, -INF
    w.v[int(w.view_cu[-1]) - 100, :, 1] = INF            # (in the last view, or the only one)
    w.v[int(w.branch_cu[1]) - 4, :, 20] = -INF           # (in the first branch)
    _compare(w, ld, cuda_device)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", sorted(LAYOUTS))
def test_infinite_keys_over_tiles_and_pieces(cuda_device, layout, dtype):
    """k_ti = inf: row i of the state, with v's signs; where v is 0, inf times 0."""
    w, ld = _workload(layout, dtype, 42)
    w.v = w.v.abs() + 0.1
    w.v[:, :, 40] *= -1
    w.k[5, :, 2] = INF
    w.v[5, :, 11] = 0
    w.k[int(w.view_cu[1]) - 1, 0, 17] = INF              # (in the first view's last row, whose factor is 1)
    _compare(w, ld, cuda_device)
