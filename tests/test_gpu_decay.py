"""Decayed packed passes against the float64 recurrence.

Tolerances, from the arithmetic.  Let A be the same sums over absolute values:
A_t = sum_j a^(t-j) sum_i |q_i k_i| |v|, an upper bound of every partial sum of
o_t, and n the rows the sum runs over.

* fp32: each of at most n + 64 additions, two factors and one product of a term
  round by 2^-24 of the partial sum, and a factor a^m is off by a few 2^-24:
  |error| <= (2 n + 128) 2^-24 A.
* bf16: every term of the sum passes one rounding to bf16 (2^-8 of it: the
  masked score of its own tile, or the state entering the tile), and the output
  is rounded once (2^-8 of it): |error| <= 2.02 * 2^-8 A + the fp32 part.  For
  random data these roundings are independent and each at most 2^-8 / sqrt(3) in
  the mean square, so the 2-norm of the error is also at most 5e-3 of the
  output's.
* states are fp32 in both: |error| <= (2 n + 128) 2^-24 A_S.
"""
import math
import threading

import numpy as np
import pytest
import torch

from hybrid_linear_attention_packed_gb300 import (SpanLAError, ViewStateCache, packed_positions, rope_inv_freq, span_la_check,
                                                  span_la_decay_branches_from_state, span_la_decay_pass, span_la_decay_step,
                                                  span_la_pass, span_la_qk_norm_rope, spanla, workloads)
from oracle.decay_oracle import oracle_decay_pass, oracle_norm_rope

pytestmark = pytest.mark.gpu

INF = float("inf")
U32, U16 = 2.0 ** -24, 2.0 ** -8


def _f64(t):
    return t.detach().double().cpu().numpy()


def _longest(view_cu, branch_cu, parent):
    v = np.diff(view_cu) if len(view_cu) > 1 else np.zeros(1)
    n = int(v.max(initial=0))
    for b in range(max(len(branch_cu) - 1, 0)):
        before = v[parent[b]] if len(view_cu) > 1 else 0
        n = max(n, int(before + branch_cu[b + 1] - branch_cu[b]))
    return n


def _check(w, ld, out, state, kept=None, extra=0):
    """out and state of the workload's pass against the oracle, within the bounds of the module's text."""
    q, k, v = (_f64(x) for x in (w.q, w.k, w.v))
    vcu = [] if kept is not None else w.view_cu
    ref, ref_s = oracle_decay_pass(q, k, v, ld, vcu, w.branch_cu, w.branch_parent, kept)
    absum, absum_s = oracle_decay_pass(abs(q), abs(k), abs(v), ld, vcu, w.branch_cu, w.branch_parent,
                                       None if kept is None else abs(kept))
    rows = ~np.isnan(ref[:, 0, 0])
    got = _f64(out)
    n = _longest(vcu, w.branch_cu, w.branch_parent) + extra
    part32 = (2 * n + 128) * U32
    tol = part32 if w.dtype == "f32" else 2.02 * U16 + part32
    err = abs(got[rows] - ref[rows])
    assert np.all(err <= tol * absum[rows] + 1e-30), float((err / (absum[rows] + 1e-30)).max() / tol)
    assert np.isnan(got[~rows]).all()          # rows in no segment: left as they were
    if rows.any() and w.dtype == "bf16" and rows.sum() > 32:
        assert np.linalg.norm(got[rows] - ref[rows]) <= 5e-3 * np.linalg.norm(ref[rows])
    if state is not None and state.numel():
        serr = abs(_f64(state) - ref_s)
        assert np.all(serr <= part32 * absum_s + 1e-30), float((serr / (absum_s + 1e-30)).max() / part32)


def _decays(H, kind):
    pool = {"slopes": [-(2.0 ** (-8.0 * (h + 1) / max(H, 2))) for h in range(H)],
            "weak": [-(2.0 ** -(6 + h)) for h in range(H)],
            "edges": [(0.0, -INF, -6.0, -90.0, -1e-6)[h % 5] for h in range(H)]}
    return np.asarray(pool[kind], dtype=np.float32)


def _put(w, dev):
    """Inputs on the device; rows in no segment hold NaN."""
    live = np.zeros(w.T, dtype=bool)
    for cu in (w.view_cu, w.branch_cu):
        if len(cu) > 1:
            live[cu[0]:cu[-1]] = True
    m = torch.from_numpy(~live).to(dev)
    ts = []
    for x in (w.q, w.k, w.v):
        x = x.to(dev).contiguous()
        x[m] = float("nan")
        ts.append(x)
    return ts


def _run(w, ld, dev, stream=None):
    q, k, v = _put(w, dev)
    out, state = span_la_decay_pass(q, k, v, torch.from_numpy(ld).to(dev), w.view_cu, w.branch_cu, w.branch_parent,
                                    out=torch.full_like(q, float("nan")), stream=stream)
    span_la_check(stream)
    return out, state


LAYOUTS = {
    "one row": ([1], [1], [0]),
    "empty view": ([0], [3, 0, 5], [0, 0, 0]),
    "no branches": ([129], [], []),
    "chunk ends": ([15, 16, 17, 1, 2], [16, 15, 17, 1], [0, 1, 2, 4]),
    "tile ends": ([127, 128, 129], [127, 128, 129, 1, 64, 63], [0, 1, 2, 2, 1, 0]),
    "siblings": ([70], [5] * 40, [0] * 40),
    "short and long branches": ([200, 0, 40], [30, 300, 7, 129, 260, 1], [0, 0, 2, 1, 2, 2]),
    "several pieces": ([900, 515], [700, 20], [1, 0]),
}


@pytest.mark.parametrize("kind", ["slopes", "weak", "edges"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("layout", sorted(LAYOUTS))
def test_pass_against_the_recurrence(cuda_device, layout, dtype, kind):
    views, branches, parent = LAYOUTS[layout]
    H = {"slopes": 3, "weak": 1, "edges": 5}[kind]
    w = workloads.make_pass(views, branches, parent, H=H, dtype=dtype, seed=11, lead_rows=3, mid_rows=2, tail_rows=5)
    out, state = _run(w, _decays(H, kind), cuda_device)
    _check(w, _decays(H, kind), out, state)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("H", [16, 24, 200])
def test_many_heads(cuda_device, H, dtype):
    w = workloads.make_pass([260, 30], [20, 140, 3], [0, 1, 1], H=H, dtype=dtype, seed=5)
    ld = _decays(H, "slopes")
    out, state = _run(w, ld, cuda_device)
    _check(w, ld, out, state)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_growing_heads_follow_the_formula(cuda_device, dtype):
    """A positive log decay (a state that grows) is computed as written."""
    w = workloads.make_pass([150], [40], [0], H=1, dtype=dtype, seed=6)
    ld = np.float32([0.02])
    out, state = _run(w, ld, cuda_device)
    _check(w, ld, out, state)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_slow_decay_keeps_its_factors_over_a_long_view(cuda_device, dtype):
    """a = exp(-2^-11), off by up to 2^-25 once rounded: a product of 2,048 rounded factors would leave the state
    6e-5 off, where the bound at the effective length 1 / (1 - a) gives (2 * 2048 + 128) 2^-24 = 2.5e-4 of the sum
    of absolute values but the mean-square error of independent roundings stays below sqrt(n) 2^-24 < 1e-5."""
    w = workloads.make_pass([6000], [10], [0], H=2, dtype=dtype, seed=7)
    ld = np.float32([-(2.0 ** -11), -(2.0 ** -11)])
    out, state = _run(w, ld, cuda_device)
    ref, ref_s = oracle_decay_pass(_f64(w.q), _f64(w.k), _f64(w.v), ld, w.view_cu, w.branch_cu, w.branch_parent)
    assert np.linalg.norm(_f64(state) - ref_s) <= 1e-5 * np.linalg.norm(ref_s)
    assert np.linalg.norm(_f64(out) - ref) <= (1e-5 if dtype == "f32" else 5e-3) * np.linalg.norm(ref)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_no_decay_agrees_with_the_undecayed_pass(cuda_device, dtype):
    w = workloads.make_pass([700, 90], [30, 200, 9], [0, 0, 1], H=4, dtype=dtype, seed=8)
    q, k, v = _put(w, cuda_device)
    out, state = span_la_decay_pass(q, k, v, torch.zeros(4, device=cuda_device), w.view_cu, w.branch_cu, w.branch_parent)
    ref, ref_state = span_la_pass(q, k, v, w.view_cu, w.branch_cu, w.branch_parent)
    span_la_check()
    # each side is within 5e-3 (bf16) of the result; fp32 inputs: the undecayed pass holds 1e-3
    assert torch.linalg.norm(out.double() - ref.double()) <= (1e-2 if dtype == "bf16" else 1e-3) * torch.linalg.norm(ref.double())
    assert torch.linalg.norm(state.double() - ref_state.double()) <= 1e-3 * torch.linalg.norm(ref_state.double())


def test_powers_of_two_are_exact(cuda_device):
    """a = 1/2 (log_decay rounded: 2^(n log2 a) is off by < 2^-22 n relative), one-hot k and v, q = e_c: o_t counts
    2^-(t-j) over the rows j that match, whose bf16 rounding is off by 2^-8 of it (one more for the score or state)."""
    rng = np.random.default_rng(9)
    T = 300
    kk, vv, qq = (rng.integers(0, 64, T) for _ in range(3))
    hot = lambda i: torch.nn.functional.one_hot(torch.from_numpy(i), 64).view(T, 1, 64).bfloat16()  # noqa: E731
    w = workloads.make_pass([T], [], [], H=1, dtype="bf16", seed=0)
    w.q, w.k, w.v = hot(qq), hot(kk), hot(vv)
    ld = np.float32([-math.log(2.0)])
    out, state = _run(w, ld, cuda_device)
    ref, ref_s = oracle_decay_pass(_f64(w.q), _f64(w.k), _f64(w.v), ld, w.view_cu, [], [])
    assert np.all(abs(_f64(out) - ref) <= (2.02 * U16 + 300 * 2.0 ** -22) * ref + 2.0 ** -126)
    assert np.all(abs(_f64(state) - ref_s) <= 300 * 2.0 ** -22 * ref_s + 2.0 ** -126)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_fork_from_kept_states(cuda_device, dtype):
    H = 4
    w = workloads.make_pass([], [5, 128, 0, 129, 700, 64, 64, 1], [2, 0, 0, 1, 2, 2, 2, 0], H=H, dtype=dtype, seed=12,
                            lead_rows=2, tail_rows=3)
    kept = torch.randn(3, H, 64, 64, generator=torch.Generator().manual_seed(1))
    ld = _decays(H, "slopes")
    q, k, v = _put(w, cuda_device)
    out = span_la_decay_branches_from_state(kept.to(cuda_device), q, k, v, torch.from_numpy(ld).to(cuda_device), w.branch_cu,
                                            w.branch_parent, out=torch.full_like(q, float("nan")))
    span_la_check()
    _check(w, ld, out, None, kept=_f64(kept))


@pytest.mark.parametrize("tiles", range(126, 134))
def test_a_branch_behind_a_branch_of_many_pieces(cuda_device, tiles):
    """One head and one kept state: a branch over some 64 SMs, and another whose first tile follows its last one on an SM.
    The first rows of the second come from the kept state, not from the first branch's."""
    w = workloads.make_pass([], [128 * tiles, 128 * (304 - tiles)], [0, 0], H=1, dtype="bf16", seed=17)
    kept = torch.randn(1, 1, 64, 64, generator=torch.Generator().manual_seed(2))
    ld = np.asarray([-1e-3], dtype=np.float32)
    q, k, v = _put(w, cuda_device)
    out = span_la_decay_branches_from_state(kept.to(cuda_device), q, k, v, torch.from_numpy(ld).to(cuda_device), w.branch_cu,
                                            w.branch_parent)
    span_la_check()
    lo = int(w.branch_cu[1])
    ref, _ = oracle_decay_pass(*(_f64(x[lo:lo + 128]) for x in (q, k, v)), ld, [], [0, 128], [0], _f64(kept))
    got = _f64(out[lo:lo + 128])
    assert np.linalg.norm(got - ref) <= 5e-3 * np.linalg.norm(ref)


@pytest.mark.parametrize("decay", [True, False])
def test_branches_behind_a_branch_of_many_pieces_in_a_pass(cuda_device, decay):
    """As above behind a view of one tile, with the first branch over some 128 SMs, decayed and not."""
    ld = np.asarray([-1e-3 if decay else 0.0], dtype=np.float32)
    for tiles in range(250, 264):
        w = workloads.make_pass([128], [128 * tiles, 128 * (303 - tiles)], [0, 0], H=1, dtype="bf16", seed=18)
        q, k, v = _put(w, cuda_device)
        args = (w.view_cu, w.branch_cu, w.branch_parent)
        if decay:
            out, _ = span_la_decay_pass(q, k, v, torch.from_numpy(ld).to(cuda_device), *args)
        else:
            out, _ = span_la_pass(q, k, v, *args)
        span_la_check()
        lo = int(w.branch_cu[1])
        both = [np.concatenate([_f64(x[:128]), _f64(x[lo:lo + 128])]) for x in (q, k, v)]
        ref, _ = oracle_decay_pass(*both, ld, [0, 128], [128, 256], [0])
        got = _f64(out[lo:lo + 128])
        assert np.linalg.norm(got - ref[128:]) <= 5e-3 * np.linalg.norm(ref[128:]), tiles


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_shards_from_a_pass_agree_with_its_branches(cuda_device, dtype):
    w = workloads.make_pass([1000], [40, 7, 90, 128, 33, 300, 64, 5], [0] * 8, H=3, dtype=dtype, seed=13)
    ld = torch.from_numpy(_decays(3, "slopes")).to(cuda_device)
    q, k, v = _put(w, cuda_device)
    out, state = span_la_decay_pass(q, k, v, ld, w.view_cu, w.branch_cu, w.branch_parent)
    shard = torch.full_like(q, float("nan"))
    for cu in workloads.shards(w, 3):
        span_la_decay_branches_from_state(state, q, k, v, ld, cu, [0] * (len(cu) - 1), out=shard)
    span_la_check()
    lo = int(w.branch_cu[0])
    a, b = out[lo:].double(), shard[lo:].double()
    assert not torch.isnan(shard[lo:]).any()
    # the same sums in another order, each rounded as the module's text says
    assert torch.linalg.norm(a - b) <= (2e-5 if dtype == "f32" else 1e-2) * torch.linalg.norm(a)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_siblings_do_not_see_one_another(cuda_device, dtype):
    """The other branches' rows do not change a branch's bits."""
    w = workloads.make_pass([300], [20, 30, 40], [0, 0, 0], H=2, dtype=dtype, seed=14)
    ld = _decays(2, "slopes")
    out, _ = _run(w, ld, cuda_device)
    lo, hi = int(w.branch_cu[1]), int(w.branch_cu[2])
    for x in (w.q, w.k, w.v):
        x[int(w.branch_cu[0]):lo] = 3.0
        x[hi:int(w.branch_cu[3])] = float("nan")
    again, _ = _run(w, ld, cuda_device)
    assert torch.equal(out[lo:hi], again[lo:hi])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_bits_do_not_depend_on_timing_or_stream(cuda_device, dtype):
    w = workloads.make_pass([2500, 300], [30] * 6 + [200], [0, 0, 1, 1, 0, 0, 1], H=16, dtype=dtype, seed=15)
    ld = torch.from_numpy(_decays(16, "slopes")).to(cuda_device)
    q, k, v = _put(w, cuda_device)
    flush = torch.empty(256 << 20, dtype=torch.uint8, device=cuda_device)
    ref, ref_s = span_la_decay_pass(q, k, v, ld, w.view_cu, w.branch_cu, w.branch_parent)
    side = torch.cuda.Stream(cuda_device)
    got = []
    for rep in range(12):
        if rep % 3 == 0:
            flush.fill_(rep)
        if rep % 3 == 1:
            side.wait_stream(torch.cuda.current_stream(cuda_device))
            with torch.cuda.stream(side):
                got.append(span_la_decay_pass(q, k, v, ld, w.view_cu, w.branch_cu, w.branch_parent, stream=side))
        else:
            got.append(span_la_decay_pass(q, k, v, ld, w.view_cu, w.branch_cu, w.branch_parent))
    torch.cuda.synchronize()
    span_la_check()
    for o, s in got:
        assert torch.equal(o, ref) and torch.equal(s, ref_s)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_graph_replays_and_eager_calls_between(cuda_device, dtype):
    """Two recorded passes, replayed in turn with an eager one between them and new contents in the buffers."""
    w = workloads.make_pass([600, 128], [30, 140], [0, 1], H=2, dtype=dtype, seed=16)
    ld = torch.from_numpy(_decays(2, "slopes")).to(cuda_device)
    q, k, v = _put(w, cuda_device)
    bufs = [tuple(torch.zeros_like(q) for _ in range(3)) for _ in range(2)]
    args = (w.view_cu, w.branch_cu, w.branch_parent)
    span_la_decay_pass(q, k, v, ld, *args)
    graphs = []
    for b in bufs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res = span_la_decay_pass(*b, ld, *args)
        graphs.append((g, res))
    for round_ in range(3):
        for (g, res), b in zip(graphs, bufs):
            scale = 1.0 + round_
            for dst, src in zip(b, (q, k, v)):
                dst.copy_(src)
            b[2].mul_(scale)
            g.replay()
            ref, ref_s = span_la_decay_pass(*b, ld, *args)
            span_la_check()
            assert torch.equal(res[0], ref) and torch.equal(res[1], ref_s)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_one_plan_on_many_streams_at_once(cuda_device, dtype):
    """Passes of one plan (which share its kept workspace) on eleven streams that nothing orders, each with inputs of its
    own, three rounds: more streams than the plan records readers for."""
    w = workloads.make_pass([1500, 700], [30] * 5 + [300], [0, 1, 0, 1, 1, 0], H=8, dtype=dtype, seed=21)
    ld = torch.from_numpy(_decays(8, "slopes")).to(cuda_device)
    q, k, v = _put(w, cuda_device)
    n = 11
    vs = [v * (1.0 + i) for i in range(n)]
    refs = [span_la_decay_pass(q, k, x, ld, w.view_cu, w.branch_cu, w.branch_parent) for x in vs]
    outs = [(torch.empty_like(q), torch.empty_like(refs[0][1])) for _ in range(n)]
    streams = [torch.cuda.Stream(cuda_device) for _ in range(n)]
    torch.cuda.synchronize()
    for _ in range(3):
        for i in range(n):
            span_la_decay_pass(q, k, vs[i], ld, w.view_cu, w.branch_cu, w.branch_parent, out=outs[i][0],
                               view_state_out=outs[i][1], stream=streams[i])
    torch.cuda.synchronize()
    span_la_check()
    for (o, s), (ro, rs) in zip(outs, refs):
        assert torch.equal(o, ro) and torch.equal(s, rs)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_plans_are_evicted_in_stream_order(cuda_device, dtype):
    """Forty layouts twice over, past the sixteen that the plan cache holds, on two streams without a synchronisation."""
    layouts = [([200 + 37 * i, 64], [20, 150 + i], [0, 1]) for i in range(40)]
    ws = [workloads.make_pass(*lay, H=2, dtype=dtype, seed=30 + i) for i, lay in enumerate(layouts)]
    ld = torch.from_numpy(_decays(2, "slopes")).to(cuda_device)
    ins = [_put(w, cuda_device) for w in ws]
    streams = [torch.cuda.Stream(cuda_device) for _ in range(2)]
    torch.cuda.synchronize()
    got = [[torch.empty_like(x[0]) for x in ins] for _ in range(2)]
    states = [[torch.empty(2, 2, 64, 64, device=cuda_device) for _ in ins] for _ in range(2)]
    for rep in range(2):
        for i, w in enumerate(ws):
            span_la_decay_pass(*ins[i], ld, w.view_cu, w.branch_cu, w.branch_parent, out=got[rep][i],
                               view_state_out=states[rep][i], stream=streams[(i + rep) % 2])
    torch.cuda.synchronize()
    span_la_check()
    for i, w in enumerate(ws):
        assert torch.equal(got[0][i], got[1][i]) and torch.equal(states[0][i], states[1][i])
        if i % 8 == 0:
            _check(w, _decays(2, "slopes"), got[0][i], states[0][i])


def test_branches_by_key_from_the_view_state_cache(cuda_device):
    w = workloads.make_pass([300, 900], [30, 7, 200, 64], [0, 1, 1, 0], H=4, dtype="bf16", seed=22)
    ld = torch.from_numpy(_decays(4, "slopes")).to(cuda_device)
    q, k, v = _put(w, cuda_device)
    _, states = span_la_decay_pass(q, k, v, ld, w.view_cu, None, None)
    keys = np.array([5, 2 ** 63 + 9], dtype=np.uint64)
    with ViewStateCache(4, 3) as cache:
        cache.put(keys, states)
        got = cache.branches(keys[w.branch_parent], q, k, v, w.branch_cu, log_decay=ld)
        ref = span_la_decay_branches_from_state(states, q, k, v, ld, w.branch_cu, w.branch_parent)
        span_la_check()
        lo = int(w.branch_cu[0])
        assert torch.equal(got[lo:], ref[lo:])
        with pytest.raises(SpanLAError, match="not cached"):
            cache.branches([5, 6, 5, 5], q, k, v, w.branch_cu, log_decay=ld)
        with pytest.raises(ValueError, match="log_decay"):
            cache.branches(keys[w.branch_parent], q, k, v, w.branch_cu, log_decay=ld[:2])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_masked_infinities_and_nans_stay_masked(cuda_device, dtype):
    """Rows after, and siblings beside: an infinite or NaN value (or key) of one row changes no earlier row and no
    other branch's bits; the rows that see it are not finite."""
    w = workloads.make_pass([200], [20, 30, 40], [0, 0, 0], H=2, dtype=dtype, seed=23)
    ld = np.float32([-0.01, -3.0])
    clean, _ = _run(w, ld, cuda_device)
    b1, b2 = int(w.branch_cu[1]), int(w.branch_cu[2])
    w.v[b1 + 10, 0, 7] = float("inf")
    w.v[b1 + 12, 1, :] = float("nan")
    w.k[b1 + 15, 0, :] = float("nan")
    w.v[150, 0, 3] = float("-inf")
    out, state = _run(w, ld, cuda_device)
    assert torch.equal(out[:150], clean[:150]) and torch.equal(out[150:, 1][:50], clean[150:, 1][:50])
    rest = [c for c in range(64) if c != 3]
    assert torch.equal(out[:b1, 0][:, rest], clean[:b1, 0][:, rest])        # the view and the first branch: column 3 only
    assert torch.equal(out[b2:, 0][:, rest], clean[b2:, 0][:, rest]) and torch.equal(out[b2:, 1], clean[b2:, 1])
    assert torch.equal(out[b1:b1 + 10, 0][:, rest], clean[b1:b1 + 10, 0][:, rest])
    assert torch.equal(out[b1:b1 + 12, 1], clean[b1:b1 + 12, 1]) and torch.isnan(out[b1 + 12, 1]).all()
    # the rows that see them: infinite by the unrolled sum, NaN by the recurrence, whose state then holds infinities of
    # both signs (k_i times one) that the output adds
    assert not torch.isfinite(out[150, 0, 3]) and not torch.isfinite(out[b1 + 10, 0, 7])
    assert not torch.isfinite(state[0, 0, :, 3]).any() and torch.isfinite(state[0, 0][:, rest]).all()


def test_allocation_failure_is_reported_and_nothing_written(cuda_device):
    w = workloads.make_pass([300], [20], [0], H=2, dtype="bf16", seed=17)
    ld = torch.from_numpy(_decays(2, "slopes")).to(cuda_device)
    q, k, v = _put(w, cuda_device)
    out = torch.full_like(q, float("nan"))
    state = torch.full((1, 2, 64, 64), float("nan"), device=cuda_device)
    spanla.fault_inject(spanla.FAULT_ALLOC, 1)
    try:
        with pytest.raises(SpanLAError) as ei:
            span_la_decay_pass(q, k, v, ld, w.view_cu, w.branch_cu, w.branch_parent, out=out, view_state_out=state)
        assert ei.value.status == 4
    finally:
        spanla.fault_inject(spanla.FAULT_ALLOC, 0)
    torch.cuda.synchronize()
    assert torch.isnan(out).all() and torch.isnan(state).all()
    span_la_decay_pass(q, k, v, ld, w.view_cu, w.branch_cu, w.branch_parent, out=out, view_state_out=state)
    span_la_check()
    _check(w, _decays(2, "slopes"), out, state)


def test_nan_of_one_head_stays_in_it(cuda_device):
    w = workloads.make_pass([200], [20], [0], H=3, dtype="bf16", seed=18)
    w.k[150, 1, 5] = float("nan")
    w.v[10, 2, 3] = float("inf")
    ld = _decays(3, "slopes")
    out, state = _run(w, ld, cuda_device)
    assert torch.isfinite(out[:, 0]).all() and torch.isfinite(state[0, 0]).all()
    assert torch.isfinite(out[:150, 1]).all() and torch.isnan(out[150:, 1]).any() and torch.isnan(state[0, 1]).any()
    # an infinite value stays in its own dimension and in later rows
    assert torch.isfinite(out[:10, 2]).all() and torch.isfinite(out[:, 2, [0, 1, 2] + list(range(4, 64))]).all()


def test_offsets_past_2_31_elements(cuda_device):
    """A pass whose last view lies past element 2^31 of every array."""
    H, rows = 16, 2_200_000
    if torch.cuda.get_device_properties(cuda_device).total_memory < 60 << 30:
        pytest.skip("needs 60 GB of device memory")
    q, k, v = workloads.draw_qkv_device(3, rows, H, cuda_device)
    view_cu = [0, 50, rows - 400, rows - 100]
    branch_cu = [rows - 100, rows - 60, rows]
    ld = _decays(H, "slopes")
    out, state = span_la_decay_pass(q, k, v, torch.from_numpy(ld).to(cuda_device), view_cu, branch_cu, [2, 2])
    span_la_check()
    lo = rows - 400
    w = workloads.make_pass([300], [40, 60], [0, 0], H=H, dtype="bf16", seed=0)
    w.q, w.k, w.v = (x[lo:].cpu() for x in (q, k, v))
    _check(w, ld, out[lo:], state[2:3])
    # the long view's last rows, from the rows that its slowest head (a = exp(-2^-8)) remembers past 1e-12
    m = 7000
    x = [t[lo - m:lo].cpu() for t in (q, k, v)]
    w2 = workloads.make_pass([m], [], [], H=H, dtype="bf16", seed=0)
    w2.q, w2.k, w2.v = x
    ref, ref_s = oracle_decay_pass(*(_f64(t) for t in x), ld, w2.view_cu, [], [])
    got = _f64(out[lo - 64:lo])
    assert np.linalg.norm(got - ref[-64:]) <= 5e-3 * np.linalg.norm(ref[-64:])
    assert np.linalg.norm(_f64(state[1]) - ref_s[0]) <= 1e-5 * np.linalg.norm(ref_s[0])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_layer_from_projection_to_next_tokens(cuda_device, dtype):
    """q and k of a fused projection, normed and rotated; the packed pass; then each view's next tokens one at a time:
    the same as a pass over the longer views."""
    H, lens, extra = 4, [150, 37], 5
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    T = sum(lens) + len(lens) * extra
    g = torch.Generator(device=cuda_device).manual_seed(4)
    rows = torch.randn(T, 3 * H * 64, generator=g, device=cuda_device).to(dt)
    v = rows[:, 2 * H * 64:].reshape(T, H, 64).contiguous()
    wq, wk = (1 + 0.1 * torch.randn(64, generator=g, device=cuda_device) for _ in range(2))
    # whole views, their new tokens in place
    cu = np.concatenate([[0], np.cumsum([n + extra for n in lens])]).astype(np.int32)
    pos_host = packed_positions(cu, None, None, T)
    pos = torch.from_numpy(pos_host).to(cuda_device)
    freq = rope_inv_freq(32)
    q, k = span_la_qk_norm_rope(rows[:, :H * 64].view(T, H, 64), rows[:, H * 64:2 * H * 64].view(T, H, 64), pos, freq, wq, wk)
    q, k = q / 8, k / 8
    ld = torch.from_numpy(_decays(H, "slopes")).to(cuda_device)
    whole, final = span_la_decay_pass(q, k, v, ld, cu, None, None)
    qn = oracle_norm_rope(_f64(rows[:, :H * 64].view(T, H, 64)), _f64(wq), pos_host, freq, 1e-6, False)
    assert np.linalg.norm(_f64(q) * 8 - qn) <= (1e-6 if dtype == "f32" else 3e-3) * np.linalg.norm(qn)
    # the prompts alone, then tokens
    parts = [np.arange(cu[s], cu[s] + n) for s, n in enumerate(lens)]
    idx = torch.from_numpy(np.concatenate(parts)).to(cuda_device)
    pcu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    _, states = span_la_decay_pass(q[idx].contiguous(), k[idx].contiguous(), v[idx].contiguous(), ld, pcu, None, None)
    for j in range(extra):
        at = torch.tensor([cu[s] + n + j for s, n in enumerate(lens)], device=cuda_device)
        out = span_la_decay_step(q[at].contiguous(), k[at].contiguous(), v[at].contiguous(), states, ld, state_index=[0, 1])
        a, b = out.double(), whole[at].double()
        assert torch.linalg.norm(a - b) <= (2e-5 if dtype == "f32" else 1e-2) * torch.linalg.norm(b)
    span_la_check()
    assert torch.linalg.norm(states.double() - final.double()) <= 1e-5 * torch.linalg.norm(final.double())


def test_calls_from_several_host_threads(cuda_device):
    """Four host threads, each on a stream of its own, with plans that they share: the results of one call after another."""
    ws = [workloads.make_pass([900, 300], [60, 5, 200], [0, 1, 0], H=3, dtype=d, seed=31) for d in ("bf16", "f32")]
    ws += [workloads.make_pass([2000], [40] * 6, [0] * 6, H=4, dtype=d, seed=32) for d in ("bf16", "f32")]
    args = []
    for w in ws:
        q, k, v = (x.to(cuda_device) for x in (w.q, w.k, w.v))
        args.append((q, k, v, torch.from_numpy(_decays(q.shape[1], "slopes")).to(cuda_device), w.view_cu, w.branch_cu,
                     w.branch_parent))
    want = [span_la_decay_pass(*a) for a in args]
    torch.cuda.synchronize()
    wrong = []

    def work(t):
        try:
            torch.cuda.set_device(cuda_device)
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                for i in range(40):
                    j = (i + t) % len(args)
                    out, state = span_la_decay_pass(*args[j])
                    if not (torch.equal(out, want[j][0]) and torch.equal(state, want[j][1])):
                        wrong.append((t, i, j))
        except Exception as e:   # noqa: BLE001 (a thread's exception would be lost)
            wrong.append(repr(e))

    threads = [threading.Thread(target=work, args=(t,)) for t in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    span_la_check()
    assert wrong == []
