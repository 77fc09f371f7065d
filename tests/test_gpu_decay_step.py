"""The single-token step against the float64 recurrence.

Bounds: a state element is a S + k v: the factor and the two operations round by
2^-24 each (factor: a few), 6 * 2^-24 of |a S| + |k v|; an output sums 64 of
them, (64 + 8) * 2^-24 of the sum of absolute values, plus 2^-8 of the output
for its rounding to bf16."""
import numpy as np
import pytest
import torch

from hybrid_linear_attention_packed_gb300 import span_la_check, span_la_decay_step, span_la_pass, workloads
from oracle.decay_oracle import oracle_decay_step

pytestmark = pytest.mark.gpu

INF = float("inf")
U32, U16 = 2.0 ** -24, 2.0 ** -8


def _f64(t):
    return t.detach().double().cpu().numpy()


def _draw(n, H, pool, dtype, dev, seed=0):
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    r = lambda *s: torch.randn(s, generator=g, device=dev)  # noqa: E731
    ld = torch.tensor([(0.0, -0.004, -0.5, -INF, -7.0)[h % 5] for h in range(H)], device=dev)
    return r(n, H, 64).to(dt), r(n, H, 64).to(dt), r(n, H, 64).to(dt), r(pool, H, 64, 64), ld


def _check(q, k, v, ld, before, index, out, states, dtype):
    ldn = np.zeros(q.shape[1]) if ld is None else _f64(ld)
    args = [_f64(x) for x in (q, k, v)]
    ref, ref_s = oracle_decay_step(*args, ldn, _f64(before), index)
    absum, absum_s = oracle_decay_step(*[abs(x) for x in args], ldn, abs(_f64(before)), index)
    got = _f64(out)
    live = np.asarray(index) >= 0
    tol = 72 * U32 * absum[live] + (U16 * 1.01 * abs(ref[live]) if dtype == "bf16" else 0)
    assert np.all(abs(got[live] - ref[live]) <= tol)
    assert np.isnan(got[~live]).all()                                   # padding: left as it was
    assert np.all(abs(_f64(states) - ref_s) <= 6 * U32 * absum_s)
    untouched = np.setdiff1d(np.arange(states.shape[0]), np.asarray(index)[live])
    assert torch.equal(states[untouched], before[untouched])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,H,pool", [(1, 1, 1), (3, 5, 7), (64, 2, 64), (65, 3, 90), (130, 16, 131), (1001, 1, 1100),
                                      (2003, 1, 2003), (4099, 1, 4100)])
def test_step_with_indices(cuda_device, n, H, pool, dtype):
    q, k, v, states, ld = _draw(n, H, pool, dtype, cuda_device)
    index = np.random.default_rng(n).permutation(pool)[:n].astype(np.int32)
    index[1::3] = -1
    before = states.clone()
    out = span_la_decay_step(q, k, v, states, ld, state_index=index, out=torch.full_like(q, float("nan")))
    span_la_check()
    _check(q, k, v, ld, before, index, out, states, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("decay", [True, False])
def test_step_in_order(cuda_device, dtype, decay):
    q, k, v, states, ld = _draw(37, 4, 40, dtype, cuda_device, seed=2)
    before = states.clone()
    out = span_la_decay_step(q, k, v, states, ld if decay else None, out=torch.full_like(q, float("nan")))
    span_la_check()
    _check(q, k, v, ld if decay else None, before, list(range(37)), out, states, dtype)


def test_all_rows_padding(cuda_device):
    q, k, v, states, ld = _draw(5, 2, 3, "bf16", cuda_device)
    before = states.clone()
    out = span_la_decay_step(q, k, v, states, ld, state_index=[-1] * 5, out=torch.full_like(q, float("nan")))
    span_la_check()
    assert torch.isnan(out).all() and torch.equal(states, before)


def test_undecayed_tokens_continue_the_undecayed_pass(cuda_device):
    """span_la_pass over 300 rows, then 4 tokens without decay, as span_la_pass over 304: bf16 outputs of both are
    within 5e-3 of the result, so within 1e-2 of each other."""
    w = workloads.make_pass([304], [], [], H=3, dtype="bf16", seed=3)
    q, k, v = (x.to(cuda_device) for x in (w.q, w.k, w.v))
    whole, final = span_la_pass(q, k, v, w.view_cu, None, None)
    _, states = span_la_pass(q, k, v, [0, 300], None, None)
    for t in range(300, 304):
        out = span_la_decay_step(q[t:t + 1], k[t:t + 1], v[t:t + 1], states)
        assert torch.linalg.norm(out[0].double() - whole[t].double()) <= 1e-2 * torch.linalg.norm(whole[t].double())
    span_la_check()
    assert torch.linalg.norm(states.double() - final.double()) <= 1e-5 * torch.linalg.norm(final.double())


def test_indices_are_kept_by_a_recorded_call(cuda_device):
    """The host index array may change after the call: replays use the recorded one.  Each replay is one more token."""
    q, k, v, states, ld = _draw(3, 2, 6, "f32", cuda_device, seed=5)
    twin = states.clone()
    index = np.array([4, 0, 2], dtype=np.int32)
    out = torch.empty_like(q)
    span_la_decay_step(q, k, v, states.clone(), ld, state_index=index, out=out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        span_la_decay_step(q, k, v, states, ld, state_index=index, out=out)
    index[:] = [1, 3, 5]
    for _ in range(3):
        g.replay()
        ref = span_la_decay_step(q, k, v, twin, ld, state_index=[4, 0, 2])
        span_la_check()
        assert torch.equal(out, ref) and torch.equal(states, twin)


def test_two_streams_on_one_pool(cuda_device):
    """Batches of different states of one pool may run at once."""
    q, k, v, states, ld = _draw(64, 16, 64, "bf16", cuda_device, seed=6)
    twin = states.clone()
    a, b = torch.cuda.Stream(cuda_device), torch.cuda.Stream(cuda_device)
    outs = [torch.empty_like(q[:32]) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        span_la_decay_step(q[:32], k[:32], v[:32], states, ld, state_index=range(0, 64, 2), out=outs[0], stream=a)
        span_la_decay_step(q[32:], k[32:], v[32:], states, ld, state_index=range(1, 64, 2), out=outs[1], stream=b)
    torch.cuda.synchronize()
    for _ in range(10):
        r0 = span_la_decay_step(q[:32], k[:32], v[:32], twin, ld, state_index=range(0, 64, 2))
        r1 = span_la_decay_step(q[32:], k[32:], v[32:], twin, ld, state_index=range(1, 64, 2))
    span_la_check()
    assert torch.equal(states, twin) and torch.equal(outs[0], r0) and torch.equal(outs[1], r1)
