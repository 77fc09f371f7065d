"""Norm and rotation of queries and keys against the float64 form.

Bounds: the mean of squares is off by (64 + 2) * 2^-24 of it at most, its root
half of that, and the products, the cosine and sine (2^-22 together) and the
sum of two products add 8 * 2^-24 of their size: |error| <= 64 * 2^-24 of
|y_a| + |y_b| in fp32, plus 2^-8 of the result where it is rounded to bf16."""
import numpy as np
import pytest
import torch

from hybrid_linear_attention_packed_gb300 import rope_inv_freq, span_la_check, span_la_qk_norm_rope
from oracle.decay_oracle import oracle_norm_rope

pytestmark = pytest.mark.gpu

U32, U16 = 2.0 ** -24, 2.0 ** -8


def _f64(t):
    return t.detach().double().cpu().numpy()


def _check(x, w, pos, freq, eps, inter, got, dtype):
    wn = None if w is None else _f64(w)
    ref = oracle_norm_rope(_f64(x), wn, pos, freq, eps, inter)
    plain = abs(oracle_norm_rope(_f64(x), wn, pos, [], eps, inter))      # norm only: the size of each pair's parts
    r = 2 * len(freq)
    size = plain.copy()
    if r:
        a, b = (slice(0, r, 2), slice(1, r, 2)) if inter else (slice(0, r // 2), slice(r // 2, r))
        size[..., a] = size[..., b] = plain[..., a] + plain[..., b]
    got = _f64(got)
    live = np.asarray(pos) >= 0
    tol = 64 * U32 * size[live] + (1.01 * U16 * abs(ref[live]) if dtype == "bf16" else 0)
    assert np.all(abs(got[live] - ref[live]) <= tol)
    assert np.isnan(got[~live]).all()


def _draw(T, Hq, Hk, dtype, dev, seed=0):
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    return [torch.randn(T, H, 64, generator=g, device=dev).to(dt) for H in (Hq, Hk)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("rotary", [0, 16, 32, 48, 64])
@pytest.mark.parametrize("T,Hq,Hk", [(1, 1, 1), (5, 16, 16), (33, 3, 7), (130, 9, 2)])
def test_norm_and_rotation(cuda_device, T, Hq, Hk, rotary, inter, dtype):
    q, k = _draw(T, Hq, Hk, dtype, cuda_device)
    rng = np.random.default_rng(T)
    pos = rng.integers(0, 2 ** 31 - 1, T).astype(np.int32)
    pos[:2] = (0, 1)[:T]
    if T > 4:
        pos[2:5] = (2 ** 31 - 1, -1, -(2 ** 31))
    freq = rope_inv_freq(rotary, 1e6)
    wq = (1 + 0.3 * torch.randn(64, device=cuda_device)).to(q.dtype)
    wk = (1 + 0.3 * torch.randn(Hk, 64, device=cuda_device)).to(q.dtype)
    outs = [torch.full_like(x, float("nan")) for x in (q, k)]
    got = span_la_qk_norm_rope(q, k, torch.from_numpy(pos).to(cuda_device), freq, wq, wk, interleaved=inter,
                               q_out=outs[0], k_out=outs[1])
    span_la_check()
    # (the oracle's own angle, position * frequency, is off by 2^-53 of it: 2^31 * 2^-53 = 2^-22 of a radian;
    # the bound's 64 * 2^-24 holds that and the kernel's)
    _check(q, wq, pos, freq, 1e-6, inter, got[0], dtype)
    _check(k, wk, pos, freq, 1e-6, inter, got[1], dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_parts_of_a_fused_projection_and_in_place(cuda_device, dtype):
    T, H = 50, 6
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    rows = torch.randn(T, 3 * H * 64 + 64, device=cuda_device).to(dt)
    q, k = rows[:, :H * 64].view(T, H, 64), rows[:, H * 64:2 * H * 64].view(T, H, 64)
    rest = rows[:, 2 * H * 64:].clone()
    pos = np.arange(T, dtype=np.int32) + 12345
    p = torch.from_numpy(pos).to(cuda_device)
    freq = rope_inv_freq(64)
    w32 = torch.rand(64, device=cuda_device) + 0.5                       # fp32 weights with either type
    a, b = span_la_qk_norm_rope(q, k, p, freq, w32, None)
    span_la_check()
    _check(q, w32, pos, freq, 1e-6, False, a, dtype)
    _check(k, None, pos, freq, 1e-6, False, b, dtype)
    span_la_qk_norm_rope(q, k, p, freq, w32, None, q_out=q, k_out=k)      # over the projection's own rows
    span_la_check()
    assert torch.equal(q, a) and torch.equal(k, b) and torch.equal(rows[:, 2 * H * 64:], rest)


def test_zero_rows_heads_and_vectors(cuda_device):
    q, k = _draw(4, 2, 2, "f32", cuda_device)
    p = torch.arange(4, dtype=torch.int32, device=cuda_device)
    q[1] = 0
    out, _ = span_la_qk_norm_rope(q, k, p, rope_inv_freq(64), eps=1e-5)
    span_la_check()
    assert torch.equal(out[1], torch.zeros_like(out[1]))
    e, _ = span_la_qk_norm_rope(q[:0], k[:0], p[:0], rope_inv_freq(64))
    assert e.shape == (0, 2, 64)
    only_q, none = span_la_qk_norm_rope(q, k[:, :0], p, rope_inv_freq(64), eps=1e-5)
    span_la_check()
    assert torch.equal(only_q, out) and none.shape == (4, 0, 64)


def test_large_and_tiny_values_and_nan(cuda_device):
    """Squares stay in range up to 1e18; a NaN stays in its own head."""
    q, k = _draw(3, 4, 4, "f32", cuda_device)
    q[0] *= 1e17
    q[1] *= 1e-15
    q[2, 1, 7] = float("nan")
    pos = np.array([3, 4, 5], dtype=np.int32)
    got, _ = span_la_qk_norm_rope(q, k, torch.from_numpy(pos).to(cuda_device), rope_inv_freq(64), eps=1e-6)
    span_la_check()
    _check(q[:2], None, pos[:2], rope_inv_freq(64), 1e-6, False, got[:2], "f32")
    assert torch.isnan(got[2, 1]).all() and torch.isfinite(got[2, [0, 2, 3]]).all()


def test_replays_use_the_recorded_frequencies(cuda_device):
    q, k = _draw(9, 2, 2, "bf16", cuda_device)
    p = torch.arange(9, dtype=torch.int32, device=cuda_device)
    freq = rope_inv_freq(64)
    ref = span_la_qk_norm_rope(q, k, p, freq)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = span_la_qk_norm_rope(q, k, p, freq)
    freq[:] = 0.0
    g.replay()
    span_la_check()
    assert all(torch.equal(a, b) for a, b in zip(got, ref))


def test_refusals_of_the_binding(cuda_device):
    q, k = _draw(4, 2, 2, "bf16", cuda_device)
    p = torch.arange(4, dtype=torch.int32, device=cuda_device)
    f = rope_inv_freq(64)
    with pytest.raises(ValueError, match="positions"):
        span_la_qk_norm_rope(q, k, p.long(), f)
    with pytest.raises(ValueError, match="next to each other"):
        span_la_qk_norm_rope(q.transpose(1, 2).contiguous().transpose(1, 2), k, p, f)
    with pytest.raises(ValueError, match="host values"):
        span_la_qk_norm_rope(q, k, p, torch.from_numpy(f).to(cuda_device))
    with pytest.raises(ValueError, match="share dtype"):
        span_la_qk_norm_rope(q, k.float(), p, f)
    with pytest.raises(ValueError, match="q_weight"):
        span_la_qk_norm_rope(q, k, p, f, q_weight=torch.ones(32, device=cuda_device, dtype=q.dtype))
