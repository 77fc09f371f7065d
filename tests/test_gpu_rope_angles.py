"""The rotation's angles at any position, against exact arithmetic.

A vector with one nonzero pair (8, 0) has a mean square of 1, so the outputs of
its pair are 8 r (cos, sin) with r near 1, and their ratio gives the angle
whatever r is.  Errors of that angle: the angle itself, at most 2^-27 of a
turn as the interface states, 2 pi 2^-27 = 0.79 * 2^-24; the cosine and the
sine, an ulp of at most 2^-24 each, sqrt(2) 2^-24 together; their product with r,
half a step each, 2^-25 sqrt(2) in the worst direction.  In all less than 3 * 2^-24
radians."""
from fractions import Fraction

import numpy as np
import pytest
import torch

from hybrid_linear_attention_packed_gb300 import rope_inv_freq, span_la_check, span_la_qk_norm_rope

pytestmark = pytest.mark.gpu


def _pi(bits=400):
    """pi as a Fraction (16 atan 1/5 - 4 atan 1/239), to 2^-bits."""
    def atan_inv(n):
        one, total, k, sign = 1 << (bits + 32), 0, 1, 1
        term = one // n
        while term:
            total += sign * (term // k)
            term //= n * n
            k, sign = k + 2, -sign
        return total
    return Fraction(16 * atan_inv(5) - 4 * atan_inv(239), 1 << (bits + 32))


def _angles(pos, freq):
    """position * frequency modulo 2 pi, in (-pi, pi], rounded once."""
    turn = 2 * _pi()
    out = np.empty((len(pos), len(freq)))
    for j, f in enumerate(freq):
        step = Fraction(float(f)) / turn
        for t, p in enumerate(pos):
            x = int(p) * step
            x -= round(x)
            out[t, j] = float(x * turn)
    return out


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("freqs", ["base 1e4", "base 1e6", "large and negative"])
def test_angles_at_any_position(cuda_device, freqs, interleaved):
    freq = {"base 1e4": rope_inv_freq(64), "base 1e6": rope_inv_freq(64, 1e6),
            "large and negative": -7.3 ** np.linspace(-9, 9, 32)}[freqs]
    rng = np.random.default_rng(6)
    pos = np.concatenate([np.arange(20), rng.integers(0, 1 << 21, 60), rng.integers(1 << 30, (1 << 31) - 1, 60),
                          [(1 << 31) - 1]]).astype(np.int32)
    T = len(pos)
    q = torch.zeros(T, 32, 64, device=cuda_device)      # head j: pair j
    for j in range(32):
        q[:, j, 2 * j if interleaved else j] = 8.0
    got, _ = span_la_qk_norm_rope(q, q[:, :1], torch.from_numpy(pos).to(cuda_device), freq, eps=0.0, interleaved=interleaved)
    span_la_check()
    x = got.double().cpu().numpy()
    heads = np.arange(32)
    c = x[:, heads, 2 * heads if interleaved else heads]
    s = x[:, heads, 2 * heads + 1 if interleaved else heads + 32]
    err = np.arctan2(s, c) - _angles(pos, freq)
    err -= 2 * np.pi * np.round(err / (2 * np.pi))
    assert np.abs(err).max() <= 3 * 2.0 ** -24, np.abs(err).max() * 2.0 ** 24
    assert np.allclose(np.hypot(c, s), 8.0, rtol=2.0 ** -20)
