"""Plain float64 forms of the decayed linear layer: the recurrence row by row
over a packed pass, one token of it, and the norm and rotation of queries and
keys.  Written from the definitions; shares no code with the CUDA library."""
from __future__ import annotations

import numpy as np


def _run(q, k, v, a, S, out):
    """Rows of one segment from state S [H, 64, 64]; a: decay [H].  Returns the final state."""
    for t in range(q.shape[0]):
        S = a[:, None, None] * S + k[t][:, :, None] * v[t][:, None, :]
        out[t] = np.einsum("hi,hij->hj", q[t], S)
    return S


def oracle_decay_pass(q, k, v, log_decay, view_cu, branch_cu, branch_parent, kept=None):
    """out [T, H, 64] (rows in no segment NaN) and the views' final states.  With ``kept`` [P, H, 64, 64]
    the branches start from those states and there are no views."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    T, H, D = q.shape
    a = np.exp(np.asarray(log_decay, dtype=np.float64))
    out = np.full((T, H, D), np.nan)
    finals = []
    if kept is not None:
        finals = list(np.asarray(kept, dtype=np.float64))
    else:
        for s in range(max(len(view_cu) - 1, 0)):
            lo, hi = int(view_cu[s]), int(view_cu[s + 1])
            finals.append(_run(q[lo:hi], k[lo:hi], v[lo:hi], a, np.zeros((H, D, D)), out[lo:hi]))
    for b in range(max(len(branch_cu) - 1, 0)):
        lo, hi = int(branch_cu[b]), int(branch_cu[b + 1])
        _run(q[lo:hi], k[lo:hi], v[lo:hi], a, finals[int(branch_parent[b])], out[lo:hi])
    return out, (np.stack(finals) if finals else np.zeros((0, H, D, D)))


def oracle_decay_step(q, k, v, log_decay, states, index):
    """(out, states) after one token of every row; rows of index -1 give NaN."""
    q, k, v, S = (np.array(x, dtype=np.float64) for x in (q, k, v, states))
    a = np.exp(np.asarray(log_decay, dtype=np.float64))
    out = np.full(q.shape, np.nan)
    for t, i in enumerate(index):
        if i >= 0:
            S[i] = _run(q[t:t + 1], k[t:t + 1], v[t:t + 1], a, S[i], out[t:t + 1])
    return out, S


def oracle_norm_rope(x, weight, positions, inv_freq, eps, interleaved):
    """x [T, H, 64], weight [64] or [H, 64] or None; rows of negative positions give NaN."""
    x = np.asarray(x, dtype=np.float64)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    if weight is not None:
        y = y * np.asarray(weight, dtype=np.float64)
    r = 2 * len(inv_freq)
    ang = np.asarray(positions, dtype=np.float64)[:, None, None] * np.asarray(inv_freq, dtype=np.float64)
    c, s = np.cos(ang), np.sin(ang)
    a = y[..., 0:r:2] if interleaved else y[..., :r // 2]
    b = y[..., 1:r:2] if interleaved else y[..., r // 2:r]
    a, b = a * c - b * s, b * c + a * s
    if interleaved:
        y[..., 0:r:2], y[..., 1:r:2] = a, b
    else:
        y[..., :r // 2], y[..., r // 2:r] = a, b
    y[np.asarray(positions) < 0] = np.nan
    return y
