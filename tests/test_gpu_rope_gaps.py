"""Weights between the rows of an output: refused only where they overlap it."""
import pytest
import torch

from hybrid_linear_attention_packed_gb300 import SpanLAError, rope_inv_freq, span_la_check, span_la_qk_norm_rope

pytestmark = pytest.mark.gpu


def test_weights_in_the_gaps_of_an_output(cuda_device):
    T, H = 12, 3
    rows = torch.randn(T, H * 64 + 128, device=cuda_device).bfloat16()
    q, k = rows[:, :H * 64].view(T, H, 64), torch.randn(T, 1, 64, device=cuda_device).bfloat16()
    w = rows[5, H * 64:H * 64 + 64]
    pos = torch.arange(T, dtype=torch.int32, device=cuda_device)
    freq = rope_inv_freq(64)
    want, _ = span_la_qk_norm_rope(q, k, pos, freq, q_weight=w.clone())
    rest = rows[:, H * 64:].clone()
    for bad in (rows[5, :64], rows[0, (H - 1) * 64:H * 64], rows[5, H * 64 - 8:H * 64 + 56]):
        with pytest.raises(SpanLAError, match="overlaps a weight"):
            span_la_qk_norm_rope(q, k, pos, freq, q_weight=bad, q_out=q)
    span_la_qk_norm_rope(q, k, pos, freq, q_weight=w, q_out=q)
    span_la_check()
    assert torch.equal(q, want) and torch.equal(rows[:, H * 64:], rest)
