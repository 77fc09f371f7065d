"""Decayed plans whose workspaces come to more than the plan cache keeps."""
import pytest
import torch

from hybrid_linear_attention_packed_gb300 import span_la_check, span_la_decay_pass, workloads

pytestmark = pytest.mark.gpu


def test_plans_past_the_bound_take_turns(cuda_device):
    """Eight layouts of some 50 MB of workspace each, three times over on two streams: the first five keep theirs, the
    others allocate it; the bits are the same every time."""
    H, rows = 16, 25_600
    q, k, v = workloads.draw_qkv_device(53, rows, H, cuda_device)
    ld = torch.full((H,), -0.01, device=cuda_device)
    cus = [[0, rows - 1000 * i] for i in range(8)]
    outs = [[(torch.empty_like(q), torch.empty(1, H, 64, 64, device=cuda_device)) for _ in cus] for _ in range(3)]
    streams = [torch.cuda.Stream(cuda_device) for _ in range(2)]
    torch.cuda.synchronize()
    for r, row in enumerate(outs):
        for i, (o, s) in enumerate(row):
            span_la_decay_pass(q, k, v, ld, cus[i], None, None, out=o, view_state_out=s, stream=streams[(i + r) % 2])
    torch.cuda.synchronize()
    span_la_check()
    for row in outs[1:]:
        for i, (o, s) in enumerate(row):
            n = cus[i][1]
            assert torch.equal(o[:n], outs[0][i][0][:n]) and torch.equal(s, outs[0][i][1])
