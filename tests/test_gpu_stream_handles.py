"""A stream's handle may come back for a new stream: plans and cached states
that calls on the first one used go on working on the second."""
import ctypes

import numpy as np
import pytest
import torch

from hybrid_linear_attention_packed_gb300 import ViewStateCache, span_la_check, span_la_decay_pass, spanla, workloads

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_calls_on_streams_created_and_destroyed_in_turn(cuda_device, dtype):
    lib = spanla.load_library()   # (its CUDA runtime)
    w = workloads.make_pass([500, 130], [100, 300, 7], [0, 1, 0], H=2, dtype=dtype, seed=95)
    q, k, v = (x.to(cuda_device) for x in (w.q, w.k, w.v))
    ld = torch.full((2,), -0.01, device=cuda_device)
    ref, ref_s = span_la_decay_pass(q, k, v, ld, w.view_cu, w.branch_cu, w.branch_parent)
    keys = np.arange(2, dtype=np.uint64)
    lo = int(w.branch_cu[0])
    outs = []
    with ViewStateCache(2, 2) as cache:
        torch.cuda.synchronize()
        shards = []
        for _ in range(6):
            handle = ctypes.c_void_p()
            assert lib.cudaStreamCreate(ctypes.byref(handle)) == 0
            s = torch.cuda.ExternalStream(handle.value, cuda_device)
            out, state, shard = torch.zeros_like(q), torch.zeros_like(ref_s), torch.zeros_like(q)
            s.wait_stream(torch.cuda.current_stream(cuda_device))
            span_la_decay_pass(q, k, v, ld, w.view_cu, w.branch_cu, w.branch_parent, out=out, view_state_out=state, stream=s)
            cache.put(keys, state, stream=s)
            cache.branches(keys[w.branch_parent], q, k, v, w.branch_cu, out=shard, log_decay=ld, stream=s)
            s.synchronize()
            outs.append((out, state))
            shards.append(shard)
            assert lib.cudaStreamDestroy(handle) == 0
        span_la_check()
    for (o, st), shard in zip(outs, shards):
        assert torch.equal(o, ref) and torch.equal(st, ref_s)
        a, b = shard[lo:].double(), ref[lo:].double()
        assert torch.equal(shard, shards[0]) and torch.linalg.norm(a - b) <= 1e-2 * torch.linalg.norm(b)
