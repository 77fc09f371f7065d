"""What plans of decayed passes hold on to, and whom they keep waiting."""
import ctypes

import pytest
import torch

from hybrid_linear_attention_packed_gb300 import (span_la_check, span_la_decay_branches_from_state, span_la_decay_pass, spanla,
                                                  workloads)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_shards_of_one_layout_do_not_wait_for_one_another(cuda_device, dtype):
    """Branches of one tile need no workspace, so two calls of their plan share nothing: one on a second stream is
    through while the first stream is still held up."""
    H = 2
    w = workloads.make_pass([], [100, 30, 128], [0, 1, 0], H=H, dtype=dtype, seed=51)
    q, k, v = (x.to(cuda_device) for x in (w.q, w.k, w.v))
    kept = torch.randn(2, H, 64, 64, device=cuda_device)
    ld = torch.full((H,), -0.01, device=cuda_device)
    outs = [torch.empty_like(q) for _ in range(3)]
    a, b = torch.cuda.Stream(cuda_device), torch.cuda.Stream(cuda_device)

    def call(i, stream=None):
        span_la_decay_branches_from_state(kept, q, k, v, ld, w.branch_cu, w.branch_parent, out=outs[i], stream=stream)

    call(0)
    torch.cuda.synchronize()
    ends = [torch.cuda.Event() for _ in range(2)]
    with torch.cuda.stream(a):
        torch.cuda._sleep(1_000_000_000)   # half a second
    call(1, a)
    ends[0].record(a)
    call(2, b)
    ends[1].record(b)
    ends[1].synchronize()
    held = not ends[0].query()
    torch.cuda.synchronize()
    span_la_check()
    assert torch.equal(outs[1], outs[0]) and torch.equal(outs[2], outs[0])
    assert held


def _pool_used(dev):
    """Bytes of the device's default memory pool that are allocated now."""
    lib = spanla.load_library()   # (its CUDA runtime)
    pool, used = ctypes.c_void_p(), ctypes.c_uint64()
    assert lib.cudaDeviceGetDefaultMemPool(ctypes.byref(pool), ctypes.c_int(dev.index or 0)) == 0
    assert lib.cudaMemPoolGetAttribute(pool, ctypes.c_int(7), ctypes.byref(used)) == 0   # cudaMemPoolAttrUsedMemCurrent
    return used.value


def test_kept_workspaces_are_bounded_in_bytes(cuda_device):
    """Twelve passes whose metadata never comes back, each with some 50 MB of workspace: their plans keep 256 MB at
    most in all (and descriptors)."""
    H, rows = 16, 25_600
    q, k, v = workloads.draw_qkv_device(52, rows, H, cuda_device)
    ld = torch.full((H,), -0.01, device=cuda_device)
    outs = []
    for i in range(12):
        outs.append(span_la_decay_pass(q, k, v, ld, [0, rows - i], None, None)[0][:rows - 64])
        torch.cuda.synchronize()
        assert _pool_used(cuda_device) <= (256 + 64) << 20, i
    span_la_check()
    for o in outs[1:]:   # (the rows before the end do not depend on it, but for the cut into runs)
        assert torch.linalg.norm(o.double() - outs[0].double()) <= 1e-2 * torch.linalg.norm(outs[0].double())
