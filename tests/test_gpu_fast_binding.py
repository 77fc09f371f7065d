"""The binding's extension module makes the same calls as ctypes: the same
bits, the same errors, the same allocations."""
import numpy as np
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

from hybrid_linear_attention_packed_gb300 import (rope_inv_freq, span_la_check, span_la_decay_branches_from_state,
                                                  span_la_decay_pass, span_la_decay_step, span_la_qk_norm_rope, spanla)

pytestmark = pytest.mark.gpu


def _calls(dev, T=300, H=4, dtype=torch.bfloat16):
    g = torch.Generator(device=dev).manual_seed(61)
    r = lambda *s: torch.randn(s, generator=g, device=dev)  # noqa: E731
    q, k, v = (r(T, H, 64).to(dtype) for _ in range(3))
    ld = torch.full((H,), -0.01, device=dev)
    vcu, bcu, par = (np.array(x, dtype=np.int32) for x in ([0, T - 40], [T - 40, T - 10, T], [0, 0]))
    kept, pool = r(2, H, 64, 64), r(4, H, 64, 64)
    index = np.full(T, -1, dtype=np.int32)
    index[[5, 7, T - 1]] = [3, 0, 2]
    pos = torch.arange(T, dtype=torch.int32, device=dev)
    freq = rope_inv_freq(64)
    return {"pass": lambda: span_la_decay_pass(q, k, v, ld, vcu, bcu, par),
            "fork": lambda: (span_la_decay_branches_from_state(kept, q, k, v, ld, bcu, par)[T - 40:],),
            "step": lambda: (span_la_decay_step(q, k, v, pool, ld, index)[torch.from_numpy(index >= 0).to(dev)], pool.clone()),
            "rope": lambda: span_la_qk_norm_rope(q, k, pos, freq)}


def _run(calls):
    res = {name: [x.clone() for x in fn()] for name, fn in calls.items()}
    span_la_check()
    return res


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_same_bits_with_and_without_the_extension(cuda_device, dtype, monkeypatch):
    spanla.load_library()
    assert spanla._fast is not None
    fast = _run(_calls(cuda_device, dtype=dtype))
    monkeypatch.setattr(spanla, "_fast", None)
    slow = _run(_calls(cuda_device, dtype=dtype))
    for name in fast:
        for a, b in zip(fast[name], slow[name]):
            assert torch.equal(a, b), name


@pytest.mark.parametrize("name", ["pass", "fork", "step", "rope"])
@pytest.mark.parametrize("fast", [True, False])
def test_out_of_memory_has_its_own_type(cuda_device, name, fast, monkeypatch):
    """An output that the caching allocator refuses (its share of the device set to nothing for the call)."""
    if not fast:
        monkeypatch.setattr(spanla, "_fast", None)
    call = _calls(cuda_device, T=40_000, H=16)[name]
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    torch.cuda.set_per_process_memory_fraction(1e-6, cuda_device)
    held = []
    try:
        with pytest.raises(torch.OutOfMemoryError):      # (what earlier tests left free in the allocator's blocks)
            while True:
                held.append(torch.empty(40_000, 16, 64, dtype=torch.bfloat16, device=cuda_device))
        with pytest.raises(torch.OutOfMemoryError):
            call()
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0, cuda_device)
        held.clear()
    call()
    span_la_check()


def _leave_ones(like):
    x = torch.ones_like(like)
    torch.cuda.synchronize()
    del x


def test_new_outputs_are_filled_where_torch_fills_them(cuda_device):
    """torch.use_deterministic_algorithms fills memory that nothing wrote: NaN in the skipped rows of a step."""
    q = torch.randn(6, 2, 64, device=cuda_device)
    pool = torch.randn(2, 2, 64, 64, device=cuda_device)
    index = np.array([-1, 1, -1, -1, 0, -1], dtype=np.int32)
    _leave_ones(q)
    torch.use_deterministic_algorithms(True)
    try:
        out = span_la_decay_step(q, q, q, pool, None, index)
    finally:
        torch.use_deterministic_algorithms(False)
    span_la_check()
    assert torch.isnan(out[torch.from_numpy(index < 0).to(cuda_device)]).all()
    assert torch.isfinite(out[[1, 4]]).all()


@pytest.mark.parametrize("name", ["pass", "fork", "step", "rope"])
def test_a_dispatch_mode_sees_the_outputs(cuda_device, name):
    class Seen(TorchDispatchMode):
        names = []

        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            self.names.append(str(func))
            return func(*args, **(kwargs or {}))

    call = _calls(cuda_device)[name]
    with Seen() as seen:
        call()
    span_la_check()
    assert any("empty" in n for n in seen.names)
