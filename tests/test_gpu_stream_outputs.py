"""Calls on another stream than the current one that allocate their outputs: no memory with work pending on either stream
is written early, or handed out early."""
import numpy as np
import pytest
import torch

from hybrid_linear_attention_packed_gb300 import (ViewStateCache, rope_inv_freq, span_la_branches_from_state, span_la_check,
                                                  span_la_decay_branches_from_state, span_la_decay_pass, span_la_decay_step,
                                                  span_la_kv_read, span_la_pass, span_la_pass_noalloc, span_la_qk_norm_rope,
                                                  span_la_softmax_branches_from_kv, span_la_softmax_paged, span_la_softmax_pass)
from hybrid_linear_attention_packed_gb300 import spanla
from paged_helpers import i32, make_pages, make_table

pytestmark = pytest.mark.gpu
T, H = 300, 4
NAMES = ["pass", "pass_noalloc", "fork", "softmax", "softmax_kv", "decay_pass", "decay_fork", "step", "rope", "cache", "kv_read", "paged"]
WAIT = 200_000_000          # cycles: a tenth of a second


def _call(name, dev):
    """A call that takes a stream and returns the outputs that it made."""
    g = torch.Generator(device=dev).manual_seed(7)
    r = lambda *s: torch.randn(s, generator=g, device=dev)  # noqa: E731
    q, k, v = (r(T, H, 64).to(torch.bfloat16) for _ in range(3))
    ld = torch.full((H,), -0.01, device=dev)
    vcu, bcu, par = (np.array(x, dtype=np.int32) for x in ([0, T - 40], [T - 40, T - 10, T], [0, 0]))
    bq, bk, bv = (x[T - 40:].contiguous() for x in (q, k, v))
    fork = (bq, bk, bv, np.array([0, 30, 40], dtype=np.int32), par)
    kept, pool = r(2, H, 64, 64), r(T, H, 64, 64)
    pos = torch.arange(T, dtype=torch.int32, device=dev)
    freq = rope_inv_freq(64)
    table, P = make_table([T], 16, 0, 0)
    c = make_pages(P, H, 16, torch.bfloat16, dev, fill=0)
    cache = (c[0], c[1], i32(table, dev), i32([T], dev), i32([0, T], dev))
    states = ViewStateCache(H, 4)
    states.put([1, 2], kept)
    one = lambda x: (x,)  # noqa: E731
    return {
        "pass": lambda s: span_la_pass(q, k, v, vcu, bcu, par, stream=s),
        "pass_noalloc": lambda s: span_la_pass_noalloc(q, k, v, vcu, bcu, par, stream=s),
        "fork": lambda s: one(span_la_branches_from_state(kept, *fork, stream=s)),
        "softmax": lambda s: one(span_la_softmax_pass(q, k, v, vcu, bcu, par, stream=s)),
        "softmax_kv": lambda s: one(span_la_softmax_branches_from_kv(k, v, [0, T], *fork, stream=s)),
        "decay_pass": lambda s: span_la_decay_pass(q, k, v, ld, vcu, bcu, par, stream=s),
        "decay_fork": lambda s: one(span_la_decay_branches_from_state(kept, *fork[:3], ld, *fork[3:], stream=s)),
        "step": lambda s: one(span_la_decay_step(q, k, v, pool.clone() if s is None else pool, ld, stream=s)),
        "rope": lambda s: span_la_qk_norm_rope(q, k, pos, freq, stream=s),
        "cache": lambda s: one(states.branches([1, 2], *fork[:4], stream=s)),
        "kv_read": lambda s: span_la_kv_read(*cache, T, stream=s),
        "paged": lambda s: one(span_la_softmax_paged(q, *cache, stream=s)),
    }[name]


@pytest.mark.parametrize("fast", [True, False])
@pytest.mark.parametrize("name", NAMES)
def test_new_outputs_on_another_stream(cuda_device, name, fast, monkeypatch):
    dev = cuda_device
    if not fast:
        monkeypatch.setattr(spanla, "_fast", None)
    call = _call(name, dev)
    here, side = torch.cuda.current_stream(dev), torch.cuda.Stream(dev)
    ref = [x.clone() for x in call(None)]
    torch.cuda.synchronize()

    def hold():   # outputs of the current stream's own memory, with work pending on it, freed
        old = [torch.empty_like(x) for x in ref]
        at = {x.data_ptr() for x in old}
        torch.cuda._sleep(WAIT)
        for x in old:
            x.fill_(7)
        return at

    pending = hold()
    first = call(side)                                         # must not be in that memory
    torch.cuda.synchronize()
    assert not pending & {x.data_ptr() for x in first}
    if name != "step":                                         # (which moves its states on)
        assert all(torch.equal(a, b) for a, b in zip(first, ref))
    got = [x.clone() for x in first]
    del first
    torch.cuda.synchronize()

    with torch.cuda.stream(side):
        torch.cuda._sleep(WAIT)
    gone = {x.data_ptr() for x in call(side)}                  # freed before the call has run
    after = [torch.empty_like(x) for x in ref]
    assert not gone & {x.data_ptr() for x in after}

    out = call(side)
    here.wait_stream(side)
    torch.cuda._sleep(WAIT)
    last = [x.clone() for x in out]                            # read by the current stream, later
    used = {x.data_ptr() for x in out}
    del out
    with torch.cuda.stream(side):
        again = [torch.empty_like(x) for x in ref]
        assert not used & {x.data_ptr() for x in again}
    torch.cuda.synchronize()
    span_la_check()
    if name != "step":
        assert all(torch.equal(a, b) for a, b in zip(last, got))


@pytest.mark.parametrize("name", ["paged", "kv_read", "rope", "pass"])
def test_the_current_stream_by_name(cuda_device, name):
    call = _call(name, cuda_device)
    ref = [x.clone() for x in call(None)]
    got = call(torch.cuda.current_stream(cuda_device))
    span_la_check()
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
