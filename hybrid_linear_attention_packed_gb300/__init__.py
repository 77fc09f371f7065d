"""Packed linear-attention pass (and the hybrid model's softmax layer over the
same packed rows) for GB300 (sm_103a).

The compute path is ``libspanla.so`` (hand-written CUDA kernels behind the C
ABI in ``include/spanla.h``); :mod:`.spanla` is its thin Python binding,
:mod:`.sharding` the host side of splitting a pass across ranks by request,
and :mod:`.workloads` the seeded synthetic inputs.
"""
from .spanla import (  # noqa: F401
    SpanLAError,
    ViewStateCache,
    kv_pages,
    load_library,
    packed_positions,
    rope_inv_freq,
    span_la_branches_from_state,
    span_la_check,
    span_la_decay_branches_from_state,
    span_la_decay_pass,
    span_la_decay_step,
    span_la_kv_read,
    span_la_kv_write,
    span_la_pass,
    span_la_pass_noalloc,
    span_la_plan_prepare,
    span_la_qk_norm_rope,
    span_la_softmax_branches_from_kv,
    span_la_softmax_paged,
    span_la_softmax_pass,
)
