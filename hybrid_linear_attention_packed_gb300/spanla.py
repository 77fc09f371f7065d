"""Thin Python binding of ``libspanla.so`` (argument marshalling only).

Every step of the pass runs in the library's CUDA kernels; this module only
checks tensor dtypes, shapes, devices and contiguity, converts host metadata to
int32 arrays and passes raw pointers and the current CUDA stream through the C
ABI declared in ``include/spanla.h``.  PyTorch is used for device memory and
streams only.  There is no fallback: if the library is missing or cannot be
loaded, every call raises.

Outputs that a call with ``stream`` makes are that stream's memory, as tensors
made under ``torch.cuda.stream(stream)`` are; whoever uses them on another
stream waits for it first, as for any of its results.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional, Sequence, Tuple

import numpy as np
import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.environ.get("SPANLA_LIB", os.path.join(_PKG, "libspanla.so"))

SPAN_LA_BF16 = 0
SPAN_LA_F32 = 1
SPAN_LA_E4M3 = 2

STATUS = {0: "SPAN_LA_OK", 1: "SPAN_LA_ERR_INVALID", 2: "SPAN_LA_ERR_UNSUPPORTED",
          3: "SPAN_LA_ERR_CUDA", 4: "SPAN_LA_ERR_NOMEM", 5: "SPAN_LA_ERR_TIMEOUT"}

EXPORTED = ("span_la_pass", "span_la_branches_from_state", "span_la_check",
            "span_la_status_string", "span_la_last_error_detail", "span_la_version",
            "span_la_selftest_wait_timeout", "span_la_profile_enable", "span_la_profile_read",
            "span_la_profile_reset", "span_la_kernel_name", "span_la_plan_stats",
            "span_la_pass_noalloc", "span_la_cache_create", "span_la_cache_destroy",
            "span_la_cache_put", "span_la_cache_contains", "span_la_cache_branches",
            "span_la_cache_stats", "span_la_softmax_pass", "span_la_softmax_branches_from_kv",
            "span_la_fault_inject", "span_la_softmax_plan_stats",
            "span_la_selftest_wait_timeout_noalloc", "span_la_pass_variant",
            "span_la_plan_prepare", "span_la_decay_pass", "span_la_decay_branches_from_state",
            "span_la_decay_step", "span_la_qk_norm_rope", "span_la_cache_decay_branches",
            "span_la_kv_write", "span_la_kv_read", "span_la_softmax_paged", "span_la_softmax_paged_workspace")
NUM_KERNELS = 20


class SpanLAError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str):
        self.status = status
        super().__init__("%s: %s (%s)" % (where, STATUS.get(status, status), detail))


class Dims(ctypes.Structure):
    _fields_ = [("total_rows", ctypes.c_int64), ("num_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class QkSide(ctypes.Structure):
    _fields_ = [("in_", ctypes.c_void_p), ("out", ctypes.c_void_p), ("weight", ctypes.c_void_p),
                ("in_row_stride", ctypes.c_int64), ("out_row_stride", ctypes.c_int64),
                ("num_heads", ctypes.c_int32), ("weight_per_head", ctypes.c_int32)]


class KvCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("page_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64), ("row_stride", ctypes.c_int64),
                ("scale_page_stride", ctypes.c_int64), ("scale_head_stride", ctypes.c_int64),
                ("num_pages", ctypes.c_int32), ("page_rows", ctypes.c_int32), ("num_heads", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("num_seqs", ctypes.c_int32), ("table_width", ctypes.c_int32),
                ("table_stride", ctypes.c_int64), ("page_table", ctypes.c_void_p), ("seq_len", ctypes.c_void_p),
                ("row_cu", ctypes.c_void_p)]


_lock = threading.Lock()
_lib = None
_fast = None   # csrc/py/fastcall.cpp bound to _lib: the usual calls without the interpreter's share


def load_library(path: Optional[str] = None):
    """Load the CUDA library (raises if it is missing: there is no fallback)."""
    global _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError("libspanla.so not found at %s: build it with "
                               "hybrid_linear_attention_packed_gb300.build.build()" % p)
        lib = ctypes.CDLL(p)
        # int32 arrays go in as addresses (c_void_p also takes ctypes pointers)
        vp = ctypes.c_void_p
        i32p = vp
        lib.span_la_pass.argtypes = [vp, vp, vp, Dims, i32p, ctypes.c_int32, i32p,
                                     ctypes.c_int32, i32p, vp, vp, vp]
        lib.span_la_pass.restype = ctypes.c_int
        lib.span_la_pass_noalloc.argtypes = [vp, vp, vp, Dims, i32p, ctypes.c_int32, i32p,
                                             ctypes.c_int32, i32p, vp, vp, vp]
        lib.span_la_pass_noalloc.restype = ctypes.c_int
        lib.span_la_branches_from_state.argtypes = [vp, ctypes.c_int32, vp, vp, vp, Dims, i32p,
                                                    ctypes.c_int32, i32p, vp, vp]
        lib.span_la_branches_from_state.restype = ctypes.c_int
        lib.span_la_check.argtypes = [vp]
        lib.span_la_check.restype = ctypes.c_int
        lib.span_la_status_string.argtypes = [ctypes.c_int]
        lib.span_la_status_string.restype = ctypes.c_char_p
        lib.span_la_last_error_detail.argtypes = []
        lib.span_la_last_error_detail.restype = ctypes.c_char_p
        lib.span_la_version.argtypes = []
        lib.span_la_version.restype = ctypes.c_int32
        lib.span_la_selftest_wait_timeout.argtypes = [ctypes.c_int32, vp]
        lib.span_la_selftest_wait_timeout.restype = ctypes.c_int
        lib.span_la_selftest_wait_timeout_noalloc.argtypes = [ctypes.c_int32, vp]
        lib.span_la_selftest_wait_timeout_noalloc.restype = ctypes.c_int
        lib.span_la_profile_enable.argtypes = [ctypes.c_int32]
        lib.span_la_profile_enable.restype = ctypes.c_int
        lib.span_la_profile_read.argtypes = [ctypes.POINTER(ctypes.c_double),
                                             ctypes.POINTER(ctypes.c_int64),
                                             ctypes.POINTER(ctypes.c_int64), ctypes.c_int32]
        lib.span_la_profile_read.restype = ctypes.c_int
        lib.span_la_profile_reset.argtypes = []
        lib.span_la_profile_reset.restype = ctypes.c_int
        lib.span_la_kernel_name.argtypes = [ctypes.c_int32]
        lib.span_la_kernel_name.restype = ctypes.c_char_p
        lib.span_la_plan_stats.argtypes = [i32p, ctypes.c_int32, i32p, ctypes.c_int32, i32p,
                                           ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                           ctypes.c_int32, ctypes.c_int32,
                                           ctypes.POINTER(ctypes.c_int64)]
        lib.span_la_plan_stats.restype = ctypes.c_int
        lib.span_la_softmax_pass.argtypes = [vp, vp, vp, Dims, i32p, ctypes.c_int32, i32p,
                                             ctypes.c_int32, i32p, ctypes.c_float, vp, vp, vp]
        lib.span_la_softmax_pass.restype = ctypes.c_int
        lib.span_la_softmax_plan_stats.argtypes = [i32p, ctypes.c_int32, i32p, ctypes.c_int32, i32p,
                                                   ctypes.c_int32, ctypes.c_int32,
                                                   ctypes.POINTER(ctypes.c_int64)]
        lib.span_la_softmax_plan_stats.restype = ctypes.c_int
        lib.span_la_pass_variant.argtypes = [ctypes.c_int32]
        lib.span_la_pass_variant.restype = ctypes.c_int
        lib.span_la_plan_prepare.argtypes = [Dims, i32p, ctypes.c_int32, i32p, ctypes.c_int32, i32p, vp]
        lib.span_la_plan_prepare.restype = ctypes.c_int
        lib.span_la_fault_inject.argtypes = [ctypes.c_int32, ctypes.c_int32]
        lib.span_la_fault_inject.restype = ctypes.c_int
        lib.span_la_softmax_branches_from_kv.argtypes = [vp, vp, ctypes.c_int64, i32p, ctypes.c_int32,
                                                         vp, vp, vp, Dims, i32p, ctypes.c_int32, i32p,
                                                         ctypes.c_float, vp, vp, vp]
        lib.span_la_softmax_branches_from_kv.restype = ctypes.c_int
        lib.span_la_decay_pass.argtypes = [vp, vp, vp, Dims, vp, i32p, ctypes.c_int32, i32p,
                                           ctypes.c_int32, i32p, vp, vp, vp]
        lib.span_la_decay_pass.restype = ctypes.c_int
        lib.span_la_decay_branches_from_state.argtypes = [vp, ctypes.c_int32, vp, vp, vp, Dims, vp, i32p,
                                                          ctypes.c_int32, i32p, vp, vp]
        lib.span_la_decay_branches_from_state.restype = ctypes.c_int
        lib.span_la_decay_step.argtypes = [vp, vp, vp, Dims, vp, vp, ctypes.c_int32, i32p, vp, vp]
        lib.span_la_decay_step.restype = ctypes.c_int
        lib.span_la_qk_norm_rope.argtypes = [QkSide, QkSide, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32,
                                             ctypes.c_float, vp, ctypes.c_int32, ctypes.c_int32, vp, vp]
        lib.span_la_qk_norm_rope.restype = ctypes.c_int
        cachep = ctypes.POINTER(KvCache)
        lib.span_la_kv_write.argtypes = [vp, vp, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int32, cachep, vp]
        lib.span_la_kv_write.restype = ctypes.c_int
        lib.span_la_kv_read.argtypes = [cachep, ctypes.c_int64, ctypes.c_int32, vp, vp, vp]
        lib.span_la_kv_read.restype = ctypes.c_int
        lib.span_la_softmax_paged.argtypes = [vp, ctypes.c_int64, ctypes.c_int64, ctypes.c_int32, cachep, ctypes.c_int32,
                                              ctypes.c_float, vp, vp, vp, vp]
        lib.span_la_softmax_paged.restype = ctypes.c_int
        lib.span_la_softmax_paged_workspace.argtypes = [ctypes.c_int64, ctypes.c_int32, cachep, ctypes.c_int32]
        lib.span_la_softmax_paged_workspace.restype = ctypes.c_int64
        lib.span_la_cache_create.argtypes = [ctypes.c_int32, ctypes.c_int32,
                                             ctypes.POINTER(ctypes.c_void_p)]
        lib.span_la_cache_create.restype = ctypes.c_int
        lib.span_la_cache_destroy.argtypes = [vp]
        lib.span_la_cache_destroy.restype = ctypes.c_int
        lib.span_la_cache_put.argtypes = [vp, vp, ctypes.c_int32, vp, vp]
        lib.span_la_cache_put.restype = ctypes.c_int
        lib.span_la_cache_contains.argtypes = [vp, vp, ctypes.c_int32, vp]
        lib.span_la_cache_contains.restype = ctypes.c_int
        lib.span_la_cache_branches.argtypes = [vp, vp, vp, vp, vp, Dims, i32p, ctypes.c_int32,
                                               vp, vp]
        lib.span_la_cache_branches.restype = ctypes.c_int
        lib.span_la_cache_decay_branches.argtypes = [vp, vp, vp, vp, vp, Dims, vp, i32p, ctypes.c_int32, vp, vp]
        lib.span_la_cache_decay_branches.restype = ctypes.c_int
        lib.span_la_cache_stats.argtypes = [vp, ctypes.POINTER(ctypes.c_int64)]
        lib.span_la_cache_stats.restype = ctypes.c_int
        if path is None:
            _lib = lib
            _bind_fast(lib)
        return lib


def _bind_fast(lib) -> None:
    global _fast
    try:
        from . import _fastcall
    except ImportError:   # not built: the same calls by way of ctypes
        return
    if getattr(_fastcall, "torch_version", None) != str(torch.__version__):   # built for another one
        return
    _fastcall.bind(*[ctypes.cast(f, ctypes.c_void_p).value
                     for f in (lib.span_la_decay_pass, lib.span_la_decay_branches_from_state, lib.span_la_decay_step,
                               lib.span_la_qk_norm_rope, lib.span_la_kv_write, lib.span_la_kv_read, lib.span_la_softmax_paged,
                               lib.span_la_softmax_paged_workspace)])
    _fast = _fastcall


def _raise(lib, status: int, where: str):
    if status != 0:
        raise SpanLAError(status, where, lib.span_la_last_error_detail().decode())


def _i32(a) -> np.ndarray:
    if a is None:
        return np.zeros(0, dtype=np.int32)
    if isinstance(a, np.ndarray) and a.dtype == np.int32 and a.ndim == 1 and a.flags.c_contiguous:
        return a
    if isinstance(a, torch.Tensor):
        a = a.detach().cpu().numpy()
    a = np.asarray(a)
    if a.size and not (a.min() >= -2 ** 31 and a.max() < 2 ** 31):
        raise ValueError("offsets and indices must fit 32 bits")
    return np.ascontiguousarray(a.reshape(-1).astype(np.int32))


def _iptr(a: np.ndarray):
    """Address of an int32 array for a ``const int32_t*`` argument (None when empty)."""
    if a.size == 0:
        return None
    if a.flags.writeable:   # (cheaper than numpy's .ctypes helper object)
        return ctypes.addressof(ctypes.c_int32.from_buffer(a))
    return a.ctypes.data


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_raw_device = getattr(torch._C, "_cuda_getDevice", None)


def _stream_handle(stream) -> int:
    """The CUDA stream handle for a call: ``stream``'s, or the current device's
    current stream."""
    if stream is None:
        if _raw_stream is not None and _raw_device is not None:
            return int(_raw_stream(_raw_device()))
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream)


def _new(shape, dtype: torch.dtype, device, stream=None) -> torch.Tensor:
    """A new output of a call on ``stream``.  On another stream than the current one it is that stream's memory, which no
    work still pending elsewhere has held, and is not handed out again before the current stream, too, has passed the
    tensor's last use."""
    if stream is not None:
        here = torch.cuda.current_stream(device)
        if int(stream.cuda_stream) != int(here.cuda_stream):
            if not isinstance(stream, torch.cuda.Stream):
                stream = torch.cuda.ExternalStream(int(stream.cuda_stream), device=device)
            with torch.cuda.stream(stream):
                x = torch.empty(shape, dtype=dtype, device=device)
            x.record_stream(here)
            return x
    return torch.empty(shape, dtype=dtype, device=device)


def _dims_of(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor) -> Dims:
    # The usual case in one expression; anything else goes through the
    # checks below, which name the problem.
    sh, dt = q.shape, q.dtype
    if (len(sh) == 3 and sh[2] == 64 and k.shape == sh and v.shape == sh and k.dtype == dt
            and v.dtype == dt and (dt == torch.bfloat16 or dt == torch.float32)
            and q.is_cuda and k.is_cuda and v.is_cuda
            and q.is_contiguous() and k.is_contiguous() and v.is_contiguous()):
        return Dims(sh[0], sh[1], 64, SPAN_LA_BF16 if dt == torch.bfloat16 else SPAN_LA_F32)
    return _dims_checked(q, k, v)


def _dims_checked(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor) -> Dims:
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not t.is_cuda:
            raise ValueError("%s must be a CUDA tensor" % name)
        if t.dim() != 3 or t.shape[2] != 64:
            raise ValueError("%s must be [T, H, 64], got %s" % (name, tuple(t.shape)))
        if not t.is_contiguous():
            raise ValueError("%s must be contiguous" % name)
    if q.shape != k.shape or q.shape != v.shape or q.dtype != k.dtype or q.dtype != v.dtype:
        raise ValueError("q, k and v must share shape and dtype")
    if q.dtype == torch.bfloat16:
        dt = SPAN_LA_BF16
    elif q.dtype == torch.float32:
        dt = SPAN_LA_F32
    else:
        raise ValueError("dtype %s not supported (bf16 or fp32)" % q.dtype)
    return Dims(q.shape[0], q.shape[1], q.shape[2], dt)


def span_la_pass(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                 view_cu_seqlens: Sequence[int], branch_cu_seqlens: Optional[Sequence[int]],
                 branch_parent: Optional[Sequence[int]],
                 out: Optional[torch.Tensor] = None,
                 view_state_out: Optional[torch.Tensor] = None,
                 stream: Optional[torch.cuda.Stream] = None,
                 _entry: str = "span_la_pass") -> Tuple[torch.Tensor, torch.Tensor]:
    """One packed pass (see ``span_la_pass`` in ``include/spanla.h``).

    Returns ``(out [T,H,64], view_state_out [V,H,64,64] fp32)``.  ``out`` is
    allocated with ``torch.empty`` when not given: rows in no segment then
    hold whatever the allocator returned.
    """
    lib = load_library()
    dims = _dims_of(q, k, v)
    vcu, bcu, par = _i32(view_cu_seqlens), _i32(branch_cu_seqlens), _i32(branch_parent)
    V = max(len(vcu) - 1, 0)
    B = max(len(bcu) - 1, 0)
    H = q.shape[1]
    if out is None:
        out = _new(q.shape, q.dtype, q.device, stream)
    if view_state_out is None:
        view_state_out = _new((V, H, 64, 64), torch.float32, q.device, stream)
    if out.shape != q.shape or out.dtype != q.dtype or not out.is_contiguous() or not out.is_cuda:
        raise ValueError("out must be a contiguous CUDA tensor like q")
    if (view_state_out.dtype != torch.float32 or not view_state_out.is_contiguous()
            or not view_state_out.is_cuda or view_state_out.numel() < V * H * 4096):
        raise ValueError("view_state_out must be a contiguous fp32 CUDA tensor [V, H, 64, 64]")
    st = getattr(lib, _entry)(q.data_ptr(), k.data_ptr(), v.data_ptr(), dims,
                              _iptr(vcu), V, _iptr(bcu), B, _iptr(par),
                              out.data_ptr(), view_state_out.data_ptr(), _stream_handle(stream))
    _raise(lib, st, _entry)
    return out, view_state_out


def span_la_plan_prepare(view_cu_seqlens: Sequence[int], branch_cu_seqlens: Optional[Sequence[int]],
                         branch_parent: Optional[Sequence[int]], total_rows: int, num_heads: int,
                         dtype: torch.dtype = torch.bfloat16,
                         stream: Optional[torch.cuda.Stream] = None) -> None:
    """Build and upload the plan of a later :func:`span_la_pass` with this
    metadata on the current device (``span_la_plan_prepare`` in
    ``include/spanla.h``), so that the pass finds it in the plan cache."""
    lib = load_library()
    if dtype == torch.bfloat16:
        dt = SPAN_LA_BF16
    elif dtype == torch.float32:
        dt = SPAN_LA_F32
    else:
        raise ValueError("dtype %s not supported (bf16 or fp32)" % dtype)
    vcu, bcu, par = _i32(view_cu_seqlens), _i32(branch_cu_seqlens), _i32(branch_parent)
    V = max(len(vcu) - 1, 0)
    B = max(len(bcu) - 1, 0)
    st = lib.span_la_plan_prepare(Dims(int(total_rows), int(num_heads), 64, dt), _iptr(vcu), V,
                                  _iptr(bcu), B, _iptr(par), _stream_handle(stream))
    _raise(lib, st, "span_la_plan_prepare")


def span_la_pass_noalloc(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                         view_cu_seqlens: Sequence[int], branch_cu_seqlens: Optional[Sequence[int]],
                         branch_parent: Optional[Sequence[int]],
                         out: Optional[torch.Tensor] = None,
                         view_state_out: Optional[torch.Tensor] = None,
                         stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """As :func:`span_la_pass`, with the workspace in the library's fixed
    scratch instead of a per-call allocation (``span_la_pass_noalloc``)."""
    return span_la_pass(q, k, v, view_cu_seqlens, branch_cu_seqlens, branch_parent, out=out,
                        view_state_out=view_state_out, stream=stream, _entry="span_la_pass_noalloc")


def span_la_branches_from_state(cached_state: torch.Tensor, q: torch.Tensor, k: torch.Tensor,
                                v: torch.Tensor, branch_cu_seqlens: Sequence[int],
                                branch_parent: Sequence[int],
                                out: Optional[torch.Tensor] = None,
                                stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Branches forking from cached view states (``span_la_branches_from_state``)."""
    lib = load_library()
    dims = _dims_of(q, k, v)
    bcu, par = _i32(branch_cu_seqlens), _i32(branch_parent)
    B = max(len(bcu) - 1, 0)
    if (cached_state.dtype != torch.float32 or not cached_state.is_contiguous()
            or not cached_state.is_cuda or cached_state.dim() != 4
            or tuple(cached_state.shape[1:]) != (q.shape[1], 64, 64)):
        raise ValueError("cached_state must be contiguous fp32 CUDA [P, H, 64, 64]")
    if out is None:
        out = _new(q.shape, q.dtype, q.device, stream)
    if out.shape != q.shape or out.dtype != q.dtype or not out.is_contiguous() or not out.is_cuda:
        raise ValueError("out must be a contiguous CUDA tensor like q")
    st = lib.span_la_branches_from_state(cached_state.data_ptr(), cached_state.shape[0],
                                         q.data_ptr(), k.data_ptr(), v.data_ptr(), dims,
                                         _iptr(bcu), B, _iptr(par), out.data_ptr(),
                                         _stream_handle(stream))
    _raise(lib, st, "span_la_branches_from_state")
    return out


def span_la_softmax_pass(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                         view_cu_seqlens: Sequence[int], branch_cu_seqlens: Sequence[int],
                         branch_parent: Sequence[int], scale: float = 0.0,
                         out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                         stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """One softmax-attention layer over the packed rows (``span_la_softmax_pass``):
    views causal, branches over their parent view plus their own causal prefix.
    ``lse`` (fp32 [T, H], optional) receives the natural-log normaliser."""
    lib = load_library()
    dims = _dims_of(q, k, v)
    vcu, bcu, par = _i32(view_cu_seqlens), _i32(branch_cu_seqlens), _i32(branch_parent)
    V = max(len(vcu) - 1, 0)
    B = max(len(bcu) - 1, 0)
    if out is None:
        out = _new(q.shape, q.dtype, q.device, stream)
    if out.shape != q.shape or out.dtype != q.dtype or not out.is_contiguous() or not out.is_cuda:
        raise ValueError("out must be a contiguous CUDA tensor like q")
    if lse is not None and (lse.dtype != torch.float32 or not lse.is_contiguous() or not lse.is_cuda
                            or tuple(lse.shape) != (q.shape[0], q.shape[1])):
        raise ValueError("lse must be contiguous fp32 CUDA [T, H]")
    st = lib.span_la_softmax_pass(q.data_ptr(), k.data_ptr(), v.data_ptr(), dims, _iptr(vcu), V,
                                  _iptr(bcu), B, _iptr(par), float(scale), out.data_ptr(),
                                  lse.data_ptr() if lse is not None else None,
                                  _stream_handle(stream))
    _raise(lib, st, "span_la_softmax_pass")
    return out


def span_la_softmax_branches_from_kv(view_k: torch.Tensor, view_v: torch.Tensor,
                                     view_cu_seqlens: Sequence[int], q: torch.Tensor, k: torch.Tensor,
                                     v: torch.Tensor, branch_cu_seqlens: Sequence[int],
                                     branch_parent: Sequence[int], scale: float = 0.0,
                                     out: Optional[torch.Tensor] = None,
                                     lse: Optional[torch.Tensor] = None,
                                     stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Softmax-layer branches over their parent views' K and V kept from an
    earlier pass (``span_la_softmax_branches_from_kv``)."""
    lib = load_library()
    dims = _dims_of(q, k, v)
    for name, t in (("view_k", view_k), ("view_v", view_v)):
        if (not t.is_cuda or t.dtype != q.dtype or not t.is_contiguous() or t.dim() != 3
                or tuple(t.shape[1:]) != tuple(q.shape[1:])):
            raise ValueError("%s must be a contiguous CUDA tensor [rows, H, 64] like q" % name)
    if view_k.shape != view_v.shape:
        raise ValueError("view_k and view_v must share shape")
    vcu, bcu, par = _i32(view_cu_seqlens), _i32(branch_cu_seqlens), _i32(branch_parent)
    V = max(len(vcu) - 1, 0)
    B = max(len(bcu) - 1, 0)
    if out is None:
        out = _new(q.shape, q.dtype, q.device, stream)
    if out.shape != q.shape or out.dtype != q.dtype or not out.is_contiguous() or not out.is_cuda:
        raise ValueError("out must be a contiguous CUDA tensor like q")
    if lse is not None and (lse.dtype != torch.float32 or not lse.is_contiguous() or not lse.is_cuda
                            or tuple(lse.shape) != (q.shape[0], q.shape[1])):
        raise ValueError("lse must be contiguous fp32 CUDA [T, H]")
    st = lib.span_la_softmax_branches_from_kv(
        view_k.data_ptr(), view_v.data_ptr(), view_k.shape[0], _iptr(vcu), V, q.data_ptr(),
        k.data_ptr(), v.data_ptr(), dims, _iptr(bcu), B, _iptr(par), float(scale), out.data_ptr(),
        lse.data_ptr() if lse is not None else None, _stream_handle(stream))
    _raise(lib, st, "span_la_softmax_branches_from_kv")
    return out


def _current_device() -> int:
    return _raw_device() if _raw_device is not None else torch.cuda.current_device()


def _on_device(dev: int, name: str, t: torch.Tensor) -> None:
    """The library runs on the current device: its tensors have to be there."""
    if t.get_device() != dev:
        raise ValueError("%s must be on the current CUDA device (%d), got %s" % (name, dev, t.device))


def _decay_args(q, k, v, log_decay, out, stream) -> Tuple[Dims, torch.Tensor, int]:
    """What the decayed calls check alike: q, k, v (as _dims_of), log_decay (may be None here) and out (allocated when
    None).  Returns the dims, out and the current device.  The usual case costs one look at each attribute."""
    dims = _dims_of(q, k, v)
    dev = _current_device()
    if q.get_device() != dev or k.get_device() != dev or v.get_device() != dev:
        for name, t in (("q", q), ("k", k), ("v", v)):
            _on_device(dev, name, t)
    if log_decay is not None:
        sh = log_decay.shape
        if (log_decay.dtype != torch.float32 or not log_decay.is_contiguous() or len(sh) != 1 or sh[0] != dims.num_heads
                or not log_decay.is_cuda):
            raise ValueError("log_decay must be contiguous fp32 CUDA [H]")
        _on_device(dev, "log_decay", log_decay)
    if out is None:
        return dims, _new(q.shape, q.dtype, q.device, stream), dev
    if out.shape != q.shape or out.dtype != q.dtype or not out.is_contiguous() or not out.is_cuda:
        raise ValueError("out must be a contiguous CUDA tensor like q")
    _on_device(dev, "out", out)
    return dims, out, dev


def _check_states(name: str, x: torch.Tensor, H: int, dev: int) -> int:
    """x as contiguous fp32 CUDA [n, H, 64, 64] on the current device; returns n."""
    sh = x.shape
    if (len(sh) != 4 or sh[1] != H or sh[2] != 64 or sh[3] != 64 or x.dtype != torch.float32 or not x.is_contiguous()
            or not x.is_cuda):
        raise ValueError("%s must be contiguous fp32 CUDA [n, H, 64, 64]" % name)
    _on_device(dev, name, x)
    return sh[0]


def span_la_decay_pass(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor,
                       view_cu_seqlens: Sequence[int], branch_cu_seqlens: Optional[Sequence[int]],
                       branch_parent: Optional[Sequence[int]], out: Optional[torch.Tensor] = None,
                       view_state_out: Optional[torch.Tensor] = None,
                       stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """One packed pass of linear attention with a decay for each head
    (``span_la_decay_pass`` in ``include/spanla.h``): ``log_decay`` is fp32
    CUDA [H], the rest as for :func:`span_la_pass`.

    Returns ``(out [T,H,64], view_state_out [V,H,64,64] fp32)``.
    """
    if _fast is not None:   # (None: an argument that the code below takes or refuses)
        r = _fast.decay_pass(q, k, v, log_decay, view_cu_seqlens, branch_cu_seqlens, branch_parent, out, view_state_out,
                             stream)
        if r is not None:
            if type(r) is int:
                _raise(_lib, r, "span_la_decay_pass")
            return r
    lib = _lib or load_library()
    if log_decay is None:
        raise ValueError("log_decay must be contiguous fp32 CUDA [H]")
    dims, out, dev = _decay_args(q, k, v, log_decay, out, stream)
    vcu, bcu, par = _i32(view_cu_seqlens), _i32(branch_cu_seqlens), _i32(branch_parent)
    V = max(len(vcu) - 1, 0)
    B = max(len(bcu) - 1, 0)
    if par.size != B:
        raise ValueError("one parent per branch")
    H = dims.num_heads
    if view_state_out is None:
        view_state_out = _new((V, H, 64, 64), torch.float32, q.device, stream)
    elif _check_states("view_state_out", view_state_out, H, dev) < V:
        raise ValueError("view_state_out must hold %d states" % V)
    st = lib.span_la_decay_pass(q.data_ptr(), k.data_ptr(), v.data_ptr(), dims, log_decay.data_ptr(), _iptr(vcu), V,
                                _iptr(bcu), B, _iptr(par), out.data_ptr(), view_state_out.data_ptr(),
                                _stream_handle(stream))
    _raise(lib, st, "span_la_decay_pass")
    return out, view_state_out


def span_la_decay_branches_from_state(cached_state: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                                      log_decay: torch.Tensor, branch_cu_seqlens: Sequence[int],
                                      branch_parent: Sequence[int], out: Optional[torch.Tensor] = None,
                                      stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Branches of a decayed pass from kept view states
    (``span_la_decay_branches_from_state``)."""
    if _fast is not None:
        r = _fast.decay_fork(cached_state, q, k, v, log_decay, branch_cu_seqlens, branch_parent, out, stream)
        if r is not None:
            if type(r) is int:
                _raise(_lib, r, "span_la_decay_branches_from_state")
            return r
    lib = _lib or load_library()
    if log_decay is None:
        raise ValueError("log_decay must be contiguous fp32 CUDA [H]")
    dims, out, dev = _decay_args(q, k, v, log_decay, out, stream)
    n = _check_states("cached_state", cached_state, dims.num_heads, dev)
    bcu, par = _i32(branch_cu_seqlens), _i32(branch_parent)
    B = max(len(bcu) - 1, 0)
    if par.size != B:
        raise ValueError("one parent per branch")
    st = lib.span_la_decay_branches_from_state(cached_state.data_ptr(), n, q.data_ptr(),
                                               k.data_ptr(), v.data_ptr(), dims, log_decay.data_ptr(), _iptr(bcu), B,
                                               _iptr(par), out.data_ptr(), _stream_handle(stream))
    _raise(lib, st, "span_la_decay_branches_from_state")
    return out


def span_la_decay_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, states: torch.Tensor,
                       log_decay: Optional[torch.Tensor] = None, state_index: Optional[Sequence[int]] = None,
                       out: Optional[torch.Tensor] = None,
                       stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """One new token of each of n sequences (``span_la_decay_step``): q, k, v
    are [n, H, 64]; ``states`` (fp32 CUDA [P, H, 64, 64]) is updated in place.
    ``state_index`` (host, n entries) names each row's state, -1 for a row to
    skip; without it row t uses state t.  Without ``log_decay`` nothing decays.
    Returns the outputs [n, H, 64]."""
    if _fast is not None:
        r = _fast.decay_step(q, k, v, states, log_decay, state_index, out, stream)
        if r is not None:
            if type(r) is int:
                _raise(_lib, r, "span_la_decay_step")
            return r
    lib = _lib or load_library()
    dims, out, dev = _decay_args(q, k, v, log_decay, out, stream)
    n = _check_states("states", states, dims.num_heads, dev)
    index = None
    if state_index is not None:
        keep = _i32(state_index)
        if keep.size != dims.total_rows:
            raise ValueError("one state index per row")
        index = _iptr(keep)
    st = lib.span_la_decay_step(q.data_ptr(), k.data_ptr(), v.data_ptr(), dims,
                                None if log_decay is None else log_decay.data_ptr(), states.data_ptr(), n, index,
                                out.data_ptr(), _stream_handle(stream))
    _raise(lib, st, "span_la_decay_step")
    return out


def rope_inv_freq(rotary_dim: int, base: float = 10000.0) -> np.ndarray:
    """The usual frequencies base^(-2 i / rotary_dim), i < rotary_dim / 2, for
    :func:`span_la_qk_norm_rope` (float64, host)."""
    return float(base) ** (-2.0 * np.arange(rotary_dim // 2, dtype=np.float64) / rotary_dim)


def packed_positions(view_cu_seqlens: Sequence[int], branch_cu_seqlens: Optional[Sequence[int]],
                     branch_parent: Optional[Sequence[int]], total_rows: int) -> np.ndarray:
    """Positions of a packed pass's rows (host int32 [total_rows]) for
    :func:`span_la_qk_norm_rope`: a view's rows count from 0, a branch's go on
    from its parent view's length, and rows in no segment get -1 (skipped)."""
    vcu, bcu, par = _i32(view_cu_seqlens), _i32(branch_cu_seqlens), _i32(branch_parent)
    V, B = max(len(vcu) - 1, 0), max(len(bcu) - 1, 0)
    if par.size != B or (B and not (0 <= par.min() and par.max() < V)):
        raise ValueError("one parent per branch, in [0, %d)" % V)
    for cu in (vcu, bcu):
        if cu.size and (cu[0] < 0 or cu[-1] > total_rows or (cu[1:] < cu[:-1]).any()):
            raise ValueError("row offsets must be non-decreasing in [0, total_rows]")
    pos = np.full(int(total_rows), -1, dtype=np.int32)
    for s in range(V):
        pos[vcu[s]:vcu[s + 1]] = np.arange(vcu[s + 1] - vcu[s], dtype=np.int32)
    for b in range(B):
        p = int(par[b])
        pos[bcu[b]:bcu[b + 1]] = np.arange(bcu[b + 1] - bcu[b], dtype=np.int32) + (vcu[p + 1] - vcu[p])
    return pos


def _row_stride(name: str, x: torch.Tensor, T: int, H: int) -> int:
    """The row stride of [T, H, 64] whose heads lie next to each other in a row."""
    s0, s1, s2 = x.stride()
    if (s2 != 1 or (s1 != 64 and H > 1)) and T > 0 and H > 0:
        raise ValueError("%s: the heads of a row must lie next to each other" % name)
    return s0 if T > 1 else H * 64


def _qk_side(name: str, x: torch.Tensor, T: int, weight: Optional[torch.Tensor], out: Optional[torch.Tensor],
             dev: int, stream) -> Tuple[QkSide, torch.Tensor]:
    """The C struct of one side of span_la_qk_norm_rope, and its output."""
    sh = x.shape
    if len(sh) != 3 or sh[2] != 64 or not x.is_cuda:
        raise ValueError("%s must be a CUDA tensor [T, H, 64], got %s" % (name, tuple(sh)))
    _on_device(dev, name, x)
    H = sh[1]
    if out is None:
        out = _new((T, H, 64), x.dtype, x.device, stream)
        out_stride = H * 64
    else:
        if out.shape != sh or out.dtype != x.dtype or not out.is_cuda:
            raise ValueError("%s_out must be a CUDA tensor of %s's shape and type" % (name, name))
        _on_device(dev, name + "_out", out)
        out_stride = _row_stride(name + "_out", out, T, H)
    per_head, wp = 0, None
    if weight is not None:
        wsh = weight.shape
        per_head = len(wsh) - 1
        if (not weight.is_cuda or not weight.is_contiguous() or wsh[-1] != 64 or per_head not in (0, 1)
                or (per_head and wsh[0] != H)):
            raise ValueError("%s_weight must be contiguous CUDA [64] or [H, 64]" % name)
        _on_device(dev, name + "_weight", weight)
        wp = weight.data_ptr()
    return QkSide(x.data_ptr(), out.data_ptr(), wp, _row_stride(name, x, T, H), out_stride, H, per_head), out


_DTYPES = {torch.bfloat16: SPAN_LA_BF16, torch.float32: SPAN_LA_F32}


def span_la_qk_norm_rope(q: torch.Tensor, k: torch.Tensor, positions: torch.Tensor, inv_freq,
                         q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None,
                         eps: float = 1e-6, interleaved: bool = False, q_out: Optional[torch.Tensor] = None,
                         k_out: Optional[torch.Tensor] = None,
                         stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """RMS norm of every head of q [T, Hq, 64] and k [T, Hk, 64], then the
    rotation by ``positions`` (CUDA int32 [T]; negative: the row is skipped)
    (``span_la_qk_norm_rope``).

    ``inv_freq`` holds rotary_dim / 2 host values in radians per position
    (:func:`rope_inv_freq`; None or empty: norm only).  q and k may be strided
    parts of a fused projection's rows; weights are [64] or [H, 64].  Returns
    (q_out, k_out), allocated contiguous when not given; an output may be its
    own input."""
    if _fast is not None:
        r = _fast.qk_norm_rope(q, k, positions, inv_freq, q_weight, k_weight, eps, interleaved, q_out, k_out, stream)
        if r is not None:
            if type(r) is int:
                _raise(_lib, r, "span_la_qk_norm_rope")
            return r
    lib = _lib or load_library()
    dt = _DTYPES.get(q.dtype)
    if dt is None:
        raise ValueError("dtype %s not supported (bf16 or fp32)" % q.dtype)
    T = q.shape[0]
    if k.dtype != q.dtype or k.shape[0] != T:
        raise ValueError("q and k must share dtype and rows")
    if not q.is_cuda or not k.is_cuda:
        raise ValueError("q and k must be CUDA tensors")
    wdt = dt
    if q_weight is not None or k_weight is not None:
        wt = (k_weight if q_weight is None else q_weight).dtype
        if wt not in _DTYPES:
            raise ValueError("weight dtype %s not supported (bf16 or fp32)" % wt)
        if k_weight is not None and k_weight.dtype != wt:
            raise ValueError("q_weight and k_weight must share dtype")
        wdt = _DTYPES[wt]
    dev = _current_device()
    qs, q_out = _qk_side("q", q, T, q_weight, q_out, dev, stream)
    ks, k_out = _qk_side("k", k, T, k_weight, k_out, dev, stream)
    psh = positions.shape
    if (positions.dtype != torch.int32 or not positions.is_contiguous() or len(psh) != 1 or psh[0] != T
            or not positions.is_cuda):
        raise ValueError("positions must be contiguous int32 CUDA [T]")
    _on_device(dev, "positions", positions)
    freq, rotary = None, 0
    if inv_freq is not None:
        if isinstance(inv_freq, torch.Tensor) and inv_freq.is_cuda:
            raise ValueError("inv_freq holds host values")
        keep = np.ascontiguousarray(inv_freq, dtype=np.float64)
        rotary = 2 * keep.size
        if rotary:
            freq = keep.ctypes.data
    st = lib.span_la_qk_norm_rope(qs, ks, T, dt, wdt, eps, freq, rotary, 1 if interleaved else 0, positions.data_ptr(),
                                  _stream_handle(stream))
    _raise(lib, st, "span_la_qk_norm_rope")
    return q_out, k_out


def kv_pages(num_pages: int, num_heads: int, page_rows: int, dtype: torch.dtype = torch.bfloat16, device=None):
    """Zeroed pages of a paged cache: ``(k_pages, v_pages, k_scale, v_scale)``,
    the pages [num_pages, num_heads, page_rows, 64] of ``dtype`` (bf16 or
    float8_e4m3fn), the scales uint8 [num_pages, num_heads, page_rows] or None."""
    if dtype not in _PAGE_DTYPES:
        raise ValueError("page dtype %s not supported (bf16 or float8_e4m3fn)" % dtype)
    dev = torch.device("cuda") if device is None else device
    shape = (int(num_pages), int(num_heads), int(page_rows))
    if dtype == torch.bfloat16:
        return tuple(torch.zeros(shape + (64,), dtype=dtype, device=dev) for _ in range(2)) + (None, None)
    pages = tuple(torch.zeros(shape + (64,), dtype=torch.uint8, device=dev).view(dtype) for _ in range(2))
    return pages + tuple(torch.full(shape, 127, dtype=torch.uint8, device=dev) for _ in range(2))


_PAGE_DTYPES = {torch.bfloat16: SPAN_LA_BF16, torch.float8_e4m3fn: SPAN_LA_E4M3}


def _i32_on(dev: int, name: str, x: torch.Tensor, shape) -> int:
    """The address of a contiguous int32 CUDA tensor of a shape."""
    if x.dtype != torch.int32 or not x.is_cuda or tuple(x.shape) != tuple(shape) or not x.is_contiguous():
        raise ValueError("%s must be contiguous int32 CUDA [%s]" % (name, ", ".join(str(n) for n in shape)))
    _on_device(dev, name, x)
    return x.data_ptr()


def _kv_cache(k_pages: torch.Tensor, v_pages: torch.Tensor, page_table: torch.Tensor, seq_len: torch.Tensor,
              row_cu: Optional[torch.Tensor], k_scale: Optional[torch.Tensor], v_scale: Optional[torch.Tensor]) -> Tuple[KvCache, int]:
    """The C struct of a paged cache, and the current device."""
    sh, st = k_pages.shape, k_pages.stride()
    for name, x in (("k_pages", k_pages), ("v_pages", v_pages)):
        if x.dim() != 4 or x.shape[3] != 64 or not x.is_cuda:
            raise ValueError("%s must be a CUDA tensor [num_pages, num_heads, page_rows, 64], got %s" % (name, tuple(x.shape)))
        if x.stride(3) != 1:
            raise ValueError("%s: the 64 elements of a row must lie next to each other" % name)
    dev = _current_device()
    _on_device(dev, "k_pages", k_pages)
    _on_device(dev, "v_pages", v_pages)
    if v_pages.shape != sh or v_pages.dtype != k_pages.dtype or v_pages.stride() != st:
        raise ValueError("k_pages and v_pages must share shape, dtype and strides")
    dt = _PAGE_DTYPES.get(k_pages.dtype)
    if dt is None:
        raise ValueError("page dtype %s not supported (bf16 or float8_e4m3fn)" % k_pages.dtype)
    if page_table.dim() != 2 or page_table.dtype != torch.int32 or not page_table.is_cuda or (
            page_table.shape[1] > 1 and page_table.stride(1) != 1):
        raise ValueError("page_table must be int32 CUDA [num_seqs, width], the entries of a row next to each other")
    _on_device(dev, "page_table", page_table)
    S, width = page_table.shape
    c = KvCache(k_pages.data_ptr(), v_pages.data_ptr(), None, None, st[0], st[1], st[2], 0, 0, sh[0], sh[2], sh[1], dt, S, width,
                page_table.stride(0) if S > 1 else width, page_table.data_ptr(), _i32_on(dev, "seq_len", seq_len, (S,)),
                None if row_cu is None else _i32_on(dev, "row_cu", row_cu, (S + 1,)))
    if dt == SPAN_LA_E4M3:
        for name, x in (("k_scale", k_scale), ("v_scale", v_scale)):
            if (x is None or x.dtype != torch.uint8 or not x.is_cuda or tuple(x.shape) != tuple(sh[:3])
                    or x.stride(2) != 1 or x.stride() != k_scale.stride()):
                raise ValueError("%s must be uint8 CUDA [num_pages, num_heads, page_rows], the bytes of a page and head next to "
                                 "each other, k_scale and v_scale of the same strides" % name)
            _on_device(dev, name, x)
        c.k_scale, c.v_scale = k_scale.data_ptr(), v_scale.data_ptr()
        c.scale_page_stride, c.scale_head_stride = k_scale.stride(0), k_scale.stride(1)
    elif k_scale is not None or v_scale is not None:
        raise ValueError("bf16 pages have no scales")
    return c, dev


def _packed(name: str, x: torch.Tensor, H: Optional[int], dev: int) -> int:
    """x as rows [T, H, 64] on the device; returns its row stride."""
    if x.dim() != 3 or x.shape[2] != 64 or not x.is_cuda or (H is not None and x.shape[1] != H):
        raise ValueError("%s must be a CUDA tensor [T, %s, 64], got %s" % (name, "H" if H is None else H, tuple(x.shape)))
    _on_device(dev, name, x)
    return _row_stride(name, x, x.shape[0], x.shape[1])


def span_la_kv_write(k: torch.Tensor, v: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, page_table: torch.Tensor,
                     seq_len: torch.Tensor, row_cu: Optional[torch.Tensor] = None, k_scale: Optional[torch.Tensor] = None,
                     v_scale: Optional[torch.Tensor] = None, stream: Optional[torch.cuda.Stream] = None) -> None:
    """New rows k, v [T, H, 64] (bf16 or fp32; parts of a fused projection's rows
    will do) into their places in the paged cache (``span_la_kv_write``).

    ``k_pages``, ``v_pages``: [num_pages, H, page_rows, 64] bf16, or float8_e4m3fn
    with uint8 scales [num_pages, H, page_rows] (:func:`kv_pages`).  On the device,
    int32: ``page_table`` [S, width], ``seq_len`` [S] (rows in the cache after the
    call) and ``row_cu`` [S + 1]: packed rows row_cu[s] .. row_cu[s + 1] are the
    last ones of sequence s (None: one row of each sequence)."""
    if _fast is not None:
        r = _fast.kv_write(k, v, k_pages, v_pages, page_table, seq_len, row_cu, k_scale, v_scale, stream)
        if r is not None:
            if r is not True:
                _raise(_lib, r, "span_la_kv_write")
            return
    lib = _lib or load_library()
    c, dev = _kv_cache(k_pages, v_pages, page_table, seq_len, row_cu, k_scale, v_scale)
    dt = _DTYPES.get(k.dtype)
    if dt is None:
        raise ValueError("dtype %s not supported (bf16 or fp32)" % k.dtype)
    if v.dtype != k.dtype or v.shape != k.shape:
        raise ValueError("k and v must share shape and dtype")
    ks, vs = _packed("k", k, c.num_heads, dev), _packed("v", v, c.num_heads, dev)
    _raise(lib, lib.span_la_kv_write(k.data_ptr(), v.data_ptr(), ks, vs, k.shape[0], dt, c, _stream_handle(stream)),
           "span_la_kv_write")


def span_la_kv_read(k_pages: torch.Tensor, v_pages: torch.Tensor, page_table: torch.Tensor, seq_len: torch.Tensor,
                    row_cu: Optional[torch.Tensor], total_rows: Optional[int] = None, k_scale: Optional[torch.Tensor] = None,
                    v_scale: Optional[torch.Tensor] = None, dtype: torch.dtype = torch.bfloat16,
                    k_out: Optional[torch.Tensor] = None, v_out: Optional[torch.Tensor] = None,
                    stream: Optional[torch.cuda.Stream] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The packed rows out of the cache (``span_la_kv_read``; the cache as for
    :func:`span_la_kv_write`): k and v [T, H, 64] of ``dtype`` (bf16 or fp32), T =
    ``total_rows`` (default: the given outputs' rows, or one a sequence).  With a
    kept view's length in row_cu and seq_len, they are the view_k and view_v of
    :func:`span_la_softmax_branches_from_kv`."""
    if _fast is not None and k_out is None and v_out is None and dtype in _DTYPES:
        r = _fast.kv_read(k_pages, v_pages, page_table, seq_len, row_cu, total_rows, k_scale, v_scale, dtype is torch.bfloat16, stream)
        if r is not None:
            if type(r) is int:
                _raise(_lib, r, "span_la_kv_read")
            return r
    lib = _lib or load_library()
    c, dev = _kv_cache(k_pages, v_pages, page_table, seq_len, row_cu, k_scale, v_scale)
    if total_rows is None:
        given = k_out if k_out is not None else v_out
        if given is None and row_cu is not None:
            raise ValueError("total_rows, or an output, says how many rows there are")
        total_rows = c.num_seqs if given is None else given.shape[0]
    outs = []
    for name, x in (("k_out", k_out), ("v_out", v_out)):
        if x is None:
            x = _new((int(total_rows), c.num_heads, 64), dtype, k_pages.device, stream)
        elif (tuple(x.shape) != (int(total_rows), c.num_heads, 64) or x.dtype != dtype or not x.is_cuda or not x.is_contiguous()):
            raise ValueError("%s must be a contiguous CUDA tensor [%d, %d, 64] of %s" % (name, total_rows, c.num_heads, dtype))
        else:
            _on_device(dev, name, x)
        outs.append(x)
    dt = _DTYPES.get(dtype)
    if dt is None:
        raise ValueError("dtype %s not supported (bf16 or fp32)" % dtype)
    _raise(lib, lib.span_la_kv_read(c, int(total_rows), dt, outs[0].data_ptr(), outs[1].data_ptr(), _stream_handle(stream)),
           "span_la_kv_read")
    return outs[0], outs[1]


def span_la_softmax_paged(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, page_table: torch.Tensor,
                          seq_len: torch.Tensor, row_cu: Optional[torch.Tensor] = None, k_scale: Optional[torch.Tensor] = None,
                          v_scale: Optional[torch.Tensor] = None, max_rows: Optional[int] = None, scale: float = 0.0,
                          out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                          stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Softmax attention of q [T, Hq, 64] (bf16; parts of a fused projection's
    rows will do) over the paged cache (``span_la_softmax_paged``; the cache as for
    :func:`span_la_kv_write`, which has written the rows' own keys and values
    before): row i of a sequence sees the sequence's rows up to itself, query head
    h the key head h // (Hq // H).  ``max_rows``: the most packed rows of a sequence
    where it is known (1 without ``row_cu``); calls of few rows, and of 2,048 row
    heads and more over e4m3 pages, are faster with it.  ``lse`` (fp32 [T, Hq], optional)
    receives the natural-log normaliser.  Returns [T, Hq, 64]."""
    if _fast is not None:
        r = _fast.softmax_paged(q, k_pages, v_pages, page_table, seq_len, row_cu, k_scale, v_scale, max_rows, scale, out, lse, stream)
        if r is not None:
            if type(r) is int:
                _raise(_lib, r, "span_la_softmax_paged")
            return r
    lib = _lib or load_library()
    c, dev = _kv_cache(k_pages, v_pages, page_table, seq_len, row_cu, k_scale, v_scale)
    qs = _packed("q", q, None, dev)
    if q.dtype != torch.bfloat16:
        raise ValueError("q must be bf16, got %s" % q.dtype)
    T, H = q.shape[0], q.shape[1]
    if out is None:
        out = _new((T, H, 64), q.dtype, q.device, stream)
    elif out.shape != q.shape or out.dtype != q.dtype or not out.is_contiguous() or not out.is_cuda:
        raise ValueError("out must be a contiguous CUDA tensor like q")
    else:
        _on_device(dev, "out", out)
    if lse is not None:
        if lse.dtype != torch.float32 or not lse.is_contiguous() or not lse.is_cuda or tuple(lse.shape) != (T, H):
            raise ValueError("lse must be contiguous fp32 CUDA [T, H]")
        _on_device(dev, "lse", lse)
    if max_rows is None:
        max_rows = 1 if row_cu is None else 0
    elif not 1 <= max_rows < 1 << 31:
        raise ValueError("max_rows must be at least 1, and below 2^31")
    # The workspace from torch's allocator on the current stream (on another one: the library's own).
    bytes_ = lib.span_la_softmax_paged_workspace(T, H, c, int(max_rows)) if stream is None else 0
    ws = torch.empty(bytes_, dtype=torch.uint8, device=q.device) if bytes_ else None
    _raise(lib, lib.span_la_softmax_paged(q.data_ptr(), qs, T, H, c, int(max_rows), float(scale), out.data_ptr(),
                                          lse.data_ptr() if lse is not None else None, ws.data_ptr() if bytes_ else None,
                                          _stream_handle(stream)), "span_la_softmax_paged")
    return out


def _keys(keys) -> np.ndarray:
    a = np.ascontiguousarray(np.asarray(keys, dtype=np.uint64).reshape(-1))
    return a


CACHE_FIELDS = ("entries", "capacity", "hits", "misses", "evictions", "puts")


class ViewStateCache:
    """Keyed least-recently-used cache of view final states in device memory
    (``span_la_cache_*``): put a pass's ``view_state_out`` rows under keys,
    then run branches (or shards of them) from the cached states by key."""

    def __init__(self, num_heads: int, capacity: int):
        self._lib = load_library()
        handle = ctypes.c_void_p()
        _raise(self._lib, self._lib.span_la_cache_create(int(num_heads), int(capacity),
                                                         ctypes.byref(handle)),
               "span_la_cache_create")
        self._handle = handle.value
        self.num_heads = int(num_heads)
        self.capacity = int(capacity)

    def close(self) -> None:
        if self._handle:
            handle, self._handle = self._handle, None
            _raise(self._lib, self._lib.span_la_cache_destroy(handle), "span_la_cache_destroy")

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _live(self):
        if not self._handle:
            raise ValueError("the cache is closed")
        return self._handle

    def put(self, keys, states: torch.Tensor, stream: Optional[torch.cuda.Stream] = None) -> None:
        """Store states[i] (fp32 CUDA [n, H, 64, 64], contiguous) under keys[i]."""
        ks = _keys(keys)
        if (states.dtype != torch.float32 or not states.is_contiguous() or not states.is_cuda
                or states.dim() != 4 or tuple(states.shape[1:]) != (self.num_heads, 64, 64)
                or states.shape[0] != ks.size):
            raise ValueError("states must be contiguous fp32 CUDA [len(keys), H, 64, 64]")
        _raise(self._lib, self._lib.span_la_cache_put(self._live(), ks.ctypes.data, ks.size,
                                                      states.data_ptr(), _stream_handle(stream)),
               "span_la_cache_put")

    def contains(self, keys) -> np.ndarray:
        ks = _keys(keys)
        present = np.zeros(ks.size, dtype=np.int32)
        _raise(self._lib, self._lib.span_la_cache_contains(
            self._live(), ks.ctypes.data if ks.size else None, ks.size,
            present.ctypes.data if ks.size else None), "span_la_cache_contains")
        return present.astype(bool)

    def branches(self, parent_keys, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                 branch_cu_seqlens: Sequence[int], out: Optional[torch.Tensor] = None,
                 stream: Optional[torch.cuda.Stream] = None,
                 log_decay: Optional[torch.Tensor] = None) -> torch.Tensor:
        """Branch b forks from the state cached under parent_keys[b]; with
        ``log_decay`` (fp32 CUDA [H]) as a branch of a decayed pass."""
        dims = _dims_of(q, k, v)
        bcu = _i32(branch_cu_seqlens)
        B = max(len(bcu) - 1, 0)
        ks = _keys(parent_keys)
        if ks.size != B:
            raise ValueError("one parent key per branch")
        if log_decay is not None:
            dims, out, _ = _decay_args(q, k, v, log_decay, out, stream)
            _raise(self._lib, self._lib.span_la_cache_decay_branches(
                self._live(), ks.ctypes.data if ks.size else None, q.data_ptr(), k.data_ptr(), v.data_ptr(), dims,
                log_decay.data_ptr(), _iptr(bcu), B, out.data_ptr(), _stream_handle(stream)),
                "span_la_cache_decay_branches")
            return out
        if out is None:
            out = _new(q.shape, q.dtype, q.device, stream)
        if out.shape != q.shape or out.dtype != q.dtype or not out.is_contiguous() or not out.is_cuda:
            raise ValueError("out must be a contiguous CUDA tensor like q")
        _raise(self._lib, self._lib.span_la_cache_branches(
            self._live(), ks.ctypes.data if ks.size else None, q.data_ptr(), k.data_ptr(),
            v.data_ptr(), dims, _iptr(bcu), B, out.data_ptr(), _stream_handle(stream)),
            "span_la_cache_branches")
        return out

    def stats(self) -> dict:
        st = (ctypes.c_int64 * len(CACHE_FIELDS))()
        _raise(self._lib, self._lib.span_la_cache_stats(self._live(), st), "span_la_cache_stats")
        return dict(zip(CACHE_FIELDS, (int(x) for x in st)))


def span_la_check(stream: Optional[torch.cuda.Stream] = None) -> None:
    """Synchronise the stream and raise on a CUDA error or a device wait timeout."""
    lib = load_library()
    _raise(lib, lib.span_la_check(_stream_handle(stream)), "span_la_check")


FAULT_ALLOC = 1


def fault_inject(kind: int, count: int) -> None:
    """Make the library's next `count` device allocations fail (kind FAULT_ALLOC)."""
    lib = load_library()
    _raise(lib, lib.span_la_fault_inject(int(kind), int(count)), "span_la_fault_inject")


def span_la_selftest_wait_timeout(limit_us: int, stream=None) -> None:
    lib = load_library()
    _raise(lib, lib.span_la_selftest_wait_timeout(int(limit_us), _stream_handle(stream)),
           "span_la_selftest_wait_timeout")


PASS_ONE_LAUNCH = 0
PASS_THREE_LAUNCHES = 1


def set_pass_variant(variant: int) -> None:
    """Process-wide structure of the bf16 pass (``span_la_pass_variant``):
    ``PASS_ONE_LAUNCH`` (default) or ``PASS_THREE_LAUNCHES``."""
    lib = load_library()
    _raise(lib, lib.span_la_pass_variant(int(variant)), "span_la_pass_variant")


def span_la_selftest_wait_timeout_noalloc(limit_us: int, stream=None) -> None:
    lib = load_library()
    _raise(lib, lib.span_la_selftest_wait_timeout_noalloc(int(limit_us), _stream_handle(stream)),
           "span_la_selftest_wait_timeout_noalloc")


PLAN_FIELDS = ("state_slots", "state_rows", "scan_segments", "final_states", "tiles",
               "tile_rows", "start_state_reads", "out_items", "run_tiles")


def plan_stats(view_cu_seqlens, branch_cu_seqlens, branch_parent, num_heads: int,
               dtype: str = "bf16", num_parents: int = 0, from_state: bool = False,
               num_sms: int = 152) -> dict:
    """Work units the library would launch for this metadata on a GPU with
    ``num_sms`` SMs (host only; every count summed over heads)."""
    lib = load_library()
    vcu, bcu, par = _i32(view_cu_seqlens), _i32(branch_cu_seqlens), _i32(branch_parent)
    V = max(len(vcu) - 1, 0)
    B = max(len(bcu) - 1, 0)
    stats = (ctypes.c_int64 * len(PLAN_FIELDS))()
    dt = SPAN_LA_BF16 if dtype == "bf16" else SPAN_LA_F32
    _raise(lib, lib.span_la_plan_stats(_iptr(vcu), V, _iptr(bcu), B, _iptr(par), int(num_parents),
                                       1 if from_state else 0, int(num_heads), dt, int(num_sms),
                                       stats),
           "span_la_plan_stats")
    return dict(zip(PLAN_FIELDS, (int(x) for x in stats)))


SOFTMAX_PLAN_FIELDS = ("items", "rows", "key_blocks", "grid")


def softmax_plan_stats(view_cu_seqlens, branch_cu_seqlens, branch_parent, num_heads: int,
                       num_sms: int = 152) -> dict:
    """Work units of the softmax layer for this metadata (host only)."""
    lib = load_library()
    vcu, bcu, par = _i32(view_cu_seqlens), _i32(branch_cu_seqlens), _i32(branch_parent)
    V = max(len(vcu) - 1, 0)
    B = max(len(bcu) - 1, 0)
    stats = (ctypes.c_int64 * len(SOFTMAX_PLAN_FIELDS))()
    _raise(lib, lib.span_la_softmax_plan_stats(_iptr(vcu), V, _iptr(bcu), B, _iptr(par), int(num_heads),
                                               int(num_sms), stats), "span_la_softmax_plan_stats")
    return dict(zip(SOFTMAX_PLAN_FIELDS, (int(x) for x in stats)))


def profile_enable(on: bool = True) -> None:
    """Time every kernel launch with CUDA events on its stream (tracing hook)."""
    lib = load_library()
    _raise(lib, lib.span_la_profile_enable(1 if on else 0), "span_la_profile_enable")


def profile_reset() -> None:
    lib = load_library()
    _raise(lib, lib.span_la_profile_reset(), "span_la_profile_reset")


def profile_read() -> dict:
    """Per kernel name: {"ms": summed event time, "timed": launches timed,
    "launches": launches counted} since the last reset."""
    lib = load_library()
    ms = (ctypes.c_double * NUM_KERNELS)()
    timed = (ctypes.c_int64 * NUM_KERNELS)()
    launches = (ctypes.c_int64 * NUM_KERNELS)()
    _raise(lib, lib.span_la_profile_read(ms, timed, launches, NUM_KERNELS), "span_la_profile_read")
    return {lib.span_la_kernel_name(k).decode(): {"ms": ms[k], "timed": timed[k],
                                                  "launches": launches[k]}
            for k in range(NUM_KERNELS)}


def version() -> int:
    return int(load_library().span_la_version())
