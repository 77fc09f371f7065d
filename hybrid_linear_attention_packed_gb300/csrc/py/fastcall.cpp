// The usual call of the decayed passes, the single-token step, the q/k norm
// and rotation and the paged cache, from Python in about two microseconds: a decode step's kernel
// takes less time than a dozen tensor attributes read through the
// interpreter.  Each function here takes the arguments of its namesake in
// spanla.py, already in order, and
//   * returns its result when everything is as it should be and the library
//     accepted the call;
//   * returns None, having done nothing, when any argument is not the usual
//     one, or torch is in a mode in which allocations are more than that:
//     spanla.py then checks them one by one and names the problem, or makes the
//     call itself;
//   * returns the library's status (an int) when the library refused.
// The library is reached through the addresses that bind() is given, so that
// it is the one that spanla.py loaded.
#include <Python.h>
#include <ATen/Context.h>
#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/core/impl/TorchDispatchModeTLS.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <exception>

#include "spanla.h"

namespace {

decltype(&span_la_decay_pass) g_pass = nullptr;
decltype(&span_la_decay_branches_from_state) g_fork = nullptr;
decltype(&span_la_decay_step) g_step = nullptr;
decltype(&span_la_qk_norm_rope) g_rope = nullptr;
decltype(&span_la_kv_write) g_write = nullptr;
decltype(&span_la_kv_read) g_read = nullptr;
decltype(&span_la_softmax_paged) g_paged = nullptr;
decltype(&span_la_softmax_paged_workspace) g_paged_bytes = nullptr;

// (without the dispatcher: about 1 us less for a call that returns two tensors;
// see usual_mode)
at::Tensor new_tensor(at::IntArrayRef size, at::ScalarType type, int dev) {
  return at::detail::empty_cuda(size, type, c10::Device(c10::kCUDA, static_cast<c10::DeviceIndex>(dev)), std::nullopt);
}

// A tensor argument; NULL when it is something else.
const at::Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

bool contiguous_on(const at::Tensor& t, int dev, at::ScalarType type) {
  return t.is_cuda() && t.get_device() == dev && t.scalar_type() == type && t.is_contiguous();
}

// Rows [T, H, 64] of q: its dims, when it is one that the library takes.
bool rows_of(const at::Tensor& q, int dev, span_la_dims* dims) {
  if (q.dim() != 3 || q.size(2) != 64 || !q.is_cuda() || q.get_device() != dev || !q.is_contiguous()) return false;
  const at::ScalarType type = q.scalar_type();
  if (type != at::kBFloat16 && type != at::kFloat) return false;
  if (q.size(1) < 1 || q.size(1) > INT32_MAX) return false;
  *dims = {q.size(0), static_cast<int32_t>(q.size(1)), 64, type == at::kBFloat16 ? SPAN_LA_BF16 : SPAN_LA_F32};
  return true;
}

bool like(const at::Tensor& t, const at::Tensor& q, int dev) {
  return contiguous_on(t, dev, q.scalar_type()) && t.sizes() == q.sizes();
}

bool states_of(const at::Tensor& t, int dev, int64_t H) {
  return t.dim() == 4 && t.size(1) == H && t.size(2) == 64 && t.size(3) == 64 && t.size(0) <= INT32_MAX &&
         contiguous_on(t, dev, at::kFloat);
}

// Contiguous 1-D host memory of `size`-byte elements whose format ends in one
// of `kinds` (a numpy array).  A view must be released by release().
struct HostArray {
  Py_buffer view{};
  bool held = false;
  int64_t n = 0;
  const void* p = nullptr;
  bool take(PyObject* o, int size, const char* kinds) {
    if (o == Py_None) return true;
    if (!PyObject_CheckBuffer(o) || THPVariable_Check(o)) return false;
    if (PyObject_GetBuffer(o, &view, PyBUF_C_CONTIGUOUS | PyBUF_FORMAT) != 0) {
      PyErr_Clear();
      return false;
    }
    held = true;
    if (view.ndim != 1 || view.itemsize != size || view.format == nullptr || view.format[0] == '\0' || view.format[1] != '\0')
      return false;
    bool known = false;
    for (const char* c = kinds; *c; ++c) known |= *c == view.format[0];
    n = view.shape[0];
    p = n > 0 ? view.buf : nullptr;
    return known;
  }
  ~HostArray() {
    if (held) PyBuffer_Release(&view);
  }
};

// The stream argument: None is the current stream, otherwise its handle.
bool stream_of(PyObject* o, int dev, cudaStream_t* s) {
  if (o == Py_None) {
    *s = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
    return true;
  }
  PyObject* h = PyObject_GetAttrString(o, "cuda_stream");
  if (h == nullptr) {
    PyErr_Clear();
    return false;
  }
  *s = static_cast<cudaStream_t>(PyLong_AsVoidPtr(h));
  Py_DECREF(h);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    return false;
  }
  return true;
}

// True where `s`, given as `o`, is another stream than the current one: new
// outputs are then made for it by spanla.py.
bool other_stream(PyObject* o, cudaStream_t s, int dev) {
  return o != Py_None && s != c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
}

PyObject* wrap(const at::Tensor& t) { return THPVariable_Wrap(t); }

// Output tensor: the given one when it is like q, or a new one.
bool output(PyObject* o, const at::Tensor& q, int dev, at::Tensor* out) {
  if (o == Py_None) {
    *out = new_tensor(q.sizes(), q.scalar_type(), dev);
    return true;
  }
  const at::Tensor* t = tensor(o);
  if (t == nullptr || !like(*t, q, dev)) return false;
  *out = *t;
  return true;
}

struct Common {   // q, k, v, log_decay (NULL where allowed) on the current device
  const at::Tensor *q, *k, *v;
  const float* log_decay = nullptr;
  span_la_dims dims{};
  int dev = 0;
  bool take(PyObject* oq, PyObject* ok, PyObject* ov, PyObject* od, bool need_decay) {
    q = tensor(oq);
    k = tensor(ok);
    v = tensor(ov);
    if (!q || !k || !v || !q->is_cuda()) return false;
    dev = c10::cuda::current_device();
    if (!rows_of(*q, dev, &dims) || !like(*k, *q, dev) || !like(*v, *q, dev)) return false;
    if (od == Py_None) return !need_decay;
    const at::Tensor* d = tensor(od);
    if (d == nullptr || d->dim() != 1 || d->size(0) != dims.num_heads || !contiguous_on(*d, dev, at::kFloat)) return false;
    log_decay = static_cast<const float*>(d->data_ptr());
    return true;
  }
};

// False where new tensors have to go through the dispatcher: a dispatch mode is to
// see them, or deterministic algorithms are asked for, which fill them.
bool usual_mode() { return !c10::impl::dispatch_mode_enabled() && !at::globalContext().deterministicAlgorithms(); }

// C++ exceptions become Python's, each the one that torch makes of it (an
// allocation that fails torch.OutOfMemoryError).
template <typename Fn>
PyObject* guarded(Fn&& fn) {
  try {
    if (!usual_mode()) Py_RETURN_NONE;
    return fn();
  } catch (...) {
    torch::translate_exception_to_python(std::current_exception());
    return nullptr;
  }
}

PyObject* none() { Py_RETURN_NONE; }

int32_t segments(const HostArray& cu) { return cu.n > 1 ? static_cast<int32_t>(cu.n - 1) : 0; }

// (q, k, v, log_decay, view_cu, branch_cu, branch_parent, out, view_state_out, stream)
PyObject* py_pass(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Common c;
    HostArray vcu, bcu, par;
    cudaStream_t stream;
    at::Tensor out, state;
    if (n != 10 || !c.take(a[0], a[1], a[2], a[3], true) || !vcu.take(a[4], 4, "i") || !bcu.take(a[5], 4, "i") ||
        !par.take(a[6], 4, "i") || par.n != segments(bcu) || !stream_of(a[9], c.dev, &stream) ||
        ((a[7] == Py_None || a[8] == Py_None) && other_stream(a[9], stream, c.dev)))
      return none();
    const int64_t V = segments(vcu);
    if (a[8] != Py_None) {
      const at::Tensor* t = tensor(a[8]);
      if (t == nullptr || !states_of(*t, c.dev, c.dims.num_heads) || t->size(0) < V) return none();
      state = *t;
    }
    if (!output(a[7], *c.q, c.dev, &out)) return none();
    if (!state.defined()) state = new_tensor({V, c.dims.num_heads, 64, 64}, at::kFloat, c.dev);
    span_la_status st;
    Py_BEGIN_ALLOW_THREADS
    st = g_pass(c.q->data_ptr(), c.k->data_ptr(), c.v->data_ptr(), c.dims, c.log_decay, static_cast<const int32_t*>(vcu.p),
                static_cast<int32_t>(V), static_cast<const int32_t*>(bcu.p), segments(bcu),
                static_cast<const int32_t*>(par.p), out.data_ptr(), static_cast<float*>(state.data_ptr()), stream);
    Py_END_ALLOW_THREADS
    if (st != SPAN_LA_OK) return PyLong_FromLong(st);
    return Py_BuildValue("(NN)", wrap(out), wrap(state));
  });
}

// (cached_state, q, k, v, log_decay, branch_cu, branch_parent, out, stream)
PyObject* py_fork(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Common c;
    HostArray bcu, par;
    cudaStream_t stream;
    at::Tensor out;
    const at::Tensor* kept = n == 9 ? tensor(a[0]) : nullptr;
    if (kept == nullptr || !c.take(a[1], a[2], a[3], a[4], true) || !states_of(*kept, c.dev, c.dims.num_heads) ||
        !bcu.take(a[5], 4, "i") || !par.take(a[6], 4, "i") || par.n != segments(bcu) || !stream_of(a[8], c.dev, &stream) ||
        (a[7] == Py_None && other_stream(a[8], stream, c.dev)) || !output(a[7], *c.q, c.dev, &out))
      return none();
    span_la_status st;
    Py_BEGIN_ALLOW_THREADS
    st = g_fork(static_cast<const float*>(kept->data_ptr()), static_cast<int32_t>(kept->size(0)), c.q->data_ptr(),
                c.k->data_ptr(), c.v->data_ptr(), c.dims, c.log_decay, static_cast<const int32_t*>(bcu.p), segments(bcu),
                static_cast<const int32_t*>(par.p), out.data_ptr(), stream);
    Py_END_ALLOW_THREADS
    return st != SPAN_LA_OK ? PyLong_FromLong(st) : wrap(out);
  });
}

// (q, k, v, states, log_decay, state_index, out, stream)
PyObject* py_step(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Common c;
    HostArray index;
    cudaStream_t stream;
    at::Tensor out;
    if (n != 8 || !c.take(a[0], a[1], a[2], a[4], false)) return none();
    const at::Tensor* states = tensor(a[3]);
    if (states == nullptr || !states_of(*states, c.dev, c.dims.num_heads) || !index.take(a[5], 4, "i") ||
        (a[5] != Py_None && (index.n != c.dims.total_rows || index.n == 0)) || !stream_of(a[7], c.dev, &stream) ||
        (a[6] == Py_None && other_stream(a[7], stream, c.dev)) || !output(a[6], *c.q, c.dev, &out))
      return none();
    span_la_status st;
    Py_BEGIN_ALLOW_THREADS
    st = g_step(c.q->data_ptr(), c.k->data_ptr(), c.v->data_ptr(), c.dims, c.log_decay,
                static_cast<float*>(states->data_ptr()), static_cast<int32_t>(states->size(0)),
                static_cast<const int32_t*>(index.p), out.data_ptr(), stream);
    Py_END_ALLOW_THREADS
    return st != SPAN_LA_OK ? PyLong_FromLong(st) : wrap(out);
  });
}

// One side of the norm and rotation; `dt` is the type of both, `wdt` the weights' (-1: none yet).
bool side_of(PyObject* ox, PyObject* ow, PyObject* oo, int dev, int64_t T, at::ScalarType dt, int* wdt, span_la_qk_side* s,
             at::Tensor* out) {
  const at::Tensor* x = tensor(ox);
  if (x == nullptr || x->dim() != 3 || x->size(0) != T || x->size(2) != 64 || x->scalar_type() != dt || !x->is_cuda() ||
      x->get_device() != dev || x->size(1) < 1 || x->size(1) > INT32_MAX || T < 1)
    return false;
  const int64_t H = x->size(1);
  auto row_stride = [&](const at::Tensor& t, int64_t* stride) {
    if (t.stride(2) != 1 || (H > 1 && t.stride(1) != 64)) return false;
    *stride = T > 1 ? t.stride(0) : H * 64;
    return true;
  };
  *s = {};
  if (!row_stride(*x, &s->in_row_stride)) return false;
  if (ow != Py_None) {
    const at::Tensor* w = tensor(ow);
    if (w == nullptr || w->dim() < 1 || w->dim() > 2 || w->size(-1) != 64 || (w->dim() == 2 && w->size(0) != H) ||
        !w->is_cuda() || w->get_device() != dev || !w->is_contiguous())
      return false;
    const int type = w->scalar_type() == at::kBFloat16 ? SPAN_LA_BF16 : w->scalar_type() == at::kFloat ? SPAN_LA_F32 : -2;
    if (type == -2 || (*wdt >= 0 && *wdt != type)) return false;
    *wdt = type;
    s->weight = w->data_ptr();
    s->weight_per_head = w->dim() == 2;
  }
  if (oo == Py_None) {
    *out = new_tensor({T, H, 64}, dt, dev);
    s->out_row_stride = H * 64;
  } else {
    const at::Tensor* t = tensor(oo);
    if (t == nullptr || t->sizes() != x->sizes() || t->scalar_type() != dt || !t->is_cuda() || t->get_device() != dev ||
        !row_stride(*t, &s->out_row_stride))
      return false;
    *out = *t;
  }
  s->in = x->data_ptr();
  s->out = out->data_ptr();
  s->num_heads = static_cast<int32_t>(H);
  return true;
}

// (q, k, positions, inv_freq, q_weight, k_weight, eps, interleaved, q_out, k_out, stream)
PyObject* py_rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const at::Tensor* q = n == 11 ? tensor(a[0]) : nullptr;
    const at::Tensor* pos = q != nullptr ? tensor(a[2]) : nullptr;
    if (pos == nullptr || q->dim() != 3 || !q->is_cuda()) return none();
    const at::ScalarType dt = q->scalar_type();
    if (dt != at::kBFloat16 && dt != at::kFloat) return none();
    const int dev = c10::cuda::current_device();
    const int64_t T = q->size(0);
    HostArray freq;
    cudaStream_t stream;
    int wdt = -1;
    span_la_qk_side sides[2];
    at::Tensor outs[2];
    if (pos->dim() != 1 || pos->size(0) != T || !contiguous_on(*pos, dev, at::kInt) || !freq.take(a[3], 8, "d") ||
        !PyFloat_Check(a[6]) || !PyBool_Check(a[7]) || !stream_of(a[10], dev, &stream) ||
        ((a[8] == Py_None || a[9] == Py_None) && other_stream(a[10], stream, dev)) ||
        !side_of(a[0], a[4], a[8], dev, T, dt, &wdt, &sides[0], &outs[0]) ||
        !side_of(a[1], a[5], a[9], dev, T, dt, &wdt, &sides[1], &outs[1]) || freq.n > 32)
      return none();
    const int32_t type = dt == at::kBFloat16 ? SPAN_LA_BF16 : SPAN_LA_F32;
    const float eps = static_cast<float>(PyFloat_AS_DOUBLE(a[6]));
    span_la_status st;
    Py_BEGIN_ALLOW_THREADS
    st = g_rope(sides[0], sides[1], T, type, wdt < 0 ? type : wdt, eps, static_cast<const double*>(freq.p),
                static_cast<int32_t>(2 * freq.n), a[7] == Py_True, static_cast<const int32_t*>(pos->data_ptr()), stream);
    Py_END_ALLOW_THREADS
    if (st != SPAN_LA_OK) return PyLong_FromLong(st);
    return Py_BuildValue("(NN)", wrap(outs[0]), wrap(outs[1]));
  });
}

// A paged cache: (k_pages, v_pages, page_table, seq_len, row_cu, k_scale, v_scale) into the library's struct.
struct Cache {
  span_la_kv_cache c{};
  int dev = 0;
  bool take(PyObject* ok, PyObject* ov, PyObject* ot, PyObject* ol, PyObject* oc, PyObject* oks, PyObject* ovs) {
    const at::Tensor *k = tensor(ok), *v = tensor(ov), *table = tensor(ot), *len = tensor(ol);
    if (!k || !v || !table || !len || !k->is_cuda() || k->dim() != 4) return false;
    dev = c10::cuda::current_device();
    const at::ScalarType type = k->scalar_type();
    if (k->get_device() != dev || !v->is_cuda() || v->get_device() != dev || v->scalar_type() != type || v->sizes() != k->sizes() ||
        v->strides() != k->strides() || k->size(3) != 64 || k->stride(3) != 1 || k->size(0) > INT32_MAX || k->size(1) > INT32_MAX ||
        k->size(2) > INT32_MAX || (type != at::kBFloat16 && type != at::kFloat8_e4m3fn))
      return false;
    if (table->dim() != 2 || table->scalar_type() != at::kInt || !table->is_cuda() || table->get_device() != dev ||
        (table->size(1) > 1 && table->stride(1) != 1) || table->size(0) > INT32_MAX || table->size(1) > INT32_MAX)
      return false;
    const int64_t S = table->size(0);
    if (len->dim() != 1 || len->size(0) != S || !contiguous_on(*len, dev, at::kInt)) return false;
    if (oc != Py_None) {
      const at::Tensor* cu = tensor(oc);
      if (!cu || cu->dim() != 1 || cu->size(0) != S + 1 || !contiguous_on(*cu, dev, at::kInt)) return false;
      c.row_cu = static_cast<const int32_t*>(cu->data_ptr());
    }
    if (type == at::kFloat8_e4m3fn) {
      const at::Tensor *ks = tensor(oks), *vs = tensor(ovs);
      if (!ks || !vs || ks->dim() != 3 || ks->scalar_type() != at::kByte || vs->scalar_type() != at::kByte || !ks->is_cuda() ||
          !vs->is_cuda() || ks->get_device() != dev || vs->get_device() != dev || ks->sizes() != k->sizes().slice(0, 3) ||
          vs->sizes() != ks->sizes() || vs->strides() != ks->strides() || ks->stride(2) != 1)
        return false;
      c.k_scale = static_cast<uint8_t*>(ks->data_ptr());
      c.v_scale = static_cast<uint8_t*>(vs->data_ptr());
      c.scale_page_stride = ks->stride(0);
      c.scale_head_stride = ks->stride(1);
      c.dtype = SPAN_LA_E4M3;
    } else {
      if (oks != Py_None || ovs != Py_None) return false;
      c.dtype = SPAN_LA_BF16;
    }
    c.k = k->data_ptr();
    c.v = v->data_ptr();
    c.page_stride = k->stride(0);
    c.head_stride = k->stride(1);
    c.row_stride = k->stride(2);
    c.num_pages = static_cast<int32_t>(k->size(0));
    c.num_heads = static_cast<int32_t>(k->size(1));
    c.page_rows = static_cast<int32_t>(k->size(2));
    c.num_seqs = static_cast<int32_t>(S);
    c.table_width = static_cast<int32_t>(table->size(1));
    c.table_stride = S > 1 ? table->stride(0) : table->size(1);
    c.page_table = static_cast<const int32_t*>(table->data_ptr());
    c.seq_len = static_cast<const int32_t*>(len->data_ptr());
    return true;
  }
};

// Rows [T, H, 64] whose heads lie next to each other in a row, and their stride.
bool packed_rows(const at::Tensor& t, int dev, int64_t* stride) {
  if (t.dim() != 3 || t.size(2) != 64 || !t.is_cuda() || t.get_device() != dev || t.size(0) < 1 || t.size(1) < 1 ||
      t.size(1) > INT32_MAX || t.stride(2) != 1 || (t.size(1) > 1 && t.stride(1) != 64))
    return false;
  *stride = t.size(0) > 1 ? t.stride(0) : t.size(1) * 64;
  return true;
}

// (k, v, k_pages, v_pages, page_table, seq_len, row_cu, k_scale, v_scale, stream): True when it is done
PyObject* py_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Cache c;
    cudaStream_t stream;
    int64_t ks, vs;
    if (n != 10 || !c.take(a[2], a[3], a[4], a[5], a[6], a[7], a[8])) return none();
    const at::Tensor *k = tensor(a[0]), *v = tensor(a[1]);
    if (!k || !v || !packed_rows(*k, c.dev, &ks) || !packed_rows(*v, c.dev, &vs) || k->sizes() != v->sizes() ||
        k->size(1) != c.c.num_heads || k->scalar_type() != v->scalar_type() || !stream_of(a[9], c.dev, &stream))
      return none();
    const at::ScalarType type = k->scalar_type();
    if (type != at::kBFloat16 && type != at::kFloat) return none();
    span_la_status st;
    Py_BEGIN_ALLOW_THREADS
    st = g_write(k->data_ptr(), v->data_ptr(), ks, vs, k->size(0), type == at::kBFloat16 ? SPAN_LA_BF16 : SPAN_LA_F32, &c.c, stream);
    Py_END_ALLOW_THREADS
    if (st != SPAN_LA_OK) return PyLong_FromLong(st);
    Py_RETURN_TRUE;
  });
}

// (k_pages, v_pages, page_table, seq_len, row_cu, total_rows, k_scale, v_scale, bf16, stream): new outputs
PyObject* py_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Cache c;
    cudaStream_t stream;
    if (n != 10 || !PyLong_CheckExact(a[5]) || !PyBool_Check(a[8]) || !c.take(a[0], a[1], a[2], a[3], a[4], a[6], a[7]) ||
        !stream_of(a[9], c.dev, &stream) || other_stream(a[9], stream, c.dev))
      return none();
    const int64_t T = PyLong_AsLongLong(a[5]);
    if (T < 1 || T > INT32_MAX) {
      PyErr_Clear();
      return none();
    }
    const bool bf16 = a[8] == Py_True;
    at::Tensor outs[2];
    for (at::Tensor& x : outs) x = new_tensor({T, c.c.num_heads, 64}, bf16 ? at::kBFloat16 : at::kFloat, c.dev);
    span_la_status st;
    Py_BEGIN_ALLOW_THREADS
    st = g_read(&c.c, T, bf16 ? SPAN_LA_BF16 : SPAN_LA_F32, outs[0].data_ptr(), outs[1].data_ptr(), stream);
    Py_END_ALLOW_THREADS
    if (st != SPAN_LA_OK) return PyLong_FromLong(st);
    return Py_BuildValue("(NN)", wrap(outs[0]), wrap(outs[1]));
  });
}

// (q, k_pages, v_pages, page_table, seq_len, row_cu, k_scale, v_scale, max_rows, scale, out, lse, stream)
PyObject* py_paged(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    Cache c;
    cudaStream_t stream;
    int64_t qs;
    if (n != 13 || !PyFloat_Check(a[9]) || !c.take(a[1], a[2], a[3], a[4], a[5], a[6], a[7])) return none();
    const at::Tensor* q = tensor(a[0]);
    if (!q || !packed_rows(*q, c.dev, &qs) || q->scalar_type() != at::kBFloat16 || !stream_of(a[12], c.dev, &stream)) return none();
    int64_t max_rows = c.c.row_cu == nullptr ? 1 : 0;
    if (a[8] != Py_None) {
      if (!PyLong_CheckExact(a[8])) return none();
      max_rows = PyLong_AsLongLong(a[8]);
      if (max_rows < 1 || max_rows > INT32_MAX) {
        PyErr_Clear();
        return none();
      }
    }
    at::Tensor out;
    if (a[10] == Py_None) {
      if (other_stream(a[12], stream, c.dev)) return none();
      out = new_tensor(q->sizes(), at::kBFloat16, c.dev);
    } else {
      const at::Tensor* t = tensor(a[10]);
      if (t == nullptr || !like(*t, *q, c.dev)) return none();
      out = *t;
    }
    float* lse = nullptr;
    if (a[11] != Py_None) {
      const at::Tensor* t = tensor(a[11]);
      if (t == nullptr || t->dim() != 2 || t->size(0) != q->size(0) || t->size(1) != q->size(1) || !contiguous_on(*t, c.dev, at::kFloat))
        return none();
      lse = static_cast<float*>(t->data_ptr());
    }
    // (on another stream than the current one, whose allocator this is, the library takes its own)
    at::Tensor ws;
    const int64_t bytes =
        a[12] == Py_None ? g_paged_bytes(q->size(0), static_cast<int32_t>(q->size(1)), &c.c, static_cast<int32_t>(max_rows)) : 0;
    if (bytes > 0) ws = new_tensor({bytes}, at::kByte, c.dev);
    span_la_status st;
    Py_BEGIN_ALLOW_THREADS
    st = g_paged(q->data_ptr(), qs, q->size(0), static_cast<int32_t>(q->size(1)), &c.c, static_cast<int32_t>(max_rows),
                 static_cast<float>(PyFloat_AS_DOUBLE(a[9])), out.data_ptr(), lse, bytes > 0 ? ws.data_ptr() : nullptr, stream);
    Py_END_ALLOW_THREADS
    return st != SPAN_LA_OK ? PyLong_FromLong(st) : wrap(out);
  });
}

// bind(addresses of span_la_decay_pass, .._branches_from_state, .._step, span_la_qk_norm_rope, span_la_kv_write, .._read,
// span_la_softmax_paged, .._workspace)
PyObject* py_bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != 8) {
    PyErr_SetString(PyExc_TypeError, "bind takes eight addresses");
    return nullptr;
  }
  void* p[8];
  for (int i = 0; i < 8; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (p[i] == nullptr) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "an address is NULL");
      return nullptr;
    }
  }
  g_pass = reinterpret_cast<decltype(g_pass)>(p[0]);
  g_fork = reinterpret_cast<decltype(g_fork)>(p[1]);
  g_step = reinterpret_cast<decltype(g_step)>(p[2]);
  g_rope = reinterpret_cast<decltype(g_rope)>(p[3]);
  g_write = reinterpret_cast<decltype(g_write)>(p[4]);
  g_read = reinterpret_cast<decltype(g_read)>(p[5]);
  g_paged = reinterpret_cast<decltype(g_paged)>(p[6]);
  g_paged_bytes = reinterpret_cast<decltype(g_paged_bytes)>(p[7]);
  Py_RETURN_NONE;
}

PyMethodDef kMethods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_bind)), METH_FASTCALL, nullptr},
    {"decay_pass", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_pass)), METH_FASTCALL, nullptr},
    {"decay_fork", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_fork)), METH_FASTCALL, nullptr},
    {"decay_step", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_step)), METH_FASTCALL, nullptr},
    {"qk_norm_rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_rope)), METH_FASTCALL, nullptr},
    {"kv_write", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_write)), METH_FASTCALL, nullptr},
    {"kv_read", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_read)), METH_FASTCALL, nullptr},
    {"softmax_paged", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(py_paged)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_fastcall", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// torch_version: the PyTorch that this was compiled against; spanla.py uses it
// with that one only.
PyMODINIT_FUNC PyInit__fastcall() {
  PyObject* m = PyModule_Create(&kModule);
  if (m != nullptr && PyModule_AddStringConstant(m, "torch_version", SPANLA_TORCH_VERSION) != 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
