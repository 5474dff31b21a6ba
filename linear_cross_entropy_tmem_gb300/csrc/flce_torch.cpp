// flce_torch.cpp — native marshalling of torch tensors for the operators on
// either side of the head and from one token to the next (Python module flce_torch).
//
// A decoding step's call does a few microseconds of GPU work, and a list of a
// hundred gradients little more; reading the tensors' fields from Python took
// 20 to 250 microseconds.  These functions read them here, allocate the outputs
// and call the C entry points.  They take the calls whose tensors are as the
// entry points want them (CUDA, one device, known types, matching shapes, rows
// of adjacent elements) and return None for any other, which head_ops.py or
// token_ops.py then views, copies or refuses with its own message.  Otherwise they return the
// outputs as a tuple, or an int: the status of a call that failed.
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <vector>

#include "flce.h"

namespace {

using at::Tensor;

// The C entry points of the library that Python has loaded.
struct Entry {
  decltype(&flce_add_rms_norm) norm;
  decltype(&flce_add_rms_norm_fp8) norm_fp8;
  decltype(&flce_add_rms_norm_workspace_size) norm_ws;
  decltype(&flce_add_rms_norm_backward) norm_bwd;
  decltype(&flce_grad_norm_workspace_size) grad_ws;
  decltype(&flce_grad_norm) grad_norm;
  decltype(&flce_clip_grad_norm) clip;
  decltype(&flce_process_logits_workspace_size) logits_ws;
  decltype(&flce_process_logits) logits;
  decltype(&flce_embedding) embedding;
  decltype(&flce_embedding_workspace_size) embedding_ws;
  decltype(&flce_embedding_backward) embedding_bwd;
  decltype(&flce_mxfp4_quantize) mx_quantize;
  decltype(&flce_mxfp4_dequantize) mx_dequantize;
  decltype(&flce_mxfp4_logits_workspace_size) mx_logits_ws;
  decltype(&flce_mxfp4_logits) mx_logits;
  decltype(&flce_sample) sample;
} g_entry;
constexpr Py_ssize_t kEntries = sizeof(Entry) / sizeof(void*);

PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != kEntries) {
    PyErr_Format(PyExc_TypeError, "bind takes %zd addresses", kEntries);
    return nullptr;
  }
  void** to = reinterpret_cast<void**>(&g_entry);
  for (Py_ssize_t i = 0; i < n; ++i) {
    to[i] = PyLong_AsVoidPtr(args[i]);
    if (!to[i] && PyErr_Occurred()) return nullptr;
  }
  Py_RETURN_NONE;
}

PyObject* status(int rc) { return PyLong_FromLong(rc); }

// FLCE_* type, or -1.
int code_of(at::ScalarType t) {
  return t == at::kFloat ? FLCE_F32 : t == at::kBFloat16 ? FLCE_BF16 : t == at::kHalf ? FLCE_F16 : -1;
}

// FLCE_* type to torch's.
constexpr at::ScalarType kTypes[] = {at::kFloat, at::kBFloat16, at::kHalf};

// An argument: a tensor of the call's device, or none.
struct Arg {
  const Tensor* t = nullptr;
  bool ok = true;
  explicit operator bool() const { return t != nullptr; }
  const Tensor* operator->() const { return t; }
  void* ptr() const { return t && t->numel() ? t->data_ptr() : nullptr; }
};
Arg arg(PyObject* o, int64_t device = -1) {
  Arg a;
  if (o == Py_None) return a;
  if (!THPVariable_Check(o)) {
    a.ok = false;
    return a;
  }
  a.t = &THPVariable_Unpack(o);
  a.ok = a.t->is_cuda() && (device < 0 || a.t->get_device() == device);
  return a;
}

// Rows of adjacent elements: a matrix, or any contiguous tensor with columns.
struct Rows {
  bool ok = false;
  int64_t n = 0, d = 0, stride = 0;
  explicit Rows(const Tensor& t) {
    const int64_t dim = t.dim();
    if (dim < 1) return;
    d = t.size(dim - 1);
    if (d < 1) return;
    if (dim == 2 && (t.stride(1) == 1 || d == 1)) {
      n = t.size(0);
      stride = t.stride(0);
      ok = true;
    } else if (t.is_contiguous()) {
      n = t.numel() / d;
      stride = d;
      ok = true;
    }
  }
};

Tensor empty(at::IntArrayRef size, at::ScalarType t, const Tensor& like) {
  return Tensor(at::detail::empty_cuda(size, t, like.device(), c10::nullopt));
}
flce_stream_t stream_of(const Tensor& t) {
  return reinterpret_cast<flce_stream_t>(c10::cuda::getCurrentCUDAStream(t.get_device()).stream());
}
PyObject* wrap(const Tensor& t) {
  if (!t.defined()) Py_RETURN_NONE;
  return THPVariable_Wrap(t);
}
PyObject* pack(std::initializer_list<Tensor> ts) {
  PyObject* r = PyTuple_New(Py_ssize_t(ts.size()));
  if (!r) return nullptr;
  Py_ssize_t i = 0;
  for (const Tensor& t : ts) {
    PyObject* o = wrap(t);
    if (!o) {
      Py_DECREF(r);
      return nullptr;
    }
    PyTuple_SET_ITEM(r, i++, o);
  }
  return r;
}
// The caller's workspace or a new one; false where the caller's does not do.
bool workspace(PyObject* o, size_t bytes, const Tensor& like, Tensor* out) {
  const Arg a = arg(o, like.get_device());
  if (!a.ok) return false;
  if (!a) {
    *out = empty({int64_t(bytes)}, at::kByte, like);
    return true;
  }
  *out = *a.t;
  return a->is_contiguous() && size_t(a->numel()) * a->element_size() >= bytes;
}
// The call has written a tensor of the caller's: autograd has to know (a backward that saved it raises, as after any
// in-place operation of torch).  Inference tensors keep no count.
void wrote(const Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}
bool vector_of(const Arg& a, int64_t n, at::ScalarType t) {
  return a->dim() == 1 && a->size(0) == n && a->scalar_type() == t && a->is_contiguous();
}

// (x, weight, residual, eps, weight_offset, need_rstd, group) -> (y or q, h, rstd or scale); group < 0: no 8 bits
PyObject* add_rms_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 7) return PyErr_Format(PyExc_TypeError, "add_rms_norm takes 7 arguments");
  const Arg x = arg(a[0]);
  if (!x || !x.ok) Py_RETURN_NONE;
  const Arg w = arg(a[1], x->get_device()), r = arg(a[2], x->get_device());
  const Rows rows(*x.t);
  const int code = code_of(x->scalar_type());
  if (!w.ok || !r.ok || !rows.ok || code < 0) Py_RETURN_NONE;
  const int wcode = w ? code_of(w->scalar_type()) : code, rcode = r ? code_of(r->scalar_type()) : code;
  if (wcode < 0 || rcode < 0 || (w && !vector_of(w, rows.d, w->scalar_type()))) Py_RETURN_NONE;
  int64_t rstride = 0;
  if (r) {
    const Rows rr(*r.t);
    if (!rr.ok || r->sizes() != x->sizes()) Py_RETURN_NONE;
    rstride = rr.stride;
  }
  const double eps = PyFloat_AsDouble(a[3]), offset = PyFloat_AsDouble(a[4]);
  const bool need_rstd = a[5] == Py_True;
  const long group = PyLong_AsLong(a[6]);
  if (PyErr_Occurred()) return nullptr;
  const flce_norm_problem p = {rows.n, rows.d, rows.stride, rstride, rows.d, rows.d, 0, code, rcode, wcode,
                               group < 0 ? 0 : int32_t(group), float(eps), float(offset)};
  const Tensor h = r ? empty(x->sizes(), r->scalar_type(), *x.t) : *x.t;
  void* hp = r && h.numel() ? h.data_ptr() : nullptr;
  Tensor y, extra;
  int rc;
  if (group < 0) {
    y = empty(x->sizes(), x->scalar_type(), *x.t);
    if (need_rstd) extra = empty({rows.n}, at::kFloat, *x.t);
    float* rstd = need_rstd && rows.n ? extra.mutable_data_ptr<float>() : nullptr;
    rc = g_entry.norm(&p, x.ptr(), r.ptr(), w.ptr(), hp, y.numel() ? y.data_ptr() : nullptr, rstd, stream_of(*x.t));
  } else {
    y = empty(x->sizes(), at::kFloat8_e4m3fn, *x.t);
    std::vector<int64_t> size = x->sizes().vec();
    size.back() = group ? (rows.d + group - 1) / group : 1;
    extra = empty(size, at::kFloat, *x.t);
    rc = g_entry.norm_fp8(&p, x.ptr(), r.ptr(), w.ptr(), hp, y.numel() ? y.data_ptr() : nullptr,
                          extra.numel() ? extra.mutable_data_ptr<float>() : nullptr, stream_of(*x.t));
  }
  if (rc != FLCE_OK) return status(rc);
  PyObject* out = pack({y, h, extra});
  if (out && !r) {  // h is x itself
    Py_INCREF(a[0]);
    PyTuple_SetItem(out, 1, a[0]);
  }
  return out;
  END_HANDLE_TH_ERRORS
}

// (dy, h, rstd, weight, dh, weight_offset, need_dx, need_dresidual, need_dweight, workspace) -> (dx, dresidual, dweight)
PyObject* add_rms_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 10) return PyErr_Format(PyExc_TypeError, "add_rms_norm_backward takes 10 arguments");
  const Arg dy = arg(a[0]);
  if (!dy || !dy.ok) Py_RETURN_NONE;
  const int64_t dev = dy->get_device();
  const Arg h = arg(a[1], dev), rstd = arg(a[2], dev), w = arg(a[3], dev), dh = arg(a[4], dev);
  if (!h || !rstd || !h.ok || !rstd.ok || !w.ok || !dh.ok) Py_RETURN_NONE;
  const Rows rows(*dy.t), hr(*h.t);
  const int code = code_of(dy->scalar_type()), rcode = code_of(h->scalar_type());
  const int wcode = w ? code_of(w->scalar_type()) : code;
  if (!rows.ok || !hr.ok || code < 0 || rcode < 0 || wcode < 0 || h->sizes() != dy->sizes()) Py_RETURN_NONE;
  if (w && !vector_of(w, rows.d, w->scalar_type())) Py_RETURN_NONE;
  if (rstd->scalar_type() != at::kFloat || rstd->numel() != rows.n || !rstd->is_contiguous()) Py_RETURN_NONE;
  int64_t dh_stride = 0;
  if (dh) {
    const Rows r(*dh.t);
    if (!r.ok || dh->sizes() != dy->sizes() || dh->scalar_type() != h->scalar_type()) Py_RETURN_NONE;
    dh_stride = r.stride;
  }
  const double offset = PyFloat_AsDouble(a[5]);
  if (PyErr_Occurred()) return nullptr;
  const bool same = code == rcode, need_dx = a[6] == Py_True, need_dr = a[7] == Py_True;
  const bool need_dw = w && a[8] == Py_True;
  if (!need_dx && !need_dr && !need_dw) Py_RETURN_NONE;
  Tensor dx, dr, dw, ws;
  if (need_dx || (need_dr && same)) dx = empty(dy->sizes(), dy->scalar_type(), *dy.t);
  if (need_dr && !same) dr = empty(h->sizes(), h->scalar_type(), *dy.t);
  const flce_norm_problem p = {rows.n, rows.d, rows.stride, dh_stride, hr.stride, rows.d, dr.defined() ? rows.d : 0,
                               code, rcode, wcode, 0, 0.f, float(offset)};
  size_t bytes = 0;
  if (need_dw) {
    const int rc = g_entry.norm_ws(&p, &bytes);
    if (rc != FLCE_OK) return status(rc);
    dw = empty(w->sizes(), w->scalar_type(), *dy.t);
    if (!workspace(a[9], bytes, *dy.t, &ws)) Py_RETURN_NONE;
  }
  auto ptr = [](const Tensor& t) { return t.defined() && t.numel() ? t.data_ptr() : nullptr; };
  const int rc = g_entry.norm_bwd(&p, dy.ptr(), h.ptr(), w.ptr(), static_cast<const float*>(rstd.ptr()), dh.ptr(),
                                  ptr(dx), ptr(dr), ptr(dw), ptr(ws), bytes, stream_of(*dy.t));
  if (rc != FLCE_OK) return status(rc);
  return pack({need_dx ? dx : Tensor(), need_dr ? (same ? dx : dr) : Tensor(), dw});
  END_HANDLE_TH_ERRORS
}

// (grads, max_norm or None, outputs or None, workspace) -> (norm,); grads and outputs are lists or tuples
PyObject* clip_grad_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 4) return PyErr_Format(PyExc_TypeError, "clip_grad_norm takes 4 arguments");
  if (!PyList_Check(a[0]) && !PyTuple_Check(a[0])) Py_RETURN_NONE;
  const bool to = a[2] != Py_None, clip = a[1] != Py_None;
  if (to && !PyList_Check(a[2]) && !PyTuple_Check(a[2])) Py_RETURN_NONE;
  const Py_ssize_t count = PySequence_Fast_GET_SIZE(a[0]);
  if (count == 0 || (to && PySequence_Fast_GET_SIZE(a[2]) != count)) Py_RETURN_NONE;
  PyObject **gs = PySequence_Fast_ITEMS(a[0]), **os = to ? PySequence_Fast_ITEMS(a[2]) : nullptr;
  std::vector<const void*> src(count);
  std::vector<void*> dst(count), live;
  std::vector<int64_t> numel(count);
  std::vector<int32_t> dtype(count);
  live.reserve(count);
  int64_t dev = -1;
  for (Py_ssize_t i = 0; i < count; ++i) {
    const Arg g = arg(gs[i], dev);
    if (!g || !g.ok || !g->is_contiguous()) Py_RETURN_NONE;
    dev = g->get_device();
    numel[i] = g->numel();
    dtype[i] = code_of(g->scalar_type());
    if (dtype[i] < 0) Py_RETURN_NONE;
    src[i] = g.ptr();
    dst[i] = g.ptr();
    if (to) {
      const Arg o = arg(os[i], dev);
      if (!o || !o.ok || !o->is_contiguous() || o->scalar_type() != g->scalar_type() || o->sizes() != g->sizes())
        Py_RETURN_NONE;
      dst[i] = o.ptr();
    }
    if (numel[i]) live.push_back(dst[i]);
  }
  std::sort(live.begin(), live.end());
  if (std::adjacent_find(live.begin(), live.end()) != live.end()) Py_RETURN_NONE;
  double max_norm = 0.0;
  if (clip) {
    max_norm = PyFloat_AsDouble(a[1]);
    if (PyErr_Occurred()) return nullptr;
  }
  const Tensor& like = THPVariable_Unpack(gs[0]);
  size_t bytes = 0;
  int rc = g_entry.grad_ws(count, &bytes);
  if (rc != FLCE_OK) return status(rc);
  Tensor ws;
  if (!workspace(a[3], bytes, like, &ws)) Py_RETURN_NONE;
  const Tensor norm = empty({}, at::kFloat, like);
  float* out = norm.mutable_data_ptr<float>();
  rc = clip ? g_entry.clip(src.data(), dst.data(), numel.data(), dtype.data(), count, float(max_norm), out,
                           ws.data_ptr(), bytes, stream_of(like))
            : g_entry.grad_norm(src.data(), numel.data(), dtype.data(), count, out, ws.data_ptr(), bytes,
                                stream_of(like));
  if (rc != FLCE_OK) return status(rc);
  for (Py_ssize_t i = 0; clip && i < count; ++i) wrote(THPVariable_Unpack(to ? os[i] : gs[i]));
  return pack({norm});
  END_HANDLE_TH_ERRORS
}

// (logits, tokens, lens, prompt_lens, repetition, presence, frequency, bias_ids, bias, mask, out, out type or -1,
//  workspace) -> (out, token, lse)
PyObject* process_logits(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 13) return PyErr_Format(PyExc_TypeError, "process_logits takes 13 arguments");
  const Arg z = arg(a[0]);
  if (!z || !z.ok || z->dim() != 2) Py_RETURN_NONE;
  const int64_t dev = z->get_device(), b = z->size(0), v = z->size(1);
  const Rows rows(*z.t);
  Arg t[10];
  for (int i = 1; i < 11; ++i) {
    t[i - 1] = arg(a[i], dev);
    if (!t[i - 1].ok) Py_RETURN_NONE;
  }
  const Arg &tokens = t[0], &bias_ids = t[6], &bias = t[7], &mask = t[8], &out_arg = t[9];
  const int code = code_of(z->scalar_type());
  if (!rows.ok || code < 0 || bool(bias_ids) != bool(bias)) Py_RETURN_NONE;
  flce_logits_problem p{};
  p.rows = b;
  p.vocab = v;
  p.logits_stride = rows.stride;
  p.logits_dtype = code;
  auto ids = [&](const Arg& x, int64_t* cols, int64_t* stride, int32_t* i64) {
    const at::ScalarType type = x->scalar_type();
    if (x->dim() != 2 || x->size(0) != b || (type != at::kLong && type != at::kInt)) return false;
    *cols = x->size(1);
    *stride = x->stride(0);
    *i64 = type == at::kLong;
    return x->numel() == 0 || x->size(1) == 1 || x->stride(1) == 1;
  };
  if (tokens) {
    if (!ids(tokens, &p.history, &p.tokens_stride, &p.tokens_i64)) Py_RETURN_NONE;
    for (int i = 1; i < 6; ++i)
      if (t[i] && !vector_of(t[i], b, i < 3 ? at::kLong : at::kFloat)) Py_RETURN_NONE;
  } else {
    for (int i = 1; i < 6; ++i)
      if (t[i]) Py_RETURN_NONE;
  }
  if (bias) {
    if (!ids(bias_ids, &p.n_bias, &p.bias_ids_stride, &p.bias_ids_i64)) Py_RETURN_NONE;
    if (bias->sizes() != bias_ids->sizes() || bias->scalar_type() != at::kFloat) Py_RETURN_NONE;
    if (bias->numel() && bias->size(1) > 1 && bias->stride(1) != 1) Py_RETURN_NONE;
    p.bias_stride = bias->stride(0);
  }
  if (mask) {
    if (mask->dim() != 2 || mask->size(0) != b || mask->size(1) != (v + 31) / 32 || mask->scalar_type() != at::kInt ||
        (mask->size(1) > 1 && mask->stride(1) != 1))
      Py_RETURN_NONE;
    p.mask_stride = mask->stride(0);
  }
  const long want = PyLong_AsLong(a[11]);
  if (PyErr_Occurred()) return nullptr;
  Tensor out;
  if (out_arg) {
    out = *out_arg.t;
    const int oc = code_of(out.scalar_type());
    if (out.sizes() != z->sizes() || oc < 0 || (want >= 0 && oc != want) || (v > 1 && out.stride(1) != 1)) Py_RETURN_NONE;
  } else {
    out = empty({b, v}, want < 0 ? z->scalar_type() : kTypes[want], *z.t);
  }
  p.out_stride = out.stride(0);
  p.out_dtype = code_of(out.scalar_type());
  size_t bytes = 0;
  int rc = g_entry.logits_ws(&p, &bytes);
  if (rc != FLCE_OK) return status(rc);
  Tensor ws;
  if (!workspace(a[12], bytes, *z.t, &ws)) Py_RETURN_NONE;
  const Tensor token = empty({b}, at::kLong, *z.t), lse = empty({b}, at::kFloat, *z.t);
  const bool hist = p.history > 0 && b > 0;
  auto use = [](bool on, const Arg& x) { return on ? x.ptr() : nullptr; };
  rc = g_entry.logits(&p, z.ptr(), use(hist, tokens), static_cast<const int64_t*>(use(hist, t[1])),
                      static_cast<const int64_t*>(use(hist, t[2])), static_cast<const float*>(use(hist, t[3])),
                      static_cast<const float*>(use(hist, t[4])), static_cast<const float*>(use(hist, t[5])),
                      bias_ids.ptr(), static_cast<const float*>(bias.ptr()), mask.ptr(),
                      out.numel() ? out.data_ptr() : nullptr, b ? token.mutable_data_ptr<int64_t>() : nullptr,
                      b ? lse.mutable_data_ptr<float>() : nullptr, ws.data_ptr(), bytes, stream_of(*z.t));
  if (rc != FLCE_OK) return status(rc);
  if (out_arg) wrote(out);
  PyObject* r = pack({out, token, lse});
  if (r && out_arg) {  // the caller's own object
    Py_INCREF(a[10]);
    PyTuple_SetItem(r, 0, a[10]);
  }
  return r;
  END_HANDLE_TH_ERRORS
}

bool ids_of(const Arg& a) {
  return (a->scalar_type() == at::kLong || a->scalar_type() == at::kInt) && a->is_contiguous();
}

// (weight, ids, scale, out type or -1) -> (out,)
PyObject* embedding(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 4) return PyErr_Format(PyExc_TypeError, "embedding takes 4 arguments");
  const Arg w = arg(a[0]);
  if (!w || !w.ok || w->dim() != 2 || w->size(0) < 1) Py_RETURN_NONE;
  const Arg ids = arg(a[1], w->get_device());
  const Rows rows(*w.t);
  const int code = code_of(w->scalar_type());
  if (!ids || !ids.ok || !ids_of(ids) || !rows.ok || code < 0) Py_RETURN_NONE;
  const double scale = PyFloat_AsDouble(a[2]);
  const long want = PyLong_AsLong(a[3]);
  if (PyErr_Occurred()) return nullptr;
  std::vector<int64_t> size = ids->sizes().vec();
  size.push_back(rows.d);
  const Tensor out = empty(size, want < 0 ? w->scalar_type() : kTypes[want], *w.t);
  const flce_embedding_problem p = {ids->numel(), rows.n, rows.d, rows.stride, rows.d, -1, code,
                                    want < 0 ? code : int32_t(want), ids->scalar_type() == at::kLong, 0, float(scale), 0};
  const int rc = g_entry.embedding(&p, ids.ptr(), w.ptr(), out.numel() ? out.data_ptr() : nullptr, stream_of(*w.t));
  if (rc != FLCE_OK) return status(rc);
  return pack({out});
  END_HANDLE_TH_ERRORS
}

// (dout, ids, vocab, scale, padding, type or -1, dweight or None, workspace) -> (dweight,)
PyObject* embedding_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 8) return PyErr_Format(PyExc_TypeError, "embedding_backward takes 8 arguments");
  const Arg d = arg(a[0]);
  if (!d || !d.ok || d->dim() < 1) Py_RETURN_NONE;
  const Arg ids = arg(a[1], d->get_device()), given = arg(a[6], d->get_device());
  const Rows rows(*d.t);
  const int code = code_of(d->scalar_type());
  if (!ids || !ids.ok || !ids_of(ids) || !given.ok || !rows.ok || code < 0) Py_RETURN_NONE;
  if (ids->sizes() != d->sizes().slice(0, d->dim() - 1)) Py_RETURN_NONE;
  const int64_t vocab = PyLong_AsLongLong(a[2]), padding = PyLong_AsLongLong(a[4]);
  const double scale = PyFloat_AsDouble(a[3]);
  const long want = PyLong_AsLong(a[5]);
  if (PyErr_Occurred()) return nullptr;
  if (vocab < 1 || vocab >= INT32_MAX) Py_RETURN_NONE;
  Tensor dw;
  if (given) {
    dw = *given.t;
    if (dw.dim() != 2 || dw.size(0) != vocab || dw.size(1) != rows.d || (rows.d > 1 && dw.stride(1) != 1) ||
        code_of(dw.scalar_type()) < 0 || (want >= 0 && code_of(dw.scalar_type()) != want))
      Py_RETURN_NONE;
  } else {
    dw = empty({vocab, rows.d}, want < 0 ? d->scalar_type() : kTypes[want], *d.t);
  }
  const flce_embedding_problem p = {rows.n, vocab, rows.d, dw.stride(0), rows.stride, padding,
                                    code_of(dw.scalar_type()), code, ids->scalar_type() == at::kLong, bool(given),
                                    float(scale), 0};
  size_t bytes = 0;
  int rc = g_entry.embedding_ws(&p, &bytes);
  if (rc != FLCE_OK) return status(rc);
  Tensor ws;
  if (!workspace(a[7], bytes, *d.t, &ws)) Py_RETURN_NONE;
  rc = g_entry.embedding_bwd(&p, ids.ptr(), d.ptr(), dw.data_ptr(), ws.data_ptr(), bytes, stream_of(*d.t));
  if (rc != FLCE_OK) return status(rc);
  if (given) wrote(dw);
  PyObject* r = pack({dw});
  if (r && given) {  // the caller's own object
    Py_INCREF(a[6]);
    PyTuple_SetItem(r, 0, a[6]);
  }
  return r;
  END_HANDLE_TH_ERRORS
}

// A matrix in 4 bits: contiguous codes and scales of the sizes that its columns ask for.
struct Mx {
  Arg codes, scales;
  int64_t n = 0, d = 0;
  bool ok = false;
  Mx(PyObject* c, PyObject* s, PyObject* cols, int64_t device) : codes(arg(c, device)) {
    d = PyLong_AsLongLong(cols);
    if (!codes || !codes.ok || codes->dim() != 2 || d < 1 || d > (1 << 24)) return;
    scales = arg(s, codes->get_device());
    n = codes->size(0);
    const int64_t blocks = (d + 31) / 32;
    ok = scales && scales.ok && codes->size(1) == blocks * 16 && scales->dim() == 5 &&
         scales->size(0) == (n + 127) / 128 && scales->size(1) == (blocks + 3) / 4 && scales->size(2) == 32 &&
         scales->size(3) == 4 && scales->size(4) == 4 && codes->scalar_type() == at::kByte &&
         scales->scalar_type() == at::kByte && codes->is_contiguous() && scales->is_contiguous();
  }
};

// (x,) -> (codes, scales)
PyObject* mxfp4_quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 1) return PyErr_Format(PyExc_TypeError, "mxfp4_quantize takes 1 argument");
  const Arg x = arg(a[0]);
  if (!x || !x.ok) Py_RETURN_NONE;
  const Rows rows(*x.t);
  const int code = code_of(x->scalar_type());
  if (!rows.ok || code < 0) Py_RETURN_NONE;
  const int64_t blocks = (rows.d + 31) / 32;
  const Tensor codes = empty({rows.n, blocks * 16}, at::kByte, *x.t);
  const Tensor scales = empty({(rows.n + 127) / 128, (blocks + 3) / 4, 32, 4, 4}, at::kByte, *x.t);
  const flce_mxfp4_problem p = {rows.n, rows.d, rows.stride, code, 0};
  const bool any = rows.n > 0;
  const int rc = g_entry.mx_quantize(&p, x.ptr(), any ? codes.data_ptr() : nullptr, any ? scales.data_ptr() : nullptr,
                                     stream_of(*x.t));
  if (rc != FLCE_OK) return status(rc);
  return pack({codes, scales});
  END_HANDLE_TH_ERRORS
}

// (codes, scales, cols, out type) -> (out,)
PyObject* mxfp4_dequantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 4) return PyErr_Format(PyExc_TypeError, "mxfp4_dequantize takes 4 arguments");
  const Mx q(a[0], a[1], a[2], -1);
  const long want = PyLong_AsLong(a[3]);
  if (PyErr_Occurred()) return nullptr;
  if (!q.ok) Py_RETURN_NONE;
  const Tensor out = empty({q.n, q.d}, kTypes[want], *q.codes.t);
  const flce_mxfp4_problem p = {q.n, q.d, q.d, int32_t(want), 0};
  const int rc = g_entry.mx_dequantize(&p, q.codes.ptr(), q.scales.ptr(), out.numel() ? out.data_ptr() : nullptr,
                                       stream_of(out));
  if (rc != FLCE_OK) return status(rc);
  return pack({out});
  END_HANDLE_TH_ERRORS
}

// (hidden, codes, scales, cols, bias, logit_scale, softcap, out type or -1, out, workspace) -> (out,)
PyObject* mxfp4_logits(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 10) return PyErr_Format(PyExc_TypeError, "mxfp4_logits takes 10 arguments");
  const Arg h = arg(a[0]);
  if (!h || !h.ok || h->dim() < 1) Py_RETURN_NONE;
  const int64_t dev = h->get_device();
  const Mx w(a[1], a[2], a[3], dev);
  const Arg bias = arg(a[4], dev), given = arg(a[8], dev);
  const Rows rows(*h.t);
  const int code = code_of(h->scalar_type()), bcode = bias ? code_of(bias->scalar_type()) : FLCE_F32;
  const double scale = PyFloat_AsDouble(a[5]), cap = PyFloat_AsDouble(a[6]);
  const long want = PyLong_AsLong(a[7]);
  if (PyErr_Occurred()) return nullptr;
  if (!w.ok || !bias.ok || !given.ok || !rows.ok || rows.d != w.d || w.n < 1 || code < 0 || bcode < 0) Py_RETURN_NONE;
  if (bias && !vector_of(bias, w.n, bias->scalar_type())) Py_RETURN_NONE;
  std::vector<int64_t> size = h->sizes().vec();
  size.back() = w.n;
  Tensor out;
  int64_t stride = w.n;
  if (given) {
    out = *given.t;
    const Rows o(out);
    if (!o.ok || out.sizes() != at::IntArrayRef(size) || code_of(out.scalar_type()) < 0 ||
        (want >= 0 && code_of(out.scalar_type()) != want))
      Py_RETURN_NONE;
    stride = o.stride;
  } else {
    out = empty(size, want < 0 ? h->scalar_type() : kTypes[want], *h.t);
  }
  const flce_mxfp4_logits_problem p = {rows.n, w.n, w.d, rows.stride, stride, code, code_of(out.scalar_type()), bcode,
                                       float(scale), float(cap), 0};
  size_t bytes = 0;
  int rc = g_entry.mx_logits_ws(&p, &bytes);
  if (rc != FLCE_OK) return status(rc);
  Tensor ws;
  if (!workspace(a[9], bytes, *h.t, &ws)) Py_RETURN_NONE;
  rc = g_entry.mx_logits(&p, h.ptr(), w.codes.ptr(), w.scales.ptr(), bias.ptr(),
                         out.numel() ? out.data_ptr() : nullptr, ws.data_ptr(), bytes, stream_of(*h.t));
  if (rc != FLCE_OK) return status(rc);
  if (given) wrote(out);
  PyObject* r = pack({out});
  if (r && given) {  // the caller's own object
    Py_INCREF(a[8]);
    PyTuple_SetItem(r, 0, a[8]);
  }
  return r;
  END_HANDLE_TH_ERRORS
}

// (logits, uniform, temperature, top_k, top_p, min_p) -> (token, logprob, kept)
PyObject* sample_tokens(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 6) return PyErr_Format(PyExc_TypeError, "sample_tokens takes 6 arguments");
  const Arg z = arg(a[0]);
  if (!z || !z.ok || z->dim() != 2) Py_RETURN_NONE;
  const Rows rows(*z.t);
  const int code = code_of(z->scalar_type());
  if (!rows.ok || code < 0) Py_RETURN_NONE;
  Arg t[5];
  for (int i = 0; i < 5; ++i) {
    t[i] = arg(a[i + 1], z->get_device());
    if (!t[i].ok || (!t[i] && i == 0) || (t[i] && !vector_of(t[i], rows.n, i == 2 ? at::kLong : at::kFloat)))
      Py_RETURN_NONE;
  }
  const Tensor token = empty({rows.n}, at::kLong, *z.t), logprob = empty({rows.n}, at::kFloat, *z.t),
               kept = empty({rows.n}, at::kLong, *z.t);
  const bool any = rows.n > 0;
  const flce_sample_problem p = {rows.n, rows.d, rows.stride, code, 0};
  auto f = [](const Arg& x) { return static_cast<const float*>(x.ptr()); };
  const int rc = g_entry.sample(&p, z.ptr(), f(t[0]), f(t[1]), static_cast<const int64_t*>(t[2].ptr()), f(t[3]), f(t[4]),
                                any ? token.mutable_data_ptr<int64_t>() : nullptr,
                                any ? logprob.mutable_data_ptr<float>() : nullptr,
                                any ? kept.mutable_data_ptr<int64_t>() : nullptr, stream_of(*z.t));
  if (rc != FLCE_OK) return status(rc);
  return pack({token, logprob, kept});
  END_HANDLE_TH_ERRORS
}

#define FLCE_METHOD(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {FLCE_METHOD(bind), FLCE_METHOD(add_rms_norm), FLCE_METHOD(add_rms_norm_backward),
                          FLCE_METHOD(clip_grad_norm), FLCE_METHOD(process_logits), FLCE_METHOD(embedding),
                          FLCE_METHOD(embedding_backward), FLCE_METHOD(mxfp4_quantize), FLCE_METHOD(mxfp4_dequantize),
                          FLCE_METHOD(mxfp4_logits), FLCE_METHOD(sample_tokens), {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "flce_torch", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit_flce_torch() { return PyModule_Create(&kModule); }
