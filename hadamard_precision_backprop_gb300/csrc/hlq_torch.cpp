// hlq_torch.cpp -- the binding's short way into libhlq for the operators
// around the layer: argument checks, output and workspace allocation and the
// call in one step, for the calls of a training step that cost the host more
// than the GPU.
//
// Each function takes what the Python entry point takes (outputs are always
// allocated here) and gives its result, or NotImplemented where an argument is
// not plainly right or the library refuses: the Python entry point then goes
// the long way, which does the call or says what is wrong.
#include <Python.h>

#include <array>
#include <cstdint>
#include <memory>
#include <vector>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "hlq.h"

namespace {

PyObject* not_implemented() {
  Py_INCREF(Py_NotImplemented);
  return Py_NotImplemented;
}

// hlq_dtype of a scalar type; -1: none.
int code_of(at::ScalarType t) {
  return t == at::kFloat ? HLQ_F32 : t == at::kBFloat16 ? HLQ_BF16 : -1;
}

// Lets other threads run: allocations may wait for the driver, and launches for
// a stream whose queue is full.  The arguments have been read before; their
// tensors are held by the entry point's frame.
struct WithoutGil {
  PyThreadState* state = PyEval_SaveThread();
  ~WithoutGil() { PyEval_RestoreThread(state); }
};

// What the arguments of one call have in common.
struct Call {
  bool ok = true;
  int device = -1;
  int64_t rows = 0, cols = 0;

  // An argument that is a tensor, or null for None.
  const at::Tensor* tensor(PyObject* o) {
    if (o == Py_None) return nullptr;
    if (!THPVariable_CheckExact(o)) {
      ok = false;
      return nullptr;
    }
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.layout() != at::kStrided || (device >= 0 && t.get_device() != device)) {
      ok = false;
      return nullptr;
    }
    return &t;
  }

  struct Rows {
    const void* p = nullptr;
    int64_t ld = 0;
    int dt = HLQ_F32;
  };
  // The call's first matrix: sets the device and the shape.
  Rows first(PyObject* o) {
    const at::Tensor* t = tensor(o);
    if (!t || t->dim() != 2 || t->get_device() != c10::cuda::current_device()) {
      ok = false;
      return {};
    }
    device = t->get_device();
    rows = t->size(0);
    cols = t->size(1);
    return matrix(o, -1);
  }
  // A matrix of that shape, of dtype `dt` if it is >= 0; nothing for None.
  Rows matrix(PyObject* o, int dt) {
    const at::Tensor* t = tensor(o);
    if (!t) return {};
    Rows r;
    r.dt = code_of(t->scalar_type());
    if (t->dim() != 2 || t->size(0) != rows || t->size(1) != cols || r.dt < 0 ||
        (dt >= 0 && r.dt != dt) || (t->stride(1) != 1 && cols > 1)) {
      ok = false;
      return {};
    }
    r.ld = t->stride(0);
    r.p = t->const_data_ptr();
    return r;
  }
  // A vector [n] of scalar type `want`.
  const void* vector(PyObject* o, int64_t n, at::ScalarType want) {
    const at::Tensor* t = tensor(o);
    if (!t) return nullptr;
    if (t->dim() != 1 || t->size(0) != n || !t->is_contiguous() || t->scalar_type() != want) {
      ok = false;
      return nullptr;
    }
    return t->const_data_ptr();
  }
  const float* floats(PyObject* o, int64_t n) {
    return static_cast<const float*>(vector(o, n, at::kFloat));
  }
  // A weight or bias [cols] of either type.
  const void* affine(PyObject* o, int* dt) {
    const at::Tensor* t = tensor(o);
    if (!t) return nullptr;
    *dt = code_of(t->scalar_type());
    if (*dt < 0) ok = false;
    return vector(o, cols, t->scalar_type());
  }
  // The scalar type of a dtype argument, `own` for None.
  at::ScalarType dtype(PyObject* o, int own) {
    if (o == Py_None) return own == HLQ_BF16 ? at::kBFloat16 : at::kFloat;
    if (!THPDtype_Check(o) || code_of(reinterpret_cast<THPDtype*>(o)->scalar_type) < 0) {
      ok = false;
      return at::kFloat;
    }
    return reinterpret_cast<THPDtype*>(o)->scalar_type;
  }
  double number(PyObject* o) {
    const double v = PyFloat_Check(o) ? PyFloat_AS_DOUBLE(o) : PyLong_Check(o) ? PyLong_AsDouble(o)
                                                                               : (ok = false, 0.0);
    if (v == -1.0 && PyErr_Occurred()) {
      PyErr_Clear();
      ok = false;
    }
    return v;
  }
  bool flag(PyObject* o) {
    if (!PyBool_Check(o)) ok = false;
    return o == Py_True;
  }
  at::Tensor empty(c10::IntArrayRef size, at::ScalarType dt) const {
    return at::Tensor(at::detail::empty_cuda(
        size, dt, c10::Device(c10::DeviceType::CUDA, (c10::DeviceIndex)device), std::nullopt));
  }
  at::Tensor workspace(size_t n) const { return empty({(int64_t)n}, at::kByte); }
  void* stream() const {
    return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
  }
};

// A tuple of tensors, None for an undefined one.
PyObject* tuple_of(std::initializer_list<at::Tensor> ts) {
  PyObject* out = PyTuple_New((Py_ssize_t)ts.size());
  if (!out) return nullptr;
  Py_ssize_t i = 0;
  for (const at::Tensor& t : ts) {
    PyObject* o = Py_None;
    if (t.defined())
      o = THPVariable_Wrap(t);
    else
      Py_INCREF(o);
    if (!o) {
      Py_DECREF(out);
      return nullptr;
    }
    PyTuple_SET_ITEM(out, i++, o);
  }
  return out;
}

// (x, weight, bias, eps, residual, out_dtype, with_stats)
PyObject* layer_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 7) return not_implemented();
  Call c;
  const Call::Rows x = c.first(a[0]);
  if (!c.ok) return not_implemented();
  int w_dt = -1, b_dt = -1;
  const void* w = c.affine(a[1], &w_dt);
  const void* b = c.affine(a[2], &b_dt);
  const double eps = c.number(a[3]);
  const Call::Rows r = c.matrix(a[4], x.dt);
  const at::ScalarType y_type = c.dtype(a[5], x.dt);
  const bool stats = c.flag(a[6]);
  if (!c.ok || (w && b && w_dt != b_dt)) return not_implemented();
  const int64_t T = c.rows, C = c.cols;
  const bool residual = a[4] != Py_None;
  at::Tensor y, h, mean, rstd;
  hlq_status st;
  {
    WithoutGil g;
    y = c.empty({T, C}, y_type);
    if (residual) h = c.empty({T, C}, x.dt == HLQ_BF16 ? at::kBFloat16 : at::kFloat);
    if (stats) mean = c.empty({T}, at::kFloat), rstd = c.empty({T}, at::kFloat);
    st = hlq_layer_norm(
        x.p, x.ld, r.p, r.ld, x.dt, w, b, w_dt >= 0 ? w_dt : b_dt >= 0 ? b_dt : HLQ_F32, T, C,
        (float)eps, y.mutable_data_ptr(), C, code_of(y_type),
        residual ? h.mutable_data_ptr() : nullptr, C,
        stats ? mean.mutable_data_ptr<float>() : nullptr,
        stats ? rstd.mutable_data_ptr<float>() : nullptr, c.stream());
  }
  if (st != HLQ_OK) return not_implemented();
  return h.defined() ? tuple_of({y, mean, rstd, h}) : tuple_of({y, mean, rstd});
  END_HANDLE_TH_ERRORS
}

// (g_y, x, mean, rstd, weight, g_residual, out_dtype, with_weight_grads)
PyObject* layer_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 8) return not_implemented();
  Call c;
  const Call::Rows x = c.first(a[1]);
  if (!c.ok) return not_implemented();
  const int64_t T = c.rows, C = c.cols;
  const Call::Rows g = c.matrix(a[0], -1);
  const float *mean = c.floats(a[2], T), *rstd = c.floats(a[3], T);
  int w_dt = HLQ_F32;
  const void* w = c.affine(a[4], &w_dt);
  const at::ScalarType gx_type = c.dtype(a[6], x.dt);
  const Call::Rows r = c.matrix(a[5], code_of(gx_type));
  const bool sums = c.flag(a[7]);
  if (!c.ok) return not_implemented();
  at::Tensor gx, gw, gb, ws;
  hlq_status st;
  {
    WithoutGil no_gil;
    gx = c.empty({T, C}, gx_type);
    size_t ws_bytes = 0;
    if (sums) {
      gw = c.empty({C}, at::kFloat), gb = c.empty({C}, at::kFloat);
      ws_bytes = hlq_layer_norm_backward_workspace_bytes(T, C);
      ws = c.workspace(ws_bytes);
    }
    st = hlq_layer_norm_backward(
        g.p, g.ld, g.dt, x.p, x.ld, x.dt, mean, rstd, w, w_dt, r.p, r.ld, T, C,
        gx.mutable_data_ptr(), C, code_of(gx_type), sums ? gw.mutable_data_ptr<float>() : nullptr,
        sums ? gb.mutable_data_ptr<float>() : nullptr, sums ? ws.mutable_data_ptr() : nullptr,
        ws_bytes, c.stream());
  }
  if (st != HLQ_OK) return not_implemented();
  return tuple_of({gx, gw, gb});
  END_HANDLE_TH_ERRORS
}

// (logits, targets, scale)
PyObject* token_logprobs(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 3) return not_implemented();
  Call c;
  const Call::Rows x = c.first(a[0]);
  if (!c.ok) return not_implemented();
  const int64_t T = c.rows;
  const int64_t* targets = static_cast<const int64_t*>(c.vector(a[1], T, at::kLong));
  const double scale = c.number(a[2]);
  if (!c.ok) return not_implemented();
  at::Tensor logp, lse;
  hlq_status st;
  {
    WithoutGil g;
    logp = c.empty({T}, at::kFloat), lse = c.empty({T}, at::kFloat);
    st = hlq_token_logprobs(x.p, x.ld, x.dt, targets, T, c.cols, (float)scale,
                            logp.mutable_data_ptr<float>(), lse.mutable_data_ptr<float>(),
                            c.stream());
  }
  return st == HLQ_OK ? tuple_of({logp, lse}) : not_implemented();
  END_HANDLE_TH_ERRORS
}

// (logits, actions, old_logp, advantages, weights, ref_logp, clip_low, clip_high, kl_coef, scale,
//  grad_scale, with_grad)
PyObject* policy_loss(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 12) return not_implemented();
  Call c;
  const Call::Rows x = c.first(a[0]);
  if (!c.ok) return not_implemented();
  const int64_t T = c.rows, V = c.cols;
  const int64_t* actions = static_cast<const int64_t*>(c.vector(a[1], T, at::kLong));
  const float *old = c.floats(a[2], T), *adv = c.floats(a[3], T), *w = c.floats(a[4], T),
              *ref = c.floats(a[5], T);
  std::array<double, 5> v;
  for (int i = 0; i < 5; ++i) v[i] = c.number(a[6 + i]);
  const bool grad = c.flag(a[11]);
  if (!c.ok) return not_implemented();
  at::Tensor stats, logp, g, ws;
  hlq_status st;
  {
    WithoutGil no_gil;
    const size_t ws_bytes = hlq_policy_loss_workspace_bytes(T, V);
    stats = c.empty({4}, at::kFloat), logp = c.empty({T}, at::kFloat);
    if (grad) g = c.empty({T, V}, x.dt == HLQ_BF16 ? at::kBFloat16 : at::kFloat);
    ws = c.workspace(ws_bytes);
    st = hlq_policy_loss(
        x.p, x.ld, x.dt, actions, old, ref, adv, w, T, V, (float)v[3], (float)v[0], (float)v[1],
        (float)v[2], (float)v[4], stats.mutable_data_ptr<float>(), logp.mutable_data_ptr<float>(),
        grad ? g.mutable_data_ptr() : nullptr, V, ws.mutable_data_ptr(), ws_bytes, c.stream());
  }
  if (st != HLQ_OK) return not_implemented();
  return tuple_of({stats, logp, g});
  END_HANDLE_TH_ERRORS
}

struct Table {
  std::vector<const void*> p;
  std::vector<int32_t> dt;
  std::vector<int64_t> n;
  // The tensors of a list or tuple, all on one device (the first's, if `c`
  // has none yet).
  bool fill(Call& c, PyObject* seq) {
    const Py_ssize_t len = PySequence_Fast_GET_SIZE(seq);
    p.resize(len), dt.resize(len), n.resize(len);
    PyObject** items = PySequence_Fast_ITEMS(seq);
    for (Py_ssize_t i = 0; i < len; ++i) {
      const at::Tensor* t = c.tensor(items[i]);
      if (!t || !t->is_contiguous()) return false;
      if (c.device < 0) c.device = t->get_device();
      dt[i] = code_of(t->scalar_type());
      if (dt[i] < 0) return false;
      p[i] = t->const_data_ptr();
      n[i] = t->numel();
    }
    return c.ok;
  }
};

// (grads, max_norm, outs, norm_only); grads and outs lists or tuples
PyObject* clip_grad_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 4) return not_implemented();
  const auto is_seq = [](PyObject* o) { return PyList_Check(o) || PyTuple_Check(o); };
  if (!is_seq(a[0]) || PySequence_Fast_GET_SIZE(a[0]) == 0) return not_implemented();
  Call c;
  const double max_norm = c.number(a[1]);
  const bool norm_only = c.flag(a[3]);
  if (!c.ok) return not_implemented();
  Table g, o;
  // whatever becomes of the caller's list of outputs (the gradients' is the
  // entry point's own)
  const std::unique_ptr<PyObject, void (*)(PyObject*)> outs(
      is_seq(a[2]) ? PySequence_Tuple(a[2]) : nullptr, [](PyObject* t) { Py_XDECREF(t); });
  if (!g.fill(c, a[0]) || c.device != c10::cuda::current_device()) return not_implemented();
  if (a[2] != Py_None && (norm_only || !outs || !o.fill(c, outs.get()) || o.n != g.n))
    return not_implemented();
  const Table& out = a[2] == Py_None ? g : o;
  const int64_t count = (int64_t)g.p.size();
  at::Tensor norm_coef, ws;
  hlq_status st;
  {
    WithoutGil no_gil;
    const size_t ws_bytes = hlq_clip_grad_norm_workspace_bytes(count);
    norm_coef = c.empty({2}, at::kFloat), ws = c.workspace(ws_bytes);
    st = hlq_clip_grad_norm(
        count, g.p.data(), g.dt.data(),
        norm_only ? nullptr : reinterpret_cast<void* const*>(const_cast<void**>(out.p.data())),
        norm_only ? nullptr : out.dt.data(), g.n.data(), (float)max_norm,
        norm_coef.mutable_data_ptr<float>(), ws.mutable_data_ptr(), ws_bytes, c.stream());
  }
  return st == HLQ_OK ? THPVariable_Wrap(norm_coef) : not_implemented();
  END_HANDLE_TH_ERRORS
}

#define METHOD(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(layer_norm),  METHOD(layer_norm_backward), METHOD(token_logprobs),
                         METHOD(policy_loss), METHOD(clip_grad_norm),      {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_hlq_torch", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__hlq_torch(void) { return PyModule_Create(&module); }
