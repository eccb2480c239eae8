// Python binding of the convolution, the scan and the gated projections: checks of the tensors,
// allocation of outputs and workspaces, and the call of the C entry points (include/sdm.h).
//
// These calls are on a decode step's path, where a kernel of two microseconds should not wait for
// twenty of argument handling in Python, so what api.py does in Python is done here on the tensors
// themselves.  Every function takes its arguments by position from its Python namesake in layers.py,
// works on the tensors' device and its current stream, and raises TypeError or ValueError for a
// tensor that does not fit; a status of the C entry point becomes an SDMError.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/core/LegacyTypeDispatch.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <cstdio>
#include <string>

#include "../../include/sdm.h"

namespace {

PyObject* sdm_error = nullptr;  // api.SDMError

// An exception of Python that has been set.
struct Raised {};
[[noreturn]] void raise(PyObject* type, const char* format, ...) {
  va_list v;
  va_start(v, format);
  PyErr_FormatV(type, format, v);
  va_end(v);
  throw Raised();
}
[[noreturn]] void raise_status(const char* fn, int status) {
  if (status == SDM_EOVERLAP) raise(PyExc_ValueError, "%s: an output overlaps another tensor of the call", fn);
  PyObject* e = PyObject_CallFunction(sdm_error, "si", fn, status);
  if (e) {
    PyErr_SetObject(sdm_error, e);
    Py_DECREF(e);
  }
  throw Raised();
}

std::string shape_text(at::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + ")";
}

const at::Tensor none;

// The tensor in `o`, or an undefined one for None.
const at::Tensor& optional(PyObject* o, const char* name) {
  if (o == Py_None) return none;
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, "%s must be a CUDA tensor", name);
  return THPVariable_Unpack(o);
}
const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) raise(PyExc_TypeError, "%s must be a CUDA tensor", name);
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda()) raise(PyExc_TypeError, "%s must be a CUDA tensor", name);
  return t;
}

int code(at::ScalarType t, const char* name) {
  if (t == at::kFloat) return SDM_F32;
  if (t == at::kBFloat16) return SDM_BF16;
  raise(PyExc_TypeError, "%s: unsupported dtype %s (float32 or bfloat16)", name, c10::toString(t));
}

struct Call {
  c10::DeviceIndex device;
  c10::cuda::CUDAGuard guard;
  at::AutoDispatchBelowAutograd below;  // outputs are plain tensors
  explicit Call(const at::Tensor& t) : device(t.device().index()), guard(t.device()) {}

  void* stream() const { return c10::cuda::getCurrentCUDAStream(device).stream(); }

  void fits(const at::Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape) const {
    if (!t.is_cuda()) raise(PyExc_TypeError, "%s must be a CUDA tensor", name);
    if (t.device().index() != device)
      raise(PyExc_ValueError, "%s is on cuda:%d, not on cuda:%d: every tensor of one call must be on the same device",
            name, int(t.device().index()), int(device));
    if (t.scalar_type() != type)
      raise(PyExc_TypeError, "%s must be %s, got %s", name, c10::toString(type), c10::toString(t.scalar_type()));
    if (t.sizes() != shape)
      raise(PyExc_ValueError, "%s must have shape %s, got %s", name, shape_text(shape).c_str(),
            shape_text(t.sizes()).c_str());
  }
  // Address of a contiguous tensor of that type and shape; null for None.
  void* dense(const at::Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape) const {
    if (!t.defined()) return nullptr;
    fits(t, name, type, shape);
    if (!t.is_contiguous()) raise(PyExc_ValueError, "%s must be contiguous", name);
    return t.data_ptr();
  }
  // Address and strides (between sequences, between tokens) of a tensor [B, T, ...] (lead 2) or [B, ...]
  // (lead 1) whose trailing dimensions are dense; a stride over one entry does not matter: 0.
  const void* rows(const at::Tensor& t, const char* name, at::ScalarType type, at::IntArrayRef shape, int lead,
                   long long* bs, long long* ts) const {
    *bs = *ts = 0;
    if (!t.defined()) return nullptr;
    fits(t, name, type, shape);
    int64_t n = 1;
    for (int k = int(shape.size()) - 1; k >= lead; --k) {
      if (shape[k] > 1 && t.stride(k) != n)
        raise(PyExc_ValueError, "%s must be dense in its last %d dimension(s)", name, int(shape.size()) - lead);
      n *= shape[k];
    }
    if (shape[0] > 1) *bs = t.stride(0);
    if (lead == 2 && shape[1] > 1) *ts = t.stride(1);
    return t.data_ptr();
  }
  at::Tensor empty(at::IntArrayRef shape, at::ScalarType type) const {
    return at::empty(shape, at::TensorOptions().dtype(type).device(at::kCUDA, device));
  }
  // Workspace of at least `need` bytes: the caller's, or one of its own.
  void* workspace(const at::Tensor& given, size_t need, at::Tensor* own, size_t* bytes) const {
    if (given.defined()) {
      if (!given.is_cuda() || given.device().index() != device || given.scalar_type() != at::kByte ||
          !given.is_contiguous())
        raise(PyExc_TypeError, "workspace must be a contiguous uint8 CUDA tensor on cuda:%d", int(device));
      *bytes = size_t(given.numel());
      return given.data_ptr();
    }
    *bytes = need;
    if (!need) return nullptr;
    *own = empty({int64_t(need)}, at::kByte);
    return own->data_ptr();
  }
};

// A size that the C entry points take as an int.
int as_int(int64_t v, const char* name) {
  if (v > 0x7FFFFFFF) raise(PyExc_ValueError, "%s is too large", name);
  return int(v);
}

struct State {
  const void* in = nullptr;
  void* out = nullptr;
  int rows = 0;
  PyObject* written = Py_None;
};
// state and state_out: in place where only `state` is given.
State state_rows(const Call& c, PyObject* o_in, PyObject* o_out, bool slots, int64_t nb, int64_t d1, int64_t d2,
                 at::ScalarType type) {
  State s;
  s.written = o_out == Py_None ? o_in : o_out;
  const at::Tensor &in = optional(o_in, "state"), &out = optional(s.written, "state_out");
  const at::Tensor& ref = in.defined() ? in : out;
  if (!ref.defined()) {
    if (slots) raise(PyExc_ValueError, "slots need a state");
    return s;
  }
  const int64_t n = ref.dim() ? ref.size(0) : 0;
  if (!slots && n != nb)
    raise(PyExc_ValueError, "state must have one row a sequence (%lld) without slots, got %lld", (long long)nb,
          (long long)n);
  s.in = c.dense(in, "state", type, {n, d1, d2});
  s.out = c.dense(out, "state_out", type, {n, d1, d2});
  s.rows = as_int(n, "state");
  return s;
}

PyObject* pair(PyObject* a, PyObject* b) {  // takes the reference to a
  PyObject* t = a ? PyTuple_New(2) : nullptr;
  if (!t) {
    Py_XDECREF(a);
    throw Raised();
  }
  PyTuple_SET_ITEM(t, 0, a);
  Py_INCREF(b);
  PyTuple_SET_ITEM(t, 1, b);
  return t;
}

// The output: the caller's tensor, or a new one.  Returns its address; *obj is a new reference.
void* output(const Call& c, PyObject* given, const char* name, at::IntArrayRef shape, at::ScalarType type,
             PyObject** obj) {
  if (given != Py_None) {
    void* p = c.dense(optional(given, name), name, type, shape);
    Py_INCREF(given);
    *obj = given;
    return p;
  }
  at::Tensor t = c.empty(shape, type);
  void* p = t.data_ptr();
  *obj = THPVariable_Wrap(std::move(t));
  if (!*obj) throw Raised();
  return p;
}

// Drops a reference where the call ends by an exception.
struct Held {
  PyObject* o = nullptr;
  ~Held() { Py_XDECREF(o); }
  PyObject* release() {
    PyObject* r = o;
    o = nullptr;
    return r;
  }
};

// conv(x, w, bias, state, state_out, act, lengths, slots, out, dev_err, lead) -> (y, state written)
PyObject* conv(PyObject* const* a) {
  const at::Tensor &x = tensor(a[0], "x"), &w = tensor(a[1], "w"), &bias = optional(a[2], "bias");
  const at::Tensor &lengths = optional(a[6], "lengths"), &slots = optional(a[7], "slots");
  const int act = int(PyLong_AsLong(a[5])), lead = int(PyLong_AsLong(a[10]));
  const Call c(x);
  if (x.dim() != lead + 1) raise(PyExc_ValueError, lead == 2 ? "x must be [B, T, D]" : "x must be [B, D]");
  if (w.dim() != 2) raise(PyExc_ValueError, "w must be [D, K]");
  const at::ScalarType ty = x.scalar_type(), wt = w.scalar_type();
  const int64_t nb = x.size(0), T = lead == 2 ? x.size(1) : 1, D = x.size(lead), K = w.size(1);
  const int dt = code(ty, "x"), wdt = code(wt, "w");
  long long bs, ts;
  const void* px = c.rows(x, "x", ty, x.sizes(), lead, &bs, &ts);
  const void* pw = c.dense(w, "w", wt, {D, K});
  const void* pb = c.dense(bias, "bias", wt, {D});
  const State st = state_rows(c, a[3], a[4], slots.defined(), nb, K - 1, D, ty);
  const void* pl = c.dense(lengths, "lengths", at::kInt, {nb});
  const void* ps = c.dense(slots, "slots", at::kInt, {nb});
  void* pe = c.dense(optional(a[9], "dev_err"), "dev_err", at::kInt, {1});
  Held y;
  void* py = output(c, a[8], "out", x.sizes(), ty, &y.o);
  if (nb == 0) return pair(y.release(), st.written);
  const int r = sdm_causal_conv(px, bs, ts, dt, pw, pb, wdt, as_int(nb, "B"), as_int(T, "T"), as_int(D, "D"),
                                as_int(K, "K"), act, st.in, st.out, st.rows, static_cast<const int32_t*>(pl),
                                static_cast<const int32_t*>(ps), py, static_cast<int*>(pe), c.stream());
  if (r != SDM_OK) raise_status("sdm_causal_conv", r);
  return pair(y.release(), st.written);
}

// scan(x, dt, A, B, C, D, z, dt_bias, state, state_out, softplus, lengths, slots, out, workspace, dev_err,
//      lead) -> (y, state written)
PyObject* scan(PyObject* const* a) {
  const at::Tensor &x = tensor(a[0], "x"), &dt = tensor(a[1], "dt"), &A = tensor(a[2], "A"), &B = tensor(a[3], "B"),
                   &C = tensor(a[4], "C"), &D = optional(a[5], "D"), &z = optional(a[6], "z"),
                   &bias = optional(a[7], "dt_bias"), &lengths = optional(a[11], "lengths"),
                   &slots = optional(a[12], "slots");
  const int lead = int(PyLong_AsLong(a[16]));
  const Call c(x);
  if (x.dim() != lead + 1) raise(PyExc_ValueError, lead == 2 ? "x must be [B, T, Dm]" : "x must be [B, Dm]");
  if (A.dim() != 2) raise(PyExc_ValueError, "A must be [Dm, N]");
  const at::ScalarType ty = x.scalar_type();
  const int64_t nb = x.size(0), T = lead == 2 ? x.size(1) : 1, Dm = x.size(lead), N = A.size(1);
  const bool grouped = B.dim() == lead + 2;
  if (!grouped && B.dim() != lead + 1)
    raise(PyExc_ValueError, lead == 2 ? "B must be [B, T, N] or [B, T, G, N]" : "B must be [B, N] or [B, G, N]");
  const int64_t G = grouped ? B.size(lead) : 1;
  int64_t bc[4];
  int n = 0;
  for (int k = 0; k < lead; ++k) bc[n++] = x.size(k);
  if (grouped) bc[n++] = G;
  bc[n++] = N;
  const at::IntArrayRef bcs(bc, size_t(n));

  sdm_ssm_args s = {};
  s.dtype = code(ty, "x");
  s.x = c.rows(x, "x", ty, x.sizes(), lead, &s.x_bs, &s.x_ts);
  s.dt = c.rows(dt, "dt", ty, x.sizes(), lead, &s.dt_bs, &s.dt_ts);
  s.Bm = c.rows(B, "B", ty, bcs, lead, &s.B_bs, &s.B_ts);
  s.Cm = c.rows(C, "C", ty, bcs, lead, &s.C_bs, &s.C_ts);
  s.z = c.rows(z, "z", ty, x.sizes(), lead, &s.z_bs, &s.z_ts);
  s.A = static_cast<const float*>(c.dense(A, "A", at::kFloat, {Dm, N}));
  s.D = static_cast<const float*>(c.dense(D, "D", at::kFloat, {Dm}));
  s.dt_bias = static_cast<const float*>(c.dense(bias, "dt_bias", at::kFloat, {Dm}));
  const State st = state_rows(c, a[8], a[9], slots.defined(), nb, Dm, N, at::kFloat);
  s.state = static_cast<const float*>(st.in);
  s.state_out = static_cast<float*>(st.out);
  s.n_slots = st.rows;
  s.lengths = static_cast<const int32_t*>(c.dense(lengths, "lengths", at::kInt, {nb}));
  s.slots = static_cast<const int32_t*>(c.dense(slots, "slots", at::kInt, {nb}));
  void* pe = c.dense(optional(a[15], "dev_err"), "dev_err", at::kInt, {1});
  s.B = as_int(nb, "B");
  s.T = as_int(T, "T");
  s.Dm = as_int(Dm, "Dm");
  s.N = as_int(N, "N");
  s.G = as_int(G, "G");
  s.softplus = PyObject_IsTrue(a[10]);
  if (s.softplus < 0) throw Raised();  // its truth is an error
  Held y;
  s.y = output(c, a[13], "out", x.sizes(), ty, &y.o);
  if (nb == 0) return pair(y.release(), st.written);
  at::Tensor own;
  size_t bytes = 0;
  void* ws = c.workspace(optional(a[14], "workspace"),
                         T > 1 ? sdm_selective_scan_workspace_size(s.B, s.T, s.Dm, s.N, s.G) : 0, &own, &bytes);
  const int r = sdm_selective_scan(&s, ws, bytes, static_cast<int*>(pe), c.stream());
  if (r != SDM_OK) raise_status("sdm_selective_scan", r);
  return pair(y.release(), st.written);
}

struct Gated {
  int64_t M, D, F;
  const void *x, *w;
};
Gated gated_operands(const Call& c, const at::Tensor& x, const at::Tensor& w) {
  if (x.dim() < 1 || w.dim() != 2 || w.size(0) % 2)
    raise(PyExc_ValueError, "x must be [..., D] and w [2 * F, D]");
  Gated g;
  g.D = x.size(-1);
  g.F = w.size(0) / 2;
  g.M = g.D ? x.numel() / g.D : 0;
  g.x = c.dense(x, "x", at::kBFloat16, x.sizes());
  g.w = c.dense(w, "w", at::kBFloat16, {2 * g.F, g.D});
  as_int(g.D, "D");
  as_int(g.F, "F");
  return g;
}

// gated(x, w, act, out, dev_err) -> h
PyObject* gated(PyObject* const* a) {
  const at::Tensor &x = tensor(a[0], "x"), &w = tensor(a[1], "w");
  const Call c(x);
  const Gated g = gated_operands(c, x, w);
  c10::SmallVector<int64_t, 6> shape(x.sizes().begin(), x.sizes().end());
  shape.back() = g.F;
  void* pe = c.dense(optional(a[4], "dev_err"), "dev_err", at::kInt, {1});
  Held h;
  void* ph = output(c, a[3], "out", shape, at::kBFloat16, &h.o);
  const int r = sdm_project_gated(g.x, g.w, g.M, int(g.D), int(g.F), int(PyLong_AsLong(a[2])), ph,
                                  static_cast<int*>(pe), c.stream());
  if (r != SDM_OK) raise_status("sdm_project_gated", r);
  return h.release();
}

// gated_grad(x, w, dh, act, dx, dw, workspace, dev_err) -> (dx, dw)
PyObject* gated_grad(PyObject* const* a) {
  const at::Tensor &x = tensor(a[0], "x"), &w = tensor(a[1], "w"), &dh = tensor(a[2], "dh");
  const Call c(x);
  const Gated g = gated_operands(c, x, w);
  c10::SmallVector<int64_t, 6> shape(x.sizes().begin(), x.sizes().end());
  shape.back() = g.F;
  const void* ph = c.dense(dh, "dh", at::kBFloat16, shape);
  void* pe = c.dense(optional(a[7], "dev_err"), "dev_err", at::kInt, {1});
  Held dx, dw;
  void* px = output(c, a[4], "dx", x.sizes(), at::kBFloat16, &dx.o);
  void* pw = output(c, a[5], "dw", w.sizes(), at::kBFloat16, &dw.o);
  at::Tensor own;
  size_t bytes = 0;
  void* ws = c.workspace(optional(a[6], "workspace"),
                         sdm_project_gated_backward_workspace_size(g.M, int(g.D), int(g.F)), &own, &bytes);
  const int r = sdm_project_gated_backward(g.x, g.w, ph, g.M, int(g.D), int(g.F), int(PyLong_AsLong(a[3])), px, pw,
                                           ws, bytes, static_cast<int*>(pe), c.stream());
  if (r != SDM_OK) raise_status("sdm_project_gated_backward", r);
  return pair(dx.release(), dw.o);
}

// torch's own exceptions become the Python errors that its own calls raise (out of memory:
// torch.OutOfMemoryError).
template <PyObject* (*F)(PyObject* const*)>
PyObject* translated(PyObject* const* args) {
  HANDLE_TH_ERRORS
  try {
    return F(args);
  } catch (const Raised&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// No C++ exception leaves an entry point.
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments are wanted, got %zd", N, n);
    return nullptr;
  }
  try {
    return translated<F>(args);
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

PyObject* set_error(PyObject*, PyObject* type) {
  Py_INCREF(type);
  Py_XDECREF(sdm_error);
  sdm_error = type;
  Py_RETURN_NONE;
}

template <PyObject* (*F)(PyObject* const*), int N>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<F, N>)), METH_FASTCALL, nullptr};
}
PyMethodDef methods[] = {method<conv, 11>("conv"),
                         method<scan, 17>("scan"),
                         method<gated, 5>("gated"),
                         method<gated_grad, 8>("gated_grad"),
                         {"set_error", set_error, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_layers", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__layers() { return PyModule_Create(&module); }
