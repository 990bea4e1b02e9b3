// CPython module over liblinear_norm.so for torch tensors: argument checks, result and workspace
// allocation and the library call of the operators in linear_norm.py, which documents them.
//
// A decode step calls these operators with a few microseconds of GPU work each; written in
// Python, the checks and allocations of one call took 12-14 us, several times the kernel.
// Positional arguments only (the Python functions give them in order); None stands for absent.
#include <Python.h>
#include <c10/core/AutogradState.h>
#include <c10/core/DeviceGuard.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <ATen/ATen.h>
#include <ATen/hip/EmptyTensor.h>
#include <ATen/hip/HIPContext.h>

#include "linear_norm.h"

namespace {

using at::Tensor;

const char* const kActivations[] = {"none", "relu", "gelu", "gelu_tanh", "silu"};

// The results carry no history, so an operand whose gradient (or tangent) would be lost is refused.
void untracked(const Tensor& t, const char* what) {
  const c10::AutogradState& mode = c10::AutogradState::get_tls_state();
  TORCH_CHECK_VALUE(!(mode.get_grad_mode() && t.requires_grad()) &&
                        !(mode.get_fw_grad_mode() && t._fw_grad(0).defined()),
                    what, " requires grad, and this function takes no part in autograd: call it "
                    "under torch.no_grad(), or in a torch.autograd.Function with its backward");
}

struct Args {
  PyObject* const* v;
  // a tensor, or an undefined one for None
  Tensor tensor(int i, const char* what) const {
    if (v[i] == Py_None) return Tensor();
    TORCH_CHECK_TYPE(THPVariable_Check(v[i]), what, " must be a tensor");
    const Tensor& t = THPVariable_Unpack(v[i]);
    untracked(t, what);
    return t;
  }
  Tensor needed(int i, const char* what) const {
    TORCH_CHECK_TYPE(v[i] != Py_None, what, " must be a tensor");
    return tensor(i, what);
  }
  bool flag(int i) const {
    const int f = PyObject_IsTrue(v[i]);
    if (f < 0) throw python_error();
    return f > 0;
  }
  bool has_dtype(int i) const {
    if (v[i] == Py_None) return false;
    TORCH_CHECK_TYPE(THPDtype_Check(v[i]), "out_dtype must be a torch.dtype");
    return true;
  }
  at::ScalarType dtype(int i) const { return ((THPDtype*)v[i])->scalar_type; }
  int activation(int i) const {
    const char* s = PyUnicode_Check(v[i]) ? PyUnicode_AsUTF8(v[i]) : nullptr;
    if (s == nullptr) PyErr_Clear();
    for (int a = 0; s != nullptr && a < 5; ++a)
      if (strcmp(s, kActivations[a]) == 0) return a;
    TORCH_CHECK_VALUE(false, "activation must be one of none, relu, gelu, gelu_tanh, silu; got ",
                      s ? s : "another object");
  }
};

// LINEAR_NORM_* code of a type, or -1
int code_of(at::ScalarType t) {
  switch (t) {
    case at::kHalf: return LINEAR_NORM_F16;
    case at::kBFloat16: return LINEAR_NORM_BF16;
    case at::kFloat8_e4m3fn: return LINEAR_NORM_E4M3;
    default: return -1;
  }
}
int code16(const Tensor& t, const char* what) {
  const int c = code_of(t.scalar_type());
  TORCH_CHECK_VALUE(c == LINEAR_NORM_F16 || c == LINEAR_NORM_BF16, what, " has dtype ",
                    t.scalar_type(), "; it must be float16 or bfloat16");
  return c;
}
void on_gpu(const Tensor& t, const char* what) {
  TORCH_CHECK_VALUE(t.is_cuda(), what, " must be a CUDA tensor");
}
void two_dim(const Tensor& t, const char* what) {
  TORCH_CHECK_VALUE(t.dim() == 2, "expected a 2-D ", what);
}
// Shape, type and device of an argument (undefined: absent, allowed).
void same(const Tensor& t, const char* what, at::IntArrayRef shape, at::ScalarType type,
          const at::Device& device) {
  if (!t.defined()) return;
  TORCH_CHECK_VALUE(t.sizes() == shape, what, " is ", t.sizes(), "; the call needs ", shape);
  TORCH_CHECK_VALUE(t.scalar_type() == type, what, " has dtype ", t.scalar_type(),
                    "; the call needs ", type);
  TORCH_CHECK_VALUE(t.device() == device, what, " is on ", t.device(), "; the call is on ",
                    device);
}
// ... with a unit stride along the last dimension.
void rows(const Tensor& t, const char* what, at::IntArrayRef shape, at::ScalarType type,
          const at::Device& device) {
  same(t, what, shape, type, device);
  if (!t.defined()) return;
  TORCH_CHECK_VALUE(t.stride(-1) == 1 || t.size(-1) <= 1, what,
                    " must be contiguous along its last dimension");
}

void* ptr(const Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
float* fptr(const Tensor& t) { return (float*)ptr(t); }
int64_t row(const Tensor& t) { return t.defined() ? t.stride(0) : 0; }

Tensor empty(at::IntArrayRef shape, at::ScalarType type, const at::Device& device) {
  return Tensor(at::detail::empty_cuda(shape, type, device, std::nullopt));
}

// Raises GemmError(code, name).
void check(int64_t code, const char* name) {
  if (code >= 0) return;
  PyObject* m = PyImport_ImportModule("dense_gemm_f16f32_amd");
  PyObject* cls = m ? PyObject_GetAttrString(m, "GemmError") : nullptr;
  PyObject* e = cls ? PyObject_CallFunction(cls, "is", (int)code, name) : nullptr;
  if (e) PyErr_SetObject(cls, e);
  Py_XDECREF(e);
  Py_XDECREF(cls);
  Py_XDECREF(m);
  throw python_error();
}

// Memory is allocated and kernels are launched on the device's current stream, so that memory
// freed on return is handed out again only to work behind them.
void* current_stream(const at::Device& d) {
  return (void*)at::hip::getCurrentHIPStreamMasqueradingAsCUDA(d.index()).stream();
}
template <class A>
void run(A& a, int64_t (*need)(const A*), int (*call)(const A*), const char* name,
         const at::Device& device) {
  const int64_t bytes = need(&a);
  check(bytes, name);
  Tensor ws;
  if (bytes > 0) {
    ws = empty({bytes}, at::kByte, device);
    a.workspace = ws.data_ptr();
    a.workspace_bytes = bytes;
  }
  check(call(&a), name);
}

PyObject* wrap(const Tensor& t) {
  if (t.defined()) return THPVariable_Wrap(t);
  Py_RETURN_NONE;
}
template <class... T>
PyObject* tuple_of(PyTypeObject* type, const T&... t) {   // a tuple type without other fields
  PyObject* r = type->tp_alloc(type, sizeof...(T));
  if (r == nullptr) throw python_error();
  Py_ssize_t i = 0;
  (PyTuple_SET_ITEM(r, i++, wrap(t)), ...);
  return r;
}

template <class... T>
PyObject* tuple(const T&... t) {
  return tuple_of(&PyTuple_Type, t...);
}

bool arity(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
  return false;
}

// linear(a, b, bias, residual, activation, scale_a, scale_b, out_dtype, with_pre, out)
PyObject* linear(PyObject*, PyObject* const* v, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  if (!arity(count, 10)) return nullptr;
  const Args x{v};
  const Tensor a = x.needed(0, "a"), b = x.needed(1, "b");
  const Tensor bias = x.tensor(2, "bias"), res = x.tensor(3, "residual");
  const Tensor sa = x.tensor(5, "scale_a"), sb = x.tensor(6, "scale_b");
  Tensor out = x.tensor(9, "out"), pre;
  on_gpu(a, "a");
  two_dim(a, "a");
  two_dim(b, "b");
  const at::Device device = a.device();
  const int64_t m = a.size(0), k = a.size(1), n = b.size(1);
  const int type = code_of(a.scalar_type());
  TORCH_CHECK_VALUE(type >= 0, "a has dtype ", a.scalar_type(),
                    "; it must be float16, bfloat16 or float8_e4m3fn");
  same(b, "b", {k, n}, a.scalar_type(), device);
  at::ScalarType ot = type == LINEAR_NORM_E4M3 ? at::kBFloat16 : a.scalar_type();
  if (x.has_dtype(7)) {
    const int oc = code_of(x.dtype(7));
    TORCH_CHECK_VALUE(type == LINEAR_NORM_E4M3 ? oc == LINEAR_NORM_F16 || oc == LINEAR_NORM_BF16
                                               : x.dtype(7) == ot,
                      "out_dtype ", x.dtype(7), " does not go with operands of ",
                      a.scalar_type());
    ot = x.dtype(7);
  }
  rows(bias, "bias", {n}, ot, device);
  rows(res, "residual", {m, n}, ot, device);
  rows(sa, "scale_a", {m}, at::kFloat, device);
  rows(sb, "scale_b", {n}, at::kFloat, device);
  rows(out, "out", {m, n}, ot, device);
  const int activation = x.activation(4);
  const c10::DeviceGuard guard(device);
  if (!out.defined()) out = empty({m, n}, ot, device);
  const bool with_pre = x.flag(8);
  if (with_pre) pre = empty({m, n}, ot, device);
  linear_forward_args p = {};
  p.m = m;
  p.n = n;
  p.k = k;
  p.type = type;
  p.out_type = code_of(ot);
  p.activation = activation;
  p.a = ptr(a);
  p.a_row = a.stride(0);
  p.a_col = a.stride(1);
  p.b = ptr(b);
  p.b_row = b.stride(0);
  p.b_col = b.stride(1);
  p.scale_a = fptr(sa);
  p.scale_b = fptr(sb);
  p.bias = ptr(bias);
  p.residual = ptr(res);
  p.residual_row = row(res);
  p.out = ptr(out);
  p.out_row = row(out);
  p.pre = ptr(pre);
  p.pre_row = row(pre);
  p.stream = current_stream(device);
  run(p, linear_forward_workspace, linear_forward, "linear_forward", device);
  if (with_pre) return tuple(out, pre);
  return wrap(out);
  END_HANDLE_TH_ERRORS
}

// linear_backward(dc, a, b, pre, activation, bias_grad, a_grad, b_grad)
PyObject* linear_bwd(PyObject*, PyObject* const* v, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  if (!arity(count, 8)) return nullptr;
  const Args x{v};
  const Tensor dc = x.needed(0, "dc"), a = x.needed(1, "a"), b = x.needed(2, "b");
  Tensor pre = x.tensor(3, "pre"), da, db, dbias;
  on_gpu(dc, "dc");
  two_dim(dc, "dc");
  two_dim(a, "a");
  two_dim(b, "b");
  const int type = code16(dc, "dc");
  const at::Device device = dc.device();
  const at::ScalarType t = dc.scalar_type();
  const int64_t m = dc.size(0), n = dc.size(1), k = a.size(1);
  rows(dc, "dc", {m, n}, t, device);
  same(a, "a", {m, k}, t, device);
  same(b, "b", {k, n}, t, device);
  const int activation = x.activation(4);
  if (activation == LINEAR_ACT_NONE) pre = Tensor();
  TORCH_CHECK_VALUE(activation == LINEAR_ACT_NONE || pre.defined(), "the gradient of ",
                    kActivations[activation], " needs pre");
  rows(pre, "pre", {m, n}, t, device);
  const c10::DeviceGuard guard(device);
  if (x.flag(6)) da = empty({m, k}, t, device);
  if (x.flag(7))
    db = b.stride(0) == 1 && b.stride(1) != 1 ? empty({n, k}, t, device).t()
                                              : empty({k, n}, t, device);
  if (x.flag(5)) dbias = empty({n}, t, device);
  linear_backward_args p = {};
  p.m = m;
  p.n = n;
  p.k = k;
  p.type = type;
  p.activation = activation;
  p.dc = ptr(dc);
  p.dc_row = dc.stride(0);
  p.a = ptr(a);
  p.a_row = a.stride(0);
  p.a_col = a.stride(1);
  p.b = ptr(b);
  p.b_row = b.stride(0);
  p.b_col = b.stride(1);
  p.pre = ptr(pre);
  p.pre_row = row(pre);
  p.da = ptr(da);
  p.da_row = row(da);
  p.db = ptr(db);
  p.db_row = row(db);
  p.db_col = db.defined() ? db.stride(1) : 0;
  p.dbias = ptr(dbias);
  p.stream = current_stream(device);
  run(p, linear_backward_workspace, linear_backward, "linear_backward", device);
  return tuple(da, db, dbias);
  END_HANDLE_TH_ERRORS
}

// rms_norm(x, weight, residual, eps, out_dtype, with_rstd, type of the result)
PyObject* norm(PyObject*, PyObject* const* v, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  if (!arity(count, 7)) return nullptr;
  const Args a{v};
  const Tensor x = a.needed(0, "x"), w = a.needed(1, "weight"), res = a.tensor(2, "residual");
  on_gpu(x, "x");
  two_dim(x, "x");
  const int type = code16(x, "x");
  const at::Device device = x.device();
  const at::ScalarType t = x.scalar_type();
  const int64_t n = x.size(0), dim = x.size(1);
  rows(x, "x", {n, dim}, t, device);
  rows(w, "weight", {dim}, t, device);
  rows(res, "residual", {n, dim}, t, device);
  const at::ScalarType ot = a.has_dtype(4) ? a.dtype(4) : t;
  const bool q8 = ot == at::kFloat8_e4m3fn;
  TORCH_CHECK_VALUE(q8 || ot == t, "out_dtype must be ", t, " or float8_e4m3fn, got ", ot);
  const double eps = PyFloat_AsDouble(v[3]);
  if (eps == -1.0 && PyErr_Occurred()) return nullptr;
  const c10::DeviceGuard guard(device);
  Tensor y, h, scale, rstd;
  if (q8) {   // rows on 16-byte boundaries, as linear's 8-bit operands have them
    const int64_t pad = (dim + 15) / 16 * 16;
    y = empty({n, pad}, ot, device);
    if (pad != dim) y = y.narrow(1, 0, dim);
    scale = empty({n}, at::kFloat, device);
  } else {
    y = empty({n, dim}, ot, device);
  }
  if (res.defined()) h = empty({n, dim}, t, device);
  if (a.flag(5)) rstd = empty({n}, at::kFloat, device);
  rms_norm_forward_args p = {};
  p.rows = n;
  p.dim = dim;
  p.type = type;
  p.out_type = code_of(ot);
  p.x = ptr(x);
  p.x_row = row(x);
  p.residual = ptr(res);
  p.residual_row = row(res);
  p.weight = ptr(w);
  p.y = ptr(y);
  p.y_row = row(y);
  p.scale = fptr(scale);
  p.h = ptr(h);
  p.h_row = row(h);
  p.rstd = fptr(rstd);
  p.eps = eps;
  p.stream = current_stream(device);
  check(rms_norm_forward(&p), "rms_norm_forward");
  TORCH_CHECK_TYPE(PyType_Check(v[6]) && PyType_IsSubtype((PyTypeObject*)v[6], &PyTuple_Type),
                   "the result's type must be a tuple");
  return tuple_of((PyTypeObject*)v[6], y, h.defined() ? h : x, rstd, scale);
  END_HANDLE_TH_ERRORS
}

// rms_norm_backward(dy, h, weight, rstd, dh, weight_grad)
PyObject* norm_bwd(PyObject*, PyObject* const* v, Py_ssize_t count) {
  HANDLE_TH_ERRORS
  if (!arity(count, 6)) return nullptr;
  const Args a{v};
  const Tensor dy = a.needed(0, "dy"), h = a.needed(1, "h"), w = a.needed(2, "weight");
  const Tensor rstd = a.needed(3, "rstd"), dh = a.tensor(4, "dh");
  on_gpu(dy, "dy");
  two_dim(dy, "dy");
  const int type = code16(dy, "dy");
  const at::Device device = dy.device();
  const at::ScalarType t = dy.scalar_type();
  const int64_t n = dy.size(0), dim = dy.size(1);
  rows(dy, "dy", {n, dim}, t, device);
  rows(h, "h", {n, dim}, t, device);
  rows(w, "weight", {dim}, t, device);
  rows(rstd, "rstd", {n}, at::kFloat, device);
  rows(dh, "dh", {n, dim}, t, device);
  const c10::DeviceGuard guard(device);
  Tensor dx = empty({n, dim}, t, device), dweight;
  if (a.flag(5)) dweight = empty({dim}, t, device);
  rms_norm_backward_args p = {};
  p.rows = n;
  p.dim = dim;
  p.type = type;
  p.dy = ptr(dy);
  p.dy_row = row(dy);
  p.h = ptr(h);
  p.h_row = row(h);
  p.weight = ptr(w);
  p.rstd = fptr(rstd);
  p.dh = ptr(dh);
  p.dh_row = row(dh);
  p.dx = ptr(dx);
  p.dx_row = row(dx);
  p.dweight = ptr(dweight);
  p.stream = current_stream(device);
  run(p, rms_norm_backward_workspace, rms_norm_backward, "rms_norm_backward", device);
  return tuple(dx, dweight);
  END_HANDLE_TH_ERRORS
}

PyMethodDef kMethods[] = {
    {"linear", (PyCFunction)(void*)linear, METH_FASTCALL, nullptr},
    {"linear_backward", (PyCFunction)(void*)linear_bwd, METH_FASTCALL, nullptr},
    {"rms_norm", (PyCFunction)(void*)norm, METH_FASTCALL, nullptr},
    {"rms_norm_backward", (PyCFunction)(void*)norm_bwd, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_linear_norm", nullptr, -1, kMethods};

}  // namespace

PyMODINIT_FUNC PyInit__linear_norm() { return PyModule_Create(&kModule); }
