// Tensor helpers of the mixture-of-experts operators: checks, output
// allocation and the call of the C interface, in one native call per
// operator (module _native).
//
// A call on few rows costs what the host spends on it: through ctypes and
// torch's Python allocation the norm of one token took 17 us of host time,
// its kernel 4 us.  No arithmetic happens here.  Errors leave as Python
// exceptions: ValueError for what the C interface cannot see (shapes, types,
// devices, row layouts), the binding's Fp8fgError for its status.
#include <ATen/core/Tensor.h>
#include <ATen/ops/empty_strided.h>
#include <c10/core/DeviceGuard.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include <initializer_list>
#include <string>

#include "fp8fg.h"

namespace {

using at::Tensor;

PyObject* g_error = nullptr;  // Fp8fgError

[[noreturn]] void refuse(const std::string& what) { TORCH_CHECK_VALUE(false, what); __builtin_unreachable(); }

void need(bool ok, const char* name, const char* what) {
  if (!ok) refuse(std::string(name) + " " + what);
}

// ---------------------------------------------------------------- arguments
const Tensor* tensor_or_none(PyObject* o, const char* name) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
  return &THPVariable_Unpack(o);
}

const Tensor& tensor(PyObject* o, const char* name) {
  const Tensor* t = tensor_or_none(o, name);
  if (!t) refuse(std::string(name) + " must be a tensor");
  return *t;
}

int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}

// An enumerator or another small number of the C interface, where -1 is refused:
// what no int holds is as well.
int small(PyObject* o) {
  const int64_t v = integer(o);
  return v == (int)v ? (int)v : -1;
}

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v != 0;
}

void* handle(PyObject* o) { return reinterpret_cast<void*>(integer(o)); }

// bf16 / f32, or -1
int xtype(const Tensor& t) {
  return t.scalar_type() == at::kBFloat16 ? FP8FG_BF16 : t.scalar_type() == at::kFloat ? FP8FG_F32 : -1;
}

// A 2-d GPU tensor with contiguous rows.
void rows2d(const Tensor& t, const char* name) {
  need(t.is_cuda(), name, "must be on the GPU");
  need(t.dim() == 2 && (t.size(1) <= 1 || t.stride(1) == 1), name, "must be 2-d with contiguous rows");
}

void like(const Tensor* t, const Tensor& x, const char* name) {
  if (!t) return;
  rows2d(*t, name);
  need(t->sizes() == x.sizes() && t->scalar_type() == x.scalar_type() && t->device() == x.device(), name,
       "does not match in shape, type or device");
}

void vec1(const Tensor* t, int64_t n, const Tensor& x, bool f32_only, const char* name) {
  if (!t) return;
  need(t->dim() == 1 && t->size(0) == n && t->is_contiguous() && t->device() == x.device() &&
           (f32_only ? t->scalar_type() == at::kFloat : xtype(*t) >= 0),
       name, f32_only ? "must be a contiguous f32 vector of its length on the same device"
                      : "must be a contiguous bf16 or f32 vector of the columns on the same device");
}

// Row pitch; a single row's stride carries no meaning.
int64_t pitch(const Tensor& t) { return t.size(0) > 1 ? t.stride(0) : t.size(1) > 1 ? t.size(1) : 1; }
int64_t pitch(const Tensor* t) { return t ? pitch(*t) : 0; }

template <typename T = void>
T* ptr(const Tensor* t) {
  return t ? reinterpret_cast<T*>(t->data_ptr()) : nullptr;
}
template <typename T = void>
T* ptr(const Tensor& t) {
  return reinterpret_cast<T*>(t.data_ptr());
}

// ------------------------------------------------------------------ outputs
Tensor make(int64_t rows, int64_t cols, at::ScalarType type, const Tensor& x) {
  return at::empty_strided({rows, cols}, {cols, 1}, x.options().dtype(type));
}
Tensor make1(int64_t n, at::ScalarType type, const Tensor& x) {
  return at::empty_strided({n}, {1}, x.options().dtype(type));
}
// Scales indexed [row][group], stored group-major or row-major.
Tensor make_scales(int64_t rows, int64_t groups, bool group_major, const Tensor& x) {
  return group_major ? at::empty_strided({rows, groups}, {1, rows}, x.options().dtype(at::kFloat))
                     : make(rows, groups, at::kFloat, x);
}

PyObject* give(std::initializer_list<const Tensor*> out) {
  THPObjectPtr tuple(PyTuple_New((Py_ssize_t)out.size()));
  if (!tuple) throw python_error();
  Py_ssize_t i = 0;
  for (const Tensor* t : out) {
    PyObject* o = t ? THPVariable_Wrap(*t) : Py_NewRef(Py_None);
    if (!o) throw python_error();
    PyTuple_SET_ITEM(tuple.get(), i++, o);
  }
  return tuple.release();
}

void check(int status, const char* func) {
  if (status == FP8FG_OK) return;
  THPObjectPtr e(g_error ? PyObject_CallFunction(g_error, "is", status, func) : nullptr);
  if (e)
    PyErr_SetObject(g_error, e.get());
  else if (!PyErr_Occurred())
    PyErr_SetString(PyExc_RuntimeError, fp8fg_status_string(status));
  throw python_error();
}

void arity(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    throw python_error();
  }
}

// ---------------------------------------------------------------- operators
// (x, gamma, residual, eps, rule, group_major, want_y, stream)
PyObject* rmsnorm_quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity(n, 8);
  const Tensor& x = tensor(a[0], "x");
  rows2d(x, "x");
  need(xtype(x) >= 0, "x", "must be bf16 or f32");
  const int64_t M = x.size(0), C = x.size(1);
  const Tensor& gamma = tensor(a[1], "gamma");
  vec1(&gamma, C, x, false, "gamma");
  const Tensor* r = tensor_or_none(a[2], "residual");
  like(r, x, "residual");
  const c10::DeviceGuard guard(x.device());
  const Tensor q = make(M, C, at::kByte, x), s = make_scales(M, C / 128, truth(a[5]), x);
  const Tensor h = r ? make(M, C, x.scalar_type(), x) : Tensor(), rstd = make1(M, at::kFloat, x);
  const bool want_y = truth(a[6]);
  const Tensor y = want_y ? make(M, C, x.scalar_type(), x) : Tensor();
  check(fp8_rmsnorm_quantize(ptr(x), xtype(x), M, C, pitch(x), ptr(r), pitch(r), ptr(gamma), xtype(gamma),
                             (float)number(a[3]), small(a[4]), r ? ptr(h) : nullptr, C,
                             want_y ? ptr(y) : nullptr, C, ptr<uint8_t>(q), C, ptr<float>(s), s.stride(0), s.stride(1),
                             ptr<float>(rstd), handle(a[7])),
        "fp8_rmsnorm_quantize");
  return give({&q, &s, r ? &h : &x, want_y ? &y : nullptr, &rstd});
  END_HANDLE_TH_ERRORS
}

// (dy, h, gamma, rstd, dh, stream)
PyObject* rmsnorm_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity(n, 6);
  const Tensor &dy = tensor(a[0], "dy"), &h = tensor(a[1], "h"), &gamma = tensor(a[2], "gamma"), &rstd = tensor(a[3], "rstd");
  const Tensor* dh = tensor_or_none(a[4], "dh");
  rows2d(h, "h");
  need(xtype(h) >= 0, "h", "must be bf16 or f32");
  like(&dy, h, "dy");
  like(dh, h, "dh");
  const int64_t M = h.size(0), C = h.size(1);
  vec1(&gamma, C, h, false, "gamma");
  vec1(&rstd, M, h, true, "rstd");
  const c10::DeviceGuard guard(h.device());
  const int64_t bytes = fp8_rmsnorm_backward_workspace(M, C);
  const Tensor dx = make(M, C, h.scalar_type(), h), dgamma = make1(C, at::kFloat, h), ws = make1(bytes + 16, at::kByte, h);
  check(fp8_rmsnorm_backward(ptr(dy), xtype(h), M, C, pitch(dy), ptr(dh), pitch(dh), ptr(h), pitch(h), ptr(gamma),
                             xtype(gamma), ptr<float>(rstd), ptr(dx), C, ptr<float>(dgamma), ptr(ws), bytes, handle(a[5])),
        "fp8_rmsnorm_backward");
  return give({&dx, &dgamma, &ws});
  END_HANDLE_TH_ERRORS
}

// (logits, k, bias, score, groups, top_groups, group_top, renorm, scale, stream)
PyObject* route(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity(n, 10);
  const Tensor& l = tensor(a[0], "logits");
  rows2d(l, "logits");
  need(xtype(l) >= 0, "logits", "must be bf16 or f32");
  const int64_t M = l.size(0), E = l.size(1), k = integer(a[1]);
  need(k >= 0, "k", "must not be negative");
  const Tensor* bias = tensor_or_none(a[2], "bias");
  vec1(bias, E, l, true, "bias");
  const c10::DeviceGuard guard(l.device());
  const int64_t slots = k <= E ? k : 0;  // (beyond: the call below refuses)
  const Tensor idx = make(M, slots, at::kInt, l), w = make(M, slots, at::kFloat, l);
  check(fp8_route(ptr(l), xtype(l), M, E, pitch(l), ptr<float>(bias), small(a[3]), integer(a[4]), integer(a[5]),
                  small(a[6]), k, truth(a[7]), (float)number(a[8]), ptr<int32_t>(idx), k, ptr<float>(w), k,
                  handle(a[9])),
        "fp8_route");
  return give({&idx, &w});
  END_HANDLE_TH_ERRORS
}

// (dw, logits, idx, score, renorm, scale, stream)
PyObject* route_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity(n, 7);
  const Tensor &dw = tensor(a[0], "dw"), &l = tensor(a[1], "logits"), &idx = tensor(a[2], "idx");
  rows2d(l, "logits");
  rows2d(idx, "idx");
  rows2d(dw, "dw");
  need(xtype(l) >= 0, "logits", "must be bf16 or f32");
  const int64_t M = l.size(0), E = l.size(1), k = idx.size(1);
  need(idx.scalar_type() == at::kInt && idx.size(0) == M && idx.device() == l.device(), "idx",
       "must be int32 [tokens][k] on the logits' device");
  need(dw.scalar_type() == at::kFloat && dw.sizes() == idx.sizes() && dw.device() == l.device(), "dw",
       "must be f32 [tokens][k] on the logits' device");
  const c10::DeviceGuard guard(l.device());
  const Tensor dl = make(M, E, l.scalar_type(), l);
  check(fp8_route_backward(ptr(l), xtype(l), M, E, pitch(l), small(a[3]), k, truth(a[4]), (float)number(a[5]),
                           ptr<int32_t>(idx), pitch(idx), ptr<float>(dw), pitch(dw), ptr(dl), E, handle(a[6])),
        "fp8_route_backward");
  return give({&dl});
  END_HANDLE_TH_ERRORS
}

// (idx, experts, x, s, group_major, stream)
PyObject* dispatch(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity(n, 6);
  const Tensor &idx = tensor(a[0], "idx"), &x = tensor(a[2], "x");
  const int64_t E = integer(a[1]);
  const Tensor* s = tensor_or_none(a[3], "s");
  rows2d(idx, "idx");
  rows2d(x, "x");
  const bool e4m3 = x.scalar_type() == at::kByte;
  const int type = e4m3 ? FP8FG_E4M3 : xtype(x);
  need(type >= 0, "x", "must be E4M3 bytes (uint8), bf16 or f32");
  const int64_t M = idx.size(0), k = idx.size(1), C = x.size(1);
  need(idx.scalar_type() == at::kInt && x.size(0) == M && idx.device() == x.device(), "idx",
       "must be int32 [tokens][k] on x's device");
  need(E >= 0, "experts", "must not be negative");
  need((s != nullptr) == e4m3, "s", "must be given for E4M3 rows and for no others");
  if (s)
    need(s->dim() == 2 && s->size(0) == M && s->size(1) == C / 128 && s->scalar_type() == at::kFloat &&
             s->device() == x.device(),
         "s", "must be the f32 [tokens][columns / 128] scales of x");
  const c10::DeviceGuard guard(x.device());
  // 0 bytes: sizes that the call below refuses, saying why; nothing of them is allocated
  const int64_t bytes = fp8_dispatch_workspace(M, k, E), rows = bytes ? M * k : 1;
  const Tensor out = make(rows, C, x.scalar_type(), x), offsets = make1(bytes ? E + 1 : 1, at::kInt, x);
  const Tensor pos = bytes ? make(M, k, at::kInt, x) : make1(1, at::kInt, x), token = make1(rows, at::kInt, x);
  const Tensor os = s ? make_scales(rows, C / 128, truth(a[4]), x) : Tensor();
  const Tensor ws = make1(bytes + 16, at::kByte, x);
  check(fp8_dispatch(ptr<int32_t>(idx), pitch(idx), M, k, E, ptr(x), type, C, pitch(x), ptr<float>(s), s ? s->stride(0) : 0,
                     s ? s->stride(1) : 0, ptr<int32_t>(offsets), ptr<int32_t>(pos), ptr<int32_t>(token), ptr(out), C,
                     s ? ptr<float>(os) : nullptr, s ? os.stride(0) : 0, s ? os.stride(1) : 0, ptr(ws), bytes, handle(a[5])),
        "fp8_dispatch");
  return give({&out, s ? &os : nullptr, &offsets, &pos, &token, &ws});
  END_HANDLE_TH_ERRORS
}

void places(const Tensor& pos, const Tensor* w, const Tensor& z) {
  need(pos.dim() == 2 && pos.scalar_type() == at::kInt && pos.is_contiguous() && pos.device() == z.device(), "pos",
       "must be contiguous int32 [tokens][k] on the rows' device");
  if (!w) return;
  rows2d(*w, "w");
  need(w->scalar_type() == at::kFloat && w->sizes() == pos.sizes() && w->device() == z.device(), "w",
       "must be f32 [tokens][k] on the rows' device");
}

// (z, pos, w, base, stream)
PyObject* combine(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity(n, 5);
  const Tensor &z = tensor(a[0], "z"), &pos = tensor(a[1], "pos");
  const Tensor *w = tensor_or_none(a[2], "w"), *base = tensor_or_none(a[3], "base");
  rows2d(z, "z");
  need(xtype(z) >= 0, "z", "must be bf16 or f32");
  places(pos, w, z);
  const int64_t M = pos.size(0), k = pos.size(1), R = z.size(0), C = z.size(1);
  const c10::DeviceGuard guard(z.device());
  const Tensor out = make(M, C, z.scalar_type(), z);
  like(base, out, "base");
  check(fp8_combine(ptr(z), xtype(z), R, M, k, C, pitch(z), ptr<int32_t>(pos), ptr<float>(w), pitch(w), ptr(base),
                    pitch(base), ptr(out), C, handle(a[4])),
        "fp8_combine");
  return give({&out});
  END_HANDLE_TH_ERRORS
}

// (dy, z, pos, w, stream)
PyObject* combine_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity(n, 5);
  const Tensor &dy = tensor(a[0], "dy"), &z = tensor(a[1], "z"), &pos = tensor(a[2], "pos");
  const Tensor* w = tensor_or_none(a[3], "w");
  rows2d(z, "z");
  rows2d(dy, "dy");
  need(xtype(z) >= 0, "z", "must be bf16 or f32");
  places(pos, w, z);
  const int64_t M = pos.size(0), k = pos.size(1), R = z.size(0), C = z.size(1);
  need(dy.size(0) == M && dy.size(1) == C && dy.scalar_type() == z.scalar_type() && dy.device() == z.device(), "dy",
       "must be [tokens][columns] of z's type and device");
  need(R == M * k, "z", "must have tokens * k rows");
  const c10::DeviceGuard guard(z.device());
  const Tensor dz = make(R, C, z.scalar_type(), z), dw = make(M, k, at::kFloat, z);
  check(fp8_combine_backward(ptr(dy), xtype(z), R, M, k, C, pitch(dy), ptr(z), pitch(z), ptr<int32_t>(pos), ptr<float>(w),
                             pitch(w), ptr(dz), C, ptr<float>(dw), k, handle(a[4])),
        "fp8_combine_backward");
  return give({&dz, &dw});
  END_HANDLE_TH_ERRORS
}

PyObject* set_error(PyObject*, PyObject* cls) {
  Py_XDECREF(g_error);
  g_error = Py_NewRef(cls);
  Py_RETURN_NONE;
}

#define FAST(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {FAST(rmsnorm_quantize),
                           FAST(rmsnorm_backward),
                           FAST(route),
                           FAST(route_backward),
                           FAST(dispatch),
                           FAST(combine),
                           FAST(combine_backward),
                           {"set_error", set_error, METH_O, nullptr},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&g_module); }
