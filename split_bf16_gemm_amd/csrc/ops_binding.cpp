// ops_binding.cpp -- Python entry of the operators of include/lowm_ops.h: checks
// a call's tensors, fills the argument struct and calls the C ABI.  Built as a
// Python extension because these calls are short: the same checks in Python take
// longer than the smallest kernels (5 us against 1).
//
// Every function takes its arguments by position (split_bf16_gemm_amd/ops.py has
// the signatures) and returns the C ABI's code; a tensor that does not fit raises
// ValueError or TypeError.  No C++ exception leaves a function.
#include <c10/core/DeviceGuard.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <string>

#include "lowm_ops.h"

namespace {

struct Refusal {
  PyObject* kind;
  std::string what;
};
[[noreturn]] void refuse(PyObject* kind, const std::string& what) { throw Refusal{kind, what}; }

std::string shape_text(const int64_t* s, int n) {
  std::string t = "[";
  for (int i = 0; i < n; ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + "]";
}

// The device of the call's first tensor, which the others have to share.
thread_local int call_device = -1;

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, std::string(name) + " must be a tensor");
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda()) refuse(PyExc_ValueError, std::string(name) + " must be on the GPU");
  const int device = t.get_device();
  if (call_device < 0) call_device = device;
  if (device != call_device)
    refuse(PyExc_ValueError, std::string(name) + " is on GPU " + std::to_string(device) +
                                 ", not on GPU " + std::to_string(call_device));
  return t;
}

// LOWM_BF16, LOWM_F32 or LOWM_I8; -1 for any other type.
int type_of(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return LOWM_BF16;
    case at::kFloat: return LOWM_F32;
    case at::kChar: return LOWM_I8;
    default: return -1;
  }
}
int real_type_of(const at::Tensor& t, const char* name) {
  const int k = type_of(t);
  if (k != LOWM_BF16 && k != LOWM_F32)
    refuse(PyExc_TypeError, std::string(name) + " must be bf16 or fp32");
  return k;
}

void has_shape(const at::Tensor& t, const char* name, std::initializer_list<int64_t> shape) {
  bool same = t.dim() == (int64_t)shape.size();
  int i = 0;
  if (same)
    for (int64_t s : shape) same = same && t.size(i++) == s;
  if (!same)
    refuse(PyExc_ValueError, std::string(name) + " has shape " +
                                 shape_text(t.sizes().data(), (int)t.dim()) + ", not " +
                                 shape_text(shape.begin(), (int)shape.size()));
}

// The row pitch of a tensor [m, d] with contiguous rows that do not overlap.
int64_t pitch(const at::Tensor& t, const char* name) {
  const int64_t m = t.size(0), d = t.size(1);
  if (d > 1 && t.stride(1) != 1)
    refuse(PyExc_ValueError, std::string(name) + " must have contiguous rows");
  if (m <= 1) return d;
  if (t.stride(0) < d) refuse(PyExc_ValueError, std::string(name) + "'s rows overlap");
  return t.stride(0);
}

void* dense(PyObject* o, const char* name, at::ScalarType type,
            std::initializer_list<int64_t> shape) {
  const at::Tensor& t = tensor(o, name);
  if (t.scalar_type() != type)
    refuse(PyExc_TypeError, std::string(name) + " must be " + c10::toString(type));
  has_shape(t, name, shape);
  if (!t.is_contiguous()) refuse(PyExc_ValueError, std::string(name) + " must be contiguous");
  return t.data_ptr();
}

int to_int(int64_t v, const char* name) {
  if (v < INT32_MIN || v > INT32_MAX)
    refuse(PyExc_ValueError, std::string(name) + " does not fit 32 bits");
  return (int)v;
}
int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refusal{nullptr, ""};
  return v;
}
float real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refusal{nullptr, ""};
  return (float)v;
}
void* stream_of(PyObject* o) {
  void* s = PyLong_AsVoidPtr(o);
  if (!s && PyErr_Occurred()) throw Refusal{nullptr, ""};
  return s;
}

// A zeroed workspace, or nothing.
void workspace(PyObject* o, void** p, size_t* bytes) {
  *p = nullptr;
  *bytes = 0;
  if (o == Py_None) return;
  const at::Tensor& t = tensor(o, "workspace");
  if (!t.is_contiguous()) refuse(PyExc_ValueError, "workspace must be contiguous");
  *p = t.data_ptr();
  *bytes = t.nbytes();
}

// Makes the call's GPU the current one while it launches: a launch goes to the
// current device, whatever memory its pointers are in and whose stream it is given.
c10::DeviceGuard on_call_device() {
  return c10::DeviceGuard(c10::Device(c10::kCUDA, (c10::DeviceIndex)call_device));
}

int residual_norm(PyObject* const* a) {
  lowm_residual_norm_args u{};
  const at::Tensor& r = tensor(a[1], "residual");
  if (r.dim() != 2) refuse(PyExc_ValueError, "residual must have two dimensions");
  const int64_t M = r.size(0), D = r.size(1);
  const at::Tensor& y = tensor(a[0], "y");
  const at::Tensor& r_out = tensor(a[2], "residual_out");
  u.flags = (int)integer(a[8]);
  u.M = to_int(M, "M");
  u.D = to_int(D, "D");
  u.r_type = real_type_of(r, "residual");
  u.y_type = real_type_of(y, "y");
  has_shape(y, "y", {M, D});
  has_shape(r_out, "residual_out", {M, D});
  if (r_out.scalar_type() != r.scalar_type())
    refuse(PyExc_TypeError, "residual_out must have the residual's type");
  u.y = y.data_ptr();
  u.r = r.data_ptr();
  u.r_out = r_out.data_ptr();
  u.ld_y = pitch(y, "y");
  u.ld_r = pitch(r, "residual");
  u.ld_r_out = pitch(r_out, "residual_out");
  if (a[3] != Py_None) {
    const at::Tensor& x = tensor(a[3], "out");
    u.x_type = type_of(x);
    if (u.x_type != (a[4] == Py_None ? LOWM_BF16 : LOWM_I8))
      refuse(PyExc_TypeError, "out must be bf16, or int8 with quantize");
    has_shape(x, "out", {M, D});
    u.x = x.data_ptr();
    u.ld_x = pitch(x, "out");
    if (a[4] != Py_None)
      u.x_scale = static_cast<float*>(dense(a[4], "scale_out", at::kFloat, {M}));
  }
  int w_type = -1;
  for (int i = 5; i < 7; ++i) {
    if (a[i] == Py_None) continue;
    const char* name = i == 5 ? "post_weight" : "pre_weight";
    const int k = real_type_of(tensor(a[i], name), name);
    if (w_type >= 0 && k != w_type)
      refuse(PyExc_TypeError, "post_weight and pre_weight must have one type");
    w_type = k;
    (i == 5 ? u.w_post : u.w_pre) =
        dense(a[i], name, k == LOWM_F32 ? at::kFloat : at::kBFloat16, {D});
  }
  u.w_type = w_type < 0 ? LOWM_BF16 : w_type;
  if (a[7] != Py_None) {
    const at::Tensor& g = tensor(a[7], "gate");
    u.gate_type = real_type_of(g, "gate");
    u.gate = g.data_ptr();
    if (g.dim() == 1 && g.size(0) == D) {
      u.gate_col = g.stride(0);
    } else if (g.dim() == 2 && (g.size(0) == 1 || g.size(0) == M) &&
               (g.size(1) == 1 || g.size(1) == D)) {
      u.gate_row = g.size(0) == 1 ? 0 : g.stride(0);
      u.gate_col = g.size(1) == 1 ? 0 : g.stride(1);
    } else {
      refuse(PyExc_ValueError, "gate has shape " + shape_text(g.sizes().data(), (int)g.dim()) +
                                   ": not [D], [M, 1] or [M, D]");
    }
    if (D == 1) u.gate_col = 0;
    if (u.gate_col != 0 && u.gate_col != 1)
      refuse(PyExc_ValueError, "gate must have contiguous rows");
  }
  u.residual_scale = real(a[9]);
  u.branch_scale = real(a[10]);
  u.eps = real(a[11]);
  const c10::DeviceGuard guard = on_call_device();
  return lowm_residual_norm(&u, stream_of(a[12]));
}

int quantize_rows(PyObject* const* a) {
  const at::Tensor& x = tensor(a[0], "x");
  const int type = real_type_of(x, "x");
  if (x.dim() != 2) refuse(PyExc_ValueError, "x must have two dimensions");
  const int64_t M = x.size(0), K = x.size(1);
  void* q = dense(a[1], "out", at::kChar, {M, K});
  void* s = dense(a[2], "scale_out", at::kFloat, {M});
  const c10::DeviceGuard guard = on_call_device();
  return lowm_quantize_rows(x.data_ptr(), type, pitch(x, "x"), to_int(M, "M"), to_int(K, "K"), q,
                            static_cast<float*>(s), stream_of(a[3]));
}

int gemm_i8(PyObject* const* a) {
  lowm_gemm_i8_args u{};
  const at::Tensor& A = tensor(a[0], "A");
  const at::Tensor& W = tensor(a[1], "W");
  if (A.dim() != 2 || W.dim() != 2 || A.size(1) != W.size(1))
    refuse(PyExc_ValueError, "shapes " + shape_text(A.sizes().data(), (int)A.dim()) + " and " +
                                 shape_text(W.sizes().data(), (int)W.dim()) + " do not chain");
  const int64_t M = A.size(0), K = A.size(1), N = W.size(0);
  u.a_type = type_of(A);
  if (u.a_type != LOWM_I8 && u.a_type != LOWM_BF16)
    refuse(PyExc_TypeError, "A must be int8 or bf16");
  u.A = dense(a[0], "A", A.scalar_type(), {M, K});
  u.W = dense(a[1], "W", at::kChar, {N, K});
  u.w_scale = static_cast<float*>(dense(a[2], "w_scale", at::kFloat, {N}));
  const at::Tensor& C = tensor(a[4], "out");
  u.c_type = real_type_of(C, "out");
  u.C = dense(a[4], "out", C.scalar_type(), {M, N});
  workspace(a[5], &u.workspace, &u.workspace_bytes);
  if (u.a_type == LOWM_I8) {
    if (a[3] == Py_None) refuse(PyExc_ValueError, "an int8 A needs a_scale");
    u.a_scale = static_cast<float*>(dense(a[3], "a_scale", at::kFloat, {M}));
  } else {
    if (a[3] != Py_None) refuse(PyExc_ValueError, "a bf16 A takes no a_scale");
    if (!u.workspace)
      refuse(PyExc_ValueError, "a bf16 A needs a zeroed workspace (make_gemm_i8_workspace)");
  }
  u.M = to_int(M, "M");
  u.N = to_int(N, "N");
  u.K = to_int(K, "K");
  const c10::DeviceGuard guard = on_call_device();
  return lowm_gemm_i8(&u, stream_of(a[6]));
}

int moe(PyObject* const* a) {
  lowm_moe_args u{};
  const at::Tensor& x = tensor(a[0], "x");
  const at::Tensor& w2 = tensor(a[4], "w2");
  if (x.dim() != 2 || w2.dim() != 3)
    refuse(PyExc_ValueError, "x must have two dimensions, w2 three");
  const int64_t T = x.size(0), D = x.size(1), E = w2.size(0), I = w2.size(2);
  const int64_t K = integer(a[9]);
  u.x = dense(a[0], "x", at::kBFloat16, {T, D});
  u.router = dense(a[1], "router", at::kBFloat16, {E, D});
  if (a[2] != Py_None) u.bias = static_cast<float*>(dense(a[2], "bias", at::kFloat, {E}));
  u.w13 = dense(a[3], "w13", at::kBFloat16, {E, 2 * I, D});
  u.w2 = dense(a[4], "w2", at::kBFloat16, {E, D, I});
  u.out = dense(a[5], "out", at::kBFloat16, {T, D});
  u.ids = static_cast<int32_t*>(dense(a[6], "ids_out", at::kInt, {T, K}));
  u.gates = static_cast<float*>(dense(a[7], "gates_out", at::kFloat, {T, K}));
  workspace(a[8], &u.workspace, &u.workspace_bytes);
  if (!u.workspace && T > 0)
    refuse(PyExc_ValueError, "moe needs a zeroed workspace (make_moe_workspace)");
  u.T = to_int(T, "T");
  u.D = to_int(D, "D");
  u.I = to_int(I, "I");
  u.E = to_int(E, "E");
  u.top_k = to_int(K, "top_k");
  u.flags = (int)integer(a[10]);
  u.routed_scale = real(a[11]);
  const c10::DeviceGuard guard = on_call_device();
  return lowm_moe(&u, stream_of(a[12]));
}

int token_logprobs(PyObject* const* a) {
  lowm_token_logprobs_args u{};
  const at::Tensor& x = tensor(a[0], "logits");
  if (x.dim() != 2) refuse(PyExc_ValueError, "logits must have two dimensions");
  const int64_t M = x.size(0), V = x.size(1), n = integer(a[2]);
  u.logits_type = real_type_of(x, "logits");
  u.logits = x.data_ptr();
  u.ld = pitch(x, "logits");
  const at::Tensor& t = tensor(a[1], "tokens");
  if (t.scalar_type() != at::kLong && t.scalar_type() != at::kInt)
    refuse(PyExc_TypeError, "tokens must be int64 or int32");
  u.tokens_bytes = (int)t.element_size();
  u.tokens = dense(a[1], "tokens", t.scalar_type(), {M});
  u.logprob = static_cast<float*>(dense(a[3], "logprob", at::kFloat, {M}));
  u.entropy = static_cast<float*>(dense(a[4], "entropy", at::kFloat, {M}));
  u.rank = static_cast<int32_t*>(dense(a[5], "rank", at::kInt, {M}));
  u.top_logprob = static_cast<float*>(dense(a[6], "top_logprob", at::kFloat, {M, n}));
  u.top_id = static_cast<int32_t*>(dense(a[7], "top_id", at::kInt, {M, n}));
  u.M = to_int(M, "M");
  u.V = to_int(V, "V");
  u.top_n = to_int(n, "top_n");
  workspace(a[8], &u.workspace, &u.workspace_bytes);
  if (!u.workspace && lowm_token_logprobs_workspace_bytes(u.M, u.V, u.top_n) > 0)
    refuse(PyExc_ValueError, "these rows need a zeroed workspace (make_token_logprobs_workspace)");
  const c10::DeviceGuard guard = on_call_device();
  return lowm_token_logprobs(&u, stream_of(a[9]));
}

template <int (*F)(PyObject* const*), int N>
PyObject* call(PyObject*, PyObject* const* a, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "%d arguments needed, %zd given", N, n);
    return nullptr;
  }
  call_device = -1;
  try {
    return PyLong_FromLong(F(a));
  } catch (const Refusal& r) {
    if (r.kind) PyErr_SetString(r.kind, r.what.c_str());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

template <int (*F)(PyObject* const*), int N>
PyCFunction fast() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&call<F, N>));
}

PyMethodDef methods[] = {
    {"residual_norm", fast<residual_norm, 13>(), METH_FASTCALL, nullptr},
    {"quantize_rows", fast<quantize_rows, 4>(), METH_FASTCALL, nullptr},
    {"gemm_i8", fast<gemm_i8, 7>(), METH_FASTCALL, nullptr},
    {"moe", fast<moe, 13>(), METH_FASTCALL, nullptr},
    {"token_logprobs", fast<token_logprobs, 10>(), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "ops_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_ops_binding() { return PyModule_Create(&module); }
