// ops_binding.cpp -- Python entry of the operators of include/lowm_ops.h and
// include/lowm_cache.h: checks
// a call's tensors, fills the argument struct and calls the C ABI.  Built as a
// Python extension because these calls are short: the same checks in Python take
// longer than the smallest kernels (5 us against 1).
//
// Every function takes its arguments by position (split_bf16_gemm_amd/ops.py and cache.py have
// the signatures) and returns the C ABI's code; a tensor that does not fit raises
// ValueError or TypeError.  No C++ exception leaves a function.
#include <c10/core/DeviceGuard.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <string>

#include "lowm_cache.h"

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

// [T, H, D] of `type` (or any of bf16 and fp32: at::ScalarType::Undefined) with contiguous
// rows of D; its strides.
struct HeadsOf {
  void* p;
  int64_t T, H, D, row, head;
  at::ScalarType type;
};
HeadsOf heads_of(PyObject* o, const char* name, at::ScalarType type) {
  const at::Tensor& t = tensor(o, name);
  if (type == at::ScalarType::Undefined)
    real_type_of(t, name);
  else if (t.scalar_type() != type)
    refuse(PyExc_TypeError, std::string(name) + " must be " + c10::toString(type));
  if (t.dim() != 3) refuse(PyExc_ValueError, std::string(name) + " must have three dimensions");
  if (t.size(2) > 1 && t.stride(2) != 1)
    refuse(PyExc_ValueError, std::string(name) + " must have contiguous rows");
  HeadsOf h{t.data_ptr(), t.size(0), t.size(1), t.size(2), t.stride(0), t.stride(1),
            t.scalar_type()};
  // a stride of a dimension of one element steps nowhere
  if (h.H == 1) h.head = h.D;
  if (h.T <= 1) h.row = h.H * (h.head > h.D ? h.head : h.D);
  return h;
}
void same_heads(const HeadsOf& x, const char* name, int64_t T, int64_t H, int64_t D) {
  if (x.T != T || x.H != H || x.D != D) {
    const int64_t got[] = {x.T, x.H, x.D}, want[] = {T, H, D};
    refuse(PyExc_ValueError, std::string(name) + " has shape " + shape_text(got, 3) + ", not " +
                                 shape_text(want, 3));
  }
}

// The cache's four tensors a[0..3]: one layer [P, H, ...] or, where `layers`, also
// several [L, P, H, ...].
lowm_kv_cache cache_of(PyObject* const* a, bool layers) {
  const at::Tensor& k = tensor(a[0], "cache.k");
  lowm_kv_cache c{};
  const bool many = k.dim() == 6;
  if (!(k.dim() == 5 || (many && layers)))
    refuse(PyExc_ValueError, layers ? "cache.k must have five dimensions, or six with layers"
                                    : "cache.k must have five dimensions (one layer)");
  const int64_t L = many ? k.size(0) : 1, P = k.size(many), H = k.size(many + 1),
                D = k.size(many + 2) * 16;
  if (k.scalar_type() == at::kChar)
    c.type = LOWM_I8;
  else if (k.scalar_type() == at::kFloat8_e4m3fn)
    c.type = LOWM_E4M3;
  else
    refuse(PyExc_TypeError, "cache.k must be int8 or float8_e4m3fn");
  const at::ScalarType type = k.scalar_type();
  if (many) {
    c.k = dense(a[0], "cache.k", type, {L, P, H, D / 16, 64, 16});
    c.v = dense(a[1], "cache.v", type, {L, P, H, 4, D, 16});
    c.k_scale = static_cast<float*>(dense(a[2], "cache.k_scale", at::kFloat, {L, P, H}));
    c.v_scale = static_cast<float*>(dense(a[3], "cache.v_scale", at::kFloat, {L, P, H}));
  } else {
    c.k = dense(a[0], "cache.k", type, {P, H, D / 16, 64, 16});
    c.v = dense(a[1], "cache.v", type, {P, H, 4, D, 16});
    c.k_scale = static_cast<float*>(dense(a[2], "cache.k_scale", at::kFloat, {P, H}));
    c.v_scale = static_cast<float*>(dense(a[3], "cache.v_scale", at::kFloat, {P, H}));
  }
  c.P = to_int(P, "pages");
  c.H = to_int(H, "heads");
  c.D = to_int(D, "head_dim");
  c.layers = to_int(L, "layers");
  return c;
}

// table a[0] [B, W], lens a[1] [B], row_starts a[2] [B + 1] or None, for T rows.
lowm_sequences sequences_of(PyObject* const* a, int64_t T) {
  lowm_sequences s{};
  const at::Tensor& t = tensor(a[0], "table");
  if (t.scalar_type() != at::kInt) refuse(PyExc_TypeError, "table must be int32");
  if (t.dim() != 2) refuse(PyExc_ValueError, "table must have two dimensions");
  const int64_t B = t.size(0), W = t.size(1);
  s.table_ld = pitch(t, "table");
  s.table = static_cast<const int32_t*>(t.data_ptr());
  s.lens = static_cast<const int32_t*>(dense(a[1], "lens", at::kInt, {B}));
  if (a[2] != Py_None)
    s.row_starts = static_cast<const int32_t*>(dense(a[2], "row_starts", at::kInt, {B + 1}));
  else if (B > 0 && T % B)
    refuse(PyExc_ValueError, std::to_string(T) + " rows are no multiple of " + std::to_string(B) +
                                 " sequences: row_starts is needed");
  s.B = to_int(B, "B");
  s.W = to_int(W, "W");
  s.T = to_int(T, "T");
  return s;
}

int rotary(PyObject* const* a) {
  lowm_rotary_args u{};
  const HeadsOf q = heads_of(a[0], "q", at::ScalarType::Undefined);
  const HeadsOf qo = heads_of(a[1], "q_out", q.type);
  same_heads(qo, "q_out", q.T, q.H, q.D);
  u.q = q.p;
  u.q_out = qo.p;
  u.q_row = q.row, u.q_head = q.head, u.q_out_row = qo.row, u.q_out_head = qo.head;
  if (a[2] != Py_None) {
    const HeadsOf k = heads_of(a[2], "k", q.type);
    const HeadsOf ko = heads_of(a[3], "k_out", q.type);
    same_heads(k, "k", q.T, k.H, q.D);
    same_heads(ko, "k_out", q.T, k.H, q.D);
    u.k = k.p;
    u.k_out = ko.p;
    u.k_row = k.row, u.k_head = k.head, u.k_out_row = ko.row, u.k_out_head = ko.head;
    u.Hk = to_int(k.H, "heads");
  }
  const at::Tensor& pos = tensor(a[4], "positions");
  if (pos.scalar_type() != at::kLong && pos.scalar_type() != at::kInt)
    refuse(PyExc_TypeError, "positions must be int64 or int32");
  u.positions = dense(a[4], "positions", pos.scalar_type(), {q.T});
  u.positions_bytes = (int)pos.element_size();
  const at::Tensor& f = tensor(a[5], "freqs");
  if (f.dim() != 1) refuse(PyExc_ValueError, "freqs must have one dimension");
  u.freqs = static_cast<const double*>(dense(a[5], "freqs", at::kDouble, {f.size(0)}));
  u.R = to_int(2 * f.size(0), "freqs");
  u.T = to_int(q.T, "T");
  u.Hq = to_int(q.H, "heads");
  u.D = to_int(q.D, "head_dim");
  u.type = q.type == at::kFloat ? LOWM_F32 : LOWM_BF16;
  u.first = to_int(integer(a[6]), "first");
  u.flags = (int)integer(a[7]);
  u.scale = real(a[8]);
  const c10::DeviceGuard guard = on_call_device();
  return lowm_rotary(&u, stream_of(a[9]));
}

int cache_append(PyObject* const* a) {
  lowm_cache_append_args u{};
  const HeadsOf k = heads_of(a[0], "k", at::ScalarType::Undefined);
  const HeadsOf v = heads_of(a[1], "v", k.type);
  u.cache = cache_of(a + 2, false);
  same_heads(k, "k", k.T, u.cache.H, u.cache.D);
  same_heads(v, "v", k.T, u.cache.H, u.cache.D);
  u.seq = sequences_of(a + 6, k.T);
  u.k = k.p;
  u.v = v.p;
  u.k_row = k.row, u.k_head = k.head, u.v_row = v.row, u.v_head = v.head;
  u.type = k.type == at::kFloat ? LOWM_F32 : LOWM_BF16;
  const c10::DeviceGuard guard = on_call_device();
  return lowm_cache_append(&u, stream_of(a[9]));
}

int cache_read(PyObject* const* a) {
  lowm_cache_read_args u{};
  u.cache = cache_of(a + 2, false);
  const at::Tensor& k = tensor(a[0], "k_out");
  const int64_t T = k.dim() == 3 ? k.size(0) : 0;
  u.k_out = dense(a[0], "k_out", at::kBFloat16, {T, u.cache.H, u.cache.D});
  u.v_out = dense(a[1], "v_out", at::kBFloat16, {T, u.cache.H, u.cache.D});
  u.seq = sequences_of(a + 6, T);
  const c10::DeviceGuard guard = on_call_device();
  return lowm_cache_read(&u, stream_of(a[9]));
}

int cache_attention(PyObject* const* a) {
  lowm_cache_attention_args u{};
  const HeadsOf q = heads_of(a[0], "q", at::kBFloat16);
  u.cache = cache_of(a + 1, false);
  same_heads(q, "q", q.T, q.H, u.cache.D);
  u.seq = sequences_of(a + 5, q.T);
  u.q = q.p;
  u.q_row = q.row, u.q_head = q.head;
  u.Hq = to_int(q.H, "heads");
  u.out = dense(a[8], "out", at::kBFloat16, {q.T, q.H, q.D});
  if (a[9] != Py_None) u.lse = static_cast<float*>(dense(a[9], "lse_out", at::kFloat, {q.T, q.H}));
  workspace(a[10], &u.workspace, &u.workspace_bytes);
  if (!u.workspace && q.T > 0)
    refuse(PyExc_ValueError,
           "cache_attention needs a workspace (make_cache_attention_workspace)");
  u.window = to_int(integer(a[11]), "window");
  u.scale = real(a[12]);
  const c10::DeviceGuard guard = on_call_device();
  return lowm_cache_attention(&u, stream_of(a[13]));
}

// A page table and what goes with it, for the calls on pages.
const int32_t* page_table(PyObject* o, const char* name, int64_t R, int64_t W) {
  return static_cast<const int32_t*>(dense(o, name, at::kInt, {R, W}));
}

int fork_pages(PyObject* const* a) {
  lowm_fork_pages_args u{};
  u.cache = cache_of(a, true);
  const at::Tensor& t = tensor(a[4], "table");
  if (t.dim() != 2) refuse(PyExc_ValueError, "table must have two dimensions");
  const int64_t R = t.size(0), W = t.size(1), P = u.cache.P;
  u.table = page_table(a[4], "table", R, W);
  u.lens = static_cast<const int32_t*>(dense(a[5], "lens", at::kInt, {R}));
  if (a[6] != Py_None)
    u.parents = static_cast<const int32_t*>(dense(a[6], "parents", at::kInt, {R}));
  if (a[7] != Py_None) u.held = static_cast<const int32_t*>(dense(a[7], "held", at::kInt, {P}));
  u.table_out = const_cast<int32_t*>(page_table(a[8], "table_out", R, W));
  u.lens_out = static_cast<int32_t*>(dense(a[9], "lens_out", at::kInt, {R}));
  u.refs_out = static_cast<int32_t*>(dense(a[10], "refs_out", at::kInt, {P}));
  u.missing_out = static_cast<int32_t*>(dense(a[11], "missing_out", at::kInt, {1}));
  workspace(a[12], &u.workspace, &u.workspace_bytes);
  if (!u.workspace)
    refuse(PyExc_ValueError, "fork_pages needs a workspace (make_pages_workspace)");
  u.R = to_int(R, "rows");
  u.W = to_int(W, "W");
  u.reserve = to_int(integer(a[13]), "reserve");
  const c10::DeviceGuard guard = on_call_device();
  return lowm_fork_pages(&u, stream_of(a[14]));
}

int compact_pages(PyObject* const* a) {
  lowm_compact_pages_args u{};
  u.cache = cache_of(a, true);
  const at::Tensor& t = tensor(a[4], "table");
  if (t.dim() != 2) refuse(PyExc_ValueError, "table must have two dimensions");
  const int64_t R = t.size(0), W = t.size(1), P = u.cache.P;
  u.table = page_table(a[4], "table", R, W);
  if (a[5] != Py_None) u.held = static_cast<const int32_t*>(dense(a[5], "held", at::kInt, {P}));
  u.table_out = const_cast<int32_t*>(page_table(a[6], "table_out", R, W));
  u.refs_out = static_cast<int32_t*>(dense(a[7], "refs_out", at::kInt, {P}));
  u.counts_out = static_cast<int32_t*>(dense(a[8], "counts_out", at::kInt, {2}));
  workspace(a[9], &u.workspace, &u.workspace_bytes);
  if (!u.workspace)
    refuse(PyExc_ValueError, "compact_pages needs a workspace (make_pages_workspace)");
  u.R = to_int(R, "rows");
  u.W = to_int(W, "W");
  const c10::DeviceGuard guard = on_call_device();
  return lowm_compact_pages(&u, stream_of(a[10]));
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
    {"rotary", fast<rotary, 10>(), METH_FASTCALL, nullptr},
    {"cache_append", fast<cache_append, 10>(), METH_FASTCALL, nullptr},
    {"cache_read", fast<cache_read, 10>(), METH_FASTCALL, nullptr},
    {"cache_attention", fast<cache_attention, 14>(), METH_FASTCALL, nullptr},
    {"fork_pages", fast<fork_pages, 15>(), METH_FASTCALL, nullptr},
    {"compact_pages", fast<compact_pages, 11>(), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "ops_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_ops_binding() { return PyModule_Create(&module); }
