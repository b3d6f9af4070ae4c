// The calls of binding.py whose kernels take a few microseconds: arguments
// checked, outputs allocated and the C entry points called from one place in
// C++. The same marshalling in Python took 9 to 12 us of host time a call
// (measured with 13.6 us for fp8_linear, of which 4 are the launch), more than
// many of the kernels. The arithmetic is all in the library; this module
// (nvfp4_block_scaled_05_gb300._tensor_calls) only passes pointers to it.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <string>

#include "nvfp4moe.h"

namespace {

PyObject* g_error = nullptr;   // binding.NVFP4Error

#define REFUSE(...)                                                     \
  do {                                                                  \
    PyErr_Format(g_error ? g_error : PyExc_RuntimeError, __VA_ARGS__);  \
    throw python_error();                                               \
  } while (0)

bool none(PyObject* o) { return o == nullptr || o == Py_None; }

int64_t integer(PyObject* o, const char* name) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    REFUSE("%s must be an integer", name);
  }
  return v;
}

const at::Tensor& on_gpu(PyObject* o, const char* name) {
  if (!THPVariable_Check(o) || !THPVariable_Unpack(o).is_cuda()) REFUSE("%s must be a CUDA tensor", name);
  const at::Tensor& t = THPVariable_Unpack(o);
  if (t.get_device() != c10::cuda::current_device()) REFUSE("%s must be on the current device", name);
  return t;
}

int float_type(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return NVFP4MOE_BF16;
    case at::kHalf: return NVFP4MOE_F16;
    case at::kFloat: return NVFP4MOE_F32;
    default: return -1;
  }
}

bool is_codes(at::ScalarType t) { return t == at::kByte || t == at::kFloat8_e4m3fn; }

// A 2-D tensor whose rows are contiguous and do not overlap.
struct Matrix {
  at::Tensor t;
  int64_t n, c, ld;
  void* p;
  int type;   // NVFP4MOE_BF16, ...; -1 for codes
};

Matrix matrix(PyObject* o, const char* name, bool codes = false) {
  const at::Tensor& t = on_gpu(o, name);
  const int type = float_type(t.scalar_type());
  if (t.dim() != 2 || (codes ? !is_codes(t.scalar_type()) : type < 0))
    REFUSE("%s must be a matrix of %s", name, codes ? "codes (uint8 or float8_e4m3fn)" : "BF16, F16 or F32");
  const int64_t n = t.size(0), c = t.size(1), ld = t.stride(0);
  if ((c > 1 && t.stride(1) != 1) || (n > 1 && ld < c))
    REFUSE("the rows of %s must be contiguous and must not overlap", name);
  // no second row keeps to a single one's stride, which any entry point then takes
  return Matrix{t, n, c, n > 1 ? ld : (c + 15) / 16 * 16, t.data_ptr(), codes ? -1 : type};
}

// Whether t, which is contiguous, is a tensor of these sizes, but for sizes of
// 1, or their elements in one dimension. (The number of elements alone would
// take a transposed one.)
bool has_sizes(const at::Tensor& t, std::initializer_list<int64_t> sizes) {
  int64_t numel = 1;
  for (const int64_t s : sizes) numel *= s;
  if (t.dim() == 1 || t.numel() != numel) return t.numel() == numel;
  int64_t d = 0;
  for (const int64_t s : sizes) {
    if (s == 1) continue;
    while (d < t.dim() && t.size(d) == 1) ++d;
    if (d == t.dim() || t.size(d++) != s) return false;
  }
  while (d < t.dim() && t.size(d) == 1) ++d;
  return d == t.dim();
}

void* flat(PyObject* o, const char* name, at::ScalarType type, std::initializer_list<int64_t> sizes) {
  const at::Tensor& t = on_gpu(o, name);
  if (!t.is_contiguous() || t.scalar_type() != type || !has_sizes(t, sizes)) {
    std::string dims;
    for (const int64_t s : sizes) dims += (dims.empty() ? "" : " x ") + std::to_string(s);
    REFUSE("%s must be contiguous, %s of %s", name, dims.c_str(), c10::toString(type));
  }
  return t.data_ptr();
}

// No call has a forward-mode derivative: operands with a tangent are refused, and so
// are outputs, whose tangent would be that of the old contents. (Whether gradients are
// recorded does not matter: torch.no_grad leaves tangents on.)
void no_tangents(std::initializer_list<PyObject*> operands) {
  for (PyObject* o : operands)
    if (!none(o) && THPVariable_Check(o) && THPVariable_Unpack(o)._fw_grad(0).defined())
      REFUSE("the call has no forward-mode derivative: give it tensors without tangents");
}

// The caller's output, or a new one.
Matrix output(PyObject* o, const char* name, int64_t n, int64_t c, const at::Tensor& like, at::ScalarType type) {
  if (none(o)) {
    at::Tensor t = at::empty({n, c}, like.options().dtype(type));
    return Matrix{t, n, c, c, t.data_ptr(), float_type(type)};
  }
  no_tangents({o});
  Matrix m = matrix(o, name);
  if (m.n != n || m.c != c || m.t.scalar_type() != type)
    REFUSE("%s must be %lld x %lld of %s", name, (long long)n, (long long)c, c10::toString(type));
  return m;
}

struct Slots {
  int64_t tokens;
  int k;
  const int32_t* f2p;
  const float* w;
};

Slots slots(PyObject* f2p, PyObject* k, PyObject* w) {
  const at::Tensor& t = on_gpu(f2p, "flat_to_perm");
  const int64_t kk = integer(k, "k"), n = t.numel();
  if (!t.is_contiguous() || t.scalar_type() != at::kInt || kk < 1 || kk > 16 || n % kk != 0 ||
      !has_sizes(t, {n / kk, kk}))
    REFUSE("flat_to_perm must be contiguous int32 with k entries a token, 1 <= k <= 16");
  return Slots{n / kk, (int)kk, static_cast<const int32_t*>(t.data_ptr()),
               none(w) ? nullptr : static_cast<const float*>(flat(w, "topk_w", at::kFloat, {n / kk, kk}))};
}

// The operand of the weights' gradient, and the gradient.
struct Dots {
  const void* p = nullptr;
  int64_t ld = 0;
  at::Tensor d_w;
  float* pd = nullptr;
};

Dots dots(PyObject* o, const char* name, int64_t n, int64_t c, const Matrix& like, const Slots& s) {
  Dots d;
  if (none(o)) return d;
  const Matrix m = matrix(o, name);
  if (m.n != n || m.c != c || m.type != like.type || !s.w)
    REFUSE("%s must be %lld x %lld of the other operand's type, given together with topk_w", name, (long long)n,
           (long long)c);
  d.p = m.p;
  d.ld = m.ld;
  d.d_w = at::empty({s.tokens, (int64_t)s.k}, like.t.options().dtype(at::kFloat));
  d.pd = static_cast<float*>(d.d_w.data_ptr());
  return d;
}

void* stream() { return c10::cuda::getCurrentCUDAStream().stream(); }

// `into`: the caller's tensors that the call writes into, or none. Their versions go
// up, as those of torch's own in-place operations do: a backward pass that saved the
// old contents then refuses. (A call that is refused has written nothing; tensors of
// inference mode have no version.)
template <typename Call>
void run(const char* what, std::initializer_list<PyObject*> into, Call call) {
  int status;
  void* s = stream();
  Py_BEGIN_ALLOW_THREADS
  status = call(s);
  Py_END_ALLOW_THREADS
  if (status == NVFP4MOE_OK || status == NVFP4MOE_ERR_LAUNCH) {
    for (PyObject* o : into) {
      if (none(o)) continue;
      const at::Tensor& t = THPVariable_Unpack(o);
      if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
    }
  }
  if (status != NVFP4MOE_OK) REFUSE("%s failed: %s (%d)", what, nvfp4moe_status_string(status), status);
}

PyObject* wrap(const at::Tensor& t) {
  if (t.defined()) return THPVariable_Wrap(t);
  Py_RETURN_NONE;
}

PyObject* pair(const at::Tensor& a, const at::Tensor& b) {
  PyObject* t = PyTuple_New(2);
  if (!t) throw python_error();
  PyTuple_SET_ITEM(t, 0, wrap(a));
  PyTuple_SET_ITEM(t, 1, wrap(b));
  return t;
}

int64_t blocks(int64_t n) { return (n + 127) / 128; }

#define CALL(name, count)                                                           \
  PyObject* name(PyObject*, PyObject* const* a, Py_ssize_t given) {                 \
    HANDLE_TH_ERRORS                                                                \
    if (given != (count)) REFUSE(#name " takes %d arguments", (int)(count));

#define END_CALL          \
  END_HANDLE_TH_ERRORS    \
  }

// Whether a call on this tensor has to be recorded for a backward pass:
// binding.py then makes it again through an autograd function (in which
// gradients are not recorded).
bool recorded(PyObject* o) {
  return !none(o) && c10::GradMode::is_enabled() && THPVariable_Check(o) && THPVariable_Unpack(o).requires_grad();
}

// x, flat_to_perm, k, topk_w, n_rows, rows
CALL(moe_sort_tokens, 6)
  no_tangents({a[0], a[3], a[5]});
  if (recorded(a[0]) || recorded(a[3])) Py_RETURN_NOTIMPLEMENTED;
  const Matrix x = matrix(a[0], "x");
  const Slots s = slots(a[1], a[2], a[3]);
  if (s.tokens != x.n) REFUSE("flat_to_perm must have k entries for each row of x");
  const int64_t n = !none(a[4]) ? integer(a[4], "n_rows") : !none(a[5]) ? matrix(a[5], "rows").n : x.n * s.k;
  if (n < 0) REFUSE("n_rows must not be negative");
  const Matrix out = output(a[5], "rows", n, x.c, x.t, x.t.scalar_type());
  run("moe_sort_tokens", {a[5]}, [&](void* st) {
    return ::moe_sort_tokens(x.p, x.type, x.n, x.c, x.ld, s.f2p, s.k, s.w, out.p, n, out.ld, st);
  });
  return wrap(out.t);
END_CALL

// d_rows, flat_to_perm, k, topk_w, x, dx
CALL(moe_sort_tokens_backward, 6)
  no_tangents({a[0], a[3], a[4]});
  const Matrix d = matrix(a[0], "d_rows");
  const Slots s = slots(a[1], a[2], a[3]);
  const Dots w = dots(a[4], "x", s.tokens, d.c, d, s);
  const Matrix out = output(a[5], "dx", s.tokens, d.c, d.t, d.t.scalar_type());
  run("moe_sort_tokens_backward", {a[5]}, [&](void* st) {
    return ::moe_sort_tokens_backward(d.p, d.type, d.n, d.c, d.ld, s.f2p, s.tokens, s.k, s.w, w.p, w.ld, out.p, out.ld,
                                      w.pd, st);
  });
  return pair(out.t, w.d_w);
END_CALL

// rows, flat_to_perm, k, topk_w, y
CALL(moe_unsort_tokens, 5)
  no_tangents({a[0], a[3], a[4]});
  if (recorded(a[0]) || recorded(a[3])) Py_RETURN_NOTIMPLEMENTED;
  const Matrix r = matrix(a[0], "rows");
  const Slots s = slots(a[1], a[2], a[3]);
  const Matrix out = output(a[4], "y", s.tokens, r.c, r.t, r.t.scalar_type());
  run("moe_unsort_tokens", {a[4]}, [&](void* st) {
    return ::moe_unsort_tokens(r.p, r.type, r.n, r.c, r.ld, s.f2p, s.tokens, s.k, s.w, out.p, out.ld, st);
  });
  return wrap(out.t);
END_CALL

// dy, flat_to_perm, k, topk_w, rows, n_rows, d_rows
CALL(moe_unsort_tokens_backward, 7)
  no_tangents({a[0], a[3], a[4]});
  const Matrix dy = matrix(a[0], "dy");
  const Slots s = slots(a[1], a[2], a[3]);
  if (s.tokens != dy.n) REFUSE("flat_to_perm must have k entries for each row of dy");
  const int64_t n = !none(a[5])   ? integer(a[5], "n_rows")
                    : !none(a[4]) ? matrix(a[4], "rows").n
                    : !none(a[6]) ? matrix(a[6], "d_rows").n
                                  : dy.n * s.k;
  if (n < 0) REFUSE("n_rows must not be negative");
  const Dots w = dots(a[4], "rows", n, dy.c, dy, s);
  const Matrix out = output(a[6], "d_rows", n, dy.c, dy.t, dy.t.scalar_type());
  run("moe_unsort_tokens_backward", {a[6]}, [&](void* st) {
    return ::moe_unsort_tokens_backward(dy.p, dy.type, dy.n, dy.c, dy.ld, s.f2p, s.k, s.w, w.p, w.ld, out.p, n, out.ld,
                                        w.pd, st);
  });
  return pair(out.t, w.d_w);
END_CALL

// Codes and scales of n rows: the caller's, or new ones.
struct Quantized {
  at::Tensor codes, sf;
  uint8_t* pc;
  float* ps;
};

Quantized quantized(PyObject* codes, PyObject* sf, int64_t n, int64_t K, const at::Tensor& like) {
  Quantized q;
  if (none(codes)) {
    q.codes = at::empty({n, K}, like.options().dtype(at::kByte));
    q.pc = static_cast<uint8_t*>(q.codes.data_ptr());
  } else {
    q.pc = static_cast<uint8_t*>(flat(codes, "codes", at::kByte, {n, K}));
    q.codes = THPVariable_Unpack(codes);
  }
  if (none(sf)) {
    q.sf = at::empty({n, blocks(K)}, like.options().dtype(at::kFloat));
    q.ps = static_cast<float*>(q.sf.data_ptr());
  } else {
    q.ps = static_cast<float*>(flat(sf, "sf", at::kFloat, {n, blocks(K)}));
    q.sf = THPVariable_Unpack(sf);
  }
  return q;
}

// x, flat_to_perm, k, out_rows, codes, sf
CALL(fp8_quantize, 6)
  const Matrix x = matrix(a[0], "x");
  Slots s{x.n, 1, nullptr, nullptr};
  if (!none(a[1])) {
    s = slots(a[1], a[2], nullptr);
    if (s.tokens != x.n) REFUSE("flat_to_perm must have k entries for each row of x");
  }
  const int64_t n = none(a[3]) ? x.n * s.k : integer(a[3], "out_rows");
  if (n < 0) REFUSE("out_rows must not be negative");
  const Quantized q = quantized(a[4], a[5], n, x.c, x.t);
  run("fp8_quantize", {a[4], a[5]}, [&](void* st) {
    return ::fp8_quantize(x.p, x.type, x.n, x.c, x.ld, s.f2p, s.k, n, q.pc, q.ps, st);
  });
  return pair(q.codes, q.sf);
END_CALL

// gate_up, codes, sf
CALL(fp8_swiglu_quantize, 3)
  const Matrix x = matrix(a[0], "gate_up");
  if (x.c % 2 != 0) REFUSE("gate_up must have as many up as gate columns");
  const Quantized q = quantized(a[1], a[2], x.n, x.c / 2, x.t);
  run("fp8_swiglu_quantize", {a[1], a[2]}, [&](void* st) {
    return ::fp8_swiglu_quantize(x.p, x.type, x.n, x.c / 2, x.ld, q.pc, q.ps, st);
  });
  return pair(q.codes, q.sf);
END_CALL

// w
CALL(fp8_quantize_weight, 1)
  const at::Tensor& w = on_gpu(a[0], "w");
  const int type = float_type(w.scalar_type());
  if (type < 0 || (w.dim() != 2 && w.dim() != 3) || !w.is_contiguous())
    REFUSE("w must be (N, K) or (E, N, K), contiguous, in BF16, F16 or F32");
  const bool many = w.dim() == 3;
  const int64_t E = many ? w.size(0) : 1, N = w.size(-2), K = w.size(-1);
  at::Tensor codes = at::empty(w.sizes(), w.options().dtype(at::kByte));
  at::Tensor sf = many ? at::empty({E, blocks(N), blocks(K)}, w.options().dtype(at::kFloat))
                       : at::empty({blocks(N), blocks(K)}, w.options().dtype(at::kFloat));
  run("fp8_quantize_weight", {}, [&](void* st) {
    return ::fp8_quantize_weight(w.data_ptr(), type, E, N, K, K, static_cast<uint8_t*>(codes.data_ptr()),
                                 static_cast<float*>(sf.data_ptr()), st);
  });
  return pair(codes, sf);
END_CALL

// ------------------------------------------------------------------ norms

double number(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    REFUSE("%s must be a number", name);
  }
  return v;
}

// A matrix of these sizes and this type that may be absent (p null).
Matrix optional(PyObject* o, const char* name, int64_t n, int64_t c, at::ScalarType type) {
  if (none(o)) return Matrix{at::Tensor(), n, c, c, nullptr, -1};
  Matrix m = matrix(o, name);
  if (m.n != n || m.c != c || m.t.scalar_type() != type)
    REFUSE("%s must be %lld x %lld of %s", name, (long long)n, (long long)c, c10::toString(type));
  return m;
}

// The operands and results that rms_norm and fp8_rms_norm_quantize share.
struct Norm {
  Matrix x, r, h;
  const float* gamma;
  float eps;
};

Norm norm(PyObject* x, PyObject* gamma, PyObject* eps, PyObject* residual, PyObject* h) {
  Norm m{matrix(x, "x"), {}, {}, nullptr, 0.0f};
  const at::ScalarType type = m.x.t.scalar_type();
  m.gamma = static_cast<const float*>(flat(gamma, "gamma", at::kFloat, {m.x.c}));
  m.eps = (float)number(eps, "eps");
  if (!(m.eps >= 0.0f)) REFUSE("eps must not be negative");
  m.r = optional(residual, "residual", m.x.n, m.x.c, type);
  if (m.r.t.defined()) {
    m.h = output(h, "h", m.x.n, m.x.c, m.x.t, type);
  } else {
    if (!none(h)) REFUSE("h is the sum of x and a residual: there is none without one");
    m.h = Matrix{m.x.t, m.x.n, m.x.c, m.x.ld, nullptr, m.x.type};
  }
  return m;
}

// x, gamma, eps, residual, y, h
CALL(rms_norm, 6)
  no_tangents({a[0], a[1], a[3], a[4], a[5]});
  if (recorded(a[0]) || recorded(a[1]) || recorded(a[3])) Py_RETURN_NOTIMPLEMENTED;
  const Norm m = norm(a[0], a[1], a[2], a[3], a[5]);
  const Matrix y = output(a[4], "y", m.x.n, m.x.c, m.x.t, m.x.t.scalar_type());
  run("rms_norm", {a[4], a[5]}, [&](void* st) {
    return ::rms_norm(m.x.p, m.x.type, m.x.n, m.x.c, m.x.ld, m.r.p, m.r.ld, m.gamma, m.eps, m.h.p, m.h.ld, y.p, y.ld,
                      st);
  });
  return pair(y.t, m.h.t);
END_CALL

// x, gamma, eps, residual, with_y, y, h, codes, sf
CALL(fp8_rms_norm_quantize, 9)
  no_tangents({a[0], a[1], a[3], a[5], a[6]});
  if (recorded(a[0]) || recorded(a[1]) || recorded(a[3])) Py_RETURN_NOTIMPLEMENTED;
  const Norm m = norm(a[0], a[1], a[2], a[3], a[6]);
  const int with_y = PyObject_IsTrue(a[4]);
  if (with_y < 0) throw python_error();
  const at::ScalarType type = m.x.t.scalar_type();
  const Matrix y = with_y || !none(a[5]) ? output(a[5], "y", m.x.n, m.x.c, m.x.t, type)
                                         : optional(a[5], "y", m.x.n, m.x.c, type);
  const Quantized q = quantized(a[7], a[8], m.x.n, m.x.c, m.x.t);
  run("fp8_rms_norm_quantize", {a[5], a[6], a[7], a[8]}, [&](void* st) {
    return ::fp8_rms_norm_quantize(m.x.p, m.x.type, m.x.n, m.x.c, m.x.ld, m.r.p, m.r.ld, m.gamma, m.eps, m.h.p, m.h.ld,
                                   y.p, y.ld, q.pc, q.ps, st);
  });
  PyObject* t = PyTuple_New(4);
  if (!t) throw python_error();
  PyTuple_SET_ITEM(t, 0, wrap(q.codes));
  PyTuple_SET_ITEM(t, 1, wrap(q.sf));
  PyTuple_SET_ITEM(t, 2, wrap(m.h.t));
  PyTuple_SET_ITEM(t, 3, wrap(y.t));
  return t;
END_CALL

// dy, h, gamma, eps, dh, dx
CALL(rms_norm_backward, 6)
  no_tangents({a[0], a[1], a[2], a[4]});
  const Matrix dy = matrix(a[0], "dy");
  const at::ScalarType type = dy.t.scalar_type();
  const Matrix h = optional(a[1], "h", dy.n, dy.c, type), dh = optional(a[4], "dh", dy.n, dy.c, type);
  if (!h.t.defined()) REFUSE("h must be a matrix of BF16, F16 or F32");
  const auto* gamma = static_cast<const float*>(flat(a[2], "gamma", at::kFloat, {dy.c}));
  const double eps = number(a[3], "eps");
  if (!(eps >= 0.0)) REFUSE("eps must not be negative");
  const Matrix dx = output(a[5], "dx", dy.n, dy.c, dy.t, type);
  at::Tensor d_gamma = at::empty({dy.c}, dy.t.options().dtype(at::kFloat));
  const int64_t bytes = (int64_t)::rms_norm_backward_workspace_size(dy.n, dy.c);
  at::Tensor ws = at::empty({bytes / 4}, d_gamma.options());
  run("rms_norm_backward", {a[5]}, [&](void* st) {
    return ::rms_norm_backward(dy.p, dy.type, dy.n, dy.c, dy.ld, h.p, h.ld, gamma, (float)eps, dh.p, dh.ld, dx.p, dx.ld,
                               static_cast<float*>(d_gamma.data_ptr()), ws.data_ptr(), (size_t)bytes, st);
  });
  return pair(dx.t, d_gamma);
END_CALL

// The type of a product: that of the caller's output, else out_dtype.
at::ScalarType product_type(PyObject* out, PyObject* dtype) {
  at::ScalarType t = at::kDouble;
  if (!none(out)) t = on_gpu(out, "out").scalar_type();
  else if (THPDtype_Check(dtype)) t = reinterpret_cast<THPDtype*>(dtype)->scalar_type;
  if (float_type(t) < 0) REFUSE("the result must be BF16, F16 or F32");
  return t;
}

// a_codes, a_sf, w_codes, w_sf, out, out_dtype
CALL(fp8_linear, 6)
  const Matrix x = matrix(a[0], "a_codes", true), w = matrix(a[2], "w_codes", true);
  if (w.c != x.c) REFUSE("a_codes and w_codes must have the same K");
  const int64_t kb = blocks(x.c);
  const auto* sx = static_cast<const float*>(flat(a[1], "a_sf", at::kFloat, {x.n, kb}));
  const auto* sw = static_cast<const float*>(flat(a[3], "w_sf", at::kFloat, {blocks(w.n), kb}));
  const Matrix out = output(a[4], "out", x.n, w.n, x.t, product_type(a[4], a[5]));
  run("fp8_linear", {a[4]}, [&](void* st) {
    return ::fp8_linear(static_cast<const uint8_t*>(x.p), sx, x.n, x.ld, static_cast<const uint8_t*>(w.p), sw, w.n,
                        x.c, w.ld, out.p, out.type, out.ld, st);
  });
  return wrap(out.t);
END_CALL

// a_codes, a_sf, w_codes, w_sf, offsets, out, out_dtype
CALL(fp8_grouped_gemm, 7)
  const Matrix x = matrix(a[0], "a_codes", true);
  const at::Tensor& w = on_gpu(a[2], "w_codes");
  if (!is_codes(w.scalar_type()) || w.dim() != 3 || !w.is_contiguous() || w.size(2) != x.c)
    REFUSE("w_codes must be contiguous (E, N, K) codes with the K of a_codes");
  const int64_t E = w.size(0), N = w.size(1), kb = blocks(x.c);
  if (E > 1024) REFUSE("at most 1024 experts");
  const auto* sx = static_cast<const float*>(flat(a[1], "a_sf", at::kFloat, {x.n, kb}));
  const auto* sw = static_cast<const float*>(flat(a[3], "w_sf", at::kFloat, {E, blocks(N), kb}));
  const auto* off = static_cast<const int32_t*>(flat(a[4], "offsets", at::kInt, {E + 1}));
  const Matrix out = output(a[5], "out", x.n, N, x.t, product_type(a[5], a[6]));
  run("fp8_grouped_gemm", {a[5]}, [&](void* st) {
    return ::fp8_grouped_gemm(static_cast<const uint8_t*>(x.p), sx, x.n, x.ld,
                              static_cast<const uint8_t*>(w.data_ptr()), sw, off, (int)E, N, x.c, x.c, out.p, out.type,
                              out.ld, st);
  });
  return wrap(out.t);
END_CALL

// Calls that are not recorded refuse operands that a gradient would be lost of.
void not_recorded(const char* what, std::initializer_list<PyObject*> operands) {
  for (PyObject* o : operands)
    if (recorded(o)) REFUSE("%s is not differentiable: call it without gradients (torch.no_grad)", what);
}

int activation(PyObject* o) {
  static const struct {
    const char* name;
    int value;
  } known[] = {{"none", NVFP4MOE_ACT_NONE},
               {"relu", NVFP4MOE_ACT_RELU},
               {"gelu", NVFP4MOE_ACT_GELU},
               {"gelu_tanh", NVFP4MOE_ACT_GELU_TANH},
               {"silu", NVFP4MOE_ACT_SILU}};
  if (PyUnicode_Check(o)) {
    for (const auto& k : known)
      if (PyUnicode_CompareWithASCIIString(o, k.name) == 0) return k.value;
  }
  REFUSE("activation must be none, relu, gelu, gelu_tanh or silu");
}

// a_codes, a_sf, w_codes, w_sf, bias, activation, residual, out, out_dtype
CALL(fp8_linear_epilogue, 9)
  no_tangents({a[4], a[6]});
  not_recorded("fp8_linear_epilogue", {a[4], a[6]});
  const Matrix x = matrix(a[0], "a_codes", true), w = matrix(a[2], "w_codes", true);
  if (w.c != x.c) REFUSE("a_codes and w_codes must have the same K");
  const int64_t kb = blocks(x.c);
  const auto* sx = static_cast<const float*>(flat(a[1], "a_sf", at::kFloat, {x.n, kb}));
  const auto* sw = static_cast<const float*>(flat(a[3], "w_sf", at::kFloat, {blocks(w.n), kb}));
  const auto* bias = none(a[4]) ? nullptr : static_cast<const float*>(flat(a[4], "bias", at::kFloat, {w.n}));
  const int act = activation(a[5]);
  const at::ScalarType type = product_type(a[7], a[8]);
  const Matrix r = optional(a[6], "residual", x.n, w.n, type);
  const Matrix out = output(a[7], "out", x.n, w.n, x.t, type);
  run("fp8_linear_epilogue", {a[7]}, [&](void* st) {
    return ::fp8_linear_epilogue(static_cast<const uint8_t*>(x.p), sx, x.n, x.ld, static_cast<const uint8_t*>(w.p), sw,
                                 w.n, x.c, w.ld, bias, act, r.p, r.ld, out.p, out.type, out.ld, st);
  });
  return wrap(out.t);
END_CALL

const at::Tensor& expert_codes(PyObject* o, const char* name) {
  const at::Tensor& t = on_gpu(o, name);
  if (!is_codes(t.scalar_type()) || t.dim() != 3 || !t.is_contiguous())
    REFUSE("%s must be contiguous codes with three dimensions", name);
  return t;
}

// x, logits, w1_codes, w1_sf, w2_codes, w2_sf, k, residual, ws, y
CALL(fp8_moe_few_tokens, 10)
  no_tangents({a[0], a[1], a[7]});
  not_recorded("fp8_moe_few_tokens", {a[0], a[1], a[7]});
  const Matrix x = matrix(a[0], "x");
  const at::ScalarType type = x.t.scalar_type();
  const at::Tensor &w1 = expert_codes(a[2], "w1_codes"), &w2 = expert_codes(a[4], "w2_codes");
  const int64_t T = x.n, K = x.c, E = w1.size(0), I = w2.size(2), k = integer(a[6], "k");
  if (w1.size(1) != 2 * I || w1.size(2) != K || w2.size(0) != E || w2.size(1) != K)
    REFUSE("w1_codes must be (E, 2I, K) and w2_codes (E, K, I), with the K of x");
  if (k < 1 || k > 16 || E < k || E > 1024) REFUSE("1 <= k <= 16 and k <= E <= 1024 are required");
  if (T > NVFP4MOE_FEW_TOKENS_MAX) REFUSE("at most %d tokens (fp8_moe_forward takes more)", NVFP4MOE_FEW_TOKENS_MAX);
  const auto* s1 = static_cast<const float*>(flat(a[3], "w1_sf", at::kFloat, {E, blocks(2 * I), blocks(K)}));
  const auto* s2 = static_cast<const float*>(flat(a[5], "w2_sf", at::kFloat, {E, blocks(K), blocks(I)}));
  const auto* logits = static_cast<const float*>(flat(a[1], "logits", at::kFloat, {T, E}));
  const Matrix r = optional(a[7], "residual", T, K, type);
  const Matrix y = output(a[9], "y", T, K, x.t, type);
  at::Tensor ws;
  if (none(a[8])) {
    ws = at::empty({(int64_t)::fp8_moe_few_tokens_workspace_size(T, K, I, (int)E, (int)k)},
                   x.t.options().dtype(at::kByte));
  } else {
    ws = on_gpu(a[8], "ws");
    if (!ws.is_contiguous()) REFUSE("ws must be contiguous");
  }
  run("fp8_moe_few_tokens", {a[8], a[9]}, [&](void* st) {
    return ::fp8_moe_few_tokens(x.p, x.type, T, K, x.ld, logits, I, (int)E, (int)k,
                                static_cast<const uint8_t*>(w1.data_ptr()), s1,
                                static_cast<const uint8_t*>(w2.data_ptr()), s2, r.p, r.ld, y.p, y.ld, ws.data_ptr(),
                                (size_t)ws.nbytes(), st);
  });
  return wrap(y.t);
END_CALL

// The type of the errors raised here.
PyObject* set_error(PyObject*, PyObject* type) {
  Py_INCREF(type);
  Py_XDECREF(g_error);
  g_error = type;
  Py_RETURN_NONE;
}

#define METHOD(name) {#name, (PyCFunction)(void*)name, METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {METHOD(moe_sort_tokens),
                           METHOD(moe_sort_tokens_backward),
                           METHOD(moe_unsort_tokens),
                           METHOD(moe_unsort_tokens_backward),
                           METHOD(fp8_quantize),
                           METHOD(fp8_swiglu_quantize),
                           METHOD(fp8_quantize_weight),
                           METHOD(fp8_linear),
                           METHOD(fp8_grouped_gemm),
                           METHOD(rms_norm),
                           METHOD(rms_norm_backward),
                           METHOD(fp8_rms_norm_quantize),
                           METHOD(fp8_linear_epilogue),
                           METHOD(fp8_moe_few_tokens),
                           {"set_error", set_error, METH_O, nullptr},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_tensor_calls", nullptr, -1, g_methods};

}  // namespace

PyMODINIT_FUNC PyInit__tensor_calls() { return PyModule_Create(&g_module); }
