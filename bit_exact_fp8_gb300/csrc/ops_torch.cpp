// ops_torch.cpp -- the operators around the 8-bit product on torch tensors: checks of arguments,
// outputs and workspaces, the current stream, and one call of the C ABI each (include/emu_fp8.h).
// Nothing is computed here.  It is C++ because the smallest calls (one token) are bound by the
// host: the same checks and allocations in Python took 22 us a call.
#include "emu_fp8.h"

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/core/AutogradState.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

namespace {

PyObject* g_unsupported = nullptr;      // UnsupportedFeatureError
PyObject* g_cuda_error = nullptr;       // EmuCudaError

struct Refused {                         // becomes the Python exception `type`
  PyObject* type;
  std::string what;
};
[[noreturn]] void bad(const std::string& what) { throw Refused{PyExc_ValueError, what}; }
[[noreturn]] void unsupported(const std::string& what) { throw Refused{g_unsupported ? g_unsupported : PyExc_ValueError, what}; }

std::string text(c10::ScalarType t) { return c10::toString(t); }
std::string text(const at::Tensor& t) {
  std::string s = text(t.scalar_type()) + " (";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + ") on " + t.device().str();
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) throw Refused{PyExc_TypeError, std::string(name) + " must be a tensor"};
  return THPVariable_Unpack(o);
}
c10::ScalarType dtype(PyObject* o, const char* name) {
  if (!THPDtype_Check(o)) throw Refused{PyExc_TypeError, std::string(name) + " must be a torch.dtype"};
  return reinterpret_cast<THPDtype*>(o)->scalar_type;
}
int64_t whole(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    throw Refused{PyExc_TypeError, std::string(name) + " must be a whole number of 64 bits"};
  }
  return v;
}

// the first tensor of a call: its device is everyone's
c10::Device first(const at::Tensor& t, const char* name) {
  if (t.dim() != 2) bad(std::string(name) + " must be 2-D");
  if (!t.is_cuda()) bad(std::string(name) + ": all tensors must be on a CUDA device (there is no CPU path)");
  return t.device();
}
emu_out_t float_type(c10::ScalarType t, const char* name) {
  if (t == at::kFloat) return EMU_OUT_F32;
  if (t == at::kBFloat16) return EMU_OUT_BF16;
  if (t == at::kHalf) return EMU_OUT_F16;
  bad(std::string(name) + ": fp32, bf16 or fp16 expected, got " + text(t));
}
// No floating input takes part in autograd: neither one that it records the calls of, nor one with a tangent
void no_grad(const at::Tensor& t) {
  if (c10::GradMode::is_enabled() && t.requires_grad())
    unsupported("not differentiable by autograd: an input requires grad under grad mode (call the _backward function)");
  if (c10::AutogradState::get_tls_state().get_fw_grad_mode() && t._fw_grad(0).defined())
    unsupported("not differentiable by autograd: an input carries a forward-mode tangent");
}
// An output of the caller's: autograd learns that its values are others now, as of any write in place.
void written(const at::Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}
// the row stride of [rows, cols] values whose rows are contiguous
int64_t rows_of(const at::Tensor& t, const char* name, int64_t rows, int64_t cols, c10::ScalarType type, c10::Device dev) {
  if (t.dim() != 2 || t.size(0) != rows || t.size(1) != cols || t.scalar_type() != type || t.device() != dev)
    bad(std::string(name) + ": expected " + text(type) + " (" + std::to_string(rows) + ", " + std::to_string(cols) +
        ") on " + dev.str() + ", got " + text(t));
  if (cols > 1 && t.stride(1) != 1) bad(std::string(name) + ": rows must be contiguous");
  if (rows <= 1) return cols;
  if (t.stride(0) < cols)
    bad(std::string(name) + ": rows must not overlap (row stride " + std::to_string(t.stride(0)) + ")");
  return t.stride(0);
}
void* vector_of(const at::Tensor& t, const char* name, int64_t count, c10::ScalarType type, c10::Device dev) {
  if (t.scalar_type() != type || t.device() != dev || t.numel() != count || !t.is_contiguous())
    bad(std::string(name) + ": expected " + std::to_string(count) + " contiguous " + text(type) + " on " + dev.str() +
        ", got " + text(t));
  return t.data_ptr();
}
// from the caching allocator on the current stream, as torch.empty, without its dispatch
at::Tensor make(at::IntArrayRef sizes, c10::ScalarType type, c10::Device dev) {
  return at::Tensor(at::detail::empty_cuda(sizes, type, dev, std::nullopt));
}
at::Tensor given(PyObject* o, const char* name, int64_t rows, int64_t cols, c10::ScalarType type, c10::Device dev) {
  const at::Tensor& t = tensor(o, name);
  no_grad(t);
  if (t.dim() != 2 || t.size(0) != rows || t.size(1) != cols || t.scalar_type() != type || !t.is_contiguous() ||
      t.device() != dev)
    bad(std::string(name) + " must be a contiguous " + text(type) + " (" + std::to_string(rows) + ", " +
        std::to_string(cols) + ") on " + dev.str() + ", got " + text(t));
  return t;
}
void check(int status, const char* what) {
  if (status == EMU_OK) return;
  const std::string msg = std::string(what) + ": " + emu_ops_last_error();
  if (status == EMU_EUNSUPPORTED) unsupported(msg);
  if (status == EMU_ECUDA) throw Refused{g_cuda_error ? g_cuda_error : PyExc_RuntimeError, msg};
  bad(msg);
}
// the device made current for the call, and its current stream
struct On {
  c10::cuda::CUDAGuard guard;
  void* stream;
  explicit On(c10::Device dev) : guard(dev), stream(c10::cuda::getCurrentCUDAStream(dev.index()).stream()) {}
};

PyObject* tuple_of(std::initializer_list<PyObject*> items) {        // takes the references
  PyObject* t = PyTuple_New((Py_ssize_t)items.size());
  Py_ssize_t i = 0;
  for (PyObject* o : items) {
    if (t) PyTuple_SET_ITEM(t, i++, o);
    else Py_XDECREF(o);
  }
  return t;
}
PyObject* same(PyObject* o) {
  Py_INCREF(o);
  return o;
}

// (x, weight, residual, eps, out_dtype, scale, out, residual_out) -> (q, scale, residual, rstd)
PyObject* norm_quant(PyObject* const* a) {
  const at::Tensor& x = tensor(a[0], "x");
  const at::Tensor& weight = tensor(a[1], "weight");
  const c10::Device dev = first(x, "x");
  no_grad(x);
  no_grad(weight);
  const int64_t T = x.size(0), H = x.size(1);
  const c10::ScalarType type = x.scalar_type();
  const emu_out_t ct = float_type(type, "x");
  const double eps = PyFloat_AsDouble(a[3]);
  if (eps == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    throw Refused{PyExc_TypeError, "eps must be a number"};
  }
  const c10::ScalarType qt = dtype(a[4], "out_dtype");
  emu_q_t fmt;
  if (qt == at::kFloat8_e4m3fn) fmt = EMU_Q_E4M3FN;
  else if (qt == at::kFloat8_e5m2) fmt = EMU_Q_E5M2;
  else if (qt == at::kChar) fmt = EMU_Q_INT8;
  else unsupported("out_dtype " + text(qt) + " is not supported");
  const int64_t ldx = rows_of(x, "x", T, H, type, dev);
  const c10::ScalarType wt = weight.scalar_type();
  if (wt != type && wt != at::kFloat) bad("weight: x's dtype or fp32 expected, got " + text(wt));
  void* wp = vector_of(weight, "weight", H, wt, dev);
  On on(dev);
  const void* rp = nullptr;
  void* op = nullptr;
  int64_t ldr = 0, ldo = 0;
  at::Tensor made, place;
  PyObject* h = a[0];
  if (a[7] != Py_None) {
    place = tensor(a[7], "residual_out");
    const at::Tensor& o = place;
    no_grad(o);
    ldo = rows_of(o, "residual_out", T, H, type, dev);
    op = o.data_ptr();
    h = a[7];
  }
  if (a[2] != Py_None) {
    const at::Tensor& r = tensor(a[2], "residual");
    no_grad(r);
    ldr = rows_of(r, "residual", T, H, type, dev);
    rp = r.data_ptr();
    if (!op) {
      made = make({T, H}, type, dev);
      op = made.data_ptr();
      ldo = H;
    }
  }
  const at::Tensor q = a[6] == Py_None ? make({T, H}, qt, dev) : given(a[6], "out", T, H, qt, dev);
  const at::Tensor rstd = make({T}, at::kFloat, dev);
  at::Tensor scales;
  const float* sp = nullptr;
  float* so = nullptr;
  if (a[5] != Py_None) {
    const at::Tensor& scale = tensor(a[5], "scale");
    no_grad(scale);
    sp = static_cast<const float*>(vector_of(scale, "scale", 1, at::kFloat, dev));
  } else {
    scales = make({T}, at::kFloat, dev);
    so = scales.data_ptr<float>();
  }
  check(emu_rms_norm_quant(x.data_ptr(), ldx, rp, ldr, wp, wt == at::kFloat ? EMU_OUT_F32 : ct, ct, T, H, (float)eps, sp,
                           fmt, q.data_ptr(), so, op, ldo, rstd.data_ptr<float>(), on.stream), "rms_norm_quant");
  if (place.defined()) written(place);
  if (a[6] != Py_None) written(q);
  return tuple_of({a[6] == Py_None ? THPVariable_Wrap(q) : same(a[6]), sp ? same(a[5]) : THPVariable_Wrap(scales),
                   made.defined() ? THPVariable_Wrap(made) : same(h), THPVariable_Wrap(rstd)});
}

// (grad_y, hidden, rstd, weight, grad_residual, workspace) -> (grad_x, grad_weight)
PyObject* norm_backward(PyObject* const* a) {
  const at::Tensor& gy = tensor(a[0], "grad_y");
  const at::Tensor& h = tensor(a[1], "hidden");
  const at::Tensor& weight = tensor(a[3], "weight");
  const c10::Device dev = first(h, "hidden");
  no_grad(gy);
  no_grad(h);
  no_grad(weight);
  const int64_t T = h.size(0), H = h.size(1);
  const c10::ScalarType type = h.scalar_type(), wt = weight.scalar_type();
  const emu_out_t ct = float_type(type, "hidden");
  const int64_t ldh = rows_of(h, "hidden", T, H, type, dev), ldy = rows_of(gy, "grad_y", T, H, type, dev);
  if (wt != type && wt != at::kFloat) bad("weight: hidden's dtype or fp32 expected, got " + text(wt));
  void* wp = vector_of(weight, "weight", H, wt, dev);
  const at::Tensor& rstd = tensor(a[2], "rstd");
  no_grad(rstd);
  const float* rp = static_cast<const float*>(vector_of(rstd, "rstd", T, at::kFloat, dev));
  const void* gp = nullptr;
  int64_t ldg = 0;
  if (a[4] != Py_None) {
    const at::Tensor& g = tensor(a[4], "grad_residual");
    no_grad(g);
    ldg = rows_of(g, "grad_residual", T, H, type, dev);
    gp = g.data_ptr();
  }
  On on(dev);
  const size_t need = emu_rms_norm_backward_workspace_bytes(T, H);
  at::Tensor ws;
  if (a[5] != Py_None) {
    ws = tensor(a[5], "workspace");
    if (ws.device() != dev || !ws.is_contiguous()) bad("workspace: a contiguous tensor on " + dev.str() + " expected");
  }
  if (need > 0 && (!ws.defined() || (size_t)ws.nbytes() < need)) ws = make({(int64_t)need}, at::kByte, dev);
  const at::Tensor gx = make({T, H}, type, dev), gw = make({H}, at::kFloat, dev);
  check(emu_rms_norm_backward(gy.data_ptr(), ldy, h.data_ptr(), ldh, rp, wp, wt == at::kFloat ? EMU_OUT_F32 : ct, gp, ldg,
                              ct, T, H, gx.data_ptr(), gw.data_ptr<float>(), need ? ws.data_ptr() : nullptr, need,
                              on.stream), "rms_norm_backward");
  return tuple_of({THPVariable_Wrap(gx), THPVariable_Wrap(gw)});
}

// (mat1, mat2, scale_a, scale_b, out_dtype, out, workspace) -> out
PyObject* int8_mm(PyObject* const* a) {
  const at::Tensor& m1 = tensor(a[0], "mat1");
  const at::Tensor& m2 = tensor(a[1], "mat2");
  const c10::Device dev = first(m1, "mat1");
  if (m2.dim() != 2) bad("mat2 must be 2-D");
  const int64_t M = m1.size(0), K = m1.size(1), N = m2.size(1);
  if (m2.size(0) != K) bad("shape mismatch: " + text(m1) + " @ " + text(m2));
  const int64_t lda = rows_of(m1, "mat1", M, K, at::kChar, dev);
  if (m2.scalar_type() != at::kChar || m2.device() != dev) bad("mat2: int8 on " + dev.str() + " expected, got " + text(m2));
  if (K > 1 && m2.stride(0) != 1) bad("mat2 must be column-major ([K, N] with K contiguous, e.g. w.t())");
  const int64_t ldb = N <= 1 ? K : m2.stride(1);
  if (ldb < K) bad("mat2: columns must not overlap (column stride " + std::to_string(ldb) + ")");
  const c10::ScalarType ot = dtype(a[4], "out_dtype");
  if (ot != at::kFloat && ot != at::kBFloat16 && ot != at::kHalf) unsupported("out_dtype " + text(ot) + " is not supported");
  const at::Tensor& sa = tensor(a[2], "scale_a");
  const at::Tensor& sb = tensor(a[3], "scale_b");
  no_grad(sa);
  no_grad(sb);
  const int64_t na = sa.numel(), nb = sb.numel();
  if (na != 1 && na != M) bad("scale_a: one value or " + std::to_string(M) + " expected, got " + std::to_string(na));
  if (nb != 1 && nb != N) bad("scale_b: one value or " + std::to_string(N) + " expected, got " + std::to_string(nb));
  const float* pa = static_cast<const float*>(vector_of(sa, "scale_a", na, at::kFloat, dev));
  const float* pb = static_cast<const float*>(vector_of(sb, "scale_b", nb, at::kFloat, dev));
  On on(dev);
  const at::Tensor out = a[5] == Py_None ? make({M, N}, ot, dev) : given(a[5], "out", M, N, ot, dev);
  const int8_t* A = m1.data_ptr<int8_t>();
  const int8_t* B = m2.data_ptr<int8_t>();
  const size_t need = emu_int8_workspace_bytes(M, N, K);
  at::Tensor ws;
  if (a[6] != Py_None) {
    ws = tensor(a[6], "workspace");
    if (ws.device() != dev || !ws.is_contiguous()) bad("workspace: a contiguous tensor on " + dev.str() + " expected");
  }
  if (need > 0 && (!ws.defined() || (size_t)ws.nbytes() < need || reinterpret_cast<uintptr_t>(ws.data_ptr()) % 256))
    ws = make({(int64_t)need}, at::kByte, dev);
  check(emu_int8_scaled_mm(A, lda, B, ldb, M, N, K, pa, na, pb, nb, out.data_ptr(),
                           ot == at::kFloat ? EMU_OUT_F32 : ot == at::kBFloat16 ? EMU_OUT_BF16 : EMU_OUT_F16,
                           need ? ws.data_ptr() : nullptr, need, on.stream), "int8_scaled_mm");
  if (a[5] != Py_None) written(out);
  return a[5] == Py_None ? THPVariable_Wrap(out) : same(a[5]);
}

// (logits, tokens, top_k, ignore_index) -> (logprob, entropy, lse, stats, top_logprobs, top_ids)
PyObject* logprobs(PyObject* const* a) {
  const at::Tensor& x = tensor(a[0], "logits");
  const c10::Device dev = first(x, "logits");
  no_grad(x);
  const int64_t T = x.size(0), V = x.size(1), k = whole(a[2], "top_k"), ignore = whole(a[3], "ignore_index");
  const emu_out_t ct = float_type(x.scalar_type(), "logits");
  const int64_t ldx = rows_of(x, "logits", T, V, x.scalar_type(), dev);
  const int64_t* tok = static_cast<const int64_t*>(vector_of(tensor(a[1], "tokens"), "tokens", T, at::kLong, dev));
  if (k < 0 || k > V) bad("top_k " + std::to_string(k) + " of " + std::to_string(V) + " logits");
  if (k > 32) unsupported("top_k above 32 is not supported");
  On on(dev);
  const at::Tensor lp = make({T}, at::kFloat, dev), en = make({T}, at::kFloat, dev), lse = make({T}, at::kFloat, dev),
                   st = make({T, 3}, at::kFloat, dev), tv = make({T, k}, at::kFloat, dev), ti = make({T, k}, at::kLong, dev);
  check(emu_token_logprobs(x.data_ptr(), ldx, ct, tok, T, V, (int32_t)k, ignore, lp.data_ptr<float>(),
                           en.data_ptr<float>(), lse.data_ptr<float>(), st.data_ptr<float>(), tv.data_ptr<float>(),
                           ti.data_ptr<int64_t>(), on.stream), "token_logprobs");
  return tuple_of({THPVariable_Wrap(lp), THPVariable_Wrap(en), THPVariable_Wrap(lse), THPVariable_Wrap(st),
                   THPVariable_Wrap(tv), THPVariable_Wrap(ti)});
}

// (logits, tokens, stats, grad_logprob, grad_entropy, ignore_index, out) -> grad_logits
PyObject* logprobs_backward(PyObject* const* a) {
  const at::Tensor& x = tensor(a[0], "logits");
  const c10::Device dev = first(x, "logits");
  no_grad(x);
  const int64_t T = x.size(0), V = x.size(1), ignore = whole(a[5], "ignore_index");
  const c10::ScalarType type = x.scalar_type();
  const emu_out_t ct = float_type(type, "logits");
  const int64_t ldx = rows_of(x, "logits", T, V, type, dev);
  const int64_t* tok = static_cast<const int64_t*>(vector_of(tensor(a[1], "tokens"), "tokens", T, at::kLong, dev));
  auto values = [&](PyObject* o, const char* name, int64_t count) -> const float* {
    const at::Tensor& t = tensor(o, name);
    no_grad(t);
    return static_cast<const float*>(vector_of(t, name, count, at::kFloat, dev));
  };
  const float* st = values(a[2], "stats", 3 * T);
  const float* gl = a[3] == Py_None ? nullptr : values(a[3], "grad_logprob", T);
  const float* ge = a[4] == Py_None ? nullptr : values(a[4], "grad_entropy", T);
  On on(dev);
  const at::Tensor gx = a[6] == Py_None ? make({T, V}, type, dev) : tensor(a[6], "out");
  no_grad(gx);
  const int64_t ldo = rows_of(gx, "out", T, V, type, dev);
  check(emu_token_logprobs_backward(x.data_ptr(), ldx, ct, tok, T, V, ignore, st, gl, ge, gx.data_ptr(), ldo, on.stream),
        "token_logprobs_backward");
  if (a[6] != Py_None) written(gx);
  return a[6] == Py_None ? THPVariable_Wrap(gx) : same(a[6]);
}

#include "ops_torch_block.h"

template <PyObject* (*F)(PyObject* const*), Py_ssize_t COUNT>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != COUNT) {
    PyErr_Format(PyExc_TypeError, "%zd arguments expected, got %zd", COUNT, n);
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Refused& r) {
    PyErr_SetString(r.type, r.what.c_str());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyObject* set_errors(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 2) {
    PyErr_SetString(PyExc_TypeError, "two exception classes expected");
    return nullptr;
  }
  Py_XSETREF(g_unsupported, same(args[0]));
  Py_XSETREF(g_cuda_error, same(args[1]));
  Py_RETURN_NONE;
}

#define EMU_METHOD(name, function) \
  {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(function)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {EMU_METHOD("rms_norm_quant", (entry<norm_quant, 8>)),
                           EMU_METHOD("rms_norm_backward", (entry<norm_backward, 6>)),
                           EMU_METHOD("int8_scaled_mm", (entry<int8_mm, 7>)),
                           EMU_METHOD("token_logprobs", (entry<logprobs, 4>)),
                           EMU_METHOD("token_logprobs_backward", (entry<logprobs_backward, 7>)),
                           EMU_METHOD("block_quant", (entry<block_quant, 4>)),
                           EMU_METHOD("swiglu_quant", (entry<swiglu_quant, 5>)),
                           EMU_METHOD("swiglu_backward", (entry<swiglu_backward, 3>)),
                           EMU_METHOD("block_scaled_mm", (entry<block_mm, 7>)),
                           EMU_METHOD("grouped_block_scaled_mm", (entry<grouped_mm, 8>)),
                           EMU_METHOD("grouped_block_scaled_wgrad", (entry<grouped_wgrad, 8>)),
                           EMU_METHOD("block_mm_workspace_bytes", (entry<block_mm_bytes, 2>)),
                           EMU_METHOD("block_wgrad_workspace_bytes", (entry<block_wgrad_bytes, 2>)),
                           EMU_METHOD("set_errors", set_errors),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_ops_torch", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ops_torch(void) {
  PyObject* m = PyModule_Create(&g_module);
  // the build and the loader look for this text in the file, to tell an extension of another torch
  if (m && PyModule_AddStringConstant(m, "built_for", EMU_OPS_BUILT_FOR) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
