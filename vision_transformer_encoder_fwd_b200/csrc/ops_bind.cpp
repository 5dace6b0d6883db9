// Python side of the operator entry points in include/vit_ops.h: reads torch tensors, checks what only
// they tell (types, shapes, devices), allocates outputs that are not given and calls the C ABI on the
// right device and stream.  The public functions and their documentation are in ops.py, which calls
// these with all arguments by position; marshalling in Python took 14-25 us a call, several times the
// device time of a single token's operators, and takes 2-3 us here.
#include <Python.h>

#include <ATen/Functions.h>
#include <ATen/core/grad_mode.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <optional>

#include "../../include/vit_ops.h"

namespace {

PyObject* g_error = nullptr;  // VitError(function, status, message)

[[noreturn]] void fail(const char* fn, int status, const char* msg) {
  const std::string name = std::string("vit_op_") + fn;
  PyObject* e = PyObject_CallFunction(g_error, "sis", name.c_str(), status, msg);
  if (e != nullptr) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw python_error();
}

void check(const char* fn, vit_status st) {
  if (st == VIT_OK) return;
  const char* m = vit_last_error();
  fail(fn, st, m != nullptr && m[0] != 0 ? m : vit_status_str(st));
}

using Opt = const at::Tensor*;

Opt tensor_or_none(const char* fn, PyObject* o) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) fail(fn, VIT_E_INVALID_ARG, "expected a tensor");
  return &THPVariable_Unpack(o);
}
const at::Tensor& tensor(const char* fn, PyObject* o) {
  Opt t = tensor_or_none(fn, o);
  if (t == nullptr) fail(fn, VIT_E_INVALID_ARG, "a tensor is missing");
  return *t;
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw python_error();
  return v;
}
long long integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}
bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw python_error();
  return v != 0;
}
int32_t int32_of(const char* fn, int64_t v) {
  if (v < INT32_MIN || v > INT32_MAX) fail(fn, VIT_E_SHAPE, "a size does not fit 32 bits");
  return static_cast<int32_t>(v);
}
void* ptr(Opt t) { return t == nullptr ? nullptr : t->data_ptr(); }
PyObject* wrap_or_none(const std::optional<at::Tensor>& t) {
  if (t.has_value()) return THPVariable_Wrap(*t);
  Py_RETURN_NONE;
}

// The operators keep no history: a call that autograd would expect one of is refused.
void need_no_history(const char* fn, Opt t) {
  if (t != nullptr && t->requires_grad() && at::GradMode::is_enabled())
    fail(fn, VIT_E_UNSUPPORTED, "forward only: a tensor requires a gradient (call under torch.no_grad(), or detach it)");
}
// A tensor of the caller's that was written: autograd sees that what it may have saved of it has changed.
void written(Opt t) {
  if (t != nullptr && !t->is_inference()) t->unsafeGetTensorImpl()->bump_version();
}

// The tensors' device, which becomes the current one, and the stream (None: the device's current one),
// which becomes the current one where it is given: allocations belong to it.
class Place {
 public:
  Place(const char* fn, PyObject* stream, std::initializer_list<Opt> tensors) {
    c10::Device dev(c10::DeviceType::CPU);
    for (Opt t : tensors) need_no_history(fn, t);
    for (Opt t : tensors) {
      if (t == nullptr) continue;
      if (!t->is_cuda()) fail(fn, VIT_E_INVALID_ARG, "tensors must be on a CUDA device");
      if (t->layout() != at::kStrided) fail(fn, VIT_E_UNSUPPORTED, "tensors must be strided");
      if (dev.is_cpu())
        dev = t->device();
      else if (t->device() != dev)
        fail(fn, VIT_E_INVALID_ARG, "tensors on different devices");
    }
    if (stream == Py_None) {
      device_.emplace(dev);
      handle_ = c10::cuda::getCurrentCUDAStream(dev.index()).stream();
    } else {
      auto part = [&](const char* name) {
        PyObject* v = PyObject_GetAttrString(stream, name);
        if (v == nullptr) throw python_error();
        const long long n = PyLong_AsLongLong(v);
        Py_DECREF(v);
        if (n == -1 && PyErr_Occurred()) throw python_error();
        return n;
      };
      const long long index = part("device_index");
      if (index != dev.index()) fail(fn, VIT_E_INVALID_ARG, "the stream is on another device than the tensors");
      const auto s = c10::cuda::CUDAStream::unpack3(part("stream_id"), static_cast<c10::DeviceIndex>(index),
                                                    static_cast<c10::DeviceType>(part("device_type")));
      stream_.emplace(s);
      handle_ = s.stream();
    }
  }
  vit_stream_t handle() const { return reinterpret_cast<vit_stream_t>(handle_); }

 private:
  std::optional<c10::cuda::CUDAGuard> device_;
  std::optional<c10::cuda::CUDAStreamGuard> stream_;
  cudaStream_t handle_ = nullptr;
};

vit_dtype type_of(const char* fn, const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return VIT_DT_BF16;
    case at::kHalf: return VIT_DT_F16;
    case at::kFloat: return VIT_DT_F32;
    case at::kFloat8_e4m3fn: return VIT_DT_E4M3;
    default: fail(fn, VIT_E_UNSUPPORTED, "unsupported type of tensor");
  }
}
void need_type(const char* fn, const at::Tensor& t, at::ScalarType want, const char* msg) {
  if (t.scalar_type() != want) fail(fn, VIT_E_UNSUPPORTED, msg);
}
// Leading dimension of a matrix with contiguous rows.
int64_t leading(const char* fn, const at::Tensor& t) {
  if (t.dim() != 2) fail(fn, VIT_E_SHAPE, "rows must be a matrix");
  if (t.size(1) > 1 && t.stride(1) != 1) fail(fn, VIT_E_INVALID_ARG, "rows must be contiguous");
  return t.size(0) > 1 ? t.stride(0) : t.size(1);
}
void need_vector(const char* fn, const at::Tensor& t, int64_t n, const char* msg) {
  if (t.dim() != 1 || t.size(0) != n || (n > 1 && t.stride(0) != 1)) fail(fn, VIT_E_SHAPE, msg);
}
void need_matrix(const char* fn, const at::Tensor& t, int64_t rows, int64_t cols, const char* msg) {
  if (t.dim() != 2 || t.size(0) != rows || t.size(1) != cols) fail(fn, VIT_E_SHAPE, msg);
}
at::Tensor make(at::IntArrayRef shape, at::ScalarType type, const at::Tensor& like) {
  return at::empty(shape, like.options().dtype(type).requires_grad(false).memory_format(at::MemoryFormat::Contiguous));
}
void need_args(Py_ssize_t got, Py_ssize_t want) {
  if (got != want) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, got);
    throw python_error();
  }
}

// (x, weight, eps, residual, residual_out, fp8, out, scales, stream) -> (out, scales, residual_out)
PyObject* rms_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const char* fn = "rms_norm";
  need_args(n, 9);
  const at::Tensor &x = tensor(fn, a[0]), &w = tensor(fn, a[1]);
  const double eps = number(a[2]);
  Opt r = tensor_or_none(fn, a[3]), h_in = tensor_or_none(fn, a[4]), out_in = tensor_or_none(fn, a[6]),
      sc_in = tensor_or_none(fn, a[7]);
  const bool fp8 = truth(a[5]);
  Place at(fn, a[8], {&x, &w, r, h_in, out_in, sc_in});
  const int64_t x_ld = leading(fn, x), rows = x.size(0), D = x.size(1);
  const at::Tensor out = out_in ? *out_in : make({rows, D}, fp8 ? at::kFloat8_e4m3fn : x.scalar_type(), x);
  need_matrix(fn, out, rows, D, "out must have x's shape");
  const bool e4m3 = out.scalar_type() == at::kFloat8_e4m3fn;
  if (fp8 && !e4m3) fail(fn, VIT_E_UNSUPPORTED, "fp8 needs an e4m3 out");
  std::optional<at::Tensor> sc, h;
  if (sc_in) sc = *sc_in;
  if (e4m3 && !sc) sc = make({rows}, at::kFloat, x);
  if (sc) {
    need_vector(fn, *sc, rows, "scales must be a contiguous vector of a value per row");
    need_type(fn, *sc, at::kFloat, "scales must be fp32");
  }
  need_vector(fn, w, D, "weight must be a contiguous vector of D");
  int64_t r_ld = 0, h_ld = 0;
  vit_dtype r_type = VIT_DT_BF16;
  if (r) {
    h = h_in ? *h_in : make({rows, D}, r->scalar_type(), x);
    need_matrix(fn, *r, rows, D, "residual must have x's shape");
    need_matrix(fn, *h, rows, D, "residual_out must have x's shape");
    need_type(fn, *h, r->scalar_type(), "residual and residual_out must have one type");
    r_type = type_of(fn, *r);
    r_ld = leading(fn, *r);
    h_ld = leading(fn, *h);
  } else if (h_in) {
    fail(fn, VIT_E_INVALID_ARG, "residual_out without residual");
  }
  check(fn, vit_op_rms_norm(x.data_ptr(), type_of(fn, x), x_ld, ptr(r), r_ld, h ? h->data_ptr() : nullptr, h_ld, r_type,
                            w.data_ptr(), type_of(fn, w), static_cast<float>(eps), rows, int32_of(fn, D), out.data_ptr(),
                            type_of(fn, out), leading(fn, out), sc ? static_cast<float*>(sc->data_ptr()) : nullptr,
                            at.handle()));
  written(out_in);
  written(sc_in);
  written(h_in);
  return Py_BuildValue("(NNN)", out_in ? Py_NewRef(a[6]) : THPVariable_Wrap(out), sc_in ? Py_NewRef(a[7]) : wrap_or_none(sc),
                       r && h_in ? Py_NewRef(a[4]) : wrap_or_none(h));
  END_HANDLE_TH_ERRORS
}

// (x, out, scales, stream) -> (out, scales)
PyObject* quant_rows(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const char* fn = "quant_rows";
  need_args(n, 4);
  const at::Tensor& x = tensor(fn, a[0]);
  Opt out_in = tensor_or_none(fn, a[1]), sc_in = tensor_or_none(fn, a[2]);
  Place at(fn, a[3], {&x, out_in, sc_in});
  const int64_t x_ld = leading(fn, x), rows = x.size(0), D = x.size(1);
  const at::Tensor out = out_in ? *out_in : make({rows, D}, at::kFloat8_e4m3fn, x);
  const at::Tensor sc = sc_in ? *sc_in : make({rows}, at::kFloat, x);
  need_type(fn, out, at::kFloat8_e4m3fn, "out must be e4m3");
  need_matrix(fn, out, rows, D, "out must have x's shape");
  need_vector(fn, sc, rows, "scales must be a contiguous vector of a value per row");
  need_type(fn, sc, at::kFloat, "scales must be fp32");
  check(fn, vit_op_quant_rows(x.data_ptr(), type_of(fn, x), x_ld, rows, int32_of(fn, D), out.data_ptr(), leading(fn, out),
                              static_cast<float*>(sc.data_ptr()), at.handle()));
  written(out_in);
  written(sc_in);
  return Py_BuildValue("(NN)", out_in ? Py_NewRef(a[1]) : THPVariable_Wrap(out),
                       sc_in ? Py_NewRef(a[2]) : THPVariable_Wrap(sc));
  END_HANDLE_TH_ERRORS
}

int32_t* status_word(const char* fn, Opt status) {
  if (status == nullptr) return nullptr;
  need_vector(fn, *status, 1, "status must be a vector of one");
  need_type(fn, *status, at::kInt, "status must be int32");
  return static_cast<int32_t*>(status->data_ptr());
}

uint64_t wait_limit(const char* fn, PyObject* o) {
  const long long v = integer(o);
  if (v < 0) fail(fn, VIT_E_INVALID_ARG, "wait_ns must not be negative (every wait is bounded; 0: the default)");
  return static_cast<uint64_t>(v);
}

// (a, a_scales, w, w_scales, bias, out, status, stream, wait_ns) -> out
PyObject* linear_fp8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const char* fn = "linear_fp8";
  need_args(n, 9);
  const at::Tensor &x = tensor(fn, a[0]), &sx = tensor(fn, a[1]), &w = tensor(fn, a[2]), &sw = tensor(fn, a[3]);
  Opt bias = tensor_or_none(fn, a[4]), out_in = tensor_or_none(fn, a[5]), status = tensor_or_none(fn, a[6]);
  const uint64_t wait_ns = wait_limit(fn, a[8]);
  Place at(fn, a[7], {&x, &sx, &w, &sw, bias, out_in, status});
  const int64_t lda = leading(fn, x), ldw = leading(fn, w), M = x.size(0), K = x.size(1), N = w.size(0);
  need_type(fn, x, at::kFloat8_e4m3fn, "a must be e4m3");
  need_type(fn, w, at::kFloat8_e4m3fn, "w must be e4m3");
  if (w.size(1) != K) fail(fn, VIT_E_SHAPE, "a and w differ in K");
  need_vector(fn, sx, M, "a_scales must be a contiguous vector of a value per row of a");
  need_vector(fn, sw, N, "w_scales must be a contiguous vector of a value per row of w");
  need_type(fn, sx, at::kFloat, "scales must be fp32");
  need_type(fn, sw, at::kFloat, "scales must be fp32");
  if (bias) {
    need_vector(fn, *bias, N, "bias must be a contiguous vector of N");
    need_type(fn, *bias, at::kFloat, "bias must be fp32");
  }
  const at::Tensor out = out_in ? *out_in : make({M, N}, at::kBFloat16, x);
  need_type(fn, out, at::kBFloat16, "out must be bf16");
  need_matrix(fn, out, M, N, "out must be [M, N]");
  check(fn, vit_op_linear_fp8(x.data_ptr(), lda, static_cast<const float*>(sx.data_ptr()), w.data_ptr(), ldw,
                              static_cast<const float*>(sw.data_ptr()), static_cast<const float*>(ptr(bias)),
                              int32_of(fn, M), int32_of(fn, N), int32_of(fn, K), out.data_ptr(), leading(fn, out),
                              status_word(fn, status), wait_ns, at.handle()));
  written(out_in);
  return out_in ? Py_NewRef(a[5]) : THPVariable_Wrap(out);
  END_HANDLE_TH_ERRORS
}

vit_rope_tensor rope_tensor(const char* fn, const at::Tensor& x, const at::Tensor& y, int64_t T) {
  if (x.dim() != 3 || x.size(0) != T || y.sizes() != x.sizes() || y.scalar_type() != x.scalar_type())
    fail(fn, VIT_E_SHAPE, "q, k and their outputs must be [T, heads, head_dim] of one type");
  if (x.size(2) > 1 && (x.stride(2) != 1 || y.stride(2) != 1))
    fail(fn, VIT_E_INVALID_ARG, "heads must be contiguous in their last dimension");
  const bool one = T == 1, single = x.size(1) == 1;  // the stride of a dimension of one says nothing
  return {x.data_ptr(), y.data_ptr(), one ? 0 : x.stride(0), single ? 0 : x.stride(1), one ? 0 : y.stride(0),
          single ? 0 : y.stride(1), int32_of(fn, x.size(1))};
}

// (q, k, positions, freqs, layout, gain, inverse, q_out, k_out, stream) -> (q_out, k_out)
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const char* fn = "rope";
  need_args(n, 10);
  const at::Tensor &q = tensor(fn, a[0]), &pos = tensor(fn, a[2]), &f = tensor(fn, a[3]);
  Opt k = tensor_or_none(fn, a[1]), qo_in = tensor_or_none(fn, a[7]), ko_in = tensor_or_none(fn, a[8]);
  const int32_t layout = int32_of(fn, integer(a[4]));
  const double gain = number(a[5]);
  const bool inverse = truth(a[6]);
  need_no_history(fn, &f);
  Place at(fn, a[9], {&q, k, &pos, qo_in, ko_in});
  if (q.dim() != 3) fail(fn, VIT_E_SHAPE, "q must be [T, heads, head_dim]");
  const int64_t T = q.size(0), d = q.size(2);
  const at::Tensor qo = qo_in ? *qo_in : make(q.sizes(), q.scalar_type(), q);
  std::optional<at::Tensor> ko;
  if (k) {
    if (k->dim() != 3 || k->size(2) != d || k->scalar_type() != q.scalar_type())
      fail(fn, VIT_E_SHAPE, "k must have q's type and head_dim");
    ko = ko_in ? *ko_in : make(k->sizes(), k->scalar_type(), *k);
  } else if (ko_in) {
    fail(fn, VIT_E_INVALID_ARG, "an output for k without k");
  }
  if (pos.scalar_type() != at::kInt && pos.scalar_type() != at::kLong)
    fail(fn, VIT_E_UNSUPPORTED, "positions must be int32 or int64");
  if (pos.dim() < 1 || pos.dim() > 2 || pos.size(-1) != T || !pos.is_contiguous())
    fail(fn, VIT_E_SHAPE, "positions must be contiguous [T] or [axes, T]");
  const int64_t axes = pos.dim() == 1 ? 1 : pos.size(0);
  if (!f.is_cpu() || f.scalar_type() != at::kDouble || f.dim() != 1 || !f.is_contiguous())
    fail(fn, VIT_E_INVALID_ARG, "freqs must be a contiguous CPU float64 vector");
  const vit_rope_tensor tq = rope_tensor(fn, q, qo, T);
  vit_rope_tensor tk{};
  if (k) tk = rope_tensor(fn, *k, *ko, T);
  check(fn, vit_op_rope(&tq, k ? &tk : nullptr, type_of(fn, q), T, int32_of(fn, d), int32_of(fn, 2 * f.size(0)),
                        pos.data_ptr(), pos.scalar_type() == at::kLong ? 1 : 0, int32_of(fn, axes),
                        static_cast<const double*>(f.data_ptr()), layout, static_cast<float>(gain), inverse ? 1 : 0,
                        at.handle()));
  written(qo_in);
  written(ko_in);
  return Py_BuildValue("(NN)", qo_in ? Py_NewRef(a[7]) : THPVariable_Wrap(qo), k && ko_in ? Py_NewRef(a[8]) : wrap_or_none(ko));
  END_HANDLE_TH_ERRORS
}

// (q, k, v, cu_q, cu_k, len_k, causal, scale, max_q, out, status, stream, wait_ns) -> out
PyObject* attention_packed(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  const char* fn = "attention_packed";
  need_args(n, 13);
  const at::Tensor &q = tensor(fn, a[0]), &k = tensor(fn, a[1]), &v = tensor(fn, a[2]), &cu_q = tensor(fn, a[3]),
                   &cu_k = tensor(fn, a[4]);
  Opt len_k = tensor_or_none(fn, a[5]), out_in = tensor_or_none(fn, a[9]), status = tensor_or_none(fn, a[10]);
  const bool causal = truth(a[6]);
  const uint64_t wait_ns = wait_limit(fn, a[12]);
  Place at(fn, a[11], {&q, &k, &v, &cu_q, &cu_k, len_k, out_in, status});
  if (q.dim() != 3 || k.dim() != 3 || v.sizes() != k.sizes() || q.size(2) != k.size(2))
    fail(fn, VIT_E_SHAPE, "q must be [Tq, heads_q, d], k and v [Tk, heads_k, d]");
  if (k.scalar_type() != q.scalar_type() || v.scalar_type() != q.scalar_type())
    fail(fn, VIT_E_UNSUPPORTED, "q, k and v must have one type");
  const at::Tensor out = out_in ? *out_in : make(q.sizes(), q.scalar_type(), q);
  if (out.sizes() != q.sizes() || out.scalar_type() != q.scalar_type())
    fail(fn, VIT_E_SHAPE, "out must have q's shape and type");
  if (cu_q.dim() != 1 || cu_q.size(0) < 1) fail(fn, VIT_E_SHAPE, "cu_q must be a vector of n + 1");
  const int64_t seqs = cu_q.size(0) - 1;
  need_vector(fn, cu_q, seqs + 1, "cu_q must be a contiguous vector of n + 1");
  need_vector(fn, cu_k, seqs + 1, "cu_k must be a contiguous vector of n + 1");
  need_type(fn, cu_q, at::kInt, "cu_q must be int32");
  need_type(fn, cu_k, at::kInt, "cu_k must be int32");
  if (len_k) {
    need_vector(fn, *len_k, seqs, "len_k must be a contiguous vector of n");
    need_type(fn, *len_k, at::kInt, "len_k must be int32");
  }
  const int64_t Tq = q.size(0), Tk = k.size(0), Hq = q.size(1), Hk = k.size(1), d = q.size(2);
  for (const at::Tensor* t : {&q, &k, &v, &out})
    if (d > 1 && t->stride(2) != 1) fail(fn, VIT_E_INVALID_ARG, "heads must be contiguous in their last dimension");
  auto token = [](const at::Tensor& t) { return t.size(0) == 1 ? int64_t{0} : t.stride(0); };
  auto head = [](const at::Tensor& t) { return t.size(1) == 1 ? int64_t{0} : t.stride(1); };
  vit_attn_packed p{};
  p.q = q.data_ptr();
  p.k = k.data_ptr();
  p.v = v.data_ptr();
  p.out = out.data_ptr();
  p.q_token = token(q);
  p.q_head = head(q);
  p.k_token = token(k);
  p.k_head = head(k);
  p.v_token = token(v);
  p.v_head = head(v);
  p.out_token = token(out);
  p.out_head = head(out);
  p.cu_q = static_cast<const int32_t*>(cu_q.data_ptr());
  p.cu_k = static_cast<const int32_t*>(cu_k.data_ptr());
  p.len_k = static_cast<const int32_t*>(ptr(len_k));
  p.Tq = Tq;
  p.Tk = Tk;
  p.n = int32_of(fn, seqs);
  p.heads_q = int32_of(fn, Hq);
  p.heads_k = int32_of(fn, Hk);
  p.head_dim = int32_of(fn, d);
  p.type = type_of(fn, q);
  p.causal = causal ? 1 : 0;
  p.max_q = int32_of(fn, integer(a[8]));
  p.scale = a[7] == Py_None ? (d > 0 ? 1.0f / std::sqrt(static_cast<float>(d)) : 0.f) : static_cast<float>(number(a[7]));
  p.status = status_word(fn, status);
  p.wait_ns = wait_ns;
  size_t need = 0;
  check(fn, vit_op_attention_packed_workspace(&p, &need));
  at::Tensor ws;
  if (need > 0) {
    ws = make({static_cast<int64_t>(need)}, at::kByte, q);
    p.workspace = ws.data_ptr();
    p.workspace_bytes = need;
  }
  check(fn, vit_op_attention_packed(&p, at.handle()));
  written(out_in);
  return out_in ? Py_NewRef(a[9]) : THPVariable_Wrap(out);
  END_HANDLE_TH_ERRORS
}

PyObject* set_error(PyObject*, PyObject* cls) {
  Py_XDECREF(g_error);
  g_error = Py_NewRef(cls);
  Py_RETURN_NONE;
}

template <typename F>
PyCFunction fast(F f) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)); }

PyMethodDef g_methods[] = {{"set_error", set_error, METH_O, nullptr},
                           {"rms_norm", fast(rms_norm), METH_FASTCALL, nullptr},
                           {"quant_rows", fast(quant_rows), METH_FASTCALL, nullptr},
                           {"linear_fp8", fast(linear_fp8), METH_FASTCALL, nullptr},
                           {"rope", fast(rope), METH_FASTCALL, nullptr},
                           {"attention_packed", fast(attention_packed), METH_FASTCALL, nullptr},
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_vit_ops", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__vit_ops() {
  PyObject* m = PyModule_Create(&g_module);
  if (m != nullptr && PyModule_AddStringConstant(m, "torch_version", VIT_TORCH_VERSION) < 0) Py_CLEAR(m);
  return m;
}
