// Compiled half of the Python binding for the fp8 block-scaled and 4-bit floating
// point layers and the grouped router: checks the tensors, allocates outputs and workspace that were not
// passed in, and calls the C entry points. A decode call's kernels take 5 to 15 us
// on a GB300; the same checks and allocations in Python took 10 to 18 us on its
// Grace host, and take 1 to 3 us here. Each function has the arguments of the
// Python function of the package that calls it, streams as handles (or None: the
// current stream of the tensors' device); wrong tensors raise ValueError before
// the library is called, a status other than W4_OK raises W4Error. What a call
// allocates belongs to its stream.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <cstdio>
#include <initializer_list>
#include <string>

#include "w4.h"

namespace {

using at::ScalarType;
using Types = std::initializer_list<ScalarType>;

const Types kFp8 = {ScalarType::Float8_e4m3fn, ScalarType::Byte};
const Types kBf16 = {ScalarType::BFloat16};
const Types kF32 = {ScalarType::Float};
const Types kI32 = {ScalarType::Int};
const Types kAct = {ScalarType::BFloat16, ScalarType::Half};
const Types kHalf = {ScalarType::Half};
const Types kByte = {ScalarType::Byte};
const Types kScaleMx = {ScalarType::Float8_e8m0fnu, ScalarType::Byte};
const Types kScaleNv = {ScalarType::Float8_e4m3fn, ScalarType::Byte};
const Types kLogit = {ScalarType::BFloat16, ScalarType::Float};

[[noreturn]] void value_error(const char* fmt, ...) {
  char text[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(text, sizeof(text), fmt, ap);
  va_end(ap);
  PyErr_SetString(PyExc_ValueError, text);
  throw python_error();   // keeps the error that is set
}

std::string shape_text(at::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + ")";
}

// `o` as a contiguous CUDA tensor of one of `types`, on `dev` when given.
const at::Tensor& tensor(PyObject* o, const char* name, const Types& types, const at::Device* dev) {
  if (o == Py_None) value_error("%s is required", name);
  if (!THPVariable_Check(o)) value_error("%s must be a contiguous CUDA tensor", name);
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda() || !t.is_contiguous()) value_error("%s must be a contiguous CUDA tensor", name);
  if (dev != nullptr && t.device() != *dev)
    value_error("%s is on %s, the call runs on %s", name, t.device().str().c_str(), dev->str().c_str());
  for (ScalarType s : types)
    if (t.scalar_type() == s) return t;
  value_error("%s has dtype %s, which the call does not take", name, c10::toString(t.scalar_type()));
}

const at::Tensor& tensor(PyObject* o, const char* name, const Types& types, const at::Device& dev, at::IntArrayRef shape) {
  const at::Tensor& t = tensor(o, name, types, &dev);
  if (t.sizes() != shape)
    value_error("%s must have shape %s, got %s", name, shape_text(shape).c_str(),
                            shape_text(t.sizes()).c_str());
  return t;
}

const at::Tensor& ranked(PyObject* o, const char* name, const Types& types, const at::Device* dev, int64_t dim) {
  const at::Tensor& t = tensor(o, name, types, dev);
  if (t.dim() != dim) value_error("%s must be a contiguous %d-D CUDA tensor", name, static_cast<int>(dim));
  return t;
}

// The stream of a call: the `stream` argument (a handle), or the current one of `dev`
// for None. For as long as this lives `dev` is the current device and, where the two
// streams differ, the call's is the current stream: memory allocated here belongs to
// the stream that the kernels run on, so it is neither still in use by other work when
// they write it nor handed to other work while they read it.
class CallStream {
 public:
  CallStream(PyObject* o, const at::Device& dev) : device_(dev), caller_(c10::cuda::getCurrentCUDAStream(dev.index())) {
    handle_ = caller_.stream();
    if (o == Py_None) return;
    cudaStream_t s = static_cast<cudaStream_t>(PyLong_AsVoidPtr(o));
    if (s == nullptr && PyErr_Occurred()) throw python_error();
    if (s == handle_) return;
    handle_ = s;
    stream_.reset_stream(c10::cuda::getStreamFromExternal(s, dev.index()));
  }
  cudaStream_t handle() const { return handle_; }
  // Outputs are read on the caller's stream too (once it has waited): released there,
  // they are not handed out again before that stream is done with them.
  void keep_for_caller(const at::Tensor& t) const {
    if (handle_ != caller_.stream() && t.nbytes() > 0)
      c10::cuda::CUDACachingAllocator::recordStream(t.storage().data_ptr(), caller_);
  }

 private:
  c10::cuda::CUDAGuard device_;
  c10::cuda::OptionalCUDAStreamGuard stream_;
  c10::cuda::CUDAStream caller_;
  cudaStream_t handle_;
};

at::Tensor empty(at::IntArrayRef shape, ScalarType type, const at::Device& dev) {
  return at::detail::empty_cuda(shape, type, dev, std::nullopt);
}

// `shape` of a 4-byte type at 4-byte word `at` of `base`'s storage: a view made
// directly (through the dispatcher it costs what an allocation does).
at::Tensor words_of(const at::Tensor& base, int64_t at, at::IntArrayRef shape, ScalarType type) {
  at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(base.storage()), base.key_set(),
                                                          c10::scalarTypeToTypeMeta(type));
  t.unsafeGetTensorImpl()->set_storage_offset(at);
  t.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
  return t;
}

at::Tensor output(PyObject* o, const char* name, at::IntArrayRef shape, ScalarType type, const Types& types,
                  const at::Device& dev, const CallStream& stream) {
  if (o != Py_None) return tensor(o, name, types, dev, shape);
  at::Tensor t = empty(shape, type, dev);
  stream.keep_for_caller(t);
  return t;
}

struct Scratch {
  at::Tensor t;
  void* p = nullptr;
  size_t bytes = 0;
};
// Allocated, where none is given, while the call's CallStream lives.
Scratch scratch(PyObject* o, int32_t op, int64_t M, int64_t N, int64_t K, int32_t group, const at::Device& dev) {
  Scratch s;
  if (o == Py_None) {
    s.bytes = w4_workspace_bytes(op, M, N, K, group);
    if (s.bytes == 0) return s;
    s.t = empty({static_cast<int64_t>(s.bytes)}, ScalarType::Byte, dev);
  } else {
    if (!THPVariable_Check(o)) value_error("workspace must be a contiguous CUDA tensor");
    s.t = THPVariable_Unpack(o);
    if (!s.t.is_cuda() || !s.t.is_contiguous() || s.t.device() != dev)
      value_error("workspace must be a contiguous CUDA tensor on the call's device");
    s.bytes = s.t.nbytes();   // the library checks it
  }
  s.p = s.t.data_ptr();
  return s;
}

int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw python_error();
  return v;
}
int32_t integer32(PyObject* o, const char* name) {
  const int64_t v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX) value_error("%s is out of range", name);
  return static_cast<int32_t>(v);
}

int64_t blocks(int64_t n) { return (n + 127) / 128; }
int32_t act_dtype(const at::Tensor& x) { return x.scalar_type() == ScalarType::Half ? W4_FP16 : W4_BF16; }
const float* f32(const at::Tensor& t) { return static_cast<const float*>(t.data_ptr()); }
int32_t* i32(const at::Tensor& t) { return static_cast<int32_t*>(t.data_ptr()); }

// nullptr with W4Error set unless `st` is W4_OK.
bool failed(w4_status st, const char* what) {
  if (st == W4_OK) return false;
  PyObject* m = PyImport_ImportModule("int4_weight_quantized_w4_gb300");
  if (m != nullptr) {
    PyObject* r = PyObject_CallMethod(m, "_check", "is", static_cast<int>(st), what);
    Py_XDECREF(r);
    Py_DECREF(m);
  }
  if (!PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, what);
  return true;
}

bool count(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
  return false;
}

// e4m3 [N, K], fp32 [ceil(N / 128), ceil(K / 128)] and bf16 [N] or None; N.
int64_t dense_weights(PyObject* w, PyObject* ws, PyObject* bias, int64_t K, const at::Device& dev) {
  const at::Tensor& q = ranked(w, "qweight", kFp8, &dev, 2);
  const int64_t N = q.size(0);
  if (q.size(1) != K) value_error("qweight must have the %lld columns of the activations", (long long)K);
  tensor(ws, "w_scale", kF32, dev, {blocks(N), blocks(K)});
  if (bias != Py_None) tensor(bias, "bias", kBf16, dev, {N});
  return N;
}
// The same per expert, and int32 offsets [E + 1]; N.
int64_t expert_weights(PyObject* w, PyObject* ws, PyObject* offsets, int64_t K, const at::Device& dev) {
  const at::Tensor& q = ranked(w, "qweight", kFp8, &dev, 3);
  const int64_t E = q.size(0), N = q.size(1);
  if (q.size(2) != K) value_error("qweight must have the %lld columns of the activations", (long long)K);
  if (E > INT32_MAX - 1) value_error("too many experts");
  tensor(ws, "w_scale", kF32, dev, {E, blocks(N), blocks(K)});
  tensor(offsets, "expert_offsets", kI32, dev, {E + 1});
  return N;
}
void* data(PyObject* o) { return o == Py_None ? nullptr : THPVariable_Unpack(o).data_ptr(); }

PyObject* pair(const at::Tensor& a, const at::Tensor& b) {
  PyObject* t = PyTuple_New(2);
  if (t == nullptr) return nullptr;
  PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(a));
  PyTuple_SET_ITEM(t, 1, THPVariable_Wrap(b));
  return t;
}

// logits, top_k, bias, n_group, topk_group, scoring, renormalize, scale, out, workspace, stream
PyObject* route_grouped(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count(n, 11)) return nullptr;
  const at::Tensor& x = ranked(a[0], "logits", kLogit, nullptr, 2);
  const at::Device dev = x.device();
  const int64_t T = x.size(0), E = x.size(1);
  const int32_t k = integer32(a[1], "top_k"), groups = integer32(a[3], "n_group"), keep = integer32(a[4], "topk_group");
  if (E > INT32_MAX - 1) value_error("too many experts");
  if (k < 0) value_error("top_k must not be negative");
  const double scale = PyFloat_AsDouble(a[7]);
  if (scale == -1.0 && PyErr_Occurred()) return nullptr;
  if (a[2] != Py_None) tensor(a[2], "bias", kF32, dev, {E});
  const CallStream stream(a[10], dev);
  at::Tensor o[5];
  const char* names[5] = {"topk_ids", "topk_weights", "offsets", "row_token", "row_of"};
  if (a[8] != Py_None && (!PyTuple_Check(a[8]) || PyTuple_GET_SIZE(a[8]) != 5))
    value_error("out must be the tuple (topk_ids, topk_weights, offsets, row_token, row_of)");
  // the five outputs share one allocation when none are given; a top_k that the library
  // refuses asks for no memory first
  const int64_t n_out = a[8] == Py_None && (k > E || k > 64) ? 0 : k;
  const int64_t starts[5] = {0, T * n_out, 4 * T * n_out, 2 * T * n_out, 3 * T * n_out};
  at::Tensor all;
  if (a[8] == Py_None) {
    all = empty({4 * T * n_out + E + 1}, ScalarType::Int, dev);
    stream.keep_for_caller(all);
  }
  for (int i = 0; i < 5; ++i) {
    const at::DimVector shape = i == 2   ? at::DimVector{E + 1}
                                : i == 3 ? at::DimVector{T * n_out}
                                         : at::DimVector{T, n_out};
    const ScalarType type = i == 1 ? ScalarType::Float : ScalarType::Int;
    if (a[8] == Py_None)
      o[i] = words_of(all, starts[i], shape, type);
    else
      o[i] = tensor(PyTuple_GET_ITEM(a[8], i), names[i], i == 1 ? kF32 : kI32, dev, shape);
  }
  const Scratch s = scratch(a[9], W4_OP_MOE_ROUTE_GROUPED, T, E, 1, 0, dev);
  if (failed(w4_moe_route_grouped(x.data_ptr(), x.scalar_type() == ScalarType::Float, static_cast<float*>(data(a[2])), T,
                                  static_cast<int32_t>(E), k, groups, keep, integer32(a[5], "scoring"),
                                  PyObject_IsTrue(a[6]), static_cast<float>(scale), i32(o[0]),
                                  static_cast<float*>(o[1].data_ptr()), i32(o[2]), i32(o[3]), i32(o[4]), s.p, s.bytes,
                                  stream.handle()),
             "w4_moe_route_grouped"))
    return nullptr;
  if (T == 0) o[2].zero_();   // the library writes nothing
  if (a[8] != Py_None) {
    Py_INCREF(a[8]);
    return a[8];
  }
  PyObject* t = PyTuple_New(5);
  if (t == nullptr) return nullptr;
  for (int i = 0; i < 5; ++i) PyTuple_SET_ITEM(t, i, THPVariable_Wrap(o[i]));
  return t;
  END_HANDLE_TH_ERRORS
}

// x, q, scale, stream
PyObject* quant_block(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count(n, 4)) return nullptr;
  const at::Tensor& x = ranked(a[0], "x", kAct, nullptr, 2);
  const at::Device dev = x.device();
  const int64_t M = x.size(0), K = x.size(1);
  const CallStream stream(a[3], dev);
  const at::Tensor q = output(a[1], "q", {M, K}, ScalarType::Float8_e4m3fn, kFp8, dev, stream);
  const at::Tensor s = output(a[2], "scale", {M, blocks(K)}, ScalarType::Float, kF32, dev, stream);
  if (failed(w4_quant_act_per_block(x.data_ptr(), act_dtype(x), M, K, q.data_ptr(), static_cast<float*>(s.data_ptr()),
                                    stream.handle()),
             "w4_quant_act_per_block"))
    return nullptr;
  return pair(q, s);
  END_HANDLE_TH_ERRORS
}

// h, q, scale, stream
PyObject* silu_mul_quant_block(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count(n, 4)) return nullptr;
  const at::Tensor& h = ranked(a[0], "h", kBf16, nullptr, 2);
  const at::Device dev = h.device();
  if (h.size(1) % 2) value_error("h must hold gate and up halves of equal width");
  const int64_t R = h.size(0), I = h.size(1) / 2;
  const CallStream stream(a[3], dev);
  const at::Tensor q = output(a[1], "q", {R, I}, ScalarType::Float8_e4m3fn, kFp8, dev, stream);
  const at::Tensor s = output(a[2], "scale", {R, blocks(I)}, ScalarType::Float, kF32, dev, stream);
  if (failed(w4_silu_mul_quant_block(h.data_ptr(), R, I, q.data_ptr(), static_cast<float*>(s.data_ptr()),
                                     stream.handle()),
             "w4_silu_mul_quant_block"))
    return nullptr;
  return pair(q, s);
  END_HANDLE_TH_ERRORS
}

// qx, x_scale, qweight, w_scale, bias, y, workspace, stream
PyObject* gemm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count(n, 8)) return nullptr;
  const at::Tensor& x = ranked(a[0], "qx", kFp8, nullptr, 2);
  const at::Device dev = x.device();
  const int64_t M = x.size(0), K = x.size(1), N = dense_weights(a[2], a[3], a[4], K, dev);
  const at::Tensor& xs = tensor(a[1], "x_scale", kF32, dev, {M, blocks(K)});
  const CallStream stream(a[7], dev);
  const at::Tensor y = output(a[5], "y", {M, N}, ScalarType::BFloat16, kBf16, dev, stream);
  const Scratch s = scratch(a[6], W4_OP_FP8_BLOCK, M, N, K, 0, dev);
  if (failed(w4_fp8_block_gemm(x.data_ptr(), f32(xs), data(a[2]), static_cast<const float*>(data(a[3])), data(a[4]),
                               y.data_ptr(), M, N, K, s.p, s.bytes, stream.handle()),
             "w4_fp8_block_gemm"))
    return nullptr;
  return THPVariable_Wrap(y);
  END_HANDLE_TH_ERRORS
}

// x, qweight, w_scale, bias, y, workspace, stream
PyObject* gemm_act(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count(n, 7)) return nullptr;
  const at::Tensor& x = ranked(a[0], "x", kAct, nullptr, 2);
  const at::Device dev = x.device();
  const int64_t M = x.size(0), K = x.size(1), N = dense_weights(a[1], a[2], a[3], K, dev);
  const CallStream stream(a[6], dev);
  const at::Tensor y = output(a[4], "y", {M, N}, ScalarType::BFloat16, kBf16, dev, stream);
  const Scratch s = scratch(a[5], W4_OP_FP8_BLOCK_IN, M, N, K, 0, dev);
  if (failed(w4_fp8_block_gemm_bf16in(x.data_ptr(), act_dtype(x), data(a[1]), static_cast<const float*>(data(a[2])),
                                      data(a[3]), y.data_ptr(), M, N, K, s.p, s.bytes, stream.handle()),
             "w4_fp8_block_gemm_bf16in"))
    return nullptr;
  return THPVariable_Wrap(y);
  END_HANDLE_TH_ERRORS
}

// qx, x_scale, expert_offsets, qweight, w_scale, y, stream
PyObject* moe_gemm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count(n, 7)) return nullptr;
  const at::Tensor& x = ranked(a[0], "qx", kFp8, nullptr, 2);
  const at::Device dev = x.device();
  const int64_t R = x.size(0), K = x.size(1), N = expert_weights(a[3], a[4], a[2], K, dev);
  const at::Tensor& xs = tensor(a[1], "x_scale", kF32, dev, {R, blocks(K)});
  const CallStream stream(a[6], dev);
  const at::Tensor y = output(a[5], "y", {R, N}, ScalarType::BFloat16, kBf16, dev, stream);
  if (failed(w4_fp8_block_moe_grouped_gemm(x.data_ptr(), f32(xs), static_cast<const int32_t*>(data(a[2])),
                                           static_cast<int32_t>(THPVariable_Unpack(a[3]).size(0)), data(a[3]),
                                           static_cast<const float*>(data(a[4])), y.data_ptr(), R, N, K,
                                           stream.handle()),
             "w4_fp8_block_moe_grouped_gemm"))
    return nullptr;
  return THPVariable_Wrap(y);
  END_HANDLE_TH_ERRORS
}

// x, row_token, expert_offsets, qweight, w_scale, y, workspace, stream
PyObject* moe_gemm_act(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count(n, 8)) return nullptr;
  const at::Tensor& x = ranked(a[0], "x", kBf16, nullptr, 2);
  const at::Device dev = x.device();
  const int64_t T = x.size(0), K = x.size(1), N = expert_weights(a[3], a[4], a[2], K, dev);
  const int64_t R = a[1] == Py_None ? T : tensor(a[1], "row_token", kI32, &dev).numel();
  const int32_t E = static_cast<int32_t>(THPVariable_Unpack(a[3]).size(0));
  const CallStream stream(a[7], dev);
  const at::Tensor y = output(a[5], "y", {R, N}, ScalarType::BFloat16, kBf16, dev, stream);
  const Scratch s = scratch(a[6], W4_OP_FP8_BLOCK_IN, R, N, K, E, dev);
  if (failed(w4_fp8_block_moe_gemm_bf16in(x.data_ptr(), T, static_cast<const int32_t*>(data(a[1])),
                                          static_cast<const int32_t*>(data(a[2])), E, data(a[3]),
                                          static_cast<const float*>(data(a[4])), y.data_ptr(), R, N, K, s.p, s.bytes,
                                          stream.handle()),
             "w4_fp8_block_moe_gemm_bf16in"))
    return nullptr;
  return THPVariable_Wrap(y);
  END_HANDLE_TH_ERRORS
}

// ---- 4-bit floating point ----

// W4_FMT_MXFP4 or W4_FMT_NVFP4, as the Python side checked it.
struct Format {
  int32_t id;
  int64_t block;
  const Types& scales;
  ScalarType scale;
};
Format format(PyObject* o) {
  const bool nv = integer(o) == W4_FMT_NVFP4;
  return {nv ? W4_FMT_NVFP4 : W4_FMT_MXFP4, nv ? 16 : 32, nv ? kScaleNv : kScaleMx, nv ? ScalarType::Float8_e4m3fn : ScalarType::Float8_e8m0fnu};
}
const float* global_scale(PyObject* o, const char* name, int64_t n, const at::Device& dev) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, name, kF32, &dev);
  if (t.numel() != n) value_error("%s must have %lld element(s), got %lld", name, (long long)n, (long long)t.numel());
  return f32(t);
}
// Packed [.., N, K / 2] with [.., N, K / block] scales: N.
int64_t fp4_weights(PyObject* w, PyObject* ws, int64_t dim, int64_t K, const Format& f, const at::Device& dev) {
  const at::Tensor& q = ranked(w, "qweight", kByte, &dev, dim);
  const int64_t N = q.size(dim - 2);
  if (2 * q.size(dim - 1) != K) value_error("qweight must hold the %lld columns of the activations, two in a byte", (long long)K);
  if (dim == 3) {
    if (q.size(0) > INT32_MAX - 1) value_error("too many experts");
    tensor(ws, "w_scale", f.scales, dev, {q.size(0), N, K / f.block});
  } else {
    tensor(ws, "w_scale", f.scales, dev, {N, K / f.block});
  }
  return N;
}

// x, format, global, q, scale, silu, stream
PyObject* quant_fp4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count(n, 7)) return nullptr;
  const bool silu = PyObject_IsTrue(a[5]);
  const at::Tensor& x = ranked(a[0], silu ? "h" : "x", silu ? kBf16 : kAct, nullptr, 2);
  const at::Device dev = x.device();
  if (silu && x.size(1) % 2) value_error("h must hold gate and up halves of equal width");
  const Format f = format(a[1]);
  const int64_t M = x.size(0), K = silu ? x.size(1) / 2 : x.size(1);
  const float* g = global_scale(a[2], "global_scale", 1, dev);
  const CallStream stream(a[6], dev);
  const at::Tensor q = output(a[3], "q", {M, K / 2}, ScalarType::Byte, kByte, dev, stream);
  const at::Tensor s = output(a[4], "scale", {M, K / f.block}, f.scale, f.scales, dev, stream);
  if (silu ? failed(w4_silu_mul_quant_fp4(x.data_ptr(), f.id, g, M, K, q.data_ptr(), s.data_ptr(), stream.handle()), "w4_silu_mul_quant_fp4")
           : failed(w4_quant_fp4(x.data_ptr(), act_dtype(x), f.id, g, M, K, q.data_ptr(), s.data_ptr(), stream.handle()), "w4_quant_fp4"))
    return nullptr;
  return pair(q, s);
  END_HANDLE_TH_ERRORS
}

// q, scale, format, global, fp16, out, stream
PyObject* dequant_fp4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count(n, 7)) return nullptr;
  const at::Tensor& q = ranked(a[0], "q", kByte, nullptr, 2);
  const at::Device dev = q.device();
  const Format f = format(a[2]);
  const int64_t M = q.size(0), K = 2 * q.size(1);
  const at::Tensor& s = tensor(a[1], "scale", f.scales, dev, {M, K / f.block});
  const float* g = global_scale(a[3], "global_scale", 1, dev);
  const bool half = PyObject_IsTrue(a[4]);
  const CallStream stream(a[6], dev);
  const ScalarType type = half ? ScalarType::Half : ScalarType::BFloat16;
  const at::Tensor o = output(a[5], "out", {M, K}, type, {type}, dev, stream);
  if (failed(w4_dequant_fp4(q.data_ptr(), s.data_ptr(), f.id, g, M, K, half ? W4_FP16 : W4_BF16, o.data_ptr(), stream.handle()),
             "w4_dequant_fp4"))
    return nullptr;
  return THPVariable_Wrap(o);
  END_HANDLE_TH_ERRORS
}

// qx, x_scale, qweight, w_scale, format, x_global, w_global, bias, y, stream
PyObject* fp4_gemm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count(n, 10)) return nullptr;
  const at::Tensor& x = ranked(a[0], "qx", kByte, nullptr, 2);
  const at::Device dev = x.device();
  const Format f = format(a[4]);
  const int64_t M = x.size(0), K = 2 * x.size(1), N = fp4_weights(a[2], a[3], 2, K, f, dev);
  const at::Tensor& xs = tensor(a[1], "x_scale", f.scales, dev, {M, K / f.block});
  const float* xg = global_scale(a[5], "x_global", 1, dev);
  const float* wg = global_scale(a[6], "w_global", 1, dev);
  if (a[7] != Py_None) tensor(a[7], "bias", kBf16, dev, {N});
  const CallStream stream(a[9], dev);
  const at::Tensor y = output(a[8], "y", {M, N}, ScalarType::BFloat16, kBf16, dev, stream);
  if (failed(w4_fp4_gemm(x.data_ptr(), xs.data_ptr(), xg, data(a[2]), data(a[3]), wg, f.id, data(a[7]), y.data_ptr(), M,
                         N, K, stream.handle()),
             "w4_fp4_gemm"))
    return nullptr;
  return THPVariable_Wrap(y);
  END_HANDLE_TH_ERRORS
}

// x, qweight, w_scale, format, x_global, w_global, bias, y, workspace, stream
PyObject* fp4_gemm_act(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count(n, 10)) return nullptr;
  const at::Tensor& x = ranked(a[0], "x", kAct, nullptr, 2);
  const at::Device dev = x.device();
  const Format f = format(a[3]);
  const int64_t M = x.size(0), K = x.size(1), N = fp4_weights(a[1], a[2], 2, K, f, dev);
  const float* xg = global_scale(a[4], "x_global", 1, dev);
  const float* wg = global_scale(a[5], "w_global", 1, dev);
  if (a[6] != Py_None) tensor(a[6], "bias", kBf16, dev, {N});
  const CallStream stream(a[9], dev);
  const at::Tensor y = output(a[7], "y", {M, N}, ScalarType::BFloat16, kBf16, dev, stream);
  const Scratch s = scratch(a[8], W4_OP_FP4_IN, M, N, K, static_cast<int32_t>(f.block), dev);
  if (failed(w4_fp4_gemm_bf16in(x.data_ptr(), act_dtype(x), xg, data(a[1]), data(a[2]), wg, f.id, data(a[6]),
                                y.data_ptr(), M, N, K, s.p, s.bytes, stream.handle()),
             "w4_fp4_gemm_bf16in"))
    return nullptr;
  return THPVariable_Wrap(y);
  END_HANDLE_TH_ERRORS
}

// qx, x_scale, expert_offsets, qweight, w_scale, format, x_global, w_global, y, stream
PyObject* fp4_moe_gemm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count(n, 10)) return nullptr;
  const at::Tensor& x = ranked(a[0], "qx", kByte, nullptr, 2);
  const at::Device dev = x.device();
  const Format f = format(a[5]);
  const int64_t R = x.size(0), K = 2 * x.size(1), N = fp4_weights(a[3], a[4], 3, K, f, dev);
  const int64_t E = THPVariable_Unpack(a[3]).size(0);
  const at::Tensor& xs = tensor(a[1], "x_scale", f.scales, dev, {R, K / f.block});
  tensor(a[2], "expert_offsets", kI32, dev, {E + 1});
  const float* xg = global_scale(a[6], "x_global", 1, dev);
  const float* wg = global_scale(a[7], "w_global", E, dev);
  const CallStream stream(a[9], dev);
  const at::Tensor y = output(a[8], "y", {R, N}, ScalarType::BFloat16, kBf16, dev, stream);
  if (failed(w4_fp4_moe_grouped_gemm(x.data_ptr(), xs.data_ptr(), xg, static_cast<const int32_t*>(data(a[2])),
                                     static_cast<int32_t>(E), data(a[3]), data(a[4]), wg, f.id, y.data_ptr(), R, N, K,
                                     stream.handle()),
             "w4_fp4_moe_grouped_gemm"))
    return nullptr;
  return THPVariable_Wrap(y);
  END_HANDLE_TH_ERRORS
}

// x, row_token, expert_offsets, qweight, w_scale, format, x_global, w_global, y, workspace, stream
PyObject* fp4_moe_gemm_act(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count(n, 11)) return nullptr;
  const at::Tensor& x = ranked(a[0], "x", kBf16, nullptr, 2);
  const at::Device dev = x.device();
  const Format f = format(a[5]);
  const int64_t T = x.size(0), K = x.size(1), N = fp4_weights(a[3], a[4], 3, K, f, dev);
  const int64_t E = THPVariable_Unpack(a[3]).size(0);
  tensor(a[2], "expert_offsets", kI32, dev, {E + 1});
  const int64_t R = a[1] == Py_None ? T : tensor(a[1], "row_token", kI32, &dev).numel();
  const float* xg = global_scale(a[6], "x_global", 1, dev);
  const float* wg = global_scale(a[7], "w_global", E, dev);
  const CallStream stream(a[10], dev);
  const at::Tensor y = output(a[8], "y", {R, N}, ScalarType::BFloat16, kBf16, dev, stream);
  const Scratch s = scratch(a[9], W4_OP_FP4_MOE_IN, R, N, K, static_cast<int32_t>(f.block), dev);
  if (failed(w4_fp4_moe_gemm_bf16in(x.data_ptr(), T, xg, static_cast<const int32_t*>(data(a[1])),
                                    static_cast<const int32_t*>(data(a[2])), static_cast<int32_t>(E), data(a[3]),
                                    data(a[4]), wg, f.id, y.data_ptr(), R, N, K, s.p, s.bytes, stream.handle()),
             "w4_fp4_moe_gemm_bf16in"))
    return nullptr;
  return THPVariable_Wrap(y);
  END_HANDLE_TH_ERRORS
}

// x, logits, gate_up, gate_up_scale, down, down_scale, top_k, format, gate_up_global, down_global, bias, n_group,
// topk_group, scoring, renormalize, scale, y, workspace, stream
PyObject* moe_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (!count(n, 19)) return nullptr;
  const at::Tensor& x = ranked(a[0], "x", kBf16, nullptr, 2);
  const at::Device dev = x.device();
  const at::Tensor& logits = ranked(a[1], "logits", kLogit, &dev, 2);
  const int64_t T = x.size(0), H = x.size(1), E = logits.size(1);
  if (logits.size(0) != T) value_error("logits must have the %lld tokens of x", (long long)T);
  if (E > INT32_MAX - 1) value_error("too many experts");
  const int32_t k = integer32(a[6], "top_k"), fmt = integer32(a[7], "format");
  const bool int4 = fmt == W4_FMT_INT4;
  const int64_t per = int4 ? 8 : 2;   // columns in an element of the codes
  const Types& codes = int4 ? kI32 : kByte;
  const Types& scales = int4 ? kHalf : fmt == W4_FMT_NVFP4 ? kScaleNv : kScaleMx;
  const at::Tensor& up = ranked(a[2], "gate_up", codes, &dev, 3);
  if (up.size(0) != E || up.size(1) % 2 || up.size(2) * per != H) value_error("gate_up must hold E matrices of 2I rows of H columns");
  const int64_t I = up.size(1) / 2;
  const at::Tensor& down = tensor(a[4], "down", codes, dev, {E, H, I / per});
  const at::Tensor& us = ranked(a[3], "gate_up_scale", scales, &dev, 3);
  const at::Tensor& ds = ranked(a[5], "down_scale", scales, &dev, 3);
  const int64_t block = int4 ? 0 : fmt == W4_FMT_NVFP4 ? 16 : 32;
  auto group = [&](const at::Tensor& s, const char* name, int64_t rows, int64_t K) -> int32_t {
    const int64_t G = s.size(2);
    if (s.size(0) != E || s.size(1) != rows || G < 1 || (block ? G * block != K : K % G != 0))
      value_error("%s does not match the weights: shape %s", name, shape_text(s.sizes()).c_str());
    return static_cast<int32_t>(K / G);
  };
  const int32_t ug = group(us, "gate_up_scale", 2 * I, H), dg = group(ds, "down_scale", H, I);
  const float* gu = global_scale(a[8], "gate_up_global", E, dev);
  const float* gd = global_scale(a[9], "down_global", E, dev);
  if (a[10] != Py_None) tensor(a[10], "bias", kF32, dev, {E});
  const double scale = PyFloat_AsDouble(a[15]);
  if (scale == -1.0 && PyErr_Occurred()) return nullptr;
  const CallStream stream(a[18], dev);
  const at::Tensor y = output(a[16], "y", {T, H}, ScalarType::BFloat16, kBf16, dev, stream);
  const Scratch s = scratch(a[17], W4_OP_MOE_DECODE, T, k, I, 0, dev);
  if (failed(w4_moe_decode(x.data_ptr(), logits.data_ptr(), logits.scalar_type() == ScalarType::Float,
                           static_cast<const float*>(data(a[10])), T, static_cast<int32_t>(E), k,
                           integer32(a[11], "n_group"), integer32(a[12], "topk_group"), integer32(a[13], "scoring"),
                           PyObject_IsTrue(a[14]), static_cast<float>(scale), fmt, up.data_ptr(), us.data_ptr(), gu, ug,
                           down.data_ptr(), ds.data_ptr(), gd, dg, y.data_ptr(), H, I, s.p, s.bytes, stream.handle()),
             "w4_moe_decode"))
    return nullptr;
  return THPVariable_Wrap(y);
  END_HANDLE_TH_ERRORS
}

#define W4_METHOD(f) {#f, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {W4_METHOD(route_grouped), W4_METHOD(quant_block), W4_METHOD(silu_mul_quant_block),
                          W4_METHOD(gemm),          W4_METHOD(gemm_act),    W4_METHOD(moe_gemm),
                          W4_METHOD(moe_gemm_act),  W4_METHOD(quant_fp4),   W4_METHOD(dequant_fp4),
                          W4_METHOD(fp4_gemm),      W4_METHOD(fp4_gemm_act), W4_METHOD(fp4_moe_gemm),
                          W4_METHOD(fp4_moe_gemm_act), W4_METHOD(moe_decode), {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&kModule); }
