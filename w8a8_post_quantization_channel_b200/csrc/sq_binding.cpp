// sq_binding.cpp -- native marshalling for the block-scaled and the grouped
// calls: checks tensors, allocates results on the current stream and calls
// libsq's C functions.  In Python the same steps take longer than the launch
// that they lead to (a single-token linear: 9.5 us of host time, 4.2 here).
//
// Each function returns its result, or the call's status (an int) when it is
// not SQ_OK; the Python side turns that into an SqError.  A tensor that does
// not fit raises ValueError.
#include <Python.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <sstream>

#include "sq.h"

namespace {

// What this was built from, for build.py to find in the binary.
#ifdef SQ_BUILD_KEY
[[gnu::used]] const char kBuiltFrom[] = SQ_BUILD_KEY;
#endif

struct Api {
  decltype(&sq_quant_act_e4m3_block) quant_act;
  decltype(&sq_smooth_quant_weight_e4m3_block) quant_weight;
  decltype(&sq_w8a8_linear_e4m3_block) linear_block;
  decltype(&sq_w8a8_linear_grouped) grouped_i8;
  decltype(&sq_w8a8_linear_grouped_e4m3) grouped_e4m3;
  decltype(&sq_w8a8_linear_grouped_e4m3_block) grouped_block;
} api;

int64_t blocks(int64_t n) { return (n + 127) / 128; }

sq_stream_t stream_of(const at::Device &d) { return c10::cuda::getCurrentCUDAStream(d.index()).stream(); }

// A tensor argument; nullptr for None.
const at::Tensor *tensor(PyObject *o, const char *name) {
  if (o == Py_None) return nullptr;
  TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor");
  return &THPVariable_Unpack(o);
}
const at::Tensor &need(PyObject *o, const char *name) {
  const at::Tensor *t = tensor(o, name);
  TORCH_CHECK_VALUE(t != nullptr, name, " must be a tensor, not None");
  return *t;
}

// t is a contiguous tensor of this type and shape on `device`.
void expect(const at::Tensor &t, const char *name, at::ScalarType type, at::IntArrayRef shape,
            const at::Device &device) {
  TORCH_CHECK_VALUE(t.scalar_type() == type, name, ": dtype ", t.scalar_type(), " not supported (", type, ")");
  TORCH_CHECK_VALUE(t.sizes() == shape, name, " must have shape ", shape, ", not ", t.sizes());
  TORCH_CHECK_VALUE(t.device() == device, name, " must be on ", device, ", not ", t.device());
  TORCH_CHECK_VALUE(t.is_contiguous(), name, " must be contiguous");
}

void rowmajor(const at::Tensor &t, const char *name) {
  TORCH_CHECK_VALUE(t.dim() == 2 && t.stride(1) == 1, name, " must be a 2-D tensor with unit column stride");
  TORCH_CHECK_VALUE(t.is_cuda(), name, " must be on a CUDA device");
}

sq_dtype dtype_of(at::ScalarType t, const char *name) {
  if (t == at::kFloat) return SQ_F32;
  if (t == at::kHalf) return SQ_F16;
  TORCH_CHECK_VALUE(t == at::kBFloat16, name, ": dtype ", t, " not supported (float32/float16/bfloat16)");
  return SQ_BF16;
}

// A new tensor from the caching allocator, on the current stream; without the
// dispatcher on the way.
at::Tensor fresh(at::ScalarType type, at::IntArrayRef shape, const at::Device &device) {
  return at::detail::empty_cuda(shape, type, device, std::nullopt);
}

at::Tensor given_or_new(PyObject *o, const char *name, at::ScalarType type, at::IntArrayRef shape,
                        const at::Device &device) {
  if (const at::Tensor *t = tensor(o, name)) {
    expect(*t, name, type, shape, device);
    return *t;
  }
  return fresh(type, shape, device);
}

// The library's call without the interpreter's lock, as under ctypes: a launch
// waits where the stream's queue is full, and what empties the queue may need
// another Python thread (a host callback).
struct Unlocked {
  PyThreadState *const state = PyEval_SaveThread();
  Unlocked() = default;
  Unlocked(const Unlocked &) = delete;
  ~Unlocked() { PyEval_RestoreThread(state); }
};
template <class F, class... A>
sq_status unlocked(F f, A... a) {
  const Unlocked scope;
  return f(a...);
}

PyObject *status(sq_status s) { return PyLong_FromLong((long)s); }
PyObject *wrap_or_none(const at::Tensor &t) {
  if (t.defined()) return THPVariable_Wrap(t);
  Py_RETURN_NONE;
}

void arity(Py_ssize_t n, Py_ssize_t want) { TORCH_CHECK_TYPE(n == want, "expected ", want, " arguments, got ", n); }

// init(path of libsq.so)
PyObject *init(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity(n, 1);
  const char *path = PyUnicode_AsUTF8(a[0]);
  if (path == nullptr) return nullptr;
  void *lib = dlopen(path, RTLD_NOW);
  TORCH_CHECK(lib != nullptr, "cannot load ", path, ": ", dlerror());
  auto find = [&](auto &f, const char *name) {
    f = reinterpret_cast<std::remove_reference_t<decltype(f)>>(dlsym(lib, name));
    TORCH_CHECK(f != nullptr, path, " has no ", name);
  };
  find(api.quant_act, "sq_quant_act_e4m3_block");
  find(api.quant_weight, "sq_smooth_quant_weight_e4m3_block");
  find(api.linear_block, "sq_w8a8_linear_e4m3_block");
  find(api.grouped_i8, "sq_w8a8_linear_grouped");
  find(api.grouped_e4m3, "sq_w8a8_linear_grouped_e4m3");
  find(api.grouped_block, "sq_w8a8_linear_grouped_e4m3_block");
  Py_RETURN_NONE;
  END_HANDLE_TH_ERRORS
}

// quant_act(x, inv_smooth, xq, x_scale) -> (xq, x_scale)
PyObject *quant_act(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity(n, 4);
  const at::Tensor &x = need(a[0], "x");
  rowmajor(x, "x");
  const at::Device dev = x.device();
  const c10::cuda::CUDAGuard guard(dev);
  const int64_t M = x.size(0), K = x.size(1);
  const sq_dtype dt = dtype_of(x.scalar_type(), "x");
  const at::Tensor *inv = tensor(a[1], "inv_smooth");
  if (inv != nullptr) expect(*inv, "inv_smooth", at::kFloat, {K}, dev);
  const at::Tensor q = given_or_new(a[2], "xq", at::kByte, {M, K}, dev);
  const at::Tensor s = given_or_new(a[3], "x_scale", at::kFloat, {M, blocks(K)}, dev);
  const sq_status r = unlocked(api.quant_act, x.data_ptr(), dt, M, K, M > 1 ? x.stride(0) : K,
                               inv != nullptr ? inv->const_data_ptr<float>() : nullptr,
                               static_cast<uint8_t *>(q.data_ptr()), static_cast<float *>(s.data_ptr()),
                               stream_of(dev));
  if (r != SQ_OK) return status(r);
  return Py_BuildValue("NN", THPVariable_Wrap(q), THPVariable_Wrap(s));
  END_HANDLE_TH_ERRORS
}

// quant_weight(w, amax, alpha, wq, w_scale, smooth, inv_smooth)
//   -> (wq, w_scale, smooth, inv_smooth)
PyObject *quant_weight(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity(n, 7);
  const at::Tensor &w = need(a[0], "w");
  TORCH_CHECK_VALUE((w.dim() == 2 || w.dim() == 3) && w.stride(-1) == 1,
                    "w must be a 2-D or 3-D tensor with unit column stride");
  TORCH_CHECK_VALUE(w.is_cuda(), "w must be on a CUDA device");
  const double alpha = PyFloat_AsDouble(a[2]);
  if (alpha == -1.0 && PyErr_Occurred()) return nullptr;
  const at::Device dev = w.device();
  const c10::cuda::CUDAGuard guard(dev);
  const bool many = w.dim() == 3;
  const int64_t E = many ? w.size(0) : 1, N = w.size(-2), K = w.size(-1);
  const int64_t ld = N > 1 ? w.stride(-2) : (many && E > 1 ? w.stride(0) : K);
  TORCH_CHECK_VALUE(!many || E <= 1 || w.stride(0) == N * ld,
                    "w's experts must follow one another (stride(0) == N * stride(1))");
  const sq_dtype dt = dtype_of(w.scalar_type(), "w");
  const at::Tensor *amax = tensor(a[1], "amax");
  if (amax != nullptr) expect(*amax, "amax", at::kFloat, {K}, dev);
  at::DimVector scale_shape;
  if (many) scale_shape.push_back(E);
  scale_shape.push_back(blocks(N));
  scale_shape.push_back(blocks(K));
  const at::Tensor q = given_or_new(a[3], "wq", at::kByte, w.sizes(), dev);
  const at::Tensor sc = given_or_new(a[4], "w_scale", at::kFloat, scale_shape, dev);
  at::Tensor s, inv;  // without smoothing: as they were given
  if (amax != nullptr || a[5] != Py_None) s = given_or_new(a[5], "smooth", at::kFloat, {K}, dev);
  if (amax != nullptr || a[6] != Py_None) inv = given_or_new(a[6], "inv_smooth", at::kFloat, {K}, dev);
  auto f32 = [](const at::Tensor &t) { return t.defined() ? static_cast<float *>(t.data_ptr()) : nullptr; };
  const sq_status r = unlocked(api.quant_weight, w.data_ptr(), dt, E, N, K, ld,
                               amax != nullptr ? amax->const_data_ptr<float>() : nullptr, (float)alpha,
                               static_cast<uint8_t *>(q.data_ptr()), f32(sc), f32(s), f32(inv), stream_of(dev));
  if (r != SQ_OK) return status(r);
  return Py_BuildValue("NNNN", THPVariable_Wrap(q), THPVariable_Wrap(sc), wrap_or_none(s), wrap_or_none(inv));
  END_HANDLE_TH_ERRORS
}

// linear(kind, xq, x_scale, wq, w_scale, offsets, out_dtype, y) -> y
//   kind 0: dense, block scales (offsets None); 1, 2, 3: grouped INT8, E4M3,
//   block scales
PyObject *linear(PyObject *, PyObject *const *a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  arity(n, 8);
  const long kind = PyLong_AsLong(a[0]);
  if (kind == -1 && PyErr_Occurred()) return nullptr;
  TORCH_CHECK_VALUE(kind >= 0 && kind <= 3, "kind must be 0 to 3");
  const bool grouped = kind > 0, block = kind == 0 || kind == 3;
  const at::ScalarType code = kind == 1 ? at::kChar : at::kByte;
  const at::Tensor &xq = need(a[1], "xq"), &xs = need(a[2], "x_scale"), &wq = need(a[3], "wq"),
                   &ws = need(a[4], "w_scale");
  rowmajor(xq, "xq");
  TORCH_CHECK_VALUE(wq.dim() == (grouped ? 3 : 2), "wq must be a ",
                    grouped ? "3-D tensor [E, N, K]" : "2-D tensor [N, K]");
  const at::Device dev = xq.device();
  const c10::cuda::CUDAGuard guard(dev);
  const int64_t T = xq.size(0), K = xq.size(1), E = grouped ? wq.size(0) : 1, N = wq.size(-2), KB = blocks(K);
  expect(xq, "xq", code, {T, K}, dev);
  if (grouped) {
    expect(wq, "wq", code, {E, N, K}, dev);
  } else {
    expect(wq, "wq", code, {N, K}, dev);
  }
  if (block) {
    expect(xs, "x_scale", at::kFloat, {T, KB}, dev);
  } else {
    expect(xs, "x_scale", at::kFloat, {T}, dev);
  }
  if (!grouped) {
    expect(ws, "w_scale", at::kFloat, {blocks(N), KB}, dev);
  } else if (block) {
    expect(ws, "w_scale", at::kFloat, {E, blocks(N), KB}, dev);
  } else {
    expect(ws, "w_scale", at::kFloat, {E, N}, dev);
  }
  const int32_t *off = nullptr;
  if (grouped) {
    const at::Tensor &o = need(a[5], "offsets");
    expect(o, "offsets", at::kInt, {E + 1}, dev);
    off = o.const_data_ptr<int32_t>();
  }
  at::Tensor y;
  sq_dtype yt;
  if (const at::Tensor *given = tensor(a[7], "y")) {
    y = *given;
    rowmajor(y, "y");
    yt = dtype_of(y.scalar_type(), "y");
    const int64_t shape[2] = {T, N};
    TORCH_CHECK_VALUE(y.sizes() == at::IntArrayRef(shape, 2), "y must have shape ", at::IntArrayRef(shape, 2), ", not ",
                      y.sizes());
    TORCH_CHECK_VALUE(y.device() == dev, "y must be on ", dev, ", not ", y.device());
  } else {
    TORCH_CHECK_TYPE(THPDtype_Check(a[6]), "out_dtype must be a torch.dtype");
    const at::ScalarType t = reinterpret_cast<THPDtype *>(a[6])->scalar_type;
    yt = dtype_of(t, "out_dtype");
    y = fresh(t, {T, N}, dev);
  }
  const int64_t ldy = T > 1 ? y.stride(0) : N;
  const float *px = xs.const_data_ptr<float>(), *pw = ws.const_data_ptr<float>();
  void *const q = xq.data_ptr(), *const v = wq.data_ptr(), *const out = y.data_ptr();
  const sq_stream_t st = stream_of(dev);
  auto *const q8 = static_cast<uint8_t *>(q), *const v8 = static_cast<uint8_t *>(v);
  sq_status r;
  if (kind == 0) {
    r = unlocked(api.linear_block, q8, px, v8, pw, T, N, K, out, yt, ldy, st);
  } else if (kind == 1) {
    r = unlocked(api.grouped_i8, static_cast<int8_t *>(q), px, static_cast<int8_t *>(v), pw, off, T, E, N, K, out, yt,
                 ldy, st);
  } else {
    r = unlocked(kind == 2 ? api.grouped_e4m3 : api.grouped_block, q8, px, v8, pw, off, T, E, N, K, out, yt, ldy, st);
  }
  if (r != SQ_OK) return status(r);
  return THPVariable_Wrap(y);
  END_HANDLE_TH_ERRORS
}

template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyCFunction fast() {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(F));
}

PyMethodDef methods[] = {{"init", fast<init>(), METH_FASTCALL, "init(path of libsq.so)"},
                         {"quant_act", fast<quant_act>(), METH_FASTCALL, "quant_act(x, inv_smooth, xq, x_scale)"},
                         {"quant_weight", fast<quant_weight>(), METH_FASTCALL,
                          "quant_weight(w, amax, alpha, wq, w_scale, smooth, inv_smooth)"},
                         {"linear", fast<linear>(), METH_FASTCALL,
                          "linear(kind, xq, x_scale, wq, w_scale, offsets, out_dtype, y)"},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", "Native marshalling over libsq.so.", -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
