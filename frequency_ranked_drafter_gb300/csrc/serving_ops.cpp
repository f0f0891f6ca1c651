// Python entry points of the serving operators (quantize_rows, matmul_i8,
// sample_logits, verify_draft): argument checks, output tensors, device and
// stream, then the C ABI.
//
// The kernels behind them take 2 to 10 us for a token, less than a Python
// binding needs for its checks (11 us for quantize_rows and 23 us for
// verify_draft through ctypes on a Grace core), so these four checks are
// compiled.  Types are refused with TypeError, shapes, strides and devices with
// ValueError, everything the library refuses with its own error.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/from_blob.h>
#include <ATen/ops/zeros.h>
#include <c10/cuda/CUDAGraphsC10Utils.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <string>

#include "vt.h"

namespace {

struct Api {
  decltype(&vt_quantize_rows) quantize_rows;
  decltype(&vt_matmul_i8) matmul_i8;
  decltype(&vt_matmul_i8_workspace_size) matmul_i8_workspace_size;
  decltype(&vt_sample_logits) sample_logits;
  decltype(&vt_verify_draft) verify_draft;
} api;
PyObject* check_fn = nullptr;  // check(name, status): raises the library's error

struct Refused {};  // a Python exception is set

[[noreturn]] void refuse(PyObject* kind, const std::string& why) {
  PyErr_SetString(kind, why.c_str());
  throw Refused();
}

std::string shape_text(c10::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + (s.size() == 1 ? ",)" : ")");
}

const at::Tensor& cuda_tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o) || !THPVariable_Unpack(o).is_cuda())
    refuse(PyExc_TypeError, std::string(name) + " must be a CUDA tensor");
  return THPVariable_Unpack(o);
}

void want_type(const at::Tensor& t, const char* name, at::ScalarType type) {
  if (t.scalar_type() != type)
    refuse(PyExc_TypeError, std::string(name) + " must be " + c10::toString(type) + ", got " +
                                c10::toString(t.scalar_type()));
}
void want_place(const at::Tensor& t, const char* name, c10::Device dev, c10::IntArrayRef shape) {
  if (t.device() != dev)
    refuse(PyExc_ValueError,
           std::string(name) + " is on " + t.device().str() + ", not on " + dev.str());
  if (t.sizes() != shape)
    refuse(PyExc_ValueError, std::string(name) + " must have shape " + shape_text(shape) +
                                 ", got " + shape_text(t.sizes()));
}

// A contiguous tensor of this type, place and shape.
const at::Tensor& dense(PyObject* o, const char* name, at::ScalarType type, c10::Device dev,
                        c10::IntArrayRef shape) {
  const at::Tensor& t = cuda_tensor(o, name);
  want_type(t, name, type);
  want_place(t, name, dev, shape);
  if (!t.is_contiguous())
    refuse(PyExc_ValueError, std::string(name) + " must be contiguous");
  return t;
}
template <typename T>
T* address(const at::Tensor& t) {
  return static_cast<T*>(t.data_ptr());
}
// The same, or null for None.
template <typename T>
T* maybe(PyObject* o, const char* name, at::ScalarType type, c10::Device dev,
         c10::IntArrayRef shape) {
  return o == Py_None ? nullptr : address<T>(dense(o, name, type, dev, shape));
}

// The vt_dtype of a tensor, and what it may be.
int element(const at::Tensor& t, const char* name, bool half) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return VT_BF16;
    case at::kFloat: return VT_FP32;
    case at::kHalf:
      if (half) return VT_FP16;
      break;
    default: break;
  }
  refuse(PyExc_TypeError, std::string(name) + " must be float32, bfloat16" +
                              (half ? " or float16" : "") + ", got " +
                              c10::toString(t.scalar_type()));
}

// Row stride of a matrix whose rows are contiguous (a stride along an axis of
// length 1 says nothing).
int64_t row_stride(const at::Tensor& t, const char* name) {
  if (t.dim() != 2) refuse(PyExc_ValueError, std::string(name) + " must be 2-D");
  if (t.size(1) > 1 && t.stride(1) != 1)
    refuse(PyExc_ValueError, std::string(name) + " must have unit column stride");
  return t.size(0) > 1 ? t.stride(0) : t.size(1);
}

at::Tensor fresh(c10::IntArrayRef shape, at::ScalarType type, c10::Device dev) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(dev));
}
// The caller's output, or a new one.
at::Tensor output(PyObject* o, const char* name, at::ScalarType type, c10::Device dev,
                  c10::IntArrayRef shape) {
  return o == Py_None ? fresh(shape, type, dev) : dense(o, name, type, dev, shape);
}

int32_t int32_of(int64_t v, const char* what) {
  if (v > INT32_MAX) refuse(PyExc_ValueError, std::string(what) + " is above 2^31 - 1");
  return (int32_t)v;
}

void* stream_on(c10::Device dev) {
  return c10::cuda::getCurrentCUDAStream(dev.index()).stream();
}

void done(const char* name, vt_status status) {
  if (status == VT_OK) return;
  PyObject* r = PyObject_CallFunction(check_fn, "si", name, (int)status);
  Py_XDECREF(r);
  if (r) refuse(PyExc_RuntimeError, name);
  throw Refused();
}

PyObject* wrap(const at::Tensor& t) { return THPVariable_Wrap(t); }

template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F f) {
  HANDLE_TH_ERRORS
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "%zd arguments, got %zd", want, n);
    return nullptr;
  }
  try {
    return f();
  } catch (const Refused&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// quantize_rows(X, ids, out, scale, n_invalid)
PyObject* quantize_rows(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 5, [&]() -> PyObject* {
    const at::Tensor& X = cuda_tensor(a[0], "X");
    const int type = element(X, "X", true);
    int64_t ldx = row_stride(X, "X");
    const int64_t V = X.size(0), d = X.size(1);
    if (V <= 1) ldx = (d + 7) / 8 * 8;
    const c10::Device dev = X.device();
    int64_t R = V;
    const int32_t* ids = nullptr;
    if (a[1] != Py_None) {
      R = cuda_tensor(a[1], "ids").numel();
      ids = address<int32_t>(dense(a[1], "ids", at::kInt, dev, {R}));
    }
    const at::Tensor q = output(a[2], "out", at::kChar, dev, {R, d});
    const at::Tensor s = output(a[3], "scale", at::kFloat, dev, {R});
    uint64_t* bad = maybe<uint64_t>(a[4], "n_invalid", at::kLong, dev, {1});
    const c10::cuda::CUDAGuard guard(dev);
    done("vt_quantize_rows",
         api.quantize_rows(X.data_ptr(), type, V, int32_of(d, "d"), ldx, ids,
                           int32_of(R, "rows"), address<int8_t>(q), address<float>(s), bad,
                           stream_on(dev)));
    return Py_BuildValue("(NN)", wrap(q), wrap(s));
  });
}

// A zeroed workspace of matmul_i8 that belongs to no graph, made while one is
// captured: memory of its own (the allocator's would be the graph's, free for its
// next tensor once nothing holds this one), zeroed now and not at each replay.
at::Tensor word_beside_capture(c10::Device dev) {
  const int64_t bytes = (int64_t)api.matmul_i8_workspace_size();
  const c10::cuda::CUDAStreamCaptureModeGuard relaxed(cudaStreamCaptureModeRelaxed);
  void* p = nullptr;
  cudaStream_t side;
  C10_CUDA_CHECK(cudaMalloc(&p, bytes));  // kept for the process
  C10_CUDA_CHECK(cudaStreamCreateWithFlags(&side, cudaStreamNonBlocking));
  C10_CUDA_CHECK(cudaMemsetAsync(p, 0, bytes, side));
  C10_CUDA_CHECK(cudaStreamSynchronize(side));
  C10_CUDA_CHECK(cudaStreamDestroy(side));
  return at::from_blob(p, {bytes}, at::TensorOptions().dtype(at::kByte).device(dev));
}

// The error word of this stream's calls without a workspace of their own, kept in
// the dictionary `words` under (device, stream): a call that is checked then
// sees (and clears) its own stream's word only.  Calls captured on a stream that
// has none yet share one a device, under (device, None).
at::Tensor stream_word(PyObject* words, c10::Device dev, cudaStream_t stream) {
  PyObject* key = Py_BuildValue("(iK)", (int)dev.index(),
                                (unsigned long long)reinterpret_cast<uintptr_t>(stream));
  if (!key) throw Refused();
  PyObject* known = PyDict_GetItemWithError(words, key);  // borrowed
  cudaStreamCaptureStatus status = cudaStreamCaptureStatusNone;
  if (!known && !PyErr_Occurred()) {
    C10_CUDA_CHECK(cudaStreamIsCapturing(stream, &status));
    if (status != cudaStreamCaptureStatusNone) {
      Py_DECREF(key);
      key = Py_BuildValue("(iO)", (int)dev.index(), Py_None);
      if (!key) throw Refused();
      known = PyDict_GetItemWithError(words, key);
    }
  }
  at::Tensor w;
  if (known) {
    w = THPVariable_Unpack(known);
  } else if (!PyErr_Occurred()) {
    w = status != cudaStreamCaptureStatusNone
            ? word_beside_capture(dev)
            : at::zeros({(int64_t)api.matmul_i8_workspace_size()},
                        at::TensorOptions().dtype(at::kByte).device(dev));
    PyObject* o = wrap(w);
    if (o) PyDict_SetItem(words, key, o);
    Py_XDECREF(o);
  }
  Py_DECREF(key);
  if (PyErr_Occurred()) throw Refused();
  return w;
}

// matmul_i8(Q, scale, Wq, w_scale, bias, out, out_dtype, ws, words)
PyObject* matmul_i8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    const at::Tensor& Q = cuda_tensor(a[0], "Q");
    const at::Tensor& W = cuda_tensor(a[2], "Wq");
    if (Q.dim() != 2 || W.dim() != 2) refuse(PyExc_ValueError, "Q and Wq must be 2-D");
    const int64_t M = Q.size(0), d = Q.size(1), N = W.size(0);
    const c10::Device dev = Q.device();
    dense(a[0], "Q", at::kChar, dev, {M, d});
    dense(a[2], "Wq", at::kChar, dev, {N, d});
    const float* xs = address<float>(dense(a[1], "scale", at::kFloat, dev, {M}));
    const float* ws = address<float>(dense(a[3], "w_scale", at::kFloat, dev, {N}));
    const float* bias = maybe<float>(a[4], "bias", at::kFloat, dev, {N});
    at::Tensor y;
    int64_t ldo = N;
    if (a[5] == Py_None) {
      const at::ScalarType t = THPDtype_Check(a[6])
                                   ? reinterpret_cast<THPDtype*>(a[6])->scalar_type
                                   : at::ScalarType::Undefined;
      if (t != at::kFloat && t != at::kBFloat16)
        refuse(PyExc_TypeError, "out_dtype must be float32 or bfloat16");
      y = fresh({M, N}, t, dev);
    } else {
      y = cuda_tensor(a[5], "out");
      element(y, "out", false);
      ldo = row_stride(y, "out");
      want_place(y, "out", dev, {M, N});
    }
    const c10::cuda::CUDAGuard guard(dev);
    void* stream = stream_on(dev);
    at::Tensor w;
    if (a[7] == Py_None) {
      w = stream_word(a[8], dev, static_cast<cudaStream_t>(stream));
    } else {
      w = cuda_tensor(a[7], "ws");
      dense(a[7], "ws", at::kByte, dev, {w.numel()});
    }
    done("vt_matmul_i8",
         api.matmul_i8(address<int8_t>(Q), xs, int32_of(M, "M"), address<int8_t>(W), ws,
                       int32_of(N, "N"), int32_of(d, "d"), bias, y.data_ptr(),
                       element(y, "out", false), ldo, w.data_ptr(), (size_t)w.numel(), stream));
    return wrap(y);
  });
}

// A setting: a number, or a tensor with one value a row.
float real_setting(PyObject* o, const char* name, c10::Device dev, int64_t M, const float** rows) {
  if (THPVariable_Check(o)) {
    *rows = address<float>(dense(o, name, at::kFloat, dev, {M}));
    return 0.f;
  }
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused();
  return (float)v;
}

// sample_logits(logits, u, t2f, temperature, top_k, top_p, min_p, return_dist,
//               out_ids, out_probs, out_dist)
PyObject* sample_logits(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> PyObject* {
    const at::Tensor& x = cuda_tensor(a[0], "logits");
    const int type = element(x, "logits", true);
    const int64_t ld = row_stride(x, "logits"), M = x.size(0), len = x.size(1);
    const c10::Device dev = x.device();
    vt_sample_options o = {};
    o.temperature = real_setting(a[3], "temperature", dev, M, &o.temperature_rows);
    if (THPVariable_Check(a[4])) {
      o.top_k_rows = address<int32_t>(dense(a[4], "top_k", at::kInt, dev, {M}));
    } else {
      PyObject* k = PyNumber_Index(a[4]);
      if (!k) throw Refused();
      int over = 0;
      const long long v = PyLong_AsLongLongAndOverflow(k, &over);
      Py_DECREF(k);
      o.top_k = over > 0 || v > INT32_MAX ? INT32_MAX : over < 0 || v < -1 ? -1 : (int32_t)v;
    }
    o.top_p = real_setting(a[5], "top_p", dev, M, &o.top_p_rows);
    o.min_p = real_setting(a[6], "min_p", dev, M, &o.min_p_rows);
    const int32_t* map = maybe<int32_t>(a[2], "t2f", at::kInt, dev, {len});
    const bool draws = a[1] != Py_None;
    at::Tensor ids, probs, dist;
    const float* u = nullptr;
    if (draws) {
      u = address<float>(dense(a[1], "u", at::kFloat, dev, {M}));
      ids = output(a[8], "out_ids", at::kInt, dev, {M});
      probs = output(a[9], "out_probs", at::kFloat, dev, {M});
    } else if (a[8] != Py_None || a[9] != Py_None) {
      refuse(PyExc_ValueError, "out_ids and out_probs need u");
    }
    const int truth = PyObject_IsTrue(a[7]);
    if (truth < 0) throw Refused();
    int64_t ldd = len;
    if (a[10] != Py_None) {
      dist = cuda_tensor(a[10], "out_dist");
      want_type(dist, "out_dist", at::kFloat);
      ldd = row_stride(dist, "out_dist");
      want_place(dist, "out_dist", dev, {M, len});
    } else if (truth || !draws) {
      dist = fresh({M, len}, at::kFloat, dev);
    }
    const c10::cuda::CUDAGuard guard(dev);
    done("vt_sample_logits",
         api.sample_logits(x.data_ptr(), type, int32_of(M, "rows"), int32_of(len, "n"), ld, &o, u,
                           map, draws ? address<int32_t>(ids) : nullptr,
                           draws ? address<float>(probs) : nullptr,
                           dist.defined() ? address<float>(dist) : nullptr, ldd, stream_on(dev)));
    if (!draws) return wrap(dist);
    if (!dist.defined()) return Py_BuildValue("(NN)", wrap(ids), wrap(probs));
    return Py_BuildValue("(NNN)", wrap(ids), wrap(probs), wrap(dist));
  });
}

// A float32 [a, b, c] whose rows are contiguous, and its strides.
const float* stack(PyObject* o, const char* name, c10::Device dev, int64_t* s0, int64_t* s1,
                   int64_t* last) {
  const at::Tensor& t = cuda_tensor(o, name);
  want_type(t, name, at::kFloat);
  if (t.dim() != 3) refuse(PyExc_ValueError, std::string(name) + " must be 3-D");
  const int64_t b = t.size(1), c = t.size(2);
  if (c > 1 && t.stride(2) != 1)
    refuse(PyExc_ValueError, std::string(name) + " must have unit last stride");
  *s0 = t.size(0) > 1 ? t.stride(0) : b * c;
  *s1 = b > 1 ? t.stride(1) : c;
  *last = c;
  return address<float>(t);
}

// verify_draft(draft_ids, p, q, u, n_draft, f2t, out_accepted, out_ids)
PyObject* verify_draft(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> PyObject* {
    const at::Tensor& ids = cuda_tensor(a[0], "draft_ids");
    if (ids.dim() != 2) refuse(PyExc_ValueError, "draft_ids must be [B, K]");
    const int64_t B = ids.size(0), K = ids.size(1);
    const c10::Device dev = ids.device();
    const int32_t* draft = address<int32_t>(dense(a[0], "draft_ids", at::kInt, dev, {B, K}));
    int64_t p0, p1, V, q0 = 0, q1 = 0, Vq;
    const float* p = stack(a[1], "p", dev, &p0, &p1, &V);
    want_place(THPVariable_Unpack(a[1]), "p", dev, {B, K + 1, V});
    const float* q = nullptr;
    Vq = V;
    if (a[2] != Py_None) {
      q = stack(a[2], "q", dev, &q0, &q1, &Vq);
      want_place(THPVariable_Unpack(a[2]), "q", dev, {B, K, Vq});
    } else if (K > 0) {
      refuse(PyExc_TypeError, "q must be a CUDA tensor");
    }
    if (a[5] == Py_None && Vq != V)
      refuse(PyExc_ValueError, "q covers fewer ids than p: f2t is needed");
    const float* u = address<float>(dense(a[3], "u", at::kFloat, dev, {B, K + 1}));
    const int32_t* nd = maybe<int32_t>(a[4], "n_draft", at::kInt, dev, {B});
    const int32_t* f2t = maybe<int32_t>(a[5], "f2t", at::kInt, dev, {V});
    const at::Tensor acc = output(a[6], "out_accepted", at::kInt, dev, {B});
    const at::Tensor out = output(a[7], "out_ids", at::kInt, dev, {B, K + 1});
    const c10::cuda::CUDAGuard guard(dev);
    done("vt_verify_draft",
         api.verify_draft(draft, nd, int32_of(B, "B"), int32_of(K, "K"), int32_of(V, "V"), p, p0,
                          p1, q, q0, q1, int32_of(Vq, "Vq"), f2t, u, address<int32_t>(acc),
                          address<int32_t>(out), stream_on(dev)));
    return Py_BuildValue("(NN)", wrap(acc), wrap(out));
  });
}

// bind(path of the library, check): looks the entry points up.
PyObject* bind(PyObject*, PyObject* args) {
  const char* path;
  PyObject* check;
  if (!PyArg_ParseTuple(args, "sO", &path, &check)) return nullptr;
  void* lib = dlopen(path, RTLD_NOW | RTLD_LOCAL);
  if (!lib) {
    PyErr_SetString(PyExc_RuntimeError, dlerror());
    return nullptr;
  }
  api.quantize_rows = reinterpret_cast<decltype(api.quantize_rows)>(dlsym(lib, "vt_quantize_rows"));
  api.matmul_i8 = reinterpret_cast<decltype(api.matmul_i8)>(dlsym(lib, "vt_matmul_i8"));
  api.matmul_i8_workspace_size = reinterpret_cast<decltype(api.matmul_i8_workspace_size)>(
      dlsym(lib, "vt_matmul_i8_workspace_size"));
  api.sample_logits = reinterpret_cast<decltype(api.sample_logits)>(dlsym(lib, "vt_sample_logits"));
  api.verify_draft = reinterpret_cast<decltype(api.verify_draft)>(dlsym(lib, "vt_verify_draft"));
  if (!api.quantize_rows || !api.matmul_i8 || !api.matmul_i8_workspace_size ||
      !api.sample_logits || !api.verify_draft) {
    PyErr_SetString(PyExc_RuntimeError, "the library lacks an entry point");
    return nullptr;
  }
  Py_INCREF(check);
  Py_XDECREF(check_fn);
  check_fn = check;
  Py_RETURN_NONE;
}

#define FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL
PyMethodDef methods[] = {{"bind", bind, METH_VARARGS, nullptr},
                         {"quantize_rows", FAST(quantize_rows), nullptr},
                         {"matmul_i8", FAST(matmul_i8), nullptr},
                         {"sample_logits", FAST(sample_logits), nullptr},
                         {"verify_draft", FAST(verify_draft), nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "vt_serving_ops", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit_vt_serving_ops() {
  return PyModule_Create(&module);
}
