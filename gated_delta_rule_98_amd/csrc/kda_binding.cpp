// kda_binding.cpp - argument marshalling of include/kda_linear.h and
// include/kda_norm.h for the Python package (module kda_native). Checks the
// tensors of a call, passes their addresses and strides to the C entry point
// and returns its status; nothing is computed here.
//
// Why native: the shortest kernels here take 2 to 5 us, and the same checks in
// Python took longer (a one-row step's call 8.5 us, 2.8 us of it the HIP launch,
// for a kernel of 3.6 us).

#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/core/DeviceGuard.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <stdexcept>
#include <string>

#include "kda_linear.h"
#include "kda_norm.h"

namespace {

decltype(&kda_lin_decode_step) lin_decode_step;
decltype(&kda_lin_prefill) lin_prefill;
decltype(&kda_lin_prefill_workspace) lin_prefill_workspace;
decltype(&kda_block_norm) block_norm;
PyObject *raw_stream;    // torch: device index -> handle of its current stream
PyObject *workspace_on;  // kda.py: (bytes, device index, stream) -> tensor allocated on that stream

struct PythonError {};  // a Python exception is set

struct TypeError : std::runtime_error {
  using std::runtime_error::runtime_error;
};
struct ValueError : std::runtime_error {
  using std::runtime_error::runtime_error;
};

using Shape = std::initializer_list<int64_t>;

std::string str(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + ")";
}

bool is_bf16(at::ScalarType t) { return t == at::kBFloat16 || t == at::kShort || t == at::kUInt16; }
bool is_f32(at::ScalarType t) { return t == at::kFloat; }
bool is_i32(at::ScalarType t) { return t == at::kInt; }
bool is_out(at::ScalarType t) { return is_f32(t) || is_bf16(t); }

const at::Tensor &tensor(PyObject *o, const char *name) {
  if (!THPVariable_Check(o)) throw TypeError(std::string(name) + " must be a torch.Tensor");
  return THPVariable_Unpack(o);
}

// o as a tensor of that type and shape on GPU dev.
const at::Tensor &typed(PyObject *o, const char *name, int dev, bool (*type)(at::ScalarType), const char *types,
                        Shape shape) {
  const at::Tensor &t = tensor(o, name);
  if (!type(t.scalar_type()))
    throw TypeError(std::string(name) + " has dtype " + c10::toString(t.scalar_type()) + ", expected " + types);
  if (!t.is_cuda() || t.get_device() != dev)
    throw ValueError(std::string(name) + " must be on GPU " + std::to_string(dev) + ", got " + t.device().str());
  if (t.sizes() != at::IntArrayRef(shape))
    throw ValueError(std::string(name) + " has shape " + str(t.sizes()) + ", expected " + str(at::IntArrayRef(shape)));
  return t;
}

void *contiguous(PyObject *o, const char *name, int dev, bool (*type)(at::ScalarType), const char *types, Shape shape) {
  const at::Tensor &t = typed(o, name, dev, type, types, shape);
  if (!t.is_contiguous()) throw ValueError(std::string(name) + " must be contiguous");
  return t.data_ptr();
}

constexpr const char *kBf16 = "bfloat16 (or its bits as int16 / uint16)", *kF32 = "float32", *kI32 = "int32",
                     *kOut = "float32 or bfloat16 (or its bits as int16 / uint16)";

struct Strided {
  void *p;
  int64_t stride;
};

// bf16 [rows, heads, d], each token's heads contiguous
Strided heads(PyObject *o, const char *name, int dev, int64_t rows, int64_t n, int64_t d) {
  const at::Tensor &t = typed(o, name, dev, is_bf16, kBf16, {rows, n, d});
  if (t.stride(2) != 1 || (n > 1 && t.stride(1) != d))
    throw ValueError(std::string(name) + ": each token's heads must be contiguous, got strides " + str(t.strides()));
  return {t.data_ptr(), rows > 1 ? t.stride(0) : n * d};
}

// [rows, D], each row contiguous; null for None
Strided rows_of(PyObject *o, const char *name, int dev, bool (*type)(at::ScalarType), const char *types, int64_t rows,
                int64_t D) {
  if (o == Py_None) return {nullptr, 0};
  const at::Tensor &t = typed(o, name, dev, type, types, {rows, D});
  if (D > 1 && t.stride(1) != 1)
    throw ValueError(std::string(name) + ": each row must be contiguous, got strides " + str(t.strides()));
  return {t.data_ptr(), rows > 1 ? t.stride(0) : D};
}

struct Cache {
  float *p;
  int64_t slots, stride, H, dv, dk;
  int dev;
};

// float32 [num_slots, H, dv, dk]; each slot contiguous, slots at stride(0)
Cache cache_of(PyObject *o) {
  const at::Tensor &t = tensor(o, "cache");
  if (!t.is_cuda() || t.scalar_type() != at::kFloat || t.dim() != 4)
    throw ValueError("cache must be a float32 GPU tensor [num_slots, H, dv, dk]");
  const int64_t H = t.size(1), dv = t.size(2), dk = t.size(3);
  if (t.stride(1) != dv * dk || t.stride(2) != dk || t.stride(3) != 1)
    throw ValueError("each cache slot must be contiguous [H, dv, dk]");
  return {static_cast<float *>(t.data_ptr()), t.size(0), t.size(0) > 1 ? t.stride(0) : H * dv * dk, H, dv, dk,
          (int)t.get_device()};
}

// Sizes are int32 in the C ABI.
int32_t i32(int64_t x) {
  if (x > INT32_MAX) throw ValueError("size " + std::to_string(x) + " does not fit 32 bits");
  return (int32_t)x;
}

int64_t rows_in(PyObject *o, const char *name) {
  const at::Tensor &t = tensor(o, name);
  if (t.dim() < 1) throw ValueError(std::string(name) + " must have dims");
  return t.size(0);
}

kda_lin_tokens tokens(const Cache &c, int64_t rows, PyObject *q, PyObject *k, PyObject *v, PyObject *alpha) {
  const at::Tensor &kt = tensor(k, "k");
  const int64_t Hk = kt.dim() == 3 ? kt.size(1) : 0;
  if (Hk < 1 || c.H % Hk)
    throw ValueError("k must be [rows, Hk, dk] with Hk dividing H = " + std::to_string(c.H));
  const Strided qs = heads(q, "q", c.dev, rows, Hk, c.dk), ks = heads(k, "k", c.dev, rows, Hk, c.dk),
                vs = heads(v, "v", c.dev, rows, c.H, c.dv);
  const bool fixed = tensor(alpha, "alpha").dim() == 1;
  const Strided as = fixed ? Strided{contiguous(alpha, "alpha", c.dev, is_f32, kF32, {c.H}), 0}
                           : rows_of(alpha, "alpha", c.dev, is_f32, kF32, rows, c.H);
  return {static_cast<const uint16_t *>(qs.p), static_cast<const uint16_t *>(ks.p), static_cast<const uint16_t *>(vs.p),
          static_cast<const float *>(as.p), qs.stride, ks.stride, vs.stride, as.stride, i32(Hk)};
}

int32_t *dev_err_of(PyObject *o, int dev) {
  if (o == Py_None) return nullptr;
  const at::Tensor &t = tensor(o, "dev_err");
  if (t.scalar_type() != at::kInt) throw TypeError("dev_err must be int32");
  if (!t.is_cuda() || t.get_device() != dev || t.numel() < 1)
    throw ValueError("dev_err must be on GPU " + std::to_string(dev));
  return static_cast<int32_t *>(t.data_ptr());
}

double number(PyObject *o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw PythonError();
  return x;
}

int64_t integer(PyObject *o) {
  const long long x = PyLong_AsLongLong(o);
  if (x == -1 && PyErr_Occurred()) throw PythonError();
  return x;
}

// While the C entry point runs, other Python threads may.
struct WithoutGil {
  PyThreadState *state = PyEval_SaveThread();
  WithoutGil() = default;
  WithoutGil(const WithoutGil &) = delete;
  ~WithoutGil() { PyEval_RestoreThread(state); }
};

// The stream's handle: None is the current stream of GPU dev.
void *stream_of(PyObject *o, int dev) {
  PyObject *h;
  if (o == Py_None) {
    PyObject *d = PyLong_FromLong(dev);
    h = d ? PyObject_CallOneArg(raw_stream, d) : nullptr;
    Py_XDECREF(d);
  } else if (PyLong_Check(o)) {
    Py_INCREF(o);
    h = o;
  } else {
    h = PyObject_GetAttrString(o, "cuda_stream");
  }
  if (!h) throw PythonError();
  void *p = PyLong_AsVoidPtr(h);
  Py_DECREF(h);
  if (!p && PyErr_Occurred()) throw PythonError();
  return p;
}

// A workspace allocated on a stream that the caller named.
at::Tensor workspace(size_t bytes, int dev, PyObject *stream) {
  PyObject *t = PyObject_CallFunction(workspace_on, "niO", (Py_ssize_t)bytes, dev, stream);
  if (!t) throw PythonError();
  const at::Tensor r = THPVariable_Unpack(t);
  Py_DECREF(t);
  return r;
}

template <class F>
PyObject *guarded(F &&f) {
  try {
    return PyLong_FromLong(f());
  } catch (const PythonError &) {
  } catch (const TypeError &e) {
    PyErr_SetString(PyExc_TypeError, e.what());
  } catch (const ValueError &e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const c10::Error &) {  // as torch raises it: OutOfMemoryError for a workspace that does not fit
    torch::translate_exception_to_python(std::current_exception());
  } catch (const std::exception &e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
  }
  return nullptr;
}

void expect(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) throw TypeError("expected " + std::to_string(want) + " arguments, got " + std::to_string(n));
}

kda_options options_of(int64_t tile_w, at::ScalarType out) {
  return {i32(tile_w), 0, is_bf16(out) ? (int32_t)KDA_OUT_BF16 : 0};
}

// (cache, slot_ids, q, k, v, alpha, out, gate, weight, eps, dev_err, tile_w, stream) -> status
PyObject *py_decode(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> int {
    expect(n, 13);
    const Cache c = cache_of(a[0]);
    const int64_t B = rows_in(a[1], "slot_ids");
    auto *slots = static_cast<int32_t *>(contiguous(a[1], "slot_ids", c.dev, is_i32, kI32, {B}));
    const kda_lin_tokens x = tokens(c, B, a[2], a[3], a[4], a[5]);
    void *out = contiguous(a[6], "out", c.dev, is_out, kOut, {B, c.H, c.dv});
    kda_epilogue epi = {nullptr, nullptr, 0.0f};
    const bool gate = a[7] != Py_None;
    if (gate) {
      epi.gate = static_cast<uint16_t *>(contiguous(a[7], "gate", c.dev, is_bf16, kBf16, {B, c.H, c.dv}));
      if (a[8] != Py_None) epi.weight = static_cast<float *>(contiguous(a[8], "weight", c.dev, is_f32, kF32, {c.dv}));
      epi.eps = (float)number(a[9]);
    } else if (a[8] != Py_None) {
      throw ValueError("weight needs a gate");
    }
    int32_t *err = dev_err_of(a[10], c.dev);
    const kda_options opts = options_of(integer(a[11]), tensor(a[6], "out").scalar_type());
    void *stream = stream_of(a[12], c.dev);
    const c10::DeviceGuard guard(c10::Device(c10::kCUDA, (c10::DeviceIndex)c.dev));
    const WithoutGil released;
    return lin_decode_step(c.p, c.slots, c.stride, slots, i32(B), i32(c.H), i32(c.dk), i32(c.dv), &x, out,
                           gate ? &epi : nullptr, err, &opts, stream);
  });
}

// (cache, slot_ids, cu_seqlens, q, k, v, alpha, out, ckpt_pos, ckpt, workspace, dev_err, stream) -> status
PyObject *py_prefill(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> int {
    expect(n, 13);
    const Cache c = cache_of(a[0]);
    const int64_t B = rows_in(a[1], "slot_ids"), n_tok = rows_in(a[5], "v");
    auto *slots = static_cast<int32_t *>(contiguous(a[1], "slot_ids", c.dev, is_i32, kI32, {B}));
    auto *cu = static_cast<int32_t *>(contiguous(a[2], "cu_seqlens", c.dev, is_i32, kI32, {B + 1}));
    const kda_lin_tokens x = tokens(c, n_tok, a[3], a[4], a[5], a[6]);
    void *out = contiguous(a[7], "out", c.dev, is_out, kOut, {n_tok, c.H, c.dv});
    int32_t *pos = nullptr;
    float *ckpt = nullptr;
    if (a[8] != Py_None) {
      pos = static_cast<int32_t *>(contiguous(a[8], "ckpt_pos", c.dev, is_i32, kI32, {B}));
      if (a[9] == Py_None) throw ValueError("ckpt_pos needs a ckpt buffer");
    }
    if (a[9] != Py_None) ckpt = static_cast<float *>(contiguous(a[9], "ckpt", c.dev, is_f32, kF32, {B, c.H, c.dv, c.dk}));
    int32_t *err = dev_err_of(a[11], c.dev);
    const kda_options opts = options_of(0, tensor(a[7], "out").scalar_type());
    void *stream = stream_of(a[12], c.dev);
    const c10::DeviceGuard guard(c10::Device(c10::kCUDA, (c10::DeviceIndex)c.dev));
    at::Tensor ws;
    size_t bytes = 0;
    if (a[10] != Py_None) {
      ws = tensor(a[10], "workspace");
      if (!ws.is_cuda() || ws.get_device() != c.dev || !ws.is_contiguous())
        throw ValueError("workspace must be a contiguous tensor on GPU " + std::to_string(c.dev));
      bytes = ws.nbytes();
    } else {
      const int rc = lin_prefill_workspace(i32(B), i32(n_tok), i32(c.H), i32(c.dk), i32(c.dv), &bytes);
      if (rc != KDA_OK) return rc;
      // allocated on the stream that uses it, so that its reuse is ordered behind this call
      if (bytes && a[12] == Py_None)
        ws = at::empty({(int64_t)bytes}, at::TensorOptions().dtype(at::kByte).device(c10::kCUDA, c.dev));
      else if (bytes)
        ws = workspace(bytes, c.dev, a[12]);
    }
    const WithoutGil released;
    return lin_prefill(c.p, c.slots, c.stride, slots, cu, i32(B), i32(n_tok), i32(c.H), i32(c.dk), i32(c.dv), &x, out,
                       pos, ckpt, bytes ? ws.data_ptr() : nullptr, bytes, err, &opts, stream);
  });
}

// (resid, z, resid_out, y, w_post, gate, res_scale, w_pre, eps, stream) -> status
PyObject *py_norm(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> int {
    expect(n, 10);
    const at::Tensor &r = tensor(a[0], "resid");
    if (!r.is_cuda() || r.dim() != 2) throw ValueError("resid must be a GPU tensor [rows, D]");
    const int dev = (int)r.get_device();
    const int64_t rows = r.size(0), D = r.size(1);
    const bool rb = is_bf16(r.scalar_type());
    const Strided rs = rows_of(a[0], "resid", dev, is_out, kOut, rows, D),
                  zs = rows_of(a[1], "z", dev, is_bf16, kBf16, rows, D),
                  os = rows_of(a[2], "resid_out", dev, rb ? is_bf16 : is_f32, "resid's", rows, D),
                  ys = rows_of(a[3], "y", dev, is_out, kOut, rows, D),
                  gs = rows_of(a[5], "gate", dev, is_bf16, kBf16, rows, D);
    const auto weight = [&](PyObject *o, const char *name) {
      return o == Py_None ? nullptr : static_cast<const float *>(contiguous(o, name, dev, is_f32, kF32, {D}));
    };
    const float *wo = weight(a[4], "w_post"), *wp = weight(a[7], "w_pre");
    const bool yb = ys.p && is_bf16(tensor(a[3], "y").scalar_type());
    const float scale = (float)number(a[6]), eps = (float)number(a[8]);
    void *stream = stream_of(a[9], dev);
    const c10::DeviceGuard guard(c10::Device(c10::kCUDA, (c10::DeviceIndex)dev));
    const WithoutGil released;
    return block_norm(rs.p, rs.stride, static_cast<const uint16_t *>(zs.p), zs.stride, os.p, os.stride, ys.p, ys.stride,
                      wo, static_cast<const uint16_t *>(gs.p), gs.stride, scale, wp, eps, i32(rows), i32(D),
                      (rb ? KDA_NORM_RESID_BF16 : 0) | (yb ? KDA_NORM_Y_BF16 : 0), stream);
  });
}

// The entry points' addresses (kda_lin_decode_step, kda_lin_prefill,
// kda_lin_prefill_workspace, kda_block_norm), torch's stream lookup and workspace_on.
PyObject *py_bind(PyObject *, PyObject *const *a, Py_ssize_t n) {
  return guarded([&]() -> int {
    expect(n, 6);
    const auto address = [&](int i) {
      void *p = PyLong_AsVoidPtr(a[i]);
      if (!p) throw ValueError("null entry point");
      return p;
    };
    lin_decode_step = reinterpret_cast<decltype(lin_decode_step)>(address(0));
    lin_prefill = reinterpret_cast<decltype(lin_prefill)>(address(1));
    lin_prefill_workspace = reinterpret_cast<decltype(lin_prefill_workspace)>(address(2));
    block_norm = reinterpret_cast<decltype(block_norm)>(address(3));
    Py_INCREF(a[4]);
    Py_XSETREF(raw_stream, a[4]);
    Py_INCREF(a[5]);
    Py_XSETREF(workspace_on, a[5]);
    return 0;
  });
}

PyMethodDef methods[] = {
    {"bind", (PyCFunction)(void *)py_bind, METH_FASTCALL, nullptr},
    {"lin_decode_step", (PyCFunction)(void *)py_decode, METH_FASTCALL, nullptr},
    {"lin_prefill", (PyCFunction)(void *)py_prefill, METH_FASTCALL, nullptr},
    {"block_norm", (PyCFunction)(void *)py_norm, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "kda_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_kda_native() { return PyModule_Create(&module); }
