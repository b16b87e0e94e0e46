// kv_binding.cpp - marshalling of the paged-cache calls for PyTorch tensors: a
// CPython module whose functions check tensors, allocate what is not given,
// and call libqsa's C entry points (whose addresses the package passes in
// once) on the current stream. These calls run once per layer and token of a
// serving loop; the same checks in Python took 10 us a call, twice the launch.
#include <Python.h>

#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <sstream>
#include <string>

#include "qsa.h"

namespace {

decltype(&qsa_kv_append) g_append = nullptr;
decltype(&qsa_kv_attend) g_attend = nullptr;
decltype(&qsa_kv_attend_workspace_bytes) g_attend_bytes = nullptr;

struct Refusal {
  PyObject* type;
  std::string text;
};

using at::IntArrayRef;
using at::ScalarType;
using at::Tensor;

[[noreturn]] void refuse(const std::string& text) { throw Refusal{PyExc_ValueError, text}; }

const Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) throw Refusal{PyExc_TypeError, std::string(name) + " must be a torch.Tensor"};
  return THPVariable_Unpack(o);
}

std::string described(const Tensor& t) {
  std::ostringstream s;
  s << ", got " << t.dtype().name() << " " << t.sizes() << " on " << t.device().str();
  return s.str();
}

bool on(const Tensor& t, int dev) { return t.is_cuda() && t.get_device() == dev; }

// A contiguous tensor of this type and shape on device `dev`; its address.
void* plain(const Tensor& t, ScalarType type, IntArrayRef shape, int dev, const char* name) {
  if (t.scalar_type() != type || t.sizes() != shape || !on(t, dev) || !t.is_contiguous()) {
    std::ostringstream s;
    s << name << " must be a contiguous " << c10::toString(type) << " tensor " << shape << " on cuda:" << dev;
    refuse(s.str() + described(t));
  }
  return t.data_ptr();
}

bool pages_contiguous(const Tensor& t) {
  int64_t want = 1;
  for (int i = 3; i > 0; --i) {
    if (t.size(i) != 1 && t.stride(i) != want) return false;
    want *= t.size(i);
  }
  return true;
}

// The cache arguments shared by both calls: args[0..5] = k_cache, v_cache,
// k_scale, v_scale, page_table, lens; n_new or None.
qsa_kv_cache cache_of(PyObject* const* args, PyObject* n_new, int* dev) {
  const Tensor &k = tensor(args[0], "k_cache"), &v = tensor(args[1], "v_cache");
  const Tensor &table = tensor(args[4], "page_table"), &lens = tensor(args[5], "lens");
  for (const Tensor* t : {&k, &v})
    if ((t->scalar_type() != ScalarType::Float8_e4m3fn && t->scalar_type() != ScalarType::Byte) || t->dim() != 4 ||
        !t->is_cuda())
      refuse("k_cache and v_cache must be CUDA float8_e4m3fn or uint8 tensors [n_pages, Hkv, block, D]" +
             described(*t));
  if (table.dim() != 2 || lens.dim() != 1) refuse("page_table must be int32 [B, max_blocks] and lens int32 [B]");
  *dev = k.get_device();
  const int64_t pages = k.size(0), heads = k.size(1), block = k.size(2), D = k.size(3), B = lens.size(0);
  if (v.sizes() != k.sizes() || !on(v, *dev) || (pages > 1 && v.stride(0) != k.stride(0)) || !pages_contiguous(k) ||
      !pages_contiguous(v))
    refuse("k_cache and v_cache must have one shape, page stride and device, and contiguous pages");
  for (int64_t x : {pages, heads, block, D, B, table.size(1)})
    if (x > INT32_MAX) refuse("a size of the cache does not fit 32 bits");
  qsa_kv_cache c{};
  c.k = static_cast<uint8_t*>(k.data_ptr());
  c.v = static_cast<uint8_t*>(v.data_ptr());
  c.k_scale = static_cast<float*>(plain(tensor(args[2], "k_scale"), ScalarType::Float, {pages, heads}, *dev, "k_scale"));
  c.v_scale = static_cast<float*>(plain(tensor(args[3], "v_scale"), ScalarType::Float, {pages, heads}, *dev, "v_scale"));
  c.page_table = static_cast<int32_t*>(plain(table, ScalarType::Int, {B, table.size(1)}, *dev, "page_table"));
  c.lens = static_cast<int32_t*>(plain(lens, ScalarType::Int, {B}, *dev, "lens"));
  if (n_new != Py_None)
    c.n_new = static_cast<int32_t*>(plain(tensor(n_new, "n_new"), ScalarType::Int, {B}, *dev, "n_new"));
  c.page_stride = pages > 1 ? k.stride(0) : heads * block * D;
  c.n_pages = static_cast<int32_t>(pages);
  c.max_blocks = static_cast<int32_t>(table.size(1));
  c.B = static_cast<int32_t>(B);
  c.Hkv = static_cast<int32_t>(heads);
  c.block = static_cast<int32_t>(block);
  c.D = static_cast<int32_t>(D);
  return c;
}

// Rows [B, n, heads, D] (n, heads < 0: any) of 16-bit floats, any strides but
// the last; `type` Undefined: f16 or bf16.
qsa_rows rows_of(const Tensor& t, int64_t B, int64_t n, int64_t heads, int64_t D, ScalarType type, int dev,
                 const char* name) {
  const ScalarType have = t.scalar_type();
  if (t.dim() != 4 || !on(t, dev) ||
      (type == ScalarType::Undefined ? have != ScalarType::Half && have != ScalarType::BFloat16 : have != type) ||
      t.size(0) != B || t.size(3) != D || (n >= 0 && t.size(1) != n) || (heads >= 0 && t.size(2) != heads)) {
    std::ostringstream s;
    s << name << " must be a " << (type == ScalarType::Undefined ? "Half or BFloat16" : c10::toString(type))
      << " tensor [" << B << ", " << (n < 0 ? "n" : std::to_string(n)) << ", "
      << (heads < 0 ? "heads" : std::to_string(heads)) << ", " << D << "] on cuda:" << dev;
    refuse(s.str() + described(t));
  }
  if (t.size(1) > INT32_MAX || t.size(2) > INT32_MAX) refuse(std::string(name) + " is too large");
  if (t.stride(3) != 1 && t.numel() > 0) refuse(std::string(name) + " must be contiguous in its last axis");
  // The stride of an axis of one element means nothing and may be anything.
  auto stride = [&](int i) { return t.size(i) == 1 ? 0 : t.stride(i); };
  return qsa_rows{t.data_ptr(), stride(0), stride(1), stride(2)};
}

qsa_stream_t stream_of(int dev) {
  return reinterpret_cast<qsa_stream_t>(
      c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream());
}

// Runs f; a Refusal or a C++ exception becomes a Python one.
template <class F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (const Refusal& r) {
    PyErr_SetString(r.type, r.text.c_str());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// (k, v, k_cache, v_cache, k_scale, v_scale, page_table, lens, cos, sin,
// interleaved, n_new, q, q_out, kb) -> q_out or None, or a status.
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t count) {
  return guarded([&]() -> PyObject* {
    if (count != 15 || !g_append) throw Refusal{PyExc_TypeError, "append takes 15 arguments, after bind()"};
    int dev = 0;
    const qsa_kv_cache c = cache_of(a + 2, a[11], &dev);
    const Tensor& k = tensor(a[0], "k");
    const qsa_rows rk = rows_of(k, c.B, -1, c.Hkv, c.D, ScalarType::Undefined, dev, "k");
    const int64_t n = k.size(1);
    const ScalarType type = k.scalar_type();
    const qsa_rows rv = rows_of(tensor(a[1], "v"), c.B, n, c.Hkv, c.D, type, dev, "v");
    const void *cos = nullptr, *sin = nullptr;
    int64_t rot = 0, max_pos = 0;
    if (a[8] != Py_None || a[9] != Py_None) {
      const Tensor &tc = tensor(a[8], "cos"), &ts = tensor(a[9], "sin");
      if (tc.dim() != 2) refuse("cos and sin must be float32 [max_pos, rot / 2]");
      cos = plain(tc, ScalarType::Float, tc.sizes(), dev, "cos");
      sin = plain(ts, ScalarType::Float, tc.sizes(), dev, "sin");
      max_pos = std::min<int64_t>(tc.size(0), INT32_MAX);
      rot = std::min<int64_t>(2 * tc.size(1), INT32_MAX);
    }
    const int interleaved = PyObject_IsTrue(a[10]);
    if (interleaved < 0) return nullptr;
    qsa_rows rq{};
    int64_t Hq = 0;
    Tensor made;
    PyObject* result = Py_None;
    void *q_to = nullptr, *kb = nullptr;
    if (a[12] != Py_None) {
      const Tensor& q = tensor(a[12], "q");
      rq = rows_of(q, c.B, n, -1, c.D, type, dev, "q");
      Hq = q.size(2);
      if (a[13] != Py_None) {
        q_to = plain(tensor(a[13], "q_out"), type, q.sizes(), dev, "q_out");
        result = a[13];
      } else {
        made = at::empty(q.sizes(), q.options());
        q_to = made.data_ptr();
      }
    } else if (a[13] != Py_None) {
      refuse("q_out needs q");
    }
    if (a[14] != Py_None)
      kb = plain(tensor(a[14], "kb"), ScalarType::Half, {c.B, c.Hkv, c.max_blocks, c.D}, dev, "kb");
    c10::cuda::OptionalCUDAGuard guard;
    if (c10::cuda::current_device() != dev) guard.set_index(static_cast<c10::DeviceIndex>(dev));
    const qsa_status st =
        g_append(&c, &rk, &rv, a[12] != Py_None ? &rq : nullptr, static_cast<int32_t>(n), static_cast<int32_t>(Hq),
                 type == ScalarType::BFloat16 ? QSA_BF16 : QSA_F16, static_cast<const float*>(cos),
                 static_cast<const float*>(sin), static_cast<int32_t>(rot), static_cast<int32_t>(max_pos), interleaved,
                 q_to, static_cast<uint16_t*>(kb), stream_of(dev));
    if (st != QSA_OK) return PyLong_FromLong(st);
    if (made.defined()) return THPVariable_Wrap(made);
    Py_INCREF(result);
    return result;
  });
}

// (q, k_cache, v_cache, k_scale, v_scale, page_table, lens, ids, scale, n_new,
// out, lse, workspace) -> out, or a status.
PyObject* attend(PyObject*, PyObject* const* a, Py_ssize_t count) {
  return guarded([&]() -> PyObject* {
    if (count != 13 || !g_attend) throw Refusal{PyExc_TypeError, "attend takes 13 arguments, after bind()"};
    int dev = 0;
    const qsa_kv_cache c = cache_of(a + 1, a[9], &dev);
    const Tensor& q = tensor(a[0], "q");
    const qsa_rows rq = rows_of(q, c.B, -1, -1, c.D, ScalarType::Undefined, dev, "q");
    const ScalarType type = q.scalar_type();
    const int64_t n = q.size(1), Hq = q.size(2);
    double scale = 1.0 / std::sqrt(static_cast<double>(c.D));
    if (a[8] != Py_None) {
      scale = PyFloat_AsDouble(a[8]);
      if (scale == -1.0 && PyErr_Occurred()) return nullptr;
    }
    const void* ids = nullptr;
    int64_t lists = 0, k = 0;
    if (a[7] != Py_None) {
      const Tensor& t = tensor(a[7], "ids");
      if (t.dim() != 4 || (t.size(1) != 1 && t.size(1) != c.Hkv) || t.size(3) < 1 || t.size(3) > INT32_MAX)
        refuse("ids must be int32 [B, 1 or Hkv, n, k]" + described(t));
      lists = t.size(1);
      k = t.size(3);
      ids = plain(t, ScalarType::Int, {c.B, lists, n, k}, dev, "ids");
    }
    Tensor made, room;
    void *out = nullptr, *lse = nullptr, *ws = nullptr;
    if (a[10] != Py_None) {
      out = plain(tensor(a[10], "out"), type, q.sizes(), dev, "out");
    } else {
      made = at::empty(q.sizes(), q.options());
      out = made.data_ptr();
    }
    if (a[11] != Py_None) lse = plain(tensor(a[11], "lse"), ScalarType::Float, {c.B, n, Hq}, dev, "lse");
    size_t size = 0;
    if (a[12] != Py_None) {
      const Tensor& t = tensor(a[12], "workspace");
      size = static_cast<size_t>(t.numel());
      ws = plain(t, ScalarType::Byte, {t.numel()}, dev, "workspace");
    } else {
      size = g_attend_bytes(c.B, static_cast<int32_t>(n), static_cast<int32_t>(Hq), c.Hkv, c.D);
      room = at::empty({static_cast<int64_t>(std::max<size_t>(size, 16))}, q.options().dtype(ScalarType::Byte));
      ws = room.data_ptr();
    }
    c10::cuda::OptionalCUDAGuard guard;
    if (c10::cuda::current_device() != dev) guard.set_index(static_cast<c10::DeviceIndex>(dev));
    const qsa_status st =
        g_attend(&c, &rq, static_cast<int32_t>(n), static_cast<int32_t>(Hq),
                 type == ScalarType::BFloat16 ? QSA_BF16 : QSA_F16, static_cast<float>(scale),
                 static_cast<const int32_t*>(ids), static_cast<int32_t>(lists), static_cast<int32_t>(k), out,
                 static_cast<float*>(lse), ws, size, stream_of(dev));
    if (st != QSA_OK) return PyLong_FromLong(st);
    if (made.defined()) return THPVariable_Wrap(made);
    Py_INCREF(a[10]);
    return a[10];
  });
}

// Takes the addresses of qsa_kv_append, qsa_kv_attend and
// qsa_kv_attend_workspace_bytes.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t count) {
  if (count != 3) {
    PyErr_SetString(PyExc_TypeError, "bind takes 3 addresses");
    return nullptr;
  }
  void* p[3];
  for (int i = 0; i < 3; ++i) {
    p[i] = PyLong_AsVoidPtr(a[i]);
    if (!p[i] && PyErr_Occurred()) return nullptr;
  }
  g_append = reinterpret_cast<decltype(g_append)>(p[0]);
  g_attend = reinterpret_cast<decltype(g_attend)>(p[1]);
  g_attend_bytes = reinterpret_cast<decltype(g_attend_bytes)>(p[2]);
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(append)), METH_FASTCALL, nullptr},
    {"attend", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(attend)), METH_FASTCALL, nullptr},
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(bind)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_qsa_kv", "Marshalling of the paged-cache calls.", -1, methods,
                          nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__qsa_kv(void) { return PyModule_Create(&module_def); }
