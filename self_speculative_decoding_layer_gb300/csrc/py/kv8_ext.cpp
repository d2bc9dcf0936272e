// Python binding of the 8-bit KV cache (ssd_kv8_* of include/ssd.h) for torch
// tensors: argument checks, output and scratch allocation, the current stream.
// A decoded token's kernels run for 3 to 7 us.  The same checks and
// marshalling in Python with ctypes took 14 to 21 us a call, and 2 to 5
// here; kv8.py is a thin layer over this module.
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cmath>
#include <new>
#include <optional>
#include <string>
#include <vector>

#include "../../../include/ssd.h"

namespace {

constexpr int kMaxRows = 64;
constexpr const char* kCapsule = "ssd.kv8";

struct Cache {
  std::vector<ssd_kv8_cache> layers;
  int index = 0;  // CUDA device
  int heads = 0, hd = 0;
  float scale = 0.f;
};

PyObject* g_error = nullptr;  // SSDError(status, message)

// Raised as SSDError.
struct Refused {
  int status;
  std::string what;
};
// A Python error is set already.
struct Raised {};

[[noreturn]] void refuse(const std::string& what) { throw Refused{SSD_ERR_INVALID_ARG, what}; }

template <typename F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (const Refused& e) {
    if (PyObject* v = Py_BuildValue("(is)", e.status, e.what.c_str())) {
      PyErr_SetObject(g_error, v);
      Py_DECREF(v);
    }
  } catch (const Raised&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

const Cache& cache_of(PyObject* o) {
  void* p = PyCapsule_GetPointer(o, kCapsule);
  if (!p) throw Raised{};
  return *static_cast<Cache*>(p);
}

const ssd_kv8_cache& layer_of(const Cache& c, PyObject* o) {
  const long i = PyLong_AsLong(o);
  if (i == -1 && PyErr_Occurred()) throw Raised{};
  if (i < 0 || i >= (long)c.layers.size()) refuse("layer " + std::to_string(i) + " of " + std::to_string(c.layers.size()));
  return c.layers[i];
}

// A Python integer as int; one that does not fit is refused.
int int_of(PyObject* o, const char* what) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    if (!PyErr_ExceptionMatches(PyExc_OverflowError)) throw Raised{};
    PyErr_Clear();
    refuse(std::string(what) + " is out of range");
  }
  if (v < INT32_MIN || v > INT32_MAX) refuse(std::string(what) + " is out of range");
  return (int)v;
}

float float_of(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return (float)v;
}

const at::Tensor& tensor_of(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) refuse(std::string(what) + " is a tensor");
  return THPVariable_Unpack(o);
}

int io_of(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return SSD_F32;
    case at::kBFloat16: return SSD_BF16;
    case at::kHalf: return SSD_FP16;
    default: return -1;
  }
}

bool here(const Cache& c, const at::Tensor& t) { return t.is_cuda() && t.get_device() == c.index; }

// Elements between the rows of a [rows, heads, head_dim] float tensor whose rows are contiguous.
int64_t row_stride(const Cache& c, const at::Tensor& t, int64_t heads, const char* what) {
  if (t.dim() != 3 || t.size(1) != heads || t.size(2) != c.hd || io_of(t.scalar_type()) < 0 || !here(c, t))
    refuse(std::string(what) + " is [rows, " + std::to_string(heads) + ", " + std::to_string(c.hd) +
           "] of float32, bfloat16 or float16 on cuda:" + std::to_string(c.index));
  if (t.stride(2) != 1 || (heads > 1 && t.stride(1) != c.hd)) refuse(std::string("the rows of ") + what + " are contiguous");
  return t.size(0) > 1 ? t.stride(0) : heads * c.hd;
}

int rows_of(const at::Tensor& t, const char* what) {
  if (t.size(0) > INT32_MAX) refuse(std::string(what) + " has too many rows");
  return (int)t.size(0);
}

at::Tensor empty(const Cache& c, at::IntArrayRef size, at::ScalarType t) {
  return at::Tensor(at::detail::empty_cuda(size, t, c10::Device(c10::kCUDA, (c10::DeviceIndex)c.index), std::nullopt));
}

// The cache's device made current for the life of the object, and its current torch stream.
struct Stream {
  std::optional<c10::cuda::CUDAGuard> guard;
  void* stream;
  explicit Stream(const Cache& c) {
    if (c10::cuda::current_device() != c.index) guard.emplace((c10::DeviceIndex)c.index);
    stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)c.index).stream();
  }
};

void check(ssd_status s, const char* what) {
  if (s != SSD_OK) throw Refused{(int)s, std::string(what) + (s == SSD_ERR_CUDA ? "" : " refused its arguments")};
}

#define ARGS(n)                                                                  \
  if (nargs != (n)) {                                                            \
    PyErr_Format(PyExc_TypeError, "%d arguments, not %zd", (n), (Py_ssize_t)nargs); \
    return nullptr;                                                              \
  }

// open(k, v, k_scale, v_scale, block_table addresses, n_layers, pool_pages, n_kv_heads, head_dim, n_pages, code,
// block_tokens, device): the capsule that the calls below take.  kv8.py has checked the tensors and keeps them alive.
PyObject* py_open(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  ARGS(13)
  return guarded([&]() -> PyObject* {
    void* p[5];
    for (int i = 0; i < 5; ++i) {
      p[i] = PyLong_AsVoidPtr(a[i]);
      if (PyErr_Occurred()) throw Raised{};
    }
    int n[8];
    for (int i = 0; i < 8; ++i) n[i] = int_of(a[5 + i], "a size");
    auto* c = new Cache;
    c->index = n[7];
    c->heads = n[2];
    c->hd = n[3];
    c->scale = (float)(1.0 / std::sqrt((double)n[3]));
    for (int i = 0; i < n[0]; ++i)
      c->layers.push_back(ssd_kv8_cache{p[0], p[1], (float*)p[2], (float*)p[3], (const int32_t*)p[4], n[4], n[1], i, n[2],
                                        n[3], n[5], n[6]});
    PyObject* cap = PyCapsule_New(c, kCapsule, [](PyObject* o) { delete static_cast<Cache*>(PyCapsule_GetPointer(o, kCapsule)); });
    if (!cap) {
      delete c;
      throw Raised{};
    }
    return cap;
  });
}

// append(cache, layer, k, v, first)
PyObject* py_append(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  ARGS(5)
  return guarded([&]() -> PyObject* {
    const Cache& c = cache_of(a[0]);
    const ssd_kv8_cache& l = layer_of(c, a[1]);
    const at::Tensor &k = tensor_of(a[2], "k"), &v = tensor_of(a[3], "v");
    const int64_t ld_k = row_stride(c, k, c.heads, "k"), ld_v = row_stride(c, v, c.heads, "v");
    if (v.scalar_type() != k.scalar_type() || v.size(0) != k.size(0)) refuse("k and v have the same rows and type");
    const ssd_kv8_rows r{k.data_ptr(), v.data_ptr(), ld_k, ld_v, io_of(k.scalar_type()), int_of(a[4], "first"), rows_of(k, "k")};
    const Stream s(c);
    check(ssd_kv8_append(&l, &r, s.stream), "ssd_kv8_append");
    Py_RETURN_NONE;
  });
}

PyObject* pair(const at::Tensor& x, const at::Tensor& y) {
  PyObject* a = THPVariable_Wrap(x);
  PyObject* b = a ? THPVariable_Wrap(y) : nullptr;
  PyObject* t = b ? PyTuple_Pack(2, a, b) : nullptr;
  Py_XDECREF(a);
  Py_XDECREF(b);
  if (!t) throw Raised{};
  return t;
}

// read(cache, layer, first, rows, ssd_dtype) -> (k, v)
PyObject* py_read(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  ARGS(5)
  return guarded([&]() -> PyObject* {
    const Cache& c = cache_of(a[0]);
    const ssd_kv8_cache& l = layer_of(c, a[1]);
    const int first = int_of(a[2], "first"), rows = int_of(a[3], "rows"), io = int_of(a[4], "dtype");
    if (rows < 1 || rows > l.n_pages * 64) refuse("rows from 1 to the table's slots");
    const at::ScalarType t = io == SSD_F32 ? at::kFloat : io == SSD_BF16 ? at::kBFloat16 : at::kHalf;
    const Stream s(c);
    const at::Tensor k = empty(c, {rows, c.heads, c.hd}, t), v = empty(c, {rows, c.heads, c.hd}, t);
    const int64_t ld = (int64_t)c.heads * c.hd;
    const ssd_kv8_rows r{k.data_ptr(), v.data_ptr(), ld, ld, io, first, rows};
    check(ssd_kv8_read(&l, &r, s.stream), "ssd_kv8_read");
    return pair(k, v);
  });
}

// The arguments that attention and weights share: a[0..5] = q, prefix, base, masks, scale, softcap.
void attention_args(const Cache& c, PyObject* const* a, ssd_kv8_attention_args* p) {
  const at::Tensor& q = tensor_of(a[0], "q");
  if (q.dim() != 3 || q.size(1) < 1 || q.size(1) % c.heads || q.size(1) > INT32_MAX)
    refuse("q is [rows, heads, head_dim], its heads a multiple of " + std::to_string(c.heads));
  p->ld_q = row_stride(c, q, q.size(1), "q");
  if (q.size(0) < 1 || q.size(0) > kMaxRows) refuse(std::to_string(q.size(0)) + " rows: 1 to 64");
  p->q = q.data_ptr();
  p->out = nullptr;
  p->lse = nullptr;
  p->ld_out = p->ld_lse = p->step_lse = 0;
  p->dtype = io_of(q.scalar_type());
  p->n_q_heads = (int)q.size(1);
  p->rows = (int)q.size(0);
  p->prefix = int_of(a[1], "prefix");
  p->base = a[2] == Py_None ? p->prefix : int_of(a[2], "base");
  p->scale = a[4] == Py_None ? c.scale : float_of(a[4]);
  p->softcap = float_of(a[5]);
  if (a[3] == Py_None) {
    for (int r = 0; r < p->rows; ++r) p->mask[r] = (2ull << r) - 1;
    return;
  }
  PyObject* seq = PySequence_Fast(a[3], "masks are a sequence of integers");
  if (!seq) throw Raised{};
  const Py_ssize_t n = PySequence_Fast_GET_SIZE(seq);
  if (n != p->rows) {
    Py_DECREF(seq);
    refuse(std::to_string(n) + " masks for " + std::to_string(p->rows) + " rows");
  }
  for (Py_ssize_t r = 0; r < n; ++r) {
    PyObject* i = PyNumber_Index(PySequence_Fast_GET_ITEM(seq, r));
    p->mask[r] = i ? PyLong_AsUnsignedLongLongMask(i) : 0;
    Py_XDECREF(i);
    if (PyErr_Occurred()) {
      Py_DECREF(seq);
      throw Raised{};
    }
  }
  Py_DECREF(seq);
}

// attention(cache, layer, q, prefix, base, masks, scale, softcap, out, return_lse) -> out or (out, lse)
PyObject* py_attention(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  ARGS(10)
  return guarded([&]() -> PyObject* {
    const Cache& c = cache_of(a[0]);
    const ssd_kv8_cache& l = layer_of(c, a[1]);
    ssd_kv8_attention_args p;
    attention_args(c, a + 2, &p);
    const at::Tensor& q = THPVariable_Unpack(a[2]);
    const int want_lse = PyObject_IsTrue(a[9]);
    if (want_lse < 0) throw Raised{};
    const Stream s(c);
    at::Tensor out, lse;
    if (a[8] == Py_None) {
      out = empty(c, q.sizes(), q.scalar_type());
      p.ld_out = (int64_t)p.n_q_heads * c.hd;
    } else {
      out = tensor_of(a[8], "out");
      if (out.sizes() != q.sizes() || out.scalar_type() != q.scalar_type()) refuse("out has the shape and type of q");
      p.ld_out = row_stride(c, out, p.n_q_heads, "out");
    }
    p.out = out.data_ptr();
    if (want_lse) {
      lse = empty(c, {p.rows, p.n_q_heads}, at::kFloat);
      p.lse = lse.data_ptr<float>();
    }
    // Scratch for each call, from the current stream's pool: calls on other streams and captured graphs share none.
    const size_t need = ssd_kv8_attention_scratch_bytes(&l, &p);
    at::Tensor scratch;
    if (need > 256) scratch = empty(c, {(int64_t)need}, at::kByte);
    check(ssd_kv8_attention(&l, &p, need > 256 ? scratch.data_ptr() : nullptr, need, s.stream), "ssd_kv8_attention");
    if (want_lse) return pair(out, lse);
    if (a[8] != Py_None) {
      Py_INCREF(a[8]);
      return a[8];
    }
    return THPVariable_Wrap(out);
  });
}

// Elements between the heads of a float32 [n_kv_heads, >= slots] tensor whose rows are contiguous.
int64_t weight_stride(const Cache& c, const at::Tensor& t, int64_t slots) {
  if (t.dim() != 2 || t.size(0) != c.heads || t.size(1) < slots || t.scalar_type() != at::kFloat || !here(c, t))
    refuse("weights are float32 [" + std::to_string(c.heads) + ", " + std::to_string(slots) + " or more] on cuda:" +
           std::to_string(c.index));
  const int64_t ld = c.heads == 1 ? t.size(1) : t.stride(0);
  if ((t.stride(1) != 1 && t.size(1) > 1) || ld < t.size(1)) refuse("the rows of weights are contiguous and apart");
  return ld;
}

// weights(cache, layer, q, prefix, base, masks, scale, softcap, lse, rows, weight, out) -> out
PyObject* py_weights(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  ARGS(12)
  return guarded([&]() -> PyObject* {
    const Cache& c = cache_of(a[0]);
    const ssd_kv8_cache& l = layer_of(c, a[1]);
    ssd_kv8_attention_args p;
    attention_args(c, a + 2, &p);
    const at::Tensor& lse = tensor_of(a[8], "lse");
    if (lse.dim() != 2 || lse.size(0) != p.rows || lse.size(1) != p.n_q_heads || lse.scalar_type() != at::kFloat || !here(c, lse))
      refuse("lse is the float32 [rows, heads] of the attention call");
    const int64_t slots = std::max<int64_t>({(int64_t)p.prefix, (int64_t)p.base + p.rows, 1});
    uint64_t take = 0;
    if (a[9] == Py_None) {
      take = p.rows == 64 ? ~0ull : (1ull << p.rows) - 1;
    } else {
      PyObject* seq = PySequence_Fast(a[9], "rows are a sequence of integers");
      if (!seq) throw Raised{};
      for (Py_ssize_t i = 0; i < PySequence_Fast_GET_SIZE(seq); ++i) {
        const Py_ssize_t r = PyNumber_AsSsize_t(PySequence_Fast_GET_ITEM(seq, i), PyExc_IndexError);
        if (PyErr_Occurred()) {
          Py_DECREF(seq);
          throw Raised{};
        }
        if (r < 0 || r >= p.rows) {
          Py_DECREF(seq);
          refuse("row " + std::to_string(r) + " of " + std::to_string(p.rows));
        }
        take |= 1ull << r;
      }
      Py_DECREF(seq);
    }
    const Stream s(c);
    p.lse = lse.data_ptr<float>();
    p.ld_lse = lse.stride(0);
    p.step_lse = lse.stride(1);
    PyObject* result = a[11] != Py_None ? a[11] : a[10];
    at::Tensor out;
    if (result == Py_None) {
      if (p.prefix < 0 || p.base < 0 || slots > (int64_t)l.n_pages * 64) refuse("a slot past the block table");
      out = empty(c, {c.heads, slots}, at::kFloat);
    } else {
      out = tensor_of(result, "out");
    }
    const int64_t ld = weight_stride(c, out, slots);
    const float* in = nullptr;
    if (a[10] != Py_None) {
      const at::Tensor& w = tensor_of(a[10], "weight");
      if (weight_stride(c, w, slots) != ld) refuse("weight and out are laid out alike");
      in = w.data_ptr<float>();
    }
    check(ssd_kv8_weights(&l, &p, take, in, out.data_ptr<float>(), ld, s.stream), "ssd_kv8_weights");
    if (result == Py_None) return THPVariable_Wrap(out);
    Py_INCREF(result);
    return result;
  });
}

// evict(cache, layer, weight, keep, recent, to, to_layer) -> (index, kept weights)
PyObject* py_evict(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  ARGS(7)
  return guarded([&]() -> PyObject* {
    const Cache& c = cache_of(a[0]);
    const Cache& d = cache_of(a[5]);
    const ssd_kv8_cache &l = layer_of(c, a[1]), &m = layer_of(d, a[6]);
    const at::Tensor& w = tensor_of(a[2], "weight");
    const int64_t ld = weight_stride(c, w, 1), n = w.size(1);
    const int keep = int_of(a[3], "keep"), recent = int_of(a[4], "recent");
    if (d.index != c.index) refuse("both caches are on one device");
    if (n > INT32_MAX || keep < 1 || keep > n || recent < 0 || recent > keep)
      refuse("0 <= recent <= keep <= " + std::to_string(n) + ", keep >= 1");
    const Stream s(c);
    const at::Tensor index = empty(c, {c.heads, keep}, at::kInt), kept = empty(c, {c.heads, keep}, at::kFloat);
    const ssd_kv8_evict_args e{w.data_ptr<float>(), ld, index.data_ptr<int32_t>(), kept.data_ptr<float>(), (int)n, keep, recent};
    check(ssd_kv8_evict(&l, &m, &e, s.stream), "ssd_kv8_evict");
    return pair(index, kept);
  });
}

// init(SSDError)
PyObject* py_init(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  ARGS(1)
  Py_INCREF(a[0]);
  Py_XSETREF(g_error, a[0]);
  Py_RETURN_NONE;
}

#define METHOD(name) {#name, (PyCFunction)(void (*)(void))py_##name, METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {METHOD(init),      METHOD(open),    METHOD(append), METHOD(read),
                           METHOD(attention), METHOD(weights), METHOD(evict),  {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_kv8", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__kv8(void) { return PyModule_Create(&g_module); }
