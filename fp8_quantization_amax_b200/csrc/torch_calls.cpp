// The paged KV cache's calls from Python (module _torch_calls): checks of the tensors, outputs and
// workspaces that are not given, the call on the tensors' device and its current stream.
//
// A decoding step makes these calls for every layer, on a dozen tensors each.  Checked from Python
// they took 11 (page update) to 17 (append) microseconds of host time a call, several times what the
// kernels of a small batch take; from here it is 3.4 to 5, most of it the launch.
//
// The C entry points are handed over by bind() (the library is loaded by the package, once).
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <initializer_list>
#include <string>

#include "fp8q.h"

namespace {

decltype(&fp8_attention_paged) g_attention = nullptr;
decltype(&fp8q_attention_workspace_bytes) g_attention_ws = nullptr;
decltype(&fp8_kv_append) g_append = nullptr;
decltype(&fp8_kv_pages_update) g_update = nullptr;
decltype(&fp8q_pages_workspace_bytes) g_update_ws = nullptr;
PyObject* g_error = nullptr;   // (function name, status) -> exception
PyObject* g_out_of_memory = nullptr;   // torch's exception type

struct Refusal {
  PyObject* type;              // nullptr: Python's error is set already
  std::string what;
};

[[noreturn]] void refuse(PyObject* type, std::string what) { throw Refusal{type, std::move(what)}; }
[[noreturn]] void wrong_value(std::string what) { refuse(PyExc_ValueError, std::move(what)); }
[[noreturn]] void wrong_type(std::string what) { refuse(PyExc_TypeError, std::move(what)); }

const at::Tensor& tensor(PyObject* o, const char* name, at::ScalarType type) {
  if (!THPVariable_Check(o)) wrong_type(std::string(name) + " must be a torch.Tensor");
  const at::Tensor& t = THPVariable_Unpack(o);
  if (t.layout() != at::kStrided) wrong_type(std::string(name) + " must be a dense tensor");
  if (t.scalar_type() != type)
    wrong_type(std::string(name) + " must be " + c10::toString(type) + ", got " + c10::toString(t.scalar_type()));
  return t;
}

std::string text(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + ")";
}

const at::Tensor& contiguous(PyObject* o, const char* name, at::ScalarType type) {
  const at::Tensor& t = tensor(o, name, type);
  if (!t.is_contiguous()) wrong_value(std::string(name) + " must be contiguous");
  return t;
}
const at::Tensor& shaped(PyObject* o, const char* name, at::ScalarType type, std::initializer_list<int64_t> shape) {
  const at::Tensor& t = tensor(o, name, type);
  const at::IntArrayRef want(shape.begin(), shape.size());
  if (t.sizes() != want) wrong_value(std::string(name) + " must be " + text(want) + ", got " + text(t.sizes()));
  if (!t.is_contiguous()) wrong_value(std::string(name) + " must be contiguous");
  return t;
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) refuse(nullptr, "");
  return v;
}
double real(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) refuse(nullptr, "");
  return v;
}

// The CUDA device on which every tensor of a call lies; current while this lives.
struct Device {
  c10::DeviceIndex index;
  c10::cuda::CUDAGuard guard;
  static c10::DeviceIndex of(const at::Tensor& t, const char* name) {
    if (!t.is_cuda()) wrong_value(std::string(name) + " must be a CUDA tensor (this library has no CPU path)");
    return (c10::DeviceIndex)t.get_device();
  }
  Device(const at::Tensor& t, const char* name) : index(of(t, name)), guard(index) {}
  void holds(std::initializer_list<const at::Tensor*> all) const {
    for (const at::Tensor* t : all)
      if (t && !(t->is_cuda() && t->get_device() == index))
        wrong_value("all tensors of a call must be on one CUDA device (this library has no CPU path)");
  }
};

// bf16 [tokens][heads][head_dim] whose heads are contiguous within a token; its token stride
int64_t token_stride(const at::Tensor& t, const char* name) {
  if (t.dim() != 3) wrong_value(std::string(name) + " must be 3-D [tokens][heads][head_dim]");
  if ((t.stride(2) != 1 && t.size(2) > 1) || (t.stride(1) != t.size(2) && t.size(1) > 1))
    wrong_value(std::string(name) + " must be contiguous within a token");
  return t.size(0) > 1 ? t.stride(0) : t.size(1) * t.size(2);
}

struct Cache {
  const at::Tensor &k, &v, &ks, &vs;
  fp8q_kv_pages c;
  // o: k_cache, v_cache, k_scales, v_scales, fmt, gran
  explicit Cache(PyObject* const* o)
      : k(tensor(o[0], "k_cache", at::kByte)), v(tensor(o[1], "v_cache", at::kByte)),
        ks(contiguous(o[2], "k_scales", at::kFloat)), vs(contiguous(o[3], "v_scales", at::kFloat)) {
    if (k.dim() != 4 || k.sizes() != v.sizes() || k.strides() != v.strides())
      wrong_value("k_cache and v_cache must both be [num_pages][page_size][heads][head_dim] with equal strides");
    if (k.stride(3) != 1) wrong_value("k_cache and v_cache must be contiguous along head_dim");
    c.k_codes = static_cast<uint8_t*>(k.data_ptr());
    c.v_codes = static_cast<uint8_t*>(v.data_ptr());
    c.k_scales = static_cast<float*>(ks.data_ptr());
    c.v_scales = static_cast<float*>(vs.data_ptr());
    c.num_pages = k.size(0);
    c.page_size = k.size(1);
    c.heads = k.size(2);
    c.head_dim = k.size(3);
    // strides of single-entry dimensions are not used
    c.page_stride = c.num_pages > 1 ? k.stride(0) : 0;
    c.token_stride = c.page_size > 1 ? k.stride(1) : 0;
    c.head_stride = c.heads > 1 ? k.stride(2) : 0;
    const int64_t fmt = integer(o[4]), gran = integer(o[5]), slots = c.num_pages * c.page_size;
    if (fmt != FP8Q_E4M3 && fmt != FP8Q_E5M2) wrong_value("fmt must be one of E4M3, E5M2");
    c.f = (fp8q_format)fmt;
    c.g = (fp8q_kv_granularity)gran;
    const int64_t one[1] = {1}, head[1] = {c.heads}, blocks[2] = {(slots + 127) / 128, c.heads}, each[2] = {c.heads, slots};
    if (gran < 0 || gran > 3) wrong_value("gran must be one of KV_PER_TENSOR, KV_PER_HEAD, KV_PER_HEAD_TOK128, KV_PER_TOKEN");
    const at::IntArrayRef want = gran == 0 ? at::IntArrayRef(one) : gran == 1 ? at::IntArrayRef(head)
                                 : gran == 2 ? at::IntArrayRef(blocks) : at::IntArrayRef(each);
    if (ks.sizes() != want) wrong_value("k_scales must be " + text(want) + ", got " + text(ks.sizes()));
    if (vs.sizes() != want) wrong_value("v_scales must be " + text(want) + ", got " + text(vs.sizes()));
  }
};

// Scratch of `bytes` bytes: the caller's, or from torch's allocator
struct Workspace {
  at::Tensor own;
  void* p = nullptr;
  size_t bytes = 0;
  Workspace(PyObject* given, size_t need, const Device& dev) {
    if (given != Py_None) {
      if (!THPVariable_Check(given)) wrong_type("ws must be a torch.Tensor");
      const at::Tensor& t = THPVariable_Unpack(given);
      dev.holds({&t});
      if (!t.is_contiguous()) wrong_value("ws must be contiguous");
      p = t.data_ptr();
      bytes = t.nbytes();
    } else if (need > 0) {
      own = at::empty({(int64_t)need}, at::TensorOptions().dtype(at::kByte).device(at::kCUDA, dev.index));
      p = own.data_ptr();
      bytes = need;
    }
  }
};

at::Tensor made(const Device& dev, at::ScalarType type, at::IntArrayRef shape) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(at::kCUDA, dev.index));
}

// Run `call(stream)` on the device's current stream.
template <class F>
void launch(const Device& dev, const char* fn, const F& call) {
  fp8q_status st;
  fp8q_stream_t stream = (fp8q_stream_t)c10::cuda::getCurrentCUDAStream(dev.index).stream();
  Py_BEGIN_ALLOW_THREADS
  st = call(stream);
  Py_END_ALLOW_THREADS
  if (st != FP8Q_OK) {
    PyObject* e = PyObject_CallFunction(g_error, "si", fn, (int)st);
    if (e) {
      PyErr_SetObject((PyObject*)Py_TYPE(e), e);
      Py_DECREF(e);
    }
    refuse(nullptr, "");
  }
}

PyObject* tuple_of(std::initializer_list<PyObject*> items) {
  PyObject* t = PyTuple_New((Py_ssize_t)items.size());
  Py_ssize_t i = 0;
  for (PyObject* o : items) {
    if (!o) {
      for (PyObject* x : items) Py_XDECREF(x);
      Py_XDECREF(t);
      return nullptr;
    }
  }
  if (!t) return nullptr;
  for (PyObject* o : items) PyTuple_SET_ITEM(t, i++, o);
  return t;
}

// The caller's tensor again, or a new one.
PyObject* result(PyObject* given, const at::Tensor& t) { return given != Py_None ? Py_NewRef(given) : THPVariable_Wrap(t); }

template <PyObject* (*F)(PyObject* const*), int N>
PyObject* guarded(PyObject*, PyObject* const* args, Py_ssize_t n) {
  try {
    if (n != N) wrong_type("wrong number of arguments");
    if (!g_error) refuse(PyExc_RuntimeError, "the library has not been bound");
    return F(args);
  } catch (const Refusal& e) {
    if (e.type) PyErr_SetString(e.type, e.what.c_str());
  } catch (const c10::OutOfMemoryError& e) {
    PyErr_SetString(g_out_of_memory, e.what_without_backtrace());
  } catch (const c10::Error& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// q, k_cache, v_cache, k_scales, v_scales, fmt, gran, block_table, lens, scale, window, sinks, out, lse, ws
PyObject* attention(PyObject* const* a) {
  const at::Tensor& q = tensor(a[0], "q", at::kBFloat16);
  const int64_t q_stride = token_stride(q, "q");
  const Cache cache(a + 1);
  const int64_t batch = q.size(0), q_heads = q.size(1), d = q.size(2), heads = cache.c.heads;
  if (d != cache.c.head_dim || q_heads == 0 || heads == 0 || q_heads % heads)
    wrong_value("q must be [batch][q_heads][head_dim] with q_heads a multiple of the cache's heads");
  const at::Tensor& table = contiguous(a[7], "block_table", at::kInt);
  if (table.dim() != 2 || table.size(0) != batch) wrong_value("block_table must be [batch][max_pages]");
  const at::Tensor& lens = shaped(a[8], "lens", at::kInt, {batch});
  const at::Tensor* given_out = nullptr;
  if (a[12] != Py_None) {
    given_out = &tensor(a[12], "out", at::kBFloat16);
    token_stride(*given_out, "out");
    if (given_out->sizes() != q.sizes()) wrong_value("out must have q's shape");
  }
  const at::Tensor* given_lse = a[13] != Py_None ? &shaped(a[13], "lse", at::kFloat, {batch, q_heads}) : nullptr;
  const Device dev(q, "q");
  dev.holds({&cache.k, &cache.v, &cache.ks, &cache.vs, &table, &lens, given_out, given_lse});
  const double scale = a[9] == Py_None ? 1.0 / std::sqrt((double)d) : real(a[9]);
  const int64_t window = integer(a[10]), sinks = integer(a[11]), max_pages = table.size(1);
  const Workspace ws(a[14], g_attention_ws(batch, max_pages * cache.c.page_size, q_heads, heads, d), dev);
  const at::Tensor out = given_out ? *given_out : made(dev, at::kBFloat16, q.sizes());
  const at::Tensor lse = given_lse ? *given_lse : made(dev, at::kFloat, {batch, q_heads});
  const int64_t out_stride = token_stride(out, "out");
  launch(dev, "fp8_attention_paged", [&](fp8q_stream_t st) {
    return g_attention(&cache.c, q.data_ptr(), q_stride, q_heads, (const int32_t*)table.data_ptr(), batch, max_pages,
                       (const int32_t*)lens.data_ptr(), (float)scale, window, sinks, out.data_ptr(), out_stride,
                       (float*)lse.data_ptr(), ws.p, ws.bytes, st);
  });
  return tuple_of({result(a[12], out), result(a[13], lse)});
}

// q, k, v, slots, k_cache, v_cache, k_scales, v_scales, fmt, gran, positions, turns, interleaved, gain, q_weight,
// k_weight, eps, q_out
PyObject* append(PyObject* const* a) {
  const at::Tensor &k = tensor(a[1], "k", at::kBFloat16), &v = tensor(a[2], "v", at::kBFloat16);
  const int64_t k_stride = token_stride(k, "k"), v_stride = token_stride(v, "v");
  const Cache cache(a + 4);
  const int64_t tokens = k.size(0), d = k.size(2);
  if (v.sizes() != k.sizes() || k.size(1) != cache.c.heads || d != cache.c.head_dim)
    wrong_value("k and v must both be [tokens][heads][head_dim] of the cache");
  const at::Tensor& slots = shaped(a[3], "slots", at::kLong, {tokens});
  const at::Tensor *q = nullptr, *given_out = nullptr;
  int64_t q_heads = 0, q_stride = 0, out_stride = 0;
  if (a[0] != Py_None) {
    q = &tensor(a[0], "q", at::kBFloat16);
    q_stride = token_stride(*q, "q");
    if (q->size(0) != tokens || q->size(2) != d) wrong_value("q must be [tokens][q_heads][head_dim]");
    q_heads = q->size(1);
    if (a[17] != Py_None) {
      given_out = &tensor(a[17], "q_out", at::kBFloat16);
      token_stride(*given_out, "q_out");
      if (given_out->sizes() != q->sizes()) wrong_value("q_out must have q's shape");
    }
  } else if (a[17] != Py_None) {
    wrong_value("q_out without q");
  }
  const at::Tensor *turns = nullptr, *positions = nullptr, *q_weight = nullptr, *k_weight = nullptr;
  int64_t rot = 0;
  if (a[11] != Py_None) {
    turns = &contiguous(a[11], "turns", at::kLong);
    rot = 2 * turns->numel();
    if (rot && a[10] == Py_None) wrong_value("turns without positions");
  }
  if (a[10] != Py_None) positions = &shaped(a[10], "positions", at::kInt, {tokens});
  if (a[14] != Py_None) q_weight = &shaped(a[14], "q_weight", at::kBFloat16, {d});
  if (a[15] != Py_None) k_weight = &shaped(a[15], "k_weight", at::kBFloat16, {d});
  const int interleaved = PyObject_IsTrue(a[12]);
  if (interleaved < 0) refuse(nullptr, "");
  const double gain = real(a[13]), eps = real(a[16]);
  const Device dev(k, "k");
  dev.holds({q, &v, &slots, &cache.k, &cache.v, &cache.ks, &cache.vs, positions, turns, q_weight, k_weight, given_out});
  at::Tensor out;
  if (q) {
    out = given_out ? *given_out : made(dev, at::kBFloat16, q->sizes());
    out_stride = token_stride(out, "q_out");
  }
  launch(dev, "fp8_kv_append", [&](fp8q_stream_t st) {
    return g_append(&cache.c, q ? q->data_ptr() : nullptr, q_stride, q_heads, k.data_ptr(), k_stride, v.data_ptr(), v_stride,
                    tokens, (const int64_t*)slots.data_ptr(), positions ? (const int32_t*)positions->data_ptr() : nullptr,
                    turns ? (const uint64_t*)turns->data_ptr() : nullptr, rot, interleaved, (float)gain,
                    q_weight ? q_weight->data_ptr() : nullptr, k_weight ? k_weight->data_ptr() : nullptr, (float)eps,
                    q ? out.data_ptr() : nullptr, out_stride, st);
  });
  if (!q) Py_RETURN_NONE;
  return result(a[17], out);
}

// block_table, lens, added, free_pages, free_count, page_size, max_tokens, slots, positions, offsets, served, lens_out,
// free_count_out, ws
PyObject* update(PyObject* const* a) {
  const at::Tensor& table = contiguous(a[0], "block_table", at::kInt);
  if (table.dim() != 2) wrong_value("block_table must be 2-D [batch][max_pages]");
  const int64_t batch = table.size(0);
  const at::Tensor &lens = shaped(a[1], "lens", at::kInt, {batch}), &added = shaped(a[2], "added", at::kInt, {batch});
  const at::Tensor &free = contiguous(a[3], "free_pages", at::kInt), &count = shaped(a[4], "free_count", at::kInt, {1});
  const int64_t page_size = integer(a[5]);
  int64_t max_tokens;
  if (a[6] != Py_None) {
    max_tokens = integer(a[6]);
    if (max_tokens < 0) wrong_value("max_tokens must not be negative");
  } else {
    if (a[7] == Py_None) wrong_value("max_tokens or slots must be given");
    max_tokens = tensor(a[7], "slots", at::kLong).numel();
  }
  const at::Tensor* slots = a[7] != Py_None ? &shaped(a[7], "slots", at::kLong, {max_tokens}) : nullptr;
  const at::Tensor* positions = a[8] != Py_None ? &shaped(a[8], "positions", at::kInt, {max_tokens}) : nullptr;
  const at::Tensor* offsets = a[9] != Py_None ? &shaped(a[9], "offsets", at::kInt, {batch + 1}) : nullptr;
  const at::Tensor* served = a[10] != Py_None ? &shaped(a[10], "served", at::kInt, {batch}) : nullptr;
  const at::Tensor* lens_out = a[11] != Py_None ? &shaped(a[11], "lens_out", at::kInt, {batch}) : &lens;
  const at::Tensor* count_out = a[12] != Py_None ? &shaped(a[12], "free_count_out", at::kInt, {1}) : &count;
  const Device dev(table, "block_table");
  dev.holds({&lens, &added, &free, &count, slots, positions, offsets, served, lens_out, count_out});
  const Workspace ws(a[13], g_update_ws(batch, max_tokens), dev);
  const at::Tensor t_slots = slots ? *slots : made(dev, at::kLong, {max_tokens});
  const at::Tensor t_positions = positions ? *positions : made(dev, at::kInt, {max_tokens});
  const at::Tensor t_offsets = offsets ? *offsets : made(dev, at::kInt, {batch + 1});
  const at::Tensor t_served = served ? *served : made(dev, at::kInt, {batch});
  launch(dev, "fp8_kv_pages_update", [&](fp8q_stream_t st) {
    return g_update((int32_t*)table.data_ptr(), batch, table.size(1), page_size, (const int32_t*)lens.data_ptr(),
                    (const int32_t*)added.data_ptr(), (int32_t*)lens_out->data_ptr(), (int32_t*)free.data_ptr(), free.numel(),
                    (const int32_t*)count.data_ptr(), (int32_t*)count_out->data_ptr(), max_tokens,
                    (int64_t*)t_slots.data_ptr(), (int32_t*)t_positions.data_ptr(), (int32_t*)t_offsets.data_ptr(),
                    (int32_t*)t_served.data_ptr(), ws.p, ws.bytes, st);
  });
  return tuple_of({result(a[7], t_slots), result(a[8], t_positions), result(a[9], t_offsets), result(a[10], t_served),
                   Py_NewRef(a[11] != Py_None ? a[11] : a[1]), Py_NewRef(a[12] != Py_None ? a[12] : a[4])});
}

// addresses of the five entry points, (name, status) -> exception, and torch's type for a failed allocation
PyObject* bind(PyObject*, PyObject* args) {
  unsigned long long p[5];
  PyObject *error, *out_of_memory;
  if (!PyArg_ParseTuple(args, "KKKKKOO", &p[0], &p[1], &p[2], &p[3], &p[4], &error, &out_of_memory)) return nullptr;
  g_attention = (decltype(g_attention))p[0];
  g_attention_ws = (decltype(g_attention_ws))p[1];
  g_append = (decltype(g_append))p[2];
  g_update = (decltype(g_update))p[3];
  g_update_ws = (decltype(g_update_ws))p[4];
  Py_XSETREF(g_error, Py_NewRef(error));
  Py_XSETREF(g_out_of_memory, Py_NewRef(out_of_memory));
  Py_RETURN_NONE;
}

PyMethodDef g_methods[] = {
    {"bind", bind, METH_VARARGS, nullptr},
    {"attention", (PyCFunction)(void (*)(void))guarded<attention, 15>, METH_FASTCALL, nullptr},
    {"append", (PyCFunction)(void (*)(void))guarded<append, 18>, METH_FASTCALL, nullptr},
    {"update", (PyCFunction)(void (*)(void))guarded<update, 14>, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_torch_calls", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch_calls(void) { return PyModule_Create(&g_module); }
