// Calls of the serving operators from Python: tensors checked and handed on as addresses, strides and the current stream.
// Argument marshalling only, as in __init__.py, whose functions call these; compiled because in Python it takes two to three
// times as long as the launch (a call of qk_norm_rope 10.2 us, of paged_kv_resize 7.6).
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <sstream>
#include <string>

#include "medusa_verify.h"

namespace {

// Thrown with the Python error set.
struct Raised {};

template <typename... T>
[[noreturn]] void refuse(const T&... parts) {
  std::ostringstream s;
  (s << ... << parts);
  PyErr_SetString(PyExc_ValueError, s.str().c_str());
  throw Raised();
}

const at::Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) {
    PyErr_Format(PyExc_TypeError, "%s: a tensor is wanted, got %s", what, Py_TYPE(o)->tp_name);
    throw Raised();
  }
  return THPVariable_Unpack(o);
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised();
  return v;
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised();
  return v;
}
int32_t int32_of(int64_t v, const char* what) {
  if (v < INT32_MIN || v > INT32_MAX) refuse(what, ": ", v, " does not fit in 32 bits");
  return (int32_t)v;
}

int device_of(const at::Tensor& t) { return t.is_cuda() ? t.get_device() : -1; }

// [tokens, heads, head_dim]
void want3(const at::Tensor& t, const char* what) {
  if (t.dim() != 3) refuse(what, ": [tokens, heads, head_dim] is wanted, got ", t.sizes());
}

// A bf16 tensor [tokens, heads, dim] on `dev`; its last dimension must be contiguous.
mv_rows rows(const at::Tensor& t, const char* what, int dev, int64_t heads, int64_t dim, int64_t tokens) {
  if (t.scalar_type() != at::kBFloat16 || t.dim() != 3 || t.size(0) != tokens || t.size(1) != heads || t.size(2) != dim ||
      dev < 0 || device_of(t) != dev || (t.stride(2) != 1 && dim != 1))
    refuse(what, ": a bf16 tensor [", tokens, ", ", heads, ", ", dim, "] on CUDA device ", dev,
           " with a contiguous last dimension is wanted, got ", t.scalar_type(), " ", t.sizes(), " on ", t.device(),
           " with strides ", t.strides());
  return {t.data_ptr(), tokens > 1 ? t.stride(0) : 0, heads > 1 ? t.stride(1) : 0};
}

// A contiguous 1-D tensor of n values of `type` on `dev`.
template <typename T>
T* vector_of(const at::Tensor& t, const char* what, int dev, int64_t n, at::ScalarType type) {
  if (t.scalar_type() != type || t.dim() != 1 || t.size(0) != n || dev < 0 || device_of(t) != dev || !t.is_contiguous())
    refuse(what, ": a contiguous tensor of ", n, " ", type, " on CUDA device ", dev, " is wanted, got ", t.scalar_type(), " ",
           t.sizes(), " on ", t.device(), " with strides ", t.strides());
  return static_cast<T*>(t.data_ptr());
}
int32_t* ints(PyObject* o, const char* what, int dev, int64_t n) {
  return vector_of<int32_t>(tensor(o, what), what, dev, n, at::kInt);
}

// block_table int32 [n_seq, pages], whose rows may lie further apart, and seq_lens int32 [n_seq].
struct Sequences {
  int32_t *table, *lens, ld, pages, n;
  Sequences(PyObject* block_table, PyObject* seq_lens, int dev) {
    const at::Tensor& t = tensor(block_table, "block_table");
    if (t.dim() != 2) refuse("block_table: [n_seq, pages] is wanted, got ", t.sizes());
    if (t.scalar_type() != at::kInt || device_of(t) != dev || !(t.is_contiguous() || t.stride(1) == 1))
      refuse("block_table: an int32 tensor on CUDA device ", dev, " with contiguous rows is wanted, got ", t.scalar_type(), " ",
             t.sizes(), " on ", t.device(), " with strides ", t.strides());
    n = int32_of(t.size(0), "block_table");
    pages = int32_of(t.size(1), "block_table");
    ld = n > 1 ? int32_of(t.stride(0), "block_table") : pages;
    table = static_cast<int32_t*>(t.data_ptr());
    lens = ints(seq_lens, "seq_lens", dev, n);
  }
};

// The stream to launch on, with its device current while this lives.
struct On {
  c10::cuda::OptionalCUDAGuard guard;
  mv_stream stream;
  On(PyObject* o, int dev, const char* name) {
    if (dev < 0) refuse(name, ": the tensors are not on a CUDA device");
    if (o == Py_None) {
      stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
    } else {
      // whatever has a device and a raw pointer: torch's streams, and those of others that say as much
      PyObject *raw = PyObject_GetAttrString(o, "cuda_stream"), *at = raw ? PyObject_GetAttrString(o, "device") : nullptr;
      PyObject* nth = at ? PyObject_GetAttrString(at, "index") : nullptr;
      const bool here = nth && PyLong_Check(nth) && PyLong_AsLongLong(nth) == dev;
      const int64_t ptr = raw ? PyLong_AsLongLong(raw) : -1;
      PyObject* is_on = nth && !here && !PyErr_Occurred() ? PyObject_Str(at) : nullptr;
      const char* text = is_on ? PyUnicode_AsUTF8(is_on) : nullptr;
      const std::string device = text ? text : "";
      Py_XDECREF(raw);
      Py_XDECREF(at);
      Py_XDECREF(nth);
      Py_XDECREF(is_on);
      if (PyErr_Occurred()) throw Raised();
      if (!here) refuse(name, ": the stream is on ", device, ", the tensors are on CUDA device ", dev);
      stream = reinterpret_cast<mv_stream>(ptr);
    }
    if (c10::cuda::current_device() != dev) guard.set_index((c10::DeviceIndex)dev);
  }
};

// f(), which throws nothing, without the interpreter's lock; its status as a Python integer.
template <typename F>
PyObject* launched(F&& f) {
  mv_status s;
  Py_BEGIN_ALLOW_THREADS
  s = f();
  Py_END_ALLOW_THREADS
  return PyLong_FromLong(s);
}

const mv_paged_kv* cache_at(PyObject* o) { return reinterpret_cast<const mv_paged_kv*>(integer(o)); }

// q, k, v, out, address of the plan, its tokens, scale, stream
PyObject* prompt(PyObject* const* a) {
  const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k");
  want3(q, "q");
  want3(k, "k");
  const int dev = device_of(q);
  const int64_t t = q.size(0), hq = q.size(1), d = q.size(2), hk = k.size(1), n = integer(a[5]);
  if (t < n) refuse("prompt_attention: the plan has ", n, " tokens, q ", t);
  const mv_rows qr = rows(q, "q", dev, hq, d, t), kr = rows(k, "k", dev, hk, d, t);
  const mv_rows vr = rows(tensor(a[2], "v"), "v", dev, hk, d, t), out = rows(tensor(a[3], "out"), "out", dev, hq, d, t);
  const auto* plan = reinterpret_cast<const mv_prompt_plan*>(integer(a[4]));
  const float scale = (float)number(a[6]);
  const int32_t heads = int32_of(hq, "q"), kv_heads = int32_of(hk, "k"), dim = int32_of(d, "q");
  const On on(a[7], dev, "prompt_attention");
  return launched([&] { return prompt_attention(qr, kr, vr, heads, kv_heads, dim, plan, scale, out, on.stream); });
}

// k, v, cu_rows, address of the cache, its device, block_table, seq_lens, stream
template <bool kWrite>
PyObject* move_rows(PyObject* const* a) {
  const mv_paged_kv* c = cache_at(a[3]);
  const int dev = (int)integer(a[4]);
  const Sequences s(a[5], a[6], dev);
  const at::Tensor& k = tensor(a[0], kWrite ? "k" : "k_out");
  want3(k, kWrite ? "k" : "k_out");
  const int64_t n = k.size(0);
  const mv_rows kr = rows(k, kWrite ? "k" : "k_out", dev, c->n_kv_heads, c->head_dim, n);
  const mv_rows vr = rows(tensor(a[1], kWrite ? "v" : "v_out"), kWrite ? "v" : "v_out", dev, c->n_kv_heads, c->head_dim, n);
  const int32_t *cu = ints(a[2], "cu_rows", dev, (int64_t)s.n + 1), n_rows = int32_of(n, "rows");
  const On on(a[7], dev, kWrite ? "paged_kv_append" : "paged_kv_read");
  return launched([&] {
    return kWrite ? paged_kv_append(kr, vr, n_rows, cu, c, s.table, s.ld, s.pages, s.lens, s.n, on.stream)
                  : paged_kv_read(c, s.table, s.ld, s.pages, s.lens, s.n, cu, n_rows, kr, vr, on.stream);
  });
}

// q, out, workspace, scale, address of the cache, its device, block_table, seq_lens, stream
PyObject* attention(PyObject* const* a) {
  const mv_paged_kv* c = cache_at(a[4]);
  const int dev = (int)integer(a[5]);
  const Sequences s(a[6], a[7], dev);
  const at::Tensor &q = tensor(a[0], "q"), &ws = tensor(a[2], "workspace");
  want3(q, "q");
  const int64_t heads = q.size(1);
  if (device_of(ws) != dev || !ws.is_contiguous())
    refuse("paged_attention: a contiguous workspace on CUDA device ", dev, " is wanted");
  const mv_rows qr = rows(q, "q", dev, heads, c->head_dim, s.n);
  const mv_rows out = rows(tensor(a[1], "out"), "out", dev, heads, c->head_dim, s.n);
  const float scale = (float)number(a[3]);
  const On on(a[8], dev, "paged_attention");
  const int32_t n_heads = int32_of(heads, "q");
  return launched([&] {
    return paged_attention(qr, n_heads, c, s.table, s.ld, s.pages, s.lens, s.n, scale, out, ws.data_ptr(), ws.nbytes(), on.stream);
  });
}

// by, free_pages, cu_rows, positions, slots, address of the cache, its device, block_table, seq_lens, stream
PyObject* resize(PyObject* const* a) {
  const mv_paged_kv* c = cache_at(a[5]);
  const int dev = (int)integer(a[6]);
  const Sequences s(a[7], a[8], dev);
  const int32_t* by = ints(a[0], "by", dev, s.n);
  int32_t* free_pages = ints(a[1], "free_pages", dev, 1 + (int64_t)c->n_pages);
  static int64_t no_rows;  // the address of tensors without elements, whose own says that they are not wanted; never used
  int32_t *cu = nullptr, *positions = nullptr;
  int64_t *slots = nullptr, n = 0;
  if (a[2] != Py_None) cu = ints(a[2], "cu_rows", dev, (int64_t)s.n + 1);
  else if (a[3] != Py_None || a[4] != Py_None) refuse("paged_kv_resize: positions and slots are of the rows that cu_rows counts");
  if (a[3] != Py_None) {
    n = tensor(a[3], "positions").numel();
    positions = ints(a[3], "positions", dev, n);
    if (!n) positions = reinterpret_cast<int32_t*>(&no_rows);
  }
  if (a[4] != Py_None) {
    const at::Tensor& t = tensor(a[4], "slots");
    if (!positions) n = t.numel();
    slots = vector_of<int64_t>(t, "slots", dev, n, at::kLong);
    if (!n) slots = &no_rows;
  }
  const int32_t n_rows = int32_of(n, "rows");
  const On on(a[9], dev, "paged_kv_resize");
  return launched([&] {
    return paged_kv_resize(by, s.n, c->page_size, c->n_pages, s.table, s.ld, s.pages, s.lens, free_pages, cu, positions, slots,
                           n_rows, on.stream);
  });
}

// q, k, q_gain, k_gain, q_out, k_out, eps, positions, turns (a tensor or None), neighbours, stream
PyObject* norm_rope(PyObject* const* a) {
  if (a[0] == Py_None && a[1] == Py_None) refuse("qk_norm_rope: q and k are both None");
  const at::Tensor& x = tensor(a[0] != Py_None ? a[0] : a[1], a[0] != Py_None ? "q" : "k");
  want3(x, a[0] != Py_None ? "q" : "k");
  const int dev = device_of(x);
  const int64_t t = x.size(0), d = x.size(2);
  const char *names[2] = {"q", "k"}, *gains[2] = {"q_gain", "k_gain"}, *outs[2] = {"q_out", "k_out"};
  mv_rows from[2] = {}, to[2] = {};
  int32_t heads[2] = {};
  const mv_bf16* gain[2] = {};
  for (int i = 0; i < 2; ++i) {
    if (a[i] == Py_None) {
      if (a[2 + i] != Py_None || a[4 + i] != Py_None) refuse("qk_norm_rope: ", names[i], " is None, its gain or output is not");
      continue;
    }
    const at::Tensor& src = tensor(a[i], names[i]);
    want3(src, names[i]);
    heads[i] = int32_of(src.size(1), names[i]);
    from[i] = to[i] = rows(src, names[i], dev, heads[i], d, t);
    if (a[2 + i] != Py_None) gain[i] = vector_of<mv_bf16>(tensor(a[2 + i], gains[i]), gains[i], dev, d, at::kBFloat16);
    if (a[4 + i] != Py_None) to[i] = rows(tensor(a[4 + i], outs[i]), outs[i], dev, heads[i], d, t);
  }
  const float eps = (float)number(a[6]);
  const int32_t* positions = a[7] == Py_None ? nullptr : ints(a[7], "positions", dev, t);
  const uint64_t* turns = nullptr;
  int32_t rot_dim = 0;
  if (a[8] != Py_None) {
    const at::Tensor& w = tensor(a[8], "rope");
    if (a[7] == Py_None) refuse("qk_norm_rope: a rotation wants positions");
    turns = vector_of<uint64_t>(w, "rope", dev, w.numel(), at::kLong);
    rot_dim = int32_of(2 * w.numel(), "rope");
  }
  const int32_t neighbours = (int32_t)integer(a[9]), n = int32_of(t, "tokens"), dim = int32_of(d, "head_dim");
  const On on(a[10], dev, "qk_norm_rope");
  return launched([&] {
    return qk_norm_rope(from[0], from[1], n, heads[0], heads[1], dim, gain[0], gain[1], eps, positions, turns, rot_dim, neighbours,
                        to[0], to[1], on.stream);
  });
}

template <PyObject* (*kF)(PyObject* const*), int kArgs>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != kArgs) return PyErr_Format(PyExc_TypeError, "%d arguments are wanted, got %zd", kArgs, n);
  try {
    return kF(args);
  } catch (const Raised&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

#define ENTRY(name, f, n) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<f, n>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ENTRY("prompt_attention", prompt, 8),
                         ENTRY("paged_kv_append", move_rows<true>, 8),
                         ENTRY("paged_kv_read", move_rows<false>, 8),
                         ENTRY("paged_attention", attention, 9),
                         ENTRY("paged_kv_resize", resize, 10),
                         ENTRY("qk_norm_rope", norm_rope, 11),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__calls() { return PyModule_Create(&module); }
