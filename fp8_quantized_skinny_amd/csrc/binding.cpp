// Python entry of the calls whose buffers are checked as torch tensors: the
// 4-bit key/value cache, the norm and rotation before it and the log probabilities.  Ten attributes of each of
// six tensors, read from Python, took longer than the kernels of a small call
// (append and read of eight rows: 23 us a pass then, 10 this way); here they
// are fields.  Every function returns the status of the C call it makes.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <sstream>
#include <string>
#include <vector>

#include "skinny.h"

namespace {

struct Refusal {
  PyObject* type;
  std::string what;
};
struct PythonError {};  // already set

[[noreturn]] void type_error(const std::string& what) { throw Refusal{PyExc_TypeError, what}; }
[[noreturn]] void value_error(const std::string& what) { throw Refusal{PyExc_ValueError, what}; }

std::string list(at::IntArrayRef v) {
  std::ostringstream s;
  s << '[';
  for (size_t i = 0; i < v.size(); ++i) s << (i ? ", " : "") << v[i];
  s << ']';
  return s.str();
}

const char* name_of(at::ScalarType t) {
  switch (t) {
    case at::kByte: return "torch.uint8";
    case at::kInt: return "torch.int32";
    case at::kHalf: return "torch.float16";
    case at::kBFloat16: return "torch.bfloat16";
    case at::kFloat: return "torch.float32";
    default: return c10::toString(t);
  }
}

// SKINNY_F16, ... of a type, -1 for others.
int type_of(at::ScalarType t) {
  return t == at::kHalf ? SKINNY_F16 : t == at::kBFloat16 ? SKINNY_BF16 : t == at::kFloat ? SKINNY_F32 : -1;
}

const at::Tensor& tensor(PyObject* o, const std::string& name) {
  if (!THPVariable_Check(o)) type_error(name + " must be a CUDA (HIP) torch tensor");
  return THPVariable_Unpack(o);
}

void on_device(const at::Tensor& t, const std::string& name, int device) {
  if (!t.is_cuda()) type_error(name + " must be a CUDA (HIP) torch tensor");
  if (t.get_device() != device)
    value_error(name + " is on " + t.device().str() + ", but the current device is cuda:" + std::to_string(device));
}

// The address of a contiguous device tensor of exactly this type and shape.
void* buffer(PyObject* o, at::ScalarType type, at::IntArrayRef shape, const std::string& name, int device) {
  const at::Tensor& t = tensor(o, name);
  on_device(t, name, device);
  if (t.scalar_type() != type) type_error(name + " must be " + name_of(type) + ", got " + name_of(t.scalar_type()));
  if (t.sizes() != shape) value_error(name + " must be " + list(shape) + ", got " + list(t.sizes()));
  if (!t.is_contiguous()) value_error(name + " must be contiguous");
  return t.data_ptr();
}
float* floats(PyObject* o, at::IntArrayRef shape, const char* name, int device) {
  return static_cast<float*>(buffer(o, at::kFloat, shape, name, device));
}
int32_t* ints(PyObject* o, at::IntArrayRef shape, const char* name, int device) {
  return static_cast<int32_t*>(buffer(o, at::kInt, shape, name, device));
}

// A [B, T, heads, D] view; the C call checks pointer and strides.
struct Rows {
  kv4_rows rows;
  at::IntArrayRef shape;
  at::ScalarType type;
};
Rows rows_of(PyObject* o, const std::string& name, int device) {
  const at::Tensor& t = tensor(o, name);
  on_device(t, name, device);
  if (type_of(t.scalar_type()) < 0 || t.dim() != 4) type_error(name + " must be float16 or bfloat16 [B, T, heads, D]");
  const auto n = t.sizes(), s = t.strides();
  if (n[0] < 1 || n[1] < 1 || n[2] < 1) value_error(name + " is empty");
  if (s[3] != 1 && n[3] > 1) value_error("the last dimension of " + name + " must be contiguous");
  // A dimension of one entry may have any stride.
  return Rows{{t.data_ptr(), n[0] > 1 ? s[0] : 0, n[1] > 1 ? s[1] : 0, n[2] > 1 ? s[2] : 0}, n, t.scalar_type()};
}

int as_int(int64_t v, const char* name) {
  if (v > INT32_MAX) value_error(std::string(name) + " is too large");
  return static_cast<int>(v);
}

kv4_cache cache_of(PyObject* cache, PyObject* table, PyObject* lens, float gk, float gv, int device,
                   const std::string& prefix = "") {
  const at::Tensor &c = tensor(cache, prefix + "cache"), &t = tensor(table, prefix + "table");
  if (c.dim() != 3 || c.size(2) % 72) value_error(prefix + "cache must be uint8 [pages, Hk, 72 * D]");
  if (t.dim() != 2) value_error(prefix + "table must be int32 [B, width]");
  kv4_cache out{};
  out.data = buffer(cache, at::kByte, c.sizes(), prefix + "cache", device);
  out.table = static_cast<int32_t*>(buffer(table, at::kInt, t.sizes(), prefix + "table", device));
  out.lens = lens ? ints(lens, {t.size(0)}, "lens", device) : nullptr;
  out.pages = as_int(c.size(0), "the number of pages");
  out.width = as_int(t.size(1), "the width of the table");
  out.B = as_int(t.size(0), "the number of sequences");
  out.Hk = as_int(c.size(1), "the number of heads");
  out.D = as_int(c.size(2) / 72, "the head size");
  out.gk = gk;
  out.gv = gv;
  return out;
}

void same_shape(const Rows& r, const char* name, const kv4_cache& c, int64_t T) {
  const int64_t want[4] = {c.B, T, c.Hk, c.D};
  if (r.shape != at::IntArrayRef(want, 4))
    value_error(std::string(name) + " must be [B, T, Hk, D] = " + list(at::IntArrayRef(want, 4)) + ", got " + list(r.shape));
}

Rows queries(PyObject* o, const kv4_cache& c, int device) {
  const Rows q = rows_of(o, "q", device);
  if (q.shape[0] != c.B || q.shape[3] != c.D)
    value_error("q must be [B, T, Hq, D] with B = " + std::to_string(c.B) + ", D = " + std::to_string(c.D) + ", got " + list(q.shape));
  return q;
}

struct Scratch {
  void* data;
  size_t bytes;
};
Scratch scratch(PyObject* o, size_t need, const char* where, int device) {
  const std::string missing = std::string(where) + ": a workspace of at least " + std::to_string(need) + " bytes is required";
  if (o == Py_None) {
    if (need) value_error(missing);
    return Scratch{nullptr, 0};
  }
  const at::Tensor& t = tensor(o, "workspace");
  if (static_cast<size_t>(t.numel()) < need) value_error(missing);
  return Scratch{buffer(o, at::kByte, t.sizes(), "workspace", device), static_cast<size_t>(t.numel())};
}

float number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw PythonError{};
  return static_cast<float>(v);
}
int integer(PyObject* o) {
  const long v = PyLong_AsLong(o);
  if (v == -1 && PyErr_Occurred()) throw PythonError{};
  if (v > INT32_MAX || v < INT32_MIN) value_error("an integer is too large");
  return static_cast<int>(v);
}

// A torch stream, a raw handle, or None for torch's current stream.
hipStream_t stream_of(PyObject* o, int device) {
  if (o == Py_None) return c10::hip::getCurrentHIPStream(static_cast<c10::DeviceIndex>(device)).stream();
  PyObject* handle = PyLong_Check(o) ? Py_NewRef(o) : PyObject_GetAttrString(o, "cuda_stream");
  if (!handle) throw PythonError{};
  void* p = PyLong_AsVoidPtr(handle);
  Py_DECREF(handle);
  if (!p && PyErr_Occurred()) throw PythonError{};
  return static_cast<hipStream_t>(p);
}

// ---- the calls: arguments in the order of kv4.py --------------------------
int append(PyObject* const* a, int dev) {  // cache, table, lens, k, v, gk, gv, stream
  const kv4_cache c = cache_of(a[0], a[1], a[2], number(a[5]), number(a[6]), dev);
  const Rows k = rows_of(a[3], "k", dev), v = rows_of(a[4], "v", dev);
  const int64_t T = k.shape[1];
  same_shape(k, "k", c, T);
  same_shape(v, "v", c, T);
  if (k.type != v.type) type_error("k and v must have one type");
  return kv4_append(&c, &k.rows, &v.rows, type_of(k.type), as_int(T, "T"), stream_of(a[7], dev));
}

int read(PyObject* const* a, int dev) {  // cache, table, lens, k, v, gk, gv, stream
  const kv4_cache c = cache_of(a[0], a[1], a[2], number(a[5]), number(a[6]), dev);
  const at::Tensor& k = tensor(a[3], "k");
  if (k.dim() != 4) value_error("k must be [B, n, Hk, D]");
  const int64_t n = k.size(1), shape[4] = {c.B, n, c.Hk, c.D};
  void* kp = buffer(a[3], k.scalar_type(), at::IntArrayRef(shape, 4), "k", dev);
  void* vp = buffer(a[4], k.scalar_type(), at::IntArrayRef(shape, 4), "v", dev);
  return kv4_read(&c, kp, vp, type_of(k.scalar_type()), as_int(n, "n"), stream_of(a[7], dev));
}

int attention(PyObject* const* a, int dev) {  // q, cache, table, lens, out, lse, scale, gk, gv, workspace, stream
  const kv4_cache c = cache_of(a[1], a[2], a[3], number(a[7]), number(a[8]), dev);
  const Rows q = queries(a[0], c, dev);
  const int T = as_int(q.shape[1], "T"), Hq = as_int(q.shape[2], "Hq");
  void* out = buffer(a[4], q.type, q.shape, "out", dev);
  float* lse = a[5] == Py_None ? nullptr : floats(a[5], {c.B, T, Hq}, "lse", dev);
  const float scale = a[6] == Py_None ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(c.D))) : number(a[6]);
  const Scratch ws = scratch(a[9], kv4_attention_workspace_bytes(c.B, T, Hq, c.Hk, c.D, c.width), "kv4_attention", dev);
  return kv4_attention(&c, &q.rows, type_of(q.type), T, Hq, scale, out, lse, ws.data, ws.bytes, stream_of(a[10], dev));
}

// q, cache, table, lens, out, window, sinks, lse, scale, gk, gv, workspace, stream
int attention_window(PyObject* const* a, int dev) {
  const kv4_cache c = cache_of(a[1], a[2], a[3], number(a[9]), number(a[10]), dev);
  const Rows q = queries(a[0], c, dev);
  const int T = as_int(q.shape[1], "T"), Hq = as_int(q.shape[2], "Hq"), window = integer(a[5]), sinks = integer(a[6]);
  void* out = buffer(a[4], q.type, q.shape, "out", dev);
  float* lse = a[7] == Py_None ? nullptr : floats(a[7], {c.B, T, Hq}, "lse", dev);
  const float scale = a[8] == Py_None ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(c.D))) : number(a[8]);
  const Scratch ws = scratch(a[11], kv4_attention_window_workspace_bytes(c.B, T, Hq, c.Hk, c.D, c.width, window, sinks),
                             "kv4_attention_window", dev);
  return kv4_attention_window(&c, &q.rows, type_of(q.type), T, Hq, scale, window, sinks, out, lse, ws.data, ws.bytes,
                              stream_of(a[12], dev));
}

// q, starts, cache, table, lens, out, lse, scale, window, sinks, gk, gv, workspace, stream
int attention_chunk(PyObject* const* a, int dev) {
  const kv4_cache c = cache_of(a[2], a[3], a[4], number(a[10]), number(a[11]), dev);
  const at::Tensor& q = tensor(a[0], "q");
  on_device(q, "q", dev);
  if (type_of(q.scalar_type()) < 0 || q.dim() != 3) type_error("q must be float16 or bfloat16 [N, Hq, D]");
  const auto n = q.sizes(), s = q.strides();
  if (n[0] < 1 || n[1] < 1) value_error("q is empty");
  if (n[2] != c.D) value_error("q must be [N, Hq, D] with D = " + std::to_string(c.D) + ", got " + list(n));
  if (s[2] != 1) value_error("the last dimension of q must be contiguous");
  const int N = as_int(n[0], "N"), Hq = as_int(n[1], "Hq"), window = integer(a[8]), sinks = integer(a[9]);
  const int32_t* starts = ints(a[1], {c.B + 1}, "starts", dev);
  void* out = buffer(a[5], q.scalar_type(), n, "out", dev);
  float* lse = a[6] == Py_None ? nullptr : floats(a[6], {N, Hq}, "lse", dev);
  const float scale = a[7] == Py_None ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(c.D))) : number(a[7]);
  const Scratch ws = scratch(a[12], kv4_attention_chunk_workspace_bytes(N, c.B, Hq, c.Hk, c.D, c.width, window, sinks),
                             "kv4_attention_chunk", dev);
  return kv4_attention_chunk(&c, q.data_ptr(), N > 1 ? s[0] : 0, Hq > 1 ? s[1] : 0, starts, N, type_of(q.scalar_type()), Hq,
                             scale, window, sinks, out, lse, ws.data, ws.bytes, stream_of(a[13], dev));
}

// q, k, positions, inv_freq, q_out, k_out, q_weight, k_weight, eps, amplitude, interleaved, stream
int norm_rope(PyObject* const* a, int dev) {
  // [N, heads, D] is one sequence of N tokens.
  const auto heads = [&](PyObject* o, const std::string& name) {
    const at::Tensor& t = tensor(o, name);
    on_device(t, name, dev);
    const auto type = type_of(t.scalar_type());
    const int64_t d = t.dim();
    if ((type != SKINNY_F16 && type != SKINNY_BF16) || (d != 3 && d != 4))
      type_error(name + " must be float16 or bfloat16 [B, T, heads, D] or [N, heads, D]");
    const auto n = t.sizes(), s = t.strides();
    for (const int64_t x : n)
      if (x < 1) value_error(name + " is empty");
    if (s[d - 1] != 1 && n[d - 1] > 1) value_error("the last dimension of " + name + " must be contiguous");
    return Rows{{t.data_ptr(), d == 4 && n[0] > 1 ? s[0] : 0, n[d - 3] > 1 ? s[d - 3] : 0, n[d - 2] > 1 ? s[d - 2] : 0}, n, t.scalar_type()};
  };
  const Rows q = heads(a[0], "q"), k = heads(a[1], "k"), qo = heads(a[4], "q_out"), ko = heads(a[5], "k_out");
  const size_t d = q.shape.size();
  const int64_t D = q.shape[d - 1];
  if (k.shape.size() != d || k.shape[d - 1] != D || k.shape.slice(0, d - 2) != q.shape.slice(0, d - 2))
    value_error("k must have q's tokens and head size " + list(q.shape) + ", got " + list(k.shape));
  if (qo.shape != q.shape) value_error("q_out must be " + list(q.shape) + ", got " + list(qo.shape));
  if (ko.shape != k.shape) value_error("k_out must be " + list(k.shape) + ", got " + list(ko.shape));
  if (k.type != q.type || qo.type != q.type || ko.type != q.type) type_error("q, k, q_out and k_out must have one type");
  const int32_t* positions = ints(a[2], q.shape.slice(0, d - 2), "positions", dev);
  const at::Tensor& f = tensor(a[3], "inv_freq");
  if (f.dim() != 1) value_error("inv_freq must be float32 [rot / 2]");
  const float* freq = floats(a[3], f.sizes(), "inv_freq", dev);
  const int rot = 2 * as_int(f.size(0) < (1 << 20) ? f.size(0) : 1 << 20, "rot");
  const float* qw = a[6] == Py_None ? nullptr : floats(a[6], {D}, "q_weight", dev);
  const float* kw = a[7] == Py_None ? nullptr : floats(a[7], {D}, "k_weight", dev);
  const int interleaved = PyObject_IsTrue(a[10]);
  if (interleaved < 0) throw PythonError{};
  return qk_norm_rope(&q.rows, &k.rows, positions, rot ? freq : nullptr, qw, kw, type_of(q.type), as_int(d == 4 ? q.shape[0] : 1, "B"),
                      as_int(q.shape[d - 3], "T"), as_int(q.shape[d - 2], "Hq"), as_int(k.shape[d - 2], "Hk"), as_int(D, "D"), rot,
                      interleaved, number(a[8]), number(a[9]), &qo.rows, &ko.rows, stream_of(a[11], dev));
}

int weights(PyObject* const* a, int dev) {  // q, cache, table, lens, lse, acc, acc_out, scale, gk, stream
  const kv4_cache c = cache_of(a[1], a[2], a[3], number(a[8]), 1.0f, dev);
  const Rows q = queries(a[0], c, dev);
  const int T = as_int(q.shape[1], "T"), Hq = as_int(q.shape[2], "Hq");
  const float* lse = floats(a[4], {c.B, T, Hq}, "lse", dev);
  const int64_t slots = int64_t{SKINNY_KV_PAGE} * c.width;
  const float* acc = floats(a[5], {c.B, c.Hk, slots}, "acc", dev);
  float* acc_out = floats(a[6], {c.B, c.Hk, slots}, "acc_out", dev);
  const float scale = a[7] == Py_None ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(c.D))) : number(a[7]);
  return kv4_attention_weights(&c, &q.rows, type_of(q.type), T, Hq, scale, lse, acc, acc_out, stream_of(a[9], dev));
}

// cache, table, lens, acc, dst_cache, dst_table, kept, new_lens, new_acc, sinks, recent, stream
int evict(PyObject* const* a, int dev) {
  const kv4_cache c = cache_of(a[0], a[1], a[2], 1.0f, 1.0f, dev), d = cache_of(a[4], a[5], nullptr, 1.0f, 1.0f, dev, "dst_");
  if (d.B != c.B || d.Hk != c.Hk || d.D != c.D)
    value_error("dst_cache and dst_table must have the cache's sequences, heads and head size");
  const at::Tensor& kept = tensor(a[6], "kept");
  if (kept.dim() != 3) value_error("kept must be int32 [B, Hk, keep]");
  const int keep = as_int(kept.size(2), "keep");
  const float* acc = floats(a[3], {c.B, c.Hk, int64_t{SKINNY_KV_PAGE} * c.width}, "acc", dev);
  int32_t* ids = ints(a[6], {c.B, c.Hk, keep}, "kept", dev);
  int32_t* lens = ints(a[7], {c.B}, "new_lens", dev);
  float* new_acc = floats(a[8], {c.B, c.Hk, int64_t{SKINNY_KV_PAGE} * d.width}, "new_acc", dev);
  return kv4_evict(&c, acc, &d, ids, lens, new_acc, keep, integer(a[9]), integer(a[10]), stream_of(a[11], dev));
}

int logprobs(PyObject* const* a, int dev) {  // logits, tokens, logprob, entropy, top_ids, top_logprobs, workspace, stream
  const at::Tensor &x = tensor(a[0], "logits"), &top = tensor(a[4], "top_ids");
  on_device(x, "logits", dev);
  if (type_of(x.scalar_type()) < 0 || x.dim() != 2) type_error("logits must be float16, bfloat16 or float32 [R, V]");
  if (x.stride(1) != 1 && x.size(1) > 1) value_error("the rows of logits must be contiguous");
  if (top.dim() != 2) value_error("top_ids must be int32 [R, k]");
  const int R = as_int(x.size(0), "R"), V = as_int(x.size(1), "V"), k = as_int(top.size(1), "k");
  const int32_t* tokens = ints(a[1], {R}, "tokens", dev);
  float *lp = floats(a[2], {R}, "logprob", dev), *entropy = floats(a[3], {R}, "entropy", dev);
  int32_t* ids = ints(a[4], {R, k}, "top_ids", dev);
  float* top_lp = floats(a[5], {R, k}, "top_logprobs", dev);
  const Scratch ws = scratch(a[6], lm_head_logprobs_workspace_bytes(R, V, k), "lm_head_logprobs", dev);
  return lm_head_logprobs(x.data_ptr(), type_of(x.scalar_type()), R > 1 ? x.stride(0) : V, tokens, lp, entropy, ids, top_lp,
                          R, V, k, ws.data, ws.bytes, stream_of(a[7], dev));
}

template <class F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (const Refusal& r) {
    PyErr_SetString(r.type, r.what.c_str());
  } catch (const PythonError&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

template <int (*CALL)(PyObject* const*, int), int COUNT>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != COUNT) type_error(std::to_string(COUNT) + " arguments are wanted");
    return PyLong_FromLong(CALL(a, c10::hip::current_device()));
  });
}

PyObject* check_buffer(PyObject*, PyObject* const* a, Py_ssize_t n) {  // tensor, dtype, shape, name, device
  return guarded([&]() -> PyObject* {
    if (n != 5 || !THPDtype_Check(a[1]) || !PyTuple_Check(a[2])) type_error("a tensor, dtype, shape, name and device are wanted");
    std::vector<int64_t> shape;
    for (Py_ssize_t i = 0; i < PyTuple_GET_SIZE(a[2]); ++i) shape.push_back(integer(PyTuple_GET_ITEM(a[2], i)));
    const char* name = PyUnicode_AsUTF8(a[3]);
    if (!name) throw PythonError{};
    return PyLong_FromVoidPtr(buffer(a[0], reinterpret_cast<THPDtype*>(a[1])->scalar_type, shape, name, integer(a[4])));
  });
}

template <class F>
PyMethodDef method(const char* name, F* f) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)), METH_FASTCALL, nullptr};
}
PyMethodDef methods[] = {method("kv4_append", entry<append, 8>),
                         method("kv4_read", entry<read, 8>),
                         method("kv4_attention", entry<attention, 11>),
                         method("kv4_attention_window", entry<attention_window, 13>),
                         method("kv4_attention_chunk", entry<attention_chunk, 14>),
                         method("qk_norm_rope", entry<norm_rope, 12>),
                         method("kv4_attention_weights", entry<weights, 10>),
                         method("kv4_evict", entry<evict, 12>),
                         method("lm_head_logprobs", entry<logprobs, 8>),
                         method("buffer", check_buffer),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// torch_version: of the headers that this was compiled with (SKINNY_TORCH_VERSION
// comes from the build).  Tensors' fields are read in place, so the loader takes
// no other.
PyMODINIT_FUNC PyInit__binding() {
  PyObject* m = PyModule_Create(&module);
  if (m && PyModule_AddStringConstant(m, "torch_version", SKINNY_TORCH_VERSION) < 0) {
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
