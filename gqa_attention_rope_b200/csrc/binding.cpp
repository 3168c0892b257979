// binding.cpp -- the Python module _binding: argument checks and calls of the
// paged-cache entry points of include/llama_attn.h.
//
// A decode step makes several of these calls, each a few microseconds of GPU
// work. Checking a dozen tensors takes the interpreter 5 to 8 us a call and
// ctypes 2 us to convert the arguments; here both take under 1 us. Nothing is
// computed: tensors become pointers and sizes, a bad one becomes a ValueError,
// and the library's status is returned. The entry points' addresses come from
// the loaded library (the package passes them), so this file links to none.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <initializer_list>
#include <limits>
#include <stdexcept>
#include <string>

#include "llama_attn.h"

namespace {

// A Python error that has been set already.
struct PythonError {};

struct Args {
  PyObject* const* at;
  Py_ssize_t n, i = 0;
  PyObject* next() {
    if (i >= n) throw std::invalid_argument("too few arguments");
    return at[i++];
  }
  const at::Tensor& tensor(const char* name) {
    PyObject* o = next();
    if (!THPVariable_Check(o)) throw std::invalid_argument(std::string(name) + ": tensor expected");
    return THPVariable_Unpack(o);
  }
  const at::Tensor* tensor_or_none(const char* name) {
    if (i < n && at[i] == Py_None) {
      ++i;
      return nullptr;
    }
    return &tensor(name);
  }
  int integer(const char* name) {
    const long x = PyLong_AsLong(next());
    if (x == -1 && PyErr_Occurred()) throw PythonError{};
    if (x < std::numeric_limits<int>::min() || x > std::numeric_limits<int>::max())
      throw std::invalid_argument(std::string(name) + ": out of range");
    return static_cast<int>(x);
  }
  float real() {
    const double x = PyFloat_AsDouble(next());
    if (x == -1.0 && PyErr_Occurred()) throw PythonError{};
    return static_cast<float>(x);
  }
  template <typename Fn>
  Fn function() {
    void* p = PyLong_AsVoidPtr(next());
    if (p == nullptr) throw PythonError{};
    return reinterpret_cast<Fn>(p);
  }
};

[[noreturn]] void refuse(const char* name, const at::Tensor& t, const std::string& expected) {
  throw std::invalid_argument(c10::str(name, ": ", expected, " expected, got ", t.sizes(), " ", t.scalar_type(), " on ",
                                       t.device(), ", strides ", t.strides()));
}
// The CUDA device of the call, from its first tensor.
int device_of(const char* name, const at::Tensor& t) {
  if (!t.is_cuda()) throw std::invalid_argument(std::string(name) + ": CUDA tensor expected");
  return t.device().index();
}
void check_dims(const char* name, const at::Tensor& t, int64_t n) {
  if (t.dim() != n) refuse(name, t, c10::str(n, " dimensions"));
}
bool on(const at::Tensor& t, int device) { return t.is_cuda() && t.device().index() == device; }
void check(const char* name, const at::Tensor& t, at::ScalarType type, std::initializer_list<int64_t> shape, int device) {
  const at::IntArrayRef want(shape.begin(), shape.size());
  if (!on(t, device) || t.scalar_type() != type || t.sizes() != want || !t.is_contiguous())
    refuse(name, t, c10::str("contiguous ", type, " tensor of shape ", want, " on CUDA device ", device));
}
template <typename T>
T* data(const at::Tensor& t) {
  return static_cast<T*>(t.data_ptr());
}
template <typename T>
T* data(const at::Tensor* t) {
  return t ? data<T>(*t) : nullptr;
}
// Sizes become C ints: none of them may be cut off.
int dim(const at::Tensor& t, int64_t i) {
  const int64_t x = t.size(i);
  if (x > std::numeric_limits<int>::max()) throw std::invalid_argument("a tensor's extent is out of range");
  return static_cast<int>(x);
}

cudaStream_t stream_of(Args& a, int device) {
  PyObject* o = a.next();
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream();
  PyObject* index = PyObject_GetAttrString(o, "device_index");
  if (!index) throw PythonError{};
  const long d = PyLong_AsLong(index);
  Py_DECREF(index);
  if (d == -1 && PyErr_Occurred()) throw PythonError{};
  if (d != device)
    throw std::invalid_argument(c10::str("stream is on device ", d, ", the tensors are on device ", device));
  PyObject* raw = PyObject_GetAttrString(o, "cuda_stream");
  if (!raw) throw PythonError{};
  void* p = PyLong_AsVoidPtr(raw);
  Py_DECREF(raw);
  if (p == nullptr && PyErr_Occurred()) throw PythonError{};
  return static_cast<cudaStream_t>(p);
}

// The interpreter's lock, given up while this lives and taken back however the scope is left.
struct Unlocked {
  PyThreadState* state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};
// Calls the library on the tensors' device without the interpreter's lock. The
// arguments are pointers and sizes by then: forming them may throw (a tensor of
// a function transform has no storage) and needs the lock.
template <typename Fn, typename... A>
int run(int device, Fn fn, A... args) {
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(device));
  const Unlocked unlocked;
  return fn(args...);
}

// A page pool and, for E4M3, its scales.
struct Pool {
  const at::Tensor *k, *v, *ks = nullptr, *vs = nullptr;
  int n_pages, heads, page_size, width;
  bool e4m3;
};
Pool take_pool(Args& a, bool e4m3, int device) {
  Pool p;
  p.e4m3 = e4m3;
  p.k = &a.tensor("kpages");
  p.v = &a.tensor("vpages");
  check_dims("kpages", *p.k, 4);
  const at::ScalarType type = p.k->scalar_type();
  if (e4m3 ? type != at::kByte && type != at::kFloat8_e4m3fn : type != at::kBFloat16)
    refuse("kpages", *p.k, e4m3 ? "uint8 or float8_e4m3fn pages" : "bfloat16 pages");
  p.n_pages = dim(*p.k, 0);
  p.heads = dim(*p.k, 1);
  p.page_size = dim(*p.k, 2);
  p.width = dim(*p.k, 3);
  check("kpages", *p.k, type, {p.n_pages, p.heads, p.page_size, p.width}, device);
  check("vpages", *p.v, type, {p.n_pages, p.heads, p.page_size, p.width}, device);
  if (e4m3) {
    p.ks = &a.tensor("k_scales");
    p.vs = &a.tensor("v_scales");
    check("k_scales", *p.ks, at::kFloat, {p.n_pages, p.heads}, device);
    check("v_scales", *p.vs, at::kFloat, {p.n_pages, p.heads}, device);
  }
  return p;
}

using AppendBf16 = decltype(&llama_attn_kv_append_paged);
using AppendE4m3 = decltype(&llama_attn_kv_append_paged_e4m3);
using DecodeE4m3 = decltype(&llama_attn_decode_paged_e4m3);
using SparseBf16 = decltype(&llama_attn_decode_paged_sparse);
using SparseE4m3 = decltype(&llama_attn_decode_paged_sparse_e4m3);
using Select = decltype(&llama_attn_select_blocks);

// (function, e4m3, k, v, kpages, vpages[, k_scales, v_scales], block_table,
// cache_lens, rope_table, new_lens, kbounds, out_lens, stream)
int append(Args& a) {
  void* fn = a.function<void*>();
  const bool e4m3 = a.integer("e4m3") != 0;
  const at::Tensor &k = a.tensor("k"), &v = a.tensor("v");
  const int device = device_of("k", k);
  check_dims("k", k, 4);
  for (const auto& [name, t] : {std::pair<const char*, const at::Tensor&>{"k", k}, {"v", v}})
    if (!on(t, device) || t.scalar_type() != at::kBFloat16 || t.sizes() != k.sizes())
      refuse(name, t, c10::str("BFloat16 tensor of shape ", k.sizes(), " on CUDA device ", device));
  const int B = dim(k, 0), T = dim(k, 1), H = dim(k, 2), D = dim(k, 3);
  int64_t row = static_cast<int64_t>(H) * D, batch = T * row;
  if (!k.is_contiguous() || !v.is_contiguous()) {
    const auto s = k.strides(), u = v.strides();
    if ((D != 1 && (s[3] != 1 || u[3] != 1)) || (H != 1 && (s[2] != D || u[2] != D)))
      throw std::invalid_argument("k and v: the heads of a token must be contiguous");
    if ((T != 1 && s[1] != u[1]) || (B != 1 && s[0] != u[0]))
      throw std::invalid_argument("k and v must have the same strides");
    if (T != 1) row = s[1];
    batch = B != 1 ? s[0] : 0;
  }
  const Pool p = take_pool(a, e4m3, device);
  if (p.heads != H || p.width != D) refuse("kpages", *p.k, c10::str("pages of ", H, " KV heads of ", D));
  const at::Tensor& table = a.tensor("block_table");
  check_dims("block_table", table, 2);
  const int blocks = dim(table, 1);
  check("block_table", table, at::kInt, {B, blocks}, device);
  const at::Tensor& lens = a.tensor("cache_lens");
  check("cache_lens", lens, at::kInt, {B}, device);
  const at::Tensor& rope = a.tensor("rope_table");
  check_dims("rope_table", rope, 3);
  const int rows = dim(rope, 0);
  check("rope_table", rope, at::kFloat, {rows, D / 2, 2}, device);
  const at::Tensor* new_lens = a.tensor_or_none("new_lens");
  if (new_lens) check("new_lens", *new_lens, at::kInt, {B}, device);
  const at::Tensor* bounds = a.tensor_or_none("kbounds");
  if (bounds) check("kbounds", *bounds, at::kBFloat16, {p.n_pages, H, 2, D}, device);
  const at::Tensor* out_lens = a.tensor_or_none("out_lens");
  if (out_lens) check("out_lens", *out_lens, at::kInt, {B}, device);
  const cudaStream_t stream = stream_of(a, device);
  if (e4m3)
    return run(device, reinterpret_cast<AppendE4m3>(fn), data<llama_attn_bf16>(k), data<llama_attn_bf16>(v), row, batch,
               data<uint8_t>(*p.k), data<uint8_t>(*p.v), data<float>(*p.ks), data<float>(*p.vs),
               data<llama_attn_bf16>(bounds), data<int32_t>(table), data<int32_t>(lens), data<int32_t>(new_lens),
               data<int32_t>(out_lens), B, T, H, D, p.page_size, blocks, p.n_pages, data<void>(rope), rows, stream);
  return run(device, reinterpret_cast<AppendBf16>(fn), data<llama_attn_bf16>(k), data<llama_attn_bf16>(v), row, batch,
             data<llama_attn_bf16>(*p.k), data<llama_attn_bf16>(*p.v), data<llama_attn_bf16>(bounds),
             data<int32_t>(table), data<int32_t>(lens), data<int32_t>(new_lens), data<int32_t>(out_lens), B, T, H, D,
             p.page_size, blocks, p.n_pages, data<void>(rope), rows, stream);
}

// (function, e4m3, sparse, q, kpages, vpages[, k_scales, v_scales], block_table[,
// block_ids], cache_lens, out, lse, workspace, q_pos_offset, rope_theta, stream);
// e4m3 and sparse belong to the function: they say which prototype it has.
int decode(Args& a) {
  void* fn = a.function<void*>();
  const bool e4m3 = a.integer("e4m3") != 0, sparse = a.integer("sparse") != 0;
  if (!e4m3 && !sparse) throw std::invalid_argument("a decode over E4M3 pages or over chosen blocks expected");
  const at::Tensor& q = a.tensor("q");
  const int device = device_of("q", q);
  check_dims("q", q, 3);
  const int B = dim(q, 0), Hq = dim(q, 1), D = dim(q, 2);
  check("q", q, at::kBFloat16, {B, Hq, D}, device);
  const Pool p = take_pool(a, e4m3, device);
  if (p.width != D) refuse("kpages", *p.k, c10::str("pages of rows of ", D));
  const at::Tensor& table = a.tensor("block_table");
  check_dims("block_table", table, 2);
  const int blocks = dim(table, 1);
  check("block_table", table, at::kInt, {B, blocks}, device);
  const at::Tensor* ids = sparse ? &a.tensor("block_ids") : nullptr;
  int n_sel = 0;
  if (sparse) {
    check_dims("block_ids", *ids, 3);
    n_sel = dim(*ids, 2);
    check("block_ids", *ids, at::kInt, {B, p.heads, n_sel}, device);
  }
  const at::Tensor& lens = a.tensor("cache_lens");
  check("cache_lens", lens, at::kInt, {B}, device);
  const at::Tensor& out = a.tensor("out");
  check("out", out, at::kBFloat16, {B, Hq, D}, device);
  const at::Tensor* lse = a.tensor_or_none("lse");
  if (lse) check("lse", *lse, at::kFloat, {B, Hq}, device);
  const at::Tensor& ws = a.tensor("workspace");
  if (!on(ws, device) || !ws.is_contiguous())
    refuse("workspace", ws, c10::str("contiguous tensor on CUDA device ", device));
  const int offset = a.integer("q_pos_offset");
  const float theta = a.real();
  const cudaStream_t stream = stream_of(a, device);
  if (!sparse)
    return run(device, reinterpret_cast<DecodeE4m3>(fn), data<llama_attn_bf16>(q), data<uint8_t>(*p.k),
               data<uint8_t>(*p.v), data<float>(*p.ks), data<float>(*p.vs), data<int32_t>(table), data<int32_t>(lens),
               data<llama_attn_bf16>(out), data<float>(lse), B, Hq, p.heads, D, p.page_size, blocks, p.n_pages, offset,
               theta, data<void>(ws), ws.nbytes(), stream);
  if (e4m3)
    return run(device, reinterpret_cast<SparseE4m3>(fn), data<llama_attn_bf16>(q), data<uint8_t>(*p.k),
               data<uint8_t>(*p.v), data<float>(*p.ks), data<float>(*p.vs), data<int32_t>(table), data<int32_t>(*ids),
               data<int32_t>(lens), data<llama_attn_bf16>(out), data<float>(lse), B, Hq, p.heads, D, p.page_size, blocks,
               p.n_pages, n_sel, offset, theta, data<void>(ws), ws.nbytes(), stream);
  return run(device, reinterpret_cast<SparseBf16>(fn), data<llama_attn_bf16>(q), data<llama_attn_bf16>(*p.k),
             data<llama_attn_bf16>(*p.v), data<int32_t>(table), data<int32_t>(*ids), data<int32_t>(lens),
             data<llama_attn_bf16>(out), data<float>(lse), B, Hq, p.heads, D, p.page_size, blocks, p.n_pages, n_sel,
             offset, theta, data<void>(ws), ws.nbytes(), stream);
}

// (function, q, kbounds, block_table, cache_lens, block_ids, page_size, n_sel,
// n_first, n_last, q_pos_offset, rope_theta, stream)
int select(Args& a) {
  const Select fn = a.function<Select>();
  const at::Tensor& q = a.tensor("q");
  const int device = device_of("q", q);
  check_dims("q", q, 3);
  const int B = dim(q, 0), Hq = dim(q, 1), D = dim(q, 2);
  check("q", q, at::kBFloat16, {B, Hq, D}, device);
  const at::Tensor& bounds = a.tensor("kbounds");
  check_dims("kbounds", bounds, 4);
  const int n_pages = dim(bounds, 0), H = dim(bounds, 1);
  check("kbounds", bounds, at::kBFloat16, {n_pages, H, 2, D}, device);
  const at::Tensor& table = a.tensor("block_table");
  check_dims("block_table", table, 2);
  const int blocks = dim(table, 1);
  check("block_table", table, at::kInt, {B, blocks}, device);
  const at::Tensor& lens = a.tensor("cache_lens");
  check("cache_lens", lens, at::kInt, {B}, device);
  const at::Tensor& ids = a.tensor("block_ids");
  const int page_size = a.integer("page_size"), n_sel = a.integer("n_sel"), n_first = a.integer("n_first"),
            n_last = a.integer("n_last"), offset = a.integer("q_pos_offset");
  check("block_ids", ids, at::kInt, {B, H, n_sel}, device);
  const float theta = a.real();
  const cudaStream_t stream = stream_of(a, device);
  return run(device, fn, data<llama_attn_bf16>(q), data<llama_attn_bf16>(bounds), data<int32_t>(table),
             data<int32_t>(lens), data<int32_t>(ids), B, Hq, H, D, page_size, blocks, n_pages, n_sel, n_first, n_last,
             offset, theta, stream);
}

template <int (*kCall)(Args&)>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  try {
    Args a{args, n};
    const int st = kCall(a);
    return PyLong_FromLong(st);
  } catch (const PythonError&) {
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
    return nullptr;
  }
}

PyMethodDef kMethods[] = {
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&call<append>)), METH_FASTCALL, nullptr},
    {"decode", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&call<decode>)), METH_FASTCALL, nullptr},
    {"select", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&call<select>)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&kModule); }
