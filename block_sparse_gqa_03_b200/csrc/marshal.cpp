// Argument marshalling of the 8-bit cache calls: checks torch tensors, fills
// msa_params_t and calls the library.  No arithmetic of the method is here.
//
// A decode step makes a few calls of 4 to 50 us of GPU time each.  Read attribute by
// attribute from Python, ten tensors cost about 9 us a call; here about 1 us.
#include <Python.h>
#include <ATen/cuda/EmptyTensor.h>
#include <ATen/ops/empty.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <initializer_list>
#include <stdexcept>
#include <string>

#include "../../include/msa.h"

namespace {

struct Api {
  decltype(&msa_workspace_size) workspace_size;
  decltype(&msa_append_kv_q8) append;
  decltype(&msa_read_kv_q8) read;
  decltype(&msa_block_scores_q8) scores;
  decltype(&msa_index_select_q8) select;
  decltype(&msa_sparse_attn_q8) attn;
  decltype(&msa_forward_q8) forward;
} api = {};

using Dims = std::initializer_list<int64_t>;

[[noreturn]] void refuse(const std::string& what) { throw std::invalid_argument(what); }

// A tensor argument; nullptr for None when optional.
const at::Tensor* tensor(PyObject* o, const char* name, bool optional = false) {
  if (o == Py_None && optional) return nullptr;
  if (!THPVariable_Check(o)) refuse(std::string(name) + " must be a tensor");
  return &THPVariable_Unpack(o);
}

std::string describe(const at::Tensor& t) {
  std::string s = "[";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + "] " + std::string(t.dtype().name()) + " on " + t.device().str();
}

bool has_shape(const at::Tensor& t, Dims shape) { return t.sizes().equals(shape); }

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse("a size must be an integer");
  }
  return v;
}

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse("softmax_scale must be a number");
  }
  return v;
}

int32_t flag(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) {
    PyErr_Clear();
    refuse("a flag must be a truth value");
  }
  return v;
}

// One call: the cache's geometry and the parameters under construction.
struct Call {
  msa_params_t p = {};
  c10::Device dev = c10::Device(c10::kCPU);
  int64_t batch = 0, planes = 0, rows = 0, nblk = 0;
  bool paged = false;
  void* ws = nullptr;
  size_t ws_bytes = 0;
  msa_stream_t stream = nullptr;

  // tail: block, seq_lens, block_table, max_kv, workspace, stream
  Call(const at::Tensor& codes, int64_t b, PyObject* const* tail) : dev(codes.device()), batch(b) {
    if (!codes.is_cuda()) refuse("the 8-bit cache calls need CUDA tensors");
    if (codes.dim() < 2) refuse("the cache has shape " + describe(codes));
    const int64_t block = integer(tail[0]);
    if (block < 1 || block > (1 << 30)) refuse("block must be positive");
    planes = codes.size(0);
    rows = codes.size(1);
    int64_t cap = rows;
    if (const at::Tensor* t = tensor(tail[2], "block_table", true)) {
      paged = true;
      if (tail[3] == Py_None) refuse("a paged KV cache needs max_kv");
      cap = integer(tail[3]);
      nblk = (cap + block - 1) / block;
      if (rows != block) refuse("a page holds block tokens: the pool has shape " + describe(codes));
      if (t->scalar_type() != at::kInt || t->device() != dev || t->dim() != 2 ||
          t->size(0) != b || t->size(1) < nblk || (t->size(1) > 1 && t->stride(1) != 1))
        refuse("block_table must be int32 [batch, >= ceil(max_kv / block)], got " + describe(*t));
      p.block_table = t->data_ptr<int32_t>();
      p.table_stride = b > 1 ? t->stride(0) : t->size(1);
      p.num_pages = planes;
    } else {
      if (planes != b)
        refuse("the cache holds " + std::to_string(planes) + " sequences, not " + std::to_string(b));
      if (tail[3] != Py_None && integer(tail[3]) != cap)
        refuse("max_kv is the cache's token axis, " + std::to_string(cap));
      nblk = (cap + block - 1) / block;
    }
    if (const at::Tensor* t = tensor(tail[1], "seq_lens", true))
      p.seq_lens = static_cast<const int32_t*>(dense("seq_lens", t, {b}, at::kInt));
    set(p.batch, b);
    set(p.max_kv, cap);
    set(p.block, block);
    if (const at::Tensor* t = tensor(tail[4], "workspace", true)) {
      if (t->device() != dev) refuse("the workspace is on another device: " + describe(*t));
      ws = t->data_ptr();
      ws_bytes = (size_t)t->numel();
    }
    stream = reinterpret_cast<msa_stream_t>((uintptr_t)integer(tail[5]));
    // what a call does not use still has to be a supported size
    p.H = p.h = 1;
    p.d = 64;
    p.d_idx = 32;
    p.topk = 1;
    p.causal = 1;
  }

  static void set(int32_t& field, int64_t v) {
    if (v < INT32_MIN || v > INT32_MAX) refuse("a size does not fit 32 bits");
    field = (int32_t)v;
  }

  void* dense(const char* name, const at::Tensor* t, Dims shape, at::ScalarType type) const {
    if (t->scalar_type() != type || t->device() != dev || !has_shape(*t, shape) ||
        !t->is_contiguous())
      refuse(std::string(name) + " must be dense, of the call's shape, type and device: got " +
             describe(*t));
    return t->data_ptr();
  }
  void* dense(const char* name, PyObject* o, Dims shape, at::ScalarType type) const {
    return dense(name, tensor(o, name), shape, type);
  }
  void* dense_or_null(const char* name, PyObject* o, Dims shape, at::ScalarType type) const {
    const at::Tensor* t = tensor(o, name, true);
    return t ? dense(name, t, shape, type) : nullptr;
  }
  float* scale(const char* name, PyObject* o, int64_t heads) const {
    const at::Tensor* t = tensor(o, name);
    if (heads > 0)
      return static_cast<float*>(paged ? dense(name, t, {planes, heads}, at::kFloat)
                                       : dense(name, t, {planes, nblk, heads}, at::kFloat));
    return static_cast<float*>(paged ? dense(name, t, {planes}, at::kFloat)
                                     : dense(name, t, {planes, nblk}, at::kFloat));
  }

  static void strides(const at::Tensor& t, int64_t* out) {
    for (int64_t i = 0; i + 1 < t.dim(); ++i) out[i] = t.stride(i);
  }
  uint8_t* codes(const char* name, PyObject* o, Dims shape, int64_t* st) const {
    const at::Tensor& t = *tensor(o, name);
    if ((t.scalar_type() != at::kFloat8_e4m3fn && t.scalar_type() != at::kByte) ||
        t.device() != dev || !has_shape(t, shape) || t.stride(-1) != 1)
      refuse(std::string(name) + " must hold e4m3 codes (float8_e4m3fn or uint8), its innermost "
                                 "axis contiguous, of the cache's shape and device: got " +
             describe(t));
    strides(t, st);
    return static_cast<uint8_t*>(t.data_ptr());
  }
  uint16_t* rows_of(const char* name, PyObject* o, Dims shape, int64_t* st) const {
    const at::Tensor& t = *tensor(o, name);
    if (t.scalar_type() != at::kBFloat16 || t.device() != dev || !has_shape(t, shape) ||
        t.stride(-1) != 1)
      refuse(std::string(name) + " must be bf16, its innermost axis contiguous, of the call's "
                                 "shape and device: got " + describe(t));
    strides(t, st);
    return static_cast<uint16_t*>(t.data_ptr());
  }

  // 0 when the workspace is large enough, else the bytes it needs, negated.
  long long short_of(msa_op_t op) const {
    size_t need = api.workspace_size(&p, op);
    if (need == 0) need = 4096;  // bad parameters: the call itself says which
    return ws != nullptr && ws_bytes >= need ? 0 : -(long long)need;
  }
};

const at::Tensor& shaped(PyObject* o, const char* name, int64_t dims) {
  const at::Tensor& t = *tensor(o, name);
  if (t.dim() != dims) refuse(std::string(name) + " has shape " + describe(t));
  return t;
}

// k, v, k_idx, k_scale, v_scale, k_idx_scale, k_new, v_new, k_idx_new, tail
long long append(PyObject* const* a) {
  const at::Tensor& k = shaped(a[0], "k", 4);
  const at::Tensor& ki = shaped(a[2], "k_idx", 3);
  const at::Tensor* ref = nullptr;
  for (int i = 6; i < 9 && !ref; ++i) ref = tensor(a[i], "new rows", true);
  if (!ref || ref->dim() < 2) refuse("no new rows");
  Call c(k, ref->size(0), a + 9);
  const int64_t b = c.batch, n = ref->size(1), h = k.size(2), d = k.size(3), di = ki.size(2);
  c.set(c.p.n_q, n);
  c.set(c.p.h, h);
  c.p.H = c.p.h;
  c.set(c.p.d, d);
  c.set(c.p.d_idx, di);
  uint8_t* kc = c.codes("k", a[0], {c.planes, c.rows, h, d}, c.p.k_strides);
  uint8_t* vc = c.codes("v", a[1], {c.planes, c.rows, h, d}, c.p.v_strides);
  uint8_t* ic = c.codes("k_idx", a[2], {c.planes, c.rows, di}, c.p.ki_strides);
  float *ks = c.scale("k_scale", a[3], h), *vs = c.scale("v_scale", a[4], h);
  float* is = c.scale("k_idx_scale", a[5], 0);
  void* kn = c.dense_or_null("k_new", a[6], {b, n, h, d}, at::kBFloat16);
  void* vn = c.dense_or_null("v_new", a[7], {b, n, h, d}, at::kBFloat16);
  void* in = c.dense_or_null("k_idx_new", a[8], {b, n, di}, at::kBFloat16);
  if (const long long s = c.short_of(MSA_OP_APPEND_KV_Q8)) return s;
  return api.append(&c.p, (uint16_t*)kn, (uint16_t*)vn, (uint16_t*)in, kc, vc, ic, ks, vs, is,
                    c.ws, c.ws_bytes, c.stream);
}

// k, v, k_idx, k_scale, v_scale, k_idx_scale, k_out, v_out, k_idx_out, token_base, tail
long long read(PyObject* const* a) {
  const at::Tensor& k = shaped(a[0], "k", 4);
  const at::Tensor& ki = shaped(a[2], "k_idx", 3);
  const at::Tensor& ko = shaped(a[6], "k_out", 4);
  Call c(k, ko.size(0), a + 10);
  const int64_t b = c.batch, n = ko.size(1), h = k.size(2), d = k.size(3), di = ki.size(2);
  c.set(c.p.n_q, n);
  c.set(c.p.h, h);
  c.p.H = c.p.h;
  c.set(c.p.d, d);
  c.set(c.p.d_idx, di);
  uint8_t* kc = c.codes("k", a[0], {c.planes, c.rows, h, d}, c.p.k_strides);
  uint8_t* vc = c.codes("v", a[1], {c.planes, c.rows, h, d}, c.p.v_strides);
  uint8_t* ic = c.codes("k_idx", a[2], {c.planes, c.rows, di}, c.p.ki_strides);
  float *ks = c.scale("k_scale", a[3], h), *vs = c.scale("v_scale", a[4], h);
  float* is = c.scale("k_idx_scale", a[5], 0);
  void* kp = c.dense("k_out", a[6], {b, n, h, d}, at::kBFloat16);
  void* vp = c.dense("v_out", a[7], {b, n, h, d}, at::kBFloat16);
  void* ip = c.dense("k_idx_out", a[8], {b, n, di}, at::kBFloat16);
  if (const long long s = c.short_of(MSA_OP_READ_KV_Q8)) return s;
  return api.read(&c.p, kc, vc, ic, ks, vs, is, integer(a[9]), (uint16_t*)kp, (uint16_t*)vp,
                  (uint16_t*)ip, c.ws, c.ws_bytes, c.stream);
}

// q_idx, k_idx, k_idx_scale, block_ids or None, block_scores or None, causal, force, tail;
// without block_ids the scores alone
long long index(PyObject* const* a) {
  const at::Tensor& q = shaped(a[0], "q_idx", 4);
  const at::Tensor& ki = shaped(a[1], "k_idx", 3);
  Call c(ki, q.size(0), a + 7);
  const int64_t b = c.batch, n = q.size(1), h = q.size(2), di = q.size(3);
  c.set(c.p.n_q, n);
  c.set(c.p.h, h);
  c.p.H = c.p.h;
  c.set(c.p.d_idx, di);
  c.p.causal = flag(a[5]);
  c.p.force_own_block = flag(a[6]);
  uint16_t* qp = c.rows_of("q_idx", a[0], {b, n, h, di}, c.p.qi_strides);
  uint8_t* ic = c.codes("k_idx", a[1], {c.planes, c.rows, di}, c.p.ki_strides);
  float* is = c.scale("k_idx_scale", a[2], 0);
  float* sc = (float*)c.dense_or_null("block_scores", a[4], {b, n, h, c.nblk}, at::kFloat);
  if (a[3] == Py_None) {
    if (const long long s = c.short_of(MSA_OP_BLOCK_SCORES_Q8)) return s;
    return api.scores(&c.p, qp, ic, is, sc, c.ws, c.ws_bytes, c.stream);
  }
  const int64_t topk = shaped(a[3], "block_ids", 4).size(3);
  c.set(c.p.topk, topk);
  int32_t* ids = (int32_t*)c.dense("block_ids", a[3], {b, n, h, topk}, at::kInt);
  if (const long long s = c.short_of(MSA_OP_INDEX_SELECT_Q8)) return s;
  return api.select(&c.p, qp, ic, is, ids, sc, c.ws, c.ws_bytes, c.stream);
}

// q, k, v, k_scale, v_scale, block_ids, out, lse or None, causal, softmax_scale, tail
long long attn(PyObject* const* a) {
  const at::Tensor& q = shaped(a[0], "q", 4);
  const at::Tensor& k = shaped(a[1], "k", 4);
  Call c(k, q.size(0), a + 10);
  const int64_t b = c.batch, n = q.size(1), H = q.size(2), d = q.size(3), h = k.size(2);
  c.set(c.p.n_q, n);
  c.set(c.p.H, H);
  c.set(c.p.h, h);
  c.set(c.p.d, d);
  c.p.causal = flag(a[8]);
  c.p.softmax_scale = (float)number(a[9]);
  const int64_t topk = shaped(a[5], "block_ids", 4).size(3);
  c.set(c.p.topk, topk);
  uint16_t* qp = c.rows_of("q", a[0], {b, n, H, d}, c.p.q_strides);
  uint8_t* kc = c.codes("k", a[1], {c.planes, c.rows, h, d}, c.p.k_strides);
  uint8_t* vc = c.codes("v", a[2], {c.planes, c.rows, h, d}, c.p.v_strides);
  float *ks = c.scale("k_scale", a[3], h), *vs = c.scale("v_scale", a[4], h);
  int32_t* ids = (int32_t*)c.dense("block_ids", a[5], {b, n, h, topk}, at::kInt);
  uint16_t* out = c.rows_of("out", a[6], {b, n, H, d}, c.p.o_strides);
  float* lse = (float*)c.dense_or_null("lse", a[7], {b, n, H}, at::kFloat);
  if (const long long s = c.short_of(MSA_OP_SPARSE_ATTN_Q8)) return s;
  return api.attn(&c.p, qp, kc, vc, ks, vs, ids, out, lse, c.ws, c.ws_bytes, c.stream);
}

// q, k, v, q_idx, k_idx, k_scale, v_scale, k_idx_scale, out, block_ids or None, block_scores
// or None, lse or None, topk, causal, force, softmax_scale, tail
long long forward(PyObject* const* a) {
  const at::Tensor& q = shaped(a[0], "q", 4);
  const at::Tensor& k = shaped(a[1], "k", 4);
  const at::Tensor& ki = shaped(a[4], "k_idx", 3);
  Call c(k, q.size(0), a + 16);
  const int64_t b = c.batch, n = q.size(1), H = q.size(2), d = q.size(3), h = k.size(2);
  const int64_t di = ki.size(2), topk = integer(a[12]);
  c.set(c.p.n_q, n);
  c.set(c.p.H, H);
  c.set(c.p.h, h);
  c.set(c.p.d, d);
  c.set(c.p.d_idx, di);
  c.set(c.p.topk, topk);
  c.p.causal = flag(a[13]);
  c.p.force_own_block = flag(a[14]);
  c.p.softmax_scale = (float)number(a[15]);
  uint16_t* qp = c.rows_of("q", a[0], {b, n, H, d}, c.p.q_strides);
  uint8_t* kc = c.codes("k", a[1], {c.planes, c.rows, h, d}, c.p.k_strides);
  uint8_t* vc = c.codes("v", a[2], {c.planes, c.rows, h, d}, c.p.v_strides);
  uint16_t* qi = c.rows_of("q_idx", a[3], {b, n, h, di}, c.p.qi_strides);
  uint8_t* ic = c.codes("k_idx", a[4], {c.planes, c.rows, di}, c.p.ki_strides);
  float *ks = c.scale("k_scale", a[5], h), *vs = c.scale("v_scale", a[6], h);
  float* is = c.scale("k_idx_scale", a[7], 0);
  uint16_t* out = c.rows_of("out", a[8], {b, n, H, d}, c.p.o_strides);
  int32_t* ids = (int32_t*)c.dense_or_null("block_ids", a[9], {b, n, h, topk}, at::kInt);
  float* sc = (float*)c.dense_or_null("block_scores", a[10], {b, n, h, c.nblk}, at::kFloat);
  float* lse = (float*)c.dense_or_null("lse", a[11], {b, n, H}, at::kFloat);
  if (const long long s = c.short_of(MSA_OP_FORWARD_Q8)) return s;
  return api.forward(&c.p, qp, kc, vc, qi, ic, ks, vs, is, out, ids, sc, lse, c.ws, c.ws_bytes,
                     c.stream);
}

// Every function returns the library's status, or minus the workspace bytes the call
// needs when it has too few (nothing was launched then).
template <long long (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  try {
    if (n != N) refuse("wrong number of arguments");
    if (api.workspace_size == nullptr) throw std::runtime_error("the library is not bound");
    return PyLong_FromLongLong(F(args));
  } catch (const std::invalid_argument& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// empty(like, lead, last, type): a new tensor of like's first `lead` sizes and, unless it
// is negative, `last`; type 0: like's own, 1: fp32, 2: int32.  A result made with
// Tensor.new_empty costs 2.8 us of a call whose kernel takes 6, here 0.75 us (at::empty: 1.2).
PyObject* empty(PyObject*, PyObject* const* args, Py_ssize_t n) {
  try {
    if (n != 4) refuse("wrong number of arguments");
    const at::Tensor& like = *tensor(args[0], "like");
    const int64_t lead = integer(args[1]), last = integer(args[2]), type = integer(args[3]);
    if (lead < 0 || lead > like.dim()) refuse("the query has shape " + describe(like));
    c10::SmallVector<int64_t, 5> shape(like.sizes().begin(), like.sizes().begin() + lead);
    if (last >= 0) shape.push_back(last);
    const at::ScalarType t = type == 0 ? like.scalar_type() : type == 1 ? at::kFloat : at::kInt;
    if (!like.is_cuda()) return THPVariable_Wrap(at::empty(shape, t));  // refused by the call
    return THPVariable_Wrap(at::Tensor(at::detail::empty_cuda(shape, t, like.device(), {})));
  } catch (const std::invalid_argument& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  } catch (const c10::OutOfMemoryError& e) {
    PyObject* torch = PyImport_ImportModule("torch");
    PyObject* type = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
    if (type) PyErr_SetString(type, e.what_without_backtrace());
    Py_XDECREF(type);
    Py_XDECREF(torch);
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// bind(addresses of the seven library functions, in Api's order)
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != 7) {
    PyErr_SetString(PyExc_TypeError, "bind() takes seven addresses");
    return nullptr;
  }
  void* p[7];
  for (int i = 0; i < 7; ++i) {
    p[i] = PyLong_AsVoidPtr(args[i]);
    if (p[i] == nullptr) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null address");
      return nullptr;
    }
  }
  api.workspace_size = reinterpret_cast<decltype(api.workspace_size)>(p[0]);
  api.append = reinterpret_cast<decltype(api.append)>(p[1]);
  api.read = reinterpret_cast<decltype(api.read)>(p[2]);
  api.scores = reinterpret_cast<decltype(api.scores)>(p[3]);
  api.select = reinterpret_cast<decltype(api.select)>(p[4]);
  api.attn = reinterpret_cast<decltype(api.attn)>(p[5]);
  api.forward = reinterpret_cast<decltype(api.forward)>(p[6]);
  Py_RETURN_NONE;
}

#define MSA_ENTRY(name, fn, n) \
  { name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<fn, n>)), METH_FASTCALL, nullptr }

PyMethodDef methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&bind)), METH_FASTCALL,
     nullptr},
    {"empty", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&empty)), METH_FASTCALL,
     nullptr},
    MSA_ENTRY("append", append, 15),
    MSA_ENTRY("read", read, 16),
    MSA_ENTRY("index", index, 13),
    MSA_ENTRY("attn", attn, 16),
    MSA_ENTRY("forward", forward, 22),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_marshal", nullptr, -1, methods,
                      nullptr,               nullptr,    nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&module); }
