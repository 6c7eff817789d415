// binding.cpp -- the serving-step calls from Python: torch tensors checked and
// marshalled into the structs of msa.h.
//
// These calls run many times per generated token and their kernels take a few
// microseconds, so what Python spends on checking a dozen tensors attribute by
// attribute (9 us of 14 for msa_plan_step on a Grace core) would be most of a step.
// Every function here takes its arguments by position (the package's functions
// of the same name give them names and defaults), raises ValueError where one does not
// fit, and returns the entry point's status.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <cstdio>
#include <string>

#include "msa.h"

namespace {

constexpr int kBk = 128;
constexpr int kD = 128;

struct Refused {
  std::string why;
};

[[noreturn]] void refuse(const char* format, ...) {
  char buf[512];
  va_list args;
  va_start(args, format);
  std::vsnprintf(buf, sizeof(buf), format, args);
  va_end(args);
  throw Refused{buf};
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse("%s: need a tensor, got %s", name, Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}

std::string shape_of(const at::Tensor& t) {
  std::string s = "[";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + "]";
}

// The CUDA device that a call's tensors are on, from the first of them.
int device_of(const at::Tensor& t, const char* name) {
  if (!t.is_cuda()) refuse("%s must be on a CUDA device, got %s", name, t.device().str().c_str());
  return t.get_device();
}

void check(const at::Tensor& t, const char* name, at::ScalarType type, int dev, int dim) {
  if (t.scalar_type() != type || !t.is_cuda() || t.get_device() != dev || t.dim() != dim)
    refuse("%s: need a %d-dimensional %s tensor on cuda:%d, got %s of %s on %s", name, dim, c10::toString(type), dev,
           shape_of(t).c_str(), c10::toString(t.scalar_type()), t.device().str().c_str());
}

// Pointer of a contiguous tensor of this type, device, number of dimensions and (where >= 0) first size.
template <class T>
T* dense(PyObject* o, const char* name, at::ScalarType type, int dev, int dim, int64_t rows = -1) {
  const at::Tensor& t = tensor(o, name);
  check(t, name, type, dev, dim);
  if (!t.is_contiguous()) refuse("%s must be contiguous", name);
  if (rows >= 0 && t.size(0) != rows)
    refuse("%s: need %lld rows, got %lld", name, static_cast<long long>(rows), static_cast<long long>(t.size(0)));
  return static_cast<T*>(t.data_ptr());
}
template <class T>
T* dense_or_null(PyObject* o, const char* name, at::ScalarType type, int dev, int dim, int64_t rows) {
  return o == Py_None ? nullptr : dense<T>(o, name, type, dev, dim, rows);
}

// Pointer and leading strides of a bf16 tensor whose innermost dimension is contiguous.
template <int DIM>
void* rows(const at::Tensor& t, const char* name, int dev, int64_t* stride) {
  check(t, name, at::kBFloat16, dev, DIM);
  if (t.stride(DIM - 1) != 1 && t.numel() > 0) refuse("%s: innermost dimension must be contiguous", name);
  for (int i = 0; i < DIM - 1; ++i) stride[i] = t.stride(i);
  return t.data_ptr();
}

void need_shape(const at::Tensor& t, const char* name, c10::IntArrayRef shape) {
  if (t.sizes() != shape) {
    std::string want = "[";
    for (size_t i = 0; i < shape.size(); ++i) want += (i ? ", " : "") + std::to_string(shape[i]);
    refuse("%s: need shape %s], got %s", name, want.c_str(), shape_of(t).c_str());
  }
}

int32_t* err_word(PyObject* o, int dev) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, "dev_err");
  if (t.scalar_type() != at::kInt || !t.is_cuda() || t.get_device() != dev || t.numel() < 1)
    refuse("dev_err: need an int32 tensor of one value on cuda:%d", dev);
  return static_cast<int32_t*>(t.data_ptr());
}

// The cudaStream_t of a call: the device's current stream, a torch.cuda.Stream of that device, or a raw pointer.
msa_stream_t stream_of(PyObject* o, int dev) {
  if (o == Py_None) return reinterpret_cast<msa_stream_t>(c10::cuda::getCurrentCUDAStream(dev).stream());
  PyObject* raw = o;
  PyObject* own = nullptr;
  if (!PyLong_Check(o)) {
    PyObject* at = PyObject_GetAttrString(o, "device_index");
    const long on = at != nullptr ? PyLong_AsLong(at) : -1;
    Py_XDECREF(at);
    own = raw = PyErr_Occurred() ? nullptr : PyObject_GetAttrString(o, "cuda_stream");
    if (PyErr_Occurred()) {
      PyErr_Clear();
      Py_XDECREF(own);
      refuse("stream: need a torch.cuda.Stream or a stream pointer, got %s", Py_TYPE(o)->tp_name);
    }
    if (on != dev) {
      Py_DECREF(own);
      refuse("the stream is on cuda:%ld, the tensors on cuda:%d", on, dev);
    }
  }
  void* p = PyLong_AsVoidPtr(raw);
  Py_XDECREF(own);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    refuse("stream: not a stream pointer");
  }
  return static_cast<msa_stream_t>(p);
}

int64_t integer(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse("%s: need an integer", name);
  }
  return v;
}
float real(PyObject* o, const char* name) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse("%s: need a number", name);
  }
  return static_cast<float>(v);
}
bool truth(PyObject* o, const char* name) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) {
    PyErr_Clear();
    refuse("%s: need a truth value", name);
  }
  return v != 0;
}

int as_int(int64_t v, const char* name) {
  if (v < INT32_MIN || v > INT32_MAX) refuse("%s = %lld", name, static_cast<long long>(v));
  return static_cast<int>(v);
}

// Q4Cache: (K_codes, K_scales, V_codes, V_scales, k_scale, v_scale).  Fills the struct; returns the heads.
int q4_cache(PyObject* o, int dev, msa_q4_cache* c) {
  if (!PyTuple_Check(o) || PyTuple_GET_SIZE(o) != 6) refuse("cache: need a Q4Cache");
  static const char* const names[4] = {"K_codes", "K_scales", "V_codes", "V_scales"};
  const at::Tensor* t[4];
  void* p[4];
  for (int i = 0; i < 4; ++i) {
    t[i] = &tensor(PyTuple_GET_ITEM(o, i), names[i]);
    check(*t[i], names[i], at::kByte, dev, 4);
    p[i] = t[i]->data_ptr();
  }
  const int64_t P = t[0]->size(0), H = t[0]->size(1);
  for (int i = 0; i < 4; ++i) {
    const int64_t last = i & 1 ? kD / 16 : kD / 2;
    need_shape(*t[i], names[i], {P, H, kBk, last});
    if (t[i]->stride(3) != 1 || t[i]->stride(2) != last) refuse("%s: a block's rows must be contiguous", names[i]);
  }
  if (t[0]->strides() != t[2]->strides() || t[1]->strides() != t[3]->strides()) refuse("cache: K and V must share strides");
  c->K_codes = p[0]; c->K_scales = p[1]; c->V_codes = p[2]; c->V_scales = p[3];
  for (int i = 0; i < 2; ++i) {
    c->code_stride[i] = t[0]->stride(i);
    c->scale_stride[i] = t[1]->stride(i);
  }
  c->num_pages = P;
  c->k_scale = real(PyTuple_GET_ITEM(o, 4), "k_scale");
  c->v_scale = real(PyTuple_GET_ITEM(o, 5), "v_scale");
  return as_int(H, "Hkv");
}

// Lets other Python threads run while it lives: a launch waits where the stream's queue is full.
struct Unlocked {
  PyThreadState* const state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};

// Runs the entry point with the tensors' device current and the interpreter's lock released.  (The arguments, and
// with them the tensors, are held by the caller.)
template <class F>
msa_status on_device(int dev, F f) {
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(dev));
  const Unlocked unlocked;
  return f();
}

// seq_len, new_len, seq_pt, free_pages, free_count, seq_len_out, free_count_out, cu, tok_slot, tok_pos, tok_seq, num_pages,
// dev_err, stream
msa_status plan_step(PyObject* const* o) {
  const at::Tensor& L = tensor(o[0], "seq_len");
  const int dev = device_of(L, "seq_len");
  if (L.dim() != 1) refuse("seq_len must be [B]");
  const int64_t B = L.size(0);
  const at::Tensor &pt = tensor(o[2], "seq_pt"), &free = tensor(o[3], "free_pages"), &slot = tensor(o[8], "tok_slot");
  if (slot.dim() != 1) refuse("tok_slot must be [N]");
  const int64_t N = slot.size(0);
  msa_plan_args a = {};
  a.B = as_int(B, "B"); a.Bk = kBk; a.N = N;
  a.seq_len = dense<int32_t>(o[0], "seq_len", at::kInt, dev, 1);
  a.new_len = dense<int32_t>(o[1], "new_len", at::kInt, dev, 1, B);
  a.seq_pt = dense<int32_t>(o[2], "seq_pt", at::kInt, dev, 2, B);
  a.max_pages = pt.size(1);
  a.free_pages = dense<int32_t>(o[3], "free_pages", at::kInt, dev, 1);
  a.free_cap = free.size(0);
  a.free_count = dense<int32_t>(o[4], "free_count", at::kInt, dev, 1, 1);
  a.num_pages = integer(o[11], "num_pages");
  a.seq_len_out = dense<int32_t>(o[5], "seq_len_out", at::kInt, dev, 1, B);
  a.free_count_out = dense<int32_t>(o[6], "free_count_out", at::kInt, dev, 1, 1);
  a.cu = dense<int32_t>(o[7], "cu", at::kInt, dev, 1, B + 1);
  a.tok_slot = dense<int64_t>(o[8], "tok_slot", at::kLong, dev, 1);
  a.tok_pos = dense<int32_t>(o[9], "tok_pos", at::kInt, dev, 1, N);
  a.tok_seq = dense_or_null<int32_t>(o[10], "tok_seq", at::kInt, dev, 1, N);
  a.dev_err = err_word(o[12], dev);
  msa_stream_t s = stream_of(o[13], dev);
  return on_device(dev, [&] { return msa_plan_step(&a, s); });
}

// seq_len, done, seq_pt, free_pages, free_count, seq_len_out, free_count_out, num_pages (None: not given), dev_err, stream
msa_status release_pages(PyObject* const* o) {
  const at::Tensor& L = tensor(o[0], "seq_len");
  const int dev = device_of(L, "seq_len");
  if (L.dim() != 1) refuse("seq_len must be [B]");
  const int64_t B = L.size(0);
  const at::Tensor &pt = tensor(o[2], "seq_pt"), &free = tensor(o[3], "free_pages");
  msa_release_args a = {};
  a.B = as_int(B, "B"); a.Bk = kBk;
  a.seq_len = dense<int32_t>(o[0], "seq_len", at::kInt, dev, 1);
  a.done = dense<int32_t>(o[1], "done", at::kInt, dev, 1, B);
  a.seq_pt = dense<int32_t>(o[2], "seq_pt", at::kInt, dev, 2, B);
  a.max_pages = pt.size(1);
  a.free_pages = dense<int32_t>(o[3], "free_pages", at::kInt, dev, 1);
  a.free_cap = free.size(0);
  a.free_count = dense<int32_t>(o[4], "free_count", at::kInt, dev, 1, 1);
  a.seq_len_out = dense<int32_t>(o[5], "seq_len_out", at::kInt, dev, 1, B);
  a.free_count_out = dense<int32_t>(o[6], "free_count_out", at::kInt, dev, 1, 1);
  if (o[7] != Py_None) {
    a.num_pages = integer(o[7], "num_pages");
    if (a.num_pages < 1) refuse("num_pages = %lld", static_cast<long long>(a.num_pages));
  }
  a.dev_err = err_word(o[8], dev);
  msa_stream_t s = stream_of(o[9], dev);
  return on_device(dev, [&] { return msa_release_pages(&a, s); });
}

// Q, K, pos, inv_freq, Q_out, K_out, V, V_out, slots, q_weight, k_weight, eps, interleaved, dev_err, stream
msa_status qk_norm_rope(PyObject* const* o) {
  const at::Tensor& Q = tensor(o[0], "Q");
  const int dev = device_of(Q, "Q");
  if (Q.dim() != 3) refuse("Q must be [N, Hq, D]");
  const int64_t N = Q.size(0), D = Q.size(2);
  msa_norm_rope_args a = {};
  a.N = N; a.Hq = as_int(Q.size(1), "Hq"); a.D = as_int(D, "D"); a.Bk = kBk;
  a.Q = rows<3>(Q, "Q", dev, a.Q_stride);
  const at::Tensor& Q_out = tensor(o[4], "Q_out");
  need_shape(Q_out, "Q_out", Q.sizes());
  a.Q_out = rows<3>(Q_out, "Q_out", dev, a.Q_out_stride);
  const bool has_k = o[1] != Py_None, has_v = o[6] != Py_None, paged = o[8] != Py_None;
  if (has_k != (o[5] != Py_None) || has_v != (o[7] != Py_None)) refuse("K comes with K_out, and V with V_out");
  if (!has_k && (has_v || paged)) refuse("V and slots need K");
  if (has_v && !paged) refuse("V and V_out need slots");
  if (has_k) {
    const at::Tensor &K = tensor(o[1], "K"), &K_out = tensor(o[5], "K_out");
    if (K.dim() != 3) refuse("K must be [N, Hkv, D]");
    const int64_t H = K.size(1);
    need_shape(K, "K", {N, H, D});
    a.Hkv = as_int(H, "Hkv");
    a.K = rows<3>(K, "K", dev, a.K_stride);
    if (paged) {
      if (K_out.dim() != 4) refuse("K_out must be a pool [P, Hkv, %d, D] with slots", kBk);
      a.num_pages = K_out.size(0);
      need_shape(K_out, "K_out", {a.num_pages, H, kBk, D});
      a.K_out = rows<4>(K_out, "K_out", dev, a.K_out_stride);
      a.slots = dense<int64_t>(o[8], "slots", at::kLong, dev, 1, N);
    } else {
      need_shape(K_out, "K_out", {N, H, D});
      a.K_out = rows<3>(K_out, "K_out", dev, a.K_out_stride);
    }
    if (has_v) {
      const at::Tensor &V = tensor(o[6], "V"), &V_out = tensor(o[7], "V_out");
      need_shape(V, "V", {N, H, D});
      need_shape(V_out, "V_out", {a.num_pages, H, kBk, D});
      a.V = rows<3>(V, "V", dev, a.V_stride);
      a.V_out = rows<4>(V_out, "V_out", dev, a.V_out_stride);
    }
  }
  a.pos = dense<int32_t>(o[2], "pos", at::kInt, dev, 1, N);
  if (o[3] != Py_None) {
    a.inv_freq = dense<float>(o[3], "inv_freq", at::kFloat, dev, 1);
    a.rot = as_int(2 * THPVariable_Unpack(o[3]).size(0), "rot");
  }
  PyObject* const first = o[9] != Py_None ? o[9] : o[10];
  if (first != Py_None) {
    const at::ScalarType type = tensor(first, "q_weight").scalar_type();
    if (type != at::kBFloat16 && type != at::kFloat) refuse("q_weight and k_weight must be bf16 or fp32");
    a.weight_fp32 = type == at::kFloat;
    a.q_weight = dense_or_null<void>(o[9], "q_weight", type, dev, 1, D);
    a.k_weight = dense_or_null<void>(o[10], "k_weight", type, dev, 1, D);
  }
  a.eps = real(o[11], "eps");
  a.interleaved = truth(o[12], "interleaved");
  a.dev_err = err_word(o[13], dev);
  msa_stream_t s = stream_of(o[14], dev);
  return on_device(dev, [&] { return msa_qk_norm_rope(&a, s); });
}

// K, V, slots, cache, dev_err, stream
msa_status cache_append_q4(PyObject* const* o) {
  const at::Tensor &K = tensor(o[0], "K"), &V = tensor(o[1], "V");
  const int dev = device_of(K, "K");
  msa_append_q4_args a = {};
  a.K = rows<3>(K, "K", dev, a.K_stride);
  a.V = rows<3>(V, "V", dev, a.V_stride);
  need_shape(V, "V", K.sizes());
  a.N = K.size(0); a.Hkv = as_int(K.size(1), "Hkv"); a.D = as_int(K.size(2), "D"); a.Bk = kBk;
  a.slots = dense<int64_t>(o[2], "slots", at::kLong, dev, 1, a.N);
  if (q4_cache(o[3], dev, &a.cache) != a.Hkv) refuse("the cache and K must have the same heads");
  a.dev_err = err_word(o[4], dev);
  msa_stream_t s = stream_of(o[5], dev);
  return on_device(dev, [&] { return msa_cache_append_q4(&a, s); });
}

// cache, pages, K_out, V_out, dev_err, stream
msa_status cache_expand_q4(PyObject* const* o) {
  const at::Tensor& pages = tensor(o[1], "pages");
  const int dev = device_of(pages, "pages");
  msa_expand_q4_args a = {};
  a.pages = dense<int32_t>(o[1], "pages", at::kInt, dev, 1);
  a.n = pages.size(0);
  a.Hkv = q4_cache(o[0], dev, &a.cache);
  a.D = kD; a.Bk = kBk;
  a.K_out = dense<void>(o[2], "K_out", at::kBFloat16, dev, 4);
  a.V_out = dense<void>(o[3], "V_out", at::kBFloat16, dev, 4);
  need_shape(THPVariable_Unpack(o[2]), "K_out", {a.n, a.Hkv, kBk, kD});
  need_shape(THPVariable_Unpack(o[3]), "V_out", {a.n, a.Hkv, kBk, kD});
  a.dev_err = err_word(o[4], dev);
  msa_stream_t s = stream_of(o[5], dev);
  return on_device(dev, [&] { return msa_cache_expand_q4(&a, s); });
}

// The fields that the two attention calls share; returns the device.
template <class Args>
int attention(PyObject* q, PyObject* cache, PyObject* out, PyObject* lse, PyObject* ws, Args* a, void** work, size_t* bytes) {
  const at::Tensor& Q = tensor(q, "Q");
  const int dev = device_of(Q, "Q");
  a->Q = rows<3>(Q, "Q", dev, a->Q_stride);
  a->B = as_int(Q.size(0), "B"); a->Hq = as_int(Q.size(1), "Hq"); a->D = as_int(Q.size(2), "D"); a->Bk = kBk;
  a->Hkv = q4_cache(cache, dev, &a->cache);
  a->O = dense<void>(out, "O", at::kBFloat16, dev, 3);
  need_shape(THPVariable_Unpack(out), "O", Q.sizes());
  if (lse != Py_None) {
    a->LSE = dense<float>(lse, "LSE", at::kFloat, dev, 2);
    need_shape(THPVariable_Unpack(lse), "LSE", {Q.size(0), Q.size(1)});
  }
  const at::Tensor& w = tensor(ws, "ws");
  if (!w.is_contiguous() || !w.is_cuda() || w.get_device() != dev) refuse("ws must be a contiguous tensor on cuda:%d", dev);
  *work = w.data_ptr();
  *bytes = w.nbytes();
  return dev;
}

// Q, cache, pt, n, last_len, O, LSE, ws, softmax_scale, dev_err, stream, scratch_zeroed
msa_status sparse_attn_decode_q4(PyObject* const* o) {
  msa_decode_q4_args a = {};
  void* work;
  size_t bytes;
  const int dev = attention(o[0], o[1], o[5], o[6], o[7], &a, &work, &bytes);
  const int64_t r = static_cast<int64_t>(a.B) * a.Hkv;
  a.pt = dense<int32_t>(o[2], "pt", at::kInt, dev, 2, r);
  a.k = as_int(THPVariable_Unpack(o[2]).size(1), "k");
  a.n = dense<int32_t>(o[3], "n", at::kInt, dev, 1, r);
  a.last_len = dense<int32_t>(o[4], "last_len", at::kInt, dev, 1, r);
  a.softmax_scale = real(o[8], "softmax_scale");
  a.dev_err = err_word(o[9], dev);
  msa_stream_t s = stream_of(o[10], dev);
  a.scratch_zeroed = truth(o[11], "scratch_zeroed");
  return on_device(dev, [&] { return msa_sparse_attn_decode_q4(&a, work, bytes, s); });
}

// Q, cache, seq_pt, seq_len, O, LSE, ws, softmax_scale, dev_err, stream, scratch_zeroed
msa_status dense_attn_decode_q4(PyObject* const* o) {
  msa_dense_decode_q4_args a = {};
  void* work;
  size_t bytes;
  const int dev = attention(o[0], o[1], o[4], o[5], o[6], &a, &work, &bytes);
  a.seq_pt = dense<int32_t>(o[2], "seq_pt", at::kInt, dev, 2, a.B);
  a.max_pages = THPVariable_Unpack(o[2]).size(1);
  a.seq_len = dense<int32_t>(o[3], "seq_len", at::kInt, dev, 1, a.B);
  a.softmax_scale = real(o[7], "softmax_scale");
  a.dev_err = err_word(o[8], dev);
  msa_stream_t s = stream_of(o[9], dev);
  a.scratch_zeroed = truth(o[10], "scratch_zeroed");
  return on_device(dev, [&] { return msa_dense_attn_decode_q4(&a, work, bytes, s); });
}

template <msa_status (*F)(PyObject* const*), int ARGS>
PyObject* call(PyObject*, PyObject* const* o, Py_ssize_t n) {
  if (n != ARGS) {
    PyErr_Format(PyExc_TypeError, "need %d arguments, got %zd", ARGS, n);
    return nullptr;
  }
  try {
    return PyLong_FromLong(F(o));
  } catch (const Refused& e) {
    PyErr_SetString(PyExc_ValueError, e.why.c_str());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

template <msa_status (*F)(PyObject* const*), int ARGS>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&call<F, ARGS>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {
    method<plan_step, 14>("plan_step"),
    method<release_pages, 10>("release_pages"),
    method<qk_norm_rope, 15>("qk_norm_rope"),
    method<cache_append_q4, 6>("cache_append_q4"),
    method<cache_expand_q4, 6>("cache_expand_q4"),
    method<sparse_attn_decode_q4, 12>("sparse_attn_decode_q4"),
    method<dense_attn_decode_q4, 11>("dense_attn_decode_q4"),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_msa_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__msa_binding(void) {
  PyObject* const m = PyModule_Create(&module);
  if (m != nullptr && PyModule_AddStringConstant(m, "built_for", MSA_BUILT_FOR) != 0) {   // the torch whose headers it has
    Py_DECREF(m);
    return nullptr;
  }
  return m;
}
