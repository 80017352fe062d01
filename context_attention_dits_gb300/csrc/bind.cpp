// bind.cpp — torch tensors to the C ABI for calls whose host time counts: the
// checks and the marshalling of a wrapper in api.py, which documents the call
// and passes its arguments on by position. A Python attribute of a tensor costs
// some 0.2 us, and such a call looks at fifty; here they are plain loads (the
// norm-and-rotation forward of 64 tokens took 27 us of host time by ctypes).
// Everything is computed in libcpattn.so, whose functions init() looks up.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>

#include "cp_attn.h"

namespace {

struct Raised {};  // a Python error is set

[[noreturn]] void refuse(PyObject* type, const char* text) {
  PyErr_SetString(type, text);
  throw Raised{};
}
[[noreturn]] void bad_value(const char* text) { refuse(PyExc_ValueError, text); }
[[noreturn]] void bad_type(const char* text) { refuse(PyExc_TypeError, text); }

const at::Tensor& tensor(PyObject* o) {
  if (!THPVariable_Check(o)) bad_type("a tensor is wanted");
  return THPVariable_Unpack(o);
}
// nullptr for None
const at::Tensor* maybe(PyObject* o) { return o == Py_None ? nullptr : &tensor(o); }

int cuda_index(const at::Tensor& t) {
  if (!t.is_cuda()) bad_value("tensors must live on a CUDA device");
  return t.get_device();
}
void on(int index, const at::Tensor& t) {
  if (!t.is_cuda() || t.get_device() != index) bad_value("all tensors must live on the device of the first one");
}
void dense_on(int index, const at::Tensor& t) {
  on(index, t);
  if (!t.is_contiguous()) bad_value("tensors must be dense");
}
cp_dtype type_of(c10::ScalarType t) {
  if (t != at::kBFloat16 && t != at::kFloat) bad_type("unsupported dtype: tensors must be bfloat16 or float32");
  return t == at::kBFloat16 ? CP_BF16 : CP_F32;
}
bool shaped(const at::Tensor& t, at::IntArrayRef shape) { return t.sizes() == shape; }
int size_of(int64_t n) {
  if (n > INT32_MAX) bad_value("a tensor is too large");
  return static_cast<int>(n);
}

// A workspace of `need` bytes: the caller's, or one of torch's for this call.
struct Workspace {
  at::Tensor own;
  void* p = nullptr;
  size_t bytes = 0;
  Workspace(PyObject* given, size_t need, int index) {
    if (given != Py_None) {
      const at::Tensor& t = tensor(given);
      dense_on(index, t);
      p = t.data_ptr();
      bytes = t.nbytes();
    } else if (need) {
      own = at::empty({static_cast<int64_t>(need)}, at::TensorOptions().dtype(at::kByte).device(at::kCUDA, index));
      p = own.data_ptr();
      bytes = need;
    }
  }
};

// The library's call, without Python's lock: a launch waits where the stream's queue is
// full, perhaps for a host function that needs the lock. (The arguments' tensors are held
// by the caller, and what `call` uses has been read from them.)
template <class F>
PyObject* unlocked(F call) {
  PyThreadState* const state = PyEval_SaveThread();
  const cp_status st = call();
  PyEval_RestoreThread(state);
  return PyLong_FromLong(st);
}

void* stream_of(int index) { return c10::cuda::getCurrentCUDAStream(index).stream(); }

#define CP_FUNCTIONS(X)                                                                         \
  X(cp_qk_norm_rope_fwd) X(cp_qk_norm_rope_bwd) X(cp_qk_norm_rope_bwd_workspace_size)           \
  X(cp_paged_kv_append_q4) X(cp_paged_kv_read_q4) X(cp_paged_attn_decode_q4)                     \
  X(cp_paged_attn_q4_workspace_size)
#define CP_DECLARE(name) decltype(&::name) name##_p = nullptr;
CP_FUNCTIONS(CP_DECLARE)
#undef CP_DECLARE

// ---------------------------------------------------------------------------
// queries and keys between their projections and the attention
// ---------------------------------------------------------------------------
struct Heads {
  void* p;  // (of an empty tensor nullptr, with which the library does nothing)
  int64_t strides[3];
};
// [B, S, heads, D] of a type, a head's values dense
void heads(Heads* h, int index, c10::ScalarType type, at::IntArrayRef shape, const at::Tensor& t) {
  if (t.scalar_type() != type) bad_type("queries and keys, before and after, must share a dtype, and so must gradients");
  if (!shaped(t, shape)) bad_value("shape mismatch");
  on(index, t);
  const auto st = t.strides();
  if (st[3] != 1) bad_value("the values of a head must be dense");
  h->p = t.data_ptr();
  for (int i = 0; i < 3; ++i) h->strides[i] = st[i];
}

void flat(int64_t* to, std::initializer_list<const Heads*> all) {
  for (const Heads* h : all)
    for (int i = 0; i < 3; ++i) *to++ = h->p ? h->strides[i] : 0;
}

struct Qk {
  int index, B, S, H, Hkv, D;
  cp_dtype dt;
  c10::ScalarType type;
  int64_t q_shape[4], k_shape[4];
  cp_qk_rule rule;

  // args: positions, freqs, axes (bytes), interleaved, eps, q_weight, k_weight
  Qk(PyObject* q_, PyObject* k_, PyObject* const* args) {
    const at::Tensor& q = tensor(q_);
    index = cuda_index(q);
    type = q.scalar_type();
    dt = type_of(type);
    if (q.dim() != 4) bad_value("q must be [B, S, H, D]");
    for (int i = 0; i < 4; ++i) q_shape[i] = k_shape[i] = q.size(i);
    B = size_of(q_shape[0]);
    S = size_of(q_shape[1]);
    H = size_of(q_shape[2]);
    D = size_of(q_shape[3]);
    Hkv = 0;
    if (const at::Tensor* k = maybe(k_)) {
      if (k->dim() != 4) bad_value("k must be [B, S, Hkv, D]");
      Hkv = size_of(k->size(2));
    }
    k_shape[2] = Hkv;
    rule = cp_qk_rule{};
    if (args[4] != Py_None) {
      rule.norm = 1;
      rule.eps = static_cast<float>(PyFloat_AsDouble(args[4]));
      if (PyErr_Occurred()) throw Raised{};
    }
    rule.weight_dt = dt;
    const at::Tensor* w[2] = {maybe(args[5]), maybe(args[6])};
    for (const at::Tensor* x : w) {
      if (!x) continue;
      if (!rule.norm) bad_value("weights need a norm (eps)");
      if (x->dim() != 1 || x->size(0) != D || (x->scalar_type() != type && x->scalar_type() != at::kFloat))
        bad_value("weights must be [D], of q's dtype or float32");
      dense_on(index, *x);
      rule.weight_dt = type_of(x->scalar_type());
    }
    if (w[0] && w[1] && w[0]->scalar_type() != w[1]->scalar_type()) bad_value("the weights must share a dtype");
    rule.q_weight = w[0] ? w[0]->data_ptr() : nullptr;
    rule.k_weight = w[1] ? w[1]->data_ptr() : nullptr;
    rule.interleaved = PyObject_IsTrue(args[3]);
    if (rule.interleaved < 0) throw Raised{};
    if (args[1] == Py_None) {
      if (args[0] != Py_None || args[2] != Py_None) bad_value("positions and axes need freqs");
      return;
    }
    if (args[0] == Py_None) bad_value("freqs need positions");
    const at::Tensor &pos = tensor(args[0]), &freqs = tensor(args[1]);
    if (freqs.scalar_type() != at::kDouble || freqs.dim() != 1) bad_value("freqs must be float64 [pairs]");
    if (pos.scalar_type() != at::kInt) bad_type("positions must be int32");
    const int n = static_cast<int>(pos.dim());
    if ((n != 2 && n != 3) || pos.size(n - 2) != S || (n == 3 && pos.size(0) != B))
      bad_value("positions must be [B, S, axes] or [S, axes]");
    dense_on(index, freqs);
    dense_on(index, pos);
    rule.pairs = size_of(freqs.size(0));
    rule.axes = size_of(pos.size(n - 1));
    rule.freqs = static_cast<const double*>(freqs.data_ptr());
    rule.positions = static_cast<const int32_t*>(pos.data_ptr());
    rule.positions_shared = n == 2;
    if (args[2] != Py_None) {
      char* text;
      Py_ssize_t len;
      if (PyBytes_AsStringAndSize(args[2], &text, &len)) throw Raised{};
      if (len != rule.pairs) bad_value("axes must name an axis for each pair");
      rule.pair_axis = reinterpret_cast<const uint8_t*>(text);
    }
  }
  at::IntArrayRef qs() const { return {q_shape, 4}; }
  at::IntArrayRef ks() const { return {k_shape, 4}; }
};

// q, k, q_out, k_out, then the rule's seven
PyObject* qk_norm_rope_fwd(PyObject* const* a) {
  if ((a[1] == Py_None) != (a[3] == Py_None)) bad_value("k and k_out come together");
  const Qk c(a[0], a[1], a + 4);
  Heads q{}, k{}, qo{}, ko{};
  heads(&q, c.index, c.type, c.qs(), tensor(a[0]));
  heads(&qo, c.index, c.type, c.qs(), tensor(a[2]));
  if (a[1] != Py_None) {
    heads(&k, c.index, c.type, c.ks(), tensor(a[1]));
    heads(&ko, c.index, c.type, c.ks(), tensor(a[3]));
  }
  int64_t st[12];
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(c.index));
  flat(st, {&q, &k, &qo, &ko});
  void* const s = stream_of(c.index);
  return unlocked([&] {
    return cp_qk_norm_rope_fwd_p(q.p, k.p, qo.p, ko.p, st, c.B, c.S, c.H, c.Hkv, c.D, &c.rule,
                                 c.dt, s);
  });
}

// q, k, dq_out, dk_out, dq, dk, the rule's seven, dq_weight, dk_weight, workspace
PyObject* qk_norm_rope_bwd(PyObject* const* a) {
  if ((a[1] == Py_None) != (a[3] == Py_None) || (a[1] == Py_None) != (a[5] == Py_None))
    bad_value("k, dk_out and dk come together");
  const Qk c(a[0], a[1], a + 6);
  const c10::ScalarType gtype = tensor(a[2]).scalar_type();
  if (gtype != c.type && gtype != at::kFloat) bad_type("dq_out and dk_out must be float32 or of q's dtype");
  Heads q{}, k{}, gq{}, gk{}, dq{}, dk{};
  heads(&q, c.index, c.type, c.qs(), tensor(a[0]));
  heads(&gq, c.index, gtype, c.qs(), tensor(a[2]));
  heads(&dq, c.index, c.type, c.qs(), tensor(a[4]));
  if (a[1] != Py_None) {
    heads(&k, c.index, c.type, c.ks(), tensor(a[1]));
    heads(&gk, c.index, gtype, c.ks(), tensor(a[3]));
    heads(&dk, c.index, c.type, c.ks(), tensor(a[5]));
  }
  float* w[2] = {nullptr, nullptr};
  for (int i = 0; i < 2; ++i)
    if (const at::Tensor* x = maybe(a[13 + i])) {
      if (x->dim() != 1 || x->size(0) != c.D || x->scalar_type() != at::kFloat)
        bad_value("weights' gradients must be float32 [D]");
      dense_on(c.index, *x);
      w[i] = static_cast<float*>(x->data_ptr());
    }
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(c.index));
  const Workspace ws(a[15], w[0] || w[1] ? cp_qk_norm_rope_bwd_workspace_size_p(c.D) : 0, c.index);
  int64_t st[18];
  flat(st, {&q, &k, &gq, &gk, &dq, &dk});
  const cp_dtype gdt = type_of(gtype);
  void* const s = stream_of(c.index);
  return unlocked([&] {
    return cp_qk_norm_rope_bwd_p(q.p, k.p, gq.p, gk.p, dq.p, dk.p, w[0], w[1], st,
                                 c.B, c.S, c.H, c.Hkv, c.D, &c.rule, ws.p, ws.bytes, c.dt, gdt, s);
  });
}

// ---------------------------------------------------------------------------
// the paged cache in 4 bits
// ---------------------------------------------------------------------------
const int32_t* ints(int index, const at::Tensor& t, at::IntArrayRef shape, const char* text) {
  if (t.scalar_type() != at::kInt) bad_type("block_table, seq_lens and new_lens must be int32");
  if (!shaped(t, shape)) bad_value(text);
  dense_on(index, t);
  return static_cast<const int32_t*>(t.data_ptr());
}

// a: k_codes, k_scales, v_codes, v_scales, block_table, of B sequences, Hkv heads of D
cp_q4_cache cache_of(PyObject* const* a, int index, int64_t B, int64_t Hkv, int64_t D) {
  const at::Tensor *t[4], &table = tensor(a[4]);
  for (int i = 0; i < 4; ++i) t[i] = &tensor(a[i]);
  if (t[0]->dim() != 4) bad_value("codes must be [num_pages, Hkv, page, D / 2]");
  const int64_t pages = t[0]->size(0), page = t[0]->size(2);
  const int64_t codes[4] = {pages, Hkv, page, D / 2}, scales[5] = {pages, Hkv, page, D / 64, 2};
  for (int i = 0; i < 4; ++i) {
    if (t[i]->scalar_type() != (i & 1 ? at::kBFloat16 : at::kByte)) bad_type("codes must be uint8, scales bfloat16");
    if (!shaped(*t[i], i & 1 ? at::IntArrayRef(scales, 5) : at::IntArrayRef(codes, 4)))
      bad_value("codes must be [num_pages, Hkv, page, D / 2], scales [num_pages, Hkv, page, D / 64, 2]");
    dense_on(index, *t[i]);
  }
  if (table.dim() != 2) bad_value("block_table must be [B, max_pages]");
  const int64_t shape[2] = {B, table.size(1)};
  cp_q4_cache c{};
  c.k_codes = static_cast<uint8_t*>(t[0]->data_ptr());
  c.k_scales = t[1]->data_ptr();
  c.v_codes = static_cast<uint8_t*>(t[2]->data_ptr());
  c.v_scales = t[3]->data_ptr();
  c.block_table = ints(index, table, {shape, 2}, "block_table must be [B, max_pages]");
  c.num_pages = size_of(pages);
  c.page_size = size_of(page);
  c.max_pages = size_of(shape[1]);
  return c;
}

// k_new, v_new, the cache's five, seq_lens, new_lens
PyObject* paged_kv_append_q4(PyObject* const* a) {
  const at::Tensor &k = tensor(a[0]), &v = tensor(a[1]);
  const int index = cuda_index(k);
  if (k.dim() != 4 || !shaped(v, k.sizes())) bad_value("k_new and v_new must be [B, T, Hkv, D]");
  if (v.scalar_type() != k.scalar_type()) bad_type("k_new and v_new must share a dtype");
  const cp_dtype dt = type_of(k.scalar_type());
  dense_on(index, k);
  dense_on(index, v);
  const int64_t B = k.size(0);
  const cp_q4_cache c = cache_of(a + 2, index, B, k.size(2), k.size(3));
  const int32_t* lens = ints(index, tensor(a[7]), {&B, 1}, "seq_lens must be [B]");
  const at::Tensor* news = maybe(a[8]);
  const int32_t* new_lens = news ? ints(index, *news, {&B, 1}, "new_lens must be [B]") : nullptr;
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(index));
  const int b = size_of(B), t = size_of(k.size(1)), hkv = size_of(k.size(2)), d = size_of(k.size(3));
  void *const kp = k.data_ptr(), *const vp = v.data_ptr(), *const s = stream_of(index);
  return unlocked([&] { return cp_paged_kv_append_q4_p(kp, vp, &c, lens, new_lens, b, t, hkv, d, dt, s); });
}

// the cache's five, seq_lens, k_out, v_out
PyObject* paged_kv_read_q4(PyObject* const* a) {
  const at::Tensor &k = tensor(a[6]), &v = tensor(a[7]);
  const int index = cuda_index(tensor(a[0]));
  if (k.dim() != 4 || !shaped(v, k.sizes())) bad_value("k_out and v_out must be [B, T, Hkv, D]");
  if (v.scalar_type() != k.scalar_type()) bad_type("k_out and v_out must share a dtype");
  const cp_dtype dt = type_of(k.scalar_type());
  dense_on(index, k);
  dense_on(index, v);
  const int64_t B = k.size(0);
  const cp_q4_cache c = cache_of(a, index, B, k.size(2), k.size(3));
  const int32_t* lens = ints(index, tensor(a[5]), {&B, 1}, "seq_lens must be [B]");
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(index));
  const int b = size_of(B), t = size_of(k.size(1)), hkv = size_of(k.size(2)), d = size_of(k.size(3));
  void *const kp = k.data_ptr(), *const vp = v.data_ptr(), *const s = stream_of(index);
  return unlocked([&] { return cp_paged_kv_read_q4_p(&c, lens, kp, vp, b, t, hkv, d, dt, s); });
}

// q, the cache's five, seq_lens, out, lse, scale, softcap, slopes, workspace
PyObject* paged_attn_decode_q4(PyObject* const* a) {
  const at::Tensor &q = tensor(a[0]), &out = tensor(a[7]), &lse = tensor(a[8]), &codes = tensor(a[1]);
  const int index = cuda_index(q);
  const c10::ScalarType type = q.scalar_type();
  const cp_dtype dt = type_of(type);
  if (q.dim() != 3 || codes.dim() != 4) bad_value("q must be [B, H, D], codes [num_pages, Hkv, page, D / 2]");
  const int64_t B = q.size(0), H = q.size(1), D = q.size(2), Hkv = codes.size(1), lse_shape[2] = {B, H};
  if (!shaped(out, q.sizes()) || !shaped(lse, {lse_shape, 2})) bad_value("shape mismatch");
  if (lse.scalar_type() != at::kFloat) bad_type("lse must be float32");
  if (out.scalar_type() != type && out.scalar_type() != at::kFloat) bad_type("out must be float32 or of q's dtype");
  dense_on(index, q);
  dense_on(index, out);
  dense_on(index, lse);
  const cp_q4_cache c = cache_of(a + 1, index, B, Hkv, D);
  const int32_t* lens = ints(index, tensor(a[6]), {&B, 1}, "seq_lens must be [B]");
  const double scale = PyFloat_AsDouble(a[9]), cap = PyFloat_AsDouble(a[10]);
  if (PyErr_Occurred()) throw Raised{};
  const float* slopes = nullptr;
  if (const at::Tensor* t = maybe(a[11])) {
    if (t->scalar_type() != at::kFloat || !shaped(*t, {&H, 1})) bad_value("slopes must be float32 [H]");
    dense_on(index, *t);
    slopes = static_cast<const float*>(t->data_ptr());
  }
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(index));
  const int b = size_of(B), h = size_of(H), hkv = size_of(Hkv), d = size_of(D);
  const Workspace ws(a[12], cp_paged_attn_q4_workspace_size_p(b, h, hkv, d, c.page_size, c.max_pages, dt), index);
  const cp_dtype out_dt = type_of(out.scalar_type());
  void *const qp = q.data_ptr(), *const op = out.data_ptr(), *const s = stream_of(index);
  float* const lp = static_cast<float*>(lse.data_ptr());
  return unlocked([&] {
    return cp_paged_attn_decode_q4_p(qp, &c, lens, op, lp, b, h, hkv, d, static_cast<float>(scale), static_cast<float>(cap),
                                     slopes, ws.p, ws.bytes, dt, out_dt, s);
  });
}

// ---------------------------------------------------------------------------
// the module
// ---------------------------------------------------------------------------
template <PyObject* (*kCall)(PyObject* const*), int kArgs>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != kArgs) {
    PyErr_Format(PyExc_TypeError, "%d arguments are wanted, %zd given", kArgs, n);
    return nullptr;
  }
  try {
    return kCall(args);
  } catch (const Raised&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// init(handle): the library as the dynamic loader knows it
PyObject* init(PyObject*, PyObject* handle) {
  void* lib = PyLong_AsVoidPtr(handle);
  if (PyErr_Occurred()) return nullptr;
#define CP_LOOK_UP(name)                                               \
  name##_p = reinterpret_cast<decltype(&::name)>(dlsym(lib, #name));   \
  if (!name##_p) {                                                     \
    PyErr_SetString(PyExc_RuntimeError, "libcpattn.so lacks " #name);  \
    return nullptr;                                                    \
  }
  CP_FUNCTIONS(CP_LOOK_UP)
#undef CP_LOOK_UP
  Py_RETURN_NONE;
}

template <PyObject* (*kCall)(PyObject* const*), int kArgs>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&entry<kCall, kArgs>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {
    {"init", init, METH_O, nullptr},
    method<qk_norm_rope_fwd, 11>("qk_norm_rope_fwd"),
    method<qk_norm_rope_bwd, 16>("qk_norm_rope_bwd"),
    method<paged_kv_append_q4, 9>("paged_kv_append_q4"),
    method<paged_kv_read_q4, 8>("paged_kv_read_q4"),
    method<paged_attn_decode_q4, 13>("paged_attn_decode_q4"),
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_cpbind", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__cpbind() { return PyModule_Create(&module); }
