// The 8-bit cache's and the shared prefix's calls as the usual program makes them, from
// tensor objects to the C entry points without the interpreter in between: these calls
// last a few microseconds on small inputs, of which checks in Python took a dozen.
//
// Each function takes the arguments of its namesake in cache_q8.py or attn.py by
// position, and returns what that returns, or None where anything is not as
// expected: the Python form then checks step by step and raises what there is to raise,
// or serves the rare case (another current device, a stride of a dimension of size 1).
// None means that the library was not called.  Once it was, its status is the answer, an
// int if it is not 0: the call may have done its work all the same (the runtime reports
// an earlier error to whoever asks next), and rows rotated in place must not be again.
// The interpreter's lock is released over allocations and the library's call.
#include <Python.h>

#include <cmath>
#include <cstring>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "rnn.h"

namespace {

decltype(&rnn_kv_append_q8) f_append = nullptr;
decltype(&rnn_kv_read_q8) f_read = nullptr;
decltype(&rnn_attn_decode_q8) f_decode = nullptr;
decltype(&rnn_attn_decode_q8_workspace_size) f_decode_need = nullptr;
decltype(&rnn_attn_decode_shared) f_shared = nullptr;
decltype(&rnn_attn_decode_shared_workspace_size) f_shared_need = nullptr;

// Other Python threads run while this lives.
struct Unlocked {
  PyThreadState* const state = PyEval_SaveThread();
  ~Unlocked() { PyEval_RestoreThread(state); }
};

// The tensors of a call, all on one device.
struct Call {
  bool ok = true, made = false;  // made: the library was called, with this status
  int device = -1, status = 0;
  const at::Tensor* tensor(PyObject* o, int64_t ndim, at::ScalarType type) {
    if (!ok || !THPVariable_CheckExact(o)) return fail();
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.dim() != ndim || t.scalar_type() != type) return fail();
    if (device < 0) device = t.get_device();
    if (t.get_device() != device) return fail();
    return &t;
  }
  const at::Tensor* fail() {
    ok = false;
    return nullptr;
  }
  bool want(bool x) { return ok = ok && x; }

  // rows of d channels whose strides and address are the usual ones
  rnn_rows rows(const at::Tensor& t, int64_t d) {
    const auto s = t.strides();
    rnn_rows r{t.data_ptr(), s[0], s[1]};
    want(s[2] == 1 && s[0] >= d && s[1] >= d && !((s[0] | s[1]) & 7) && aligned(r.data, 16));
    return r;
  }
  rnn_pages pages(const at::Tensor& t, int64_t d) {
    const auto s = t.strides();
    rnn_pages r{t.data_ptr(), s[0], s[1], s[2]};
    want(s[3] == 1 && s[0] >= d && s[1] >= d && s[2] >= d && !((s[0] | s[1] | s[2]) & 7) &&
         aligned(r.data, 16));
    return r;
  }
  const int32_t* ints(PyObject* o, int64_t n) {
    const at::Tensor* t = tensor(o, 1, at::kInt);
    if (!t || !want(t->size(0) == n && t->is_contiguous())) return nullptr;
    return t->const_data_ptr<int32_t>();
  }
  const int32_t* table(PyObject* o, int64_t B, int64_t* stride, int32_t* n) {
    const at::Tensor* t = tensor(o, 2, at::kInt);
    if (!t || !want(t->size(0) == B && t->size(1) >= 1 && t->size(1) <= INT32_MAX &&
                    (t->size(1) == 1 || t->stride(1) == 1)))
      return nullptr;
    *stride = B > 1 ? t->stride(0) : t->size(1);
    *n = static_cast<int32_t>(t->size(1));
    return t->const_data_ptr<int32_t>();
  }
  static bool aligned(const void* p, uintptr_t to) { return !(reinterpret_cast<uintptr_t>(p) % to); }

  // a value type, or none
  int dtype(PyObject* o, at::ScalarType* type) {
    if (!ok || !THPVariable_CheckExact(o)) return fail(), 0;
    *type = THPVariable_Unpack(o).scalar_type();
    want(*type == at::kHalf || *type == at::kBFloat16);
    return *type == at::kBFloat16 ? RNN_BF16 : RNN_F16;
  }
  bool here() { return want(device == c10::cuda::current_device()); }
  rnn_stream_t stream() const {
    return reinterpret_cast<rnn_stream_t>(c10::cuda::getCurrentCUDAStream(device).stream());
  }
  at::Tensor bytes(size_t n) const { return empty({static_cast<int64_t>(n)}, at::kByte); }
  at::Tensor empty(at::IntArrayRef size, at::ScalarType type) const {
    return at::empty(size, at::TensorOptions().dtype(type).device(at::kCUDA, device));
  }
  // the caller's tensor of this shape; none yet where a new one is to be made
  at::Tensor out(PyObject* o, at::IntArrayRef size, at::ScalarType type) {
    if (o == Py_None) return {};
    const at::Tensor* t = tensor(o, static_cast<int64_t>(size.size()), type);
    if (!t || !want(t->sizes() == size)) return {};
    return *t;
  }
  // the caller's workspace, or none yet
  at::Tensor scratch(PyObject* o) {
    if (o == Py_None) return {};
    const at::Tensor* t = tensor(o, 1, at::kByte);
    if (!t || !want(t->is_contiguous())) return {};
    return *t;
  }
  // the library's call
  template <typename Args>
  void call(rnn_status (*f)(const Args*, rnn_stream_t), const Args& p) {
    if (!ok) return;
    made = true;
    status = f(&p, stream());
  }
  bool done() const { return made && status == RNN_OK; }
  float scale(PyObject* o, int64_t d) {
    if (o == Py_None) return static_cast<float>(1.0 / std::sqrt(static_cast<double>(d)));
    if (!want(PyFloat_CheckExact(o))) return 0.f;
    const double s = PyFloat_AS_DOUBLE(o);
    want(s > 0.0 && s < 2e38);
    return static_cast<float>(s);
  }
  bool flag(PyObject* o) {
    want(PyBool_Check(o));
    return o == Py_True;
  }
};

// The tensors of a cache of codes.
struct Coded {
  int64_t pages = 0, size = 0, heads = 0, d = 0;
  int32_t codes = 0;
  rnn_pages k{}, v{};
  rnn_scales scales{};
};
Coded coded(Call& c, PyObject* k, PyObject* v, PyObject* s) {
  Coded r;
  if (!c.ok || !THPVariable_CheckExact(k)) return c.fail(), r;
  const at::ScalarType type = THPVariable_Unpack(k).scalar_type();
  if (!c.want(type == at::kFloat8_e4m3fn || type == at::kChar)) return r;
  const at::Tensor *kt = c.tensor(k, 4, type), *vt = c.tensor(v, 4, type);
  const at::Tensor* st = c.tensor(s, 4, at::kFloat);
  if (!kt || !vt || !st) return r;
  r.codes = type == at::kChar ? RNN_CODES_INT8 : RNN_CODES_E4M3;
  r.pages = kt->size(0), r.size = kt->size(1), r.heads = kt->size(2), r.d = kt->size(3);
  if (!c.want(kt->sizes() == vt->sizes() && r.pages >= 1 && r.size >= 1 && r.heads >= 1 &&
              r.size <= INT32_MAX && st->size(0) == r.pages && st->size(1) == r.heads &&
              st->size(2) == r.size && st->size(3) == 2))
    return r;
  const auto ss = st->strides();
  r.k = c.pages(*kt, r.d);
  r.v = c.pages(*vt, r.d);
  r.scales = rnn_scales{st->data_ptr<float>(), ss[0], ss[1]};
  c.want(ss[3] == 1 && ss[2] == 2 && ss[0] >= 2 * r.size && ss[1] >= 2 * r.size &&
         !((ss[0] | ss[1]) & 1) && Call::aligned(r.scales.data, 8));
  return r;
}

PyObject* give(const at::Tensor& out, const at::Tensor& lse) {
  PyObject* o = THPVariable_Wrap(out);
  if (!lse.defined()) return o;
  PyObject* l = THPVariable_Wrap(lse);
  PyObject* both = PyTuple_Pack(2, o, l);
  Py_XDECREF(o);
  Py_XDECREF(l);
  return both;
}

bool channels(int64_t d, int64_t most) { return d >= 8 && d % 8 == 0 && d <= most; }
bool heads(int64_t hq, int64_t hkv) {
  return hkv >= 1 && hq >= 1 && hq <= RNN_ATTN_MAX_HEADS && hq % hkv == 0;
}

// (q, k_cache, v_cache, scales, page_table, lens, scale, with_lse, out, workspace)
PyObject* decode_q8(Call& c, PyObject* const* a) {
  at::ScalarType type;
  rnn_attn_decode_q8_args p;
  std::memset(&p, 0, sizeof(p));
  p.dtype = c.dtype(a[0], &type);
  const at::Tensor* q = c.ok ? c.tensor(a[0], 3, type) : nullptr;
  const Coded cache = coded(c, a[1], a[2], a[3]);
  if (!c.ok) return nullptr;
  const int64_t B = q->size(0), hq = q->size(1), d = q->size(2);
  if (!c.want(cache.d == d && channels(d, RNN_ATTN_MAX_DIM) && heads(hq, cache.heads)) || B < 1 ||
      B > INT32_MAX - 1024 || !c.here())
    return nullptr;
  p.q = c.rows(*q, d);
  p.k_cache = cache.k, p.v_cache = cache.v, p.scales = cache.scales;
  p.lens = c.ints(a[5], B);
  p.page_table = c.table(a[4], B, &p.table_stride, &p.max_pages);
  p.scale = c.scale(a[6], d);
  const bool with_lse = c.flag(a[7]);
  if (!c.ok) return nullptr;
  at::Tensor out = c.out(a[8], q->sizes(), type), scratch = c.scratch(a[9]), lse;
  if (!c.ok) return nullptr;
  p.num_pages = cache.pages;
  p.page_size = static_cast<int32_t>(cache.size);
  p.B = static_cast<int32_t>(B), p.Hq = static_cast<int32_t>(hq);
  p.Hkv = static_cast<int32_t>(cache.heads), p.d = static_cast<int32_t>(d);
  p.codes = cache.codes;
  {
    Unlocked unlocked;
    if (!out.defined()) out = c.empty({B, hq, d}, type);
    if (!scratch.defined()) scratch = c.bytes(f_decode_need(p.B, p.Hq, p.Hkv, p.d));
    if (with_lse) lse = c.empty({B, hq}, at::kFloat), p.lse = lse.data_ptr<float>();
    p.out = c.rows(out, d);
    p.workspace = scratch.data_ptr(), p.ws_bytes = static_cast<uint64_t>(scratch.numel());
    c.call(f_decode, p);
  }
  return c.done() ? give(out, lse) : nullptr;
}

// (q, k_cache, v_cache, prefix_pages, prefix_len, page_table, lens, scale, with_lse, out, workspace)
PyObject* shared(Call& c, PyObject* const* a) {
  at::ScalarType type;
  rnn_attn_decode_shared_args p;
  std::memset(&p, 0, sizeof(p));
  p.dtype = c.dtype(a[0], &type);
  const at::Tensor* q = c.ok ? c.tensor(a[0], 3, type) : nullptr;
  const at::Tensor* k = c.ok ? c.tensor(a[1], 4, type) : nullptr;
  const at::Tensor* v = c.ok ? c.tensor(a[2], 4, type) : nullptr;
  const at::Tensor* prefix = c.ok ? c.tensor(a[3], 1, at::kInt) : nullptr;
  if (!c.ok) return nullptr;
  const int64_t B = q->size(0), hq = q->size(1), d = q->size(2), hkv = k->size(2);
  const int64_t count = prefix->size(0);
  if (!c.want(k->sizes() == v->sizes() && k->size(3) == d && k->size(0) >= 1 && k->size(1) >= 1 &&
              k->size(1) <= INT32_MAX && channels(d, RNN_ATTN_MAX_DIM) && heads(hq, hkv) &&
              count >= 1 && count <= INT32_MAX && prefix->is_contiguous()) ||
      B < 1 || B > INT32_MAX - 1024 || !c.here())
    return nullptr;
  p.q = c.rows(*q, d);
  p.k_cache = c.pages(*k, d), p.v_cache = c.pages(*v, d);
  p.prefix_pages = prefix->const_data_ptr<int32_t>();
  p.prefix_len = c.ints(a[4], 1);
  p.page_table = c.table(a[5], B, &p.table_stride, &p.max_pages);
  p.lens = c.ints(a[6], B);
  p.scale = c.scale(a[7], d);
  const bool with_lse = c.flag(a[8]);
  if (!c.ok) return nullptr;
  at::Tensor out = c.out(a[9], q->sizes(), type), scratch = c.scratch(a[10]), lse;
  if (!c.ok) return nullptr;
  p.num_pages = k->size(0);
  p.page_size = static_cast<int32_t>(k->size(1));
  p.prefix_pages_count = static_cast<int32_t>(count);
  p.B = static_cast<int32_t>(B), p.Hq = static_cast<int32_t>(hq);
  p.Hkv = static_cast<int32_t>(hkv), p.d = static_cast<int32_t>(d);
  {
    Unlocked unlocked;
    if (!out.defined()) out = c.empty({B, hq, d}, type);
    if (!scratch.defined())
      scratch = c.bytes(f_shared_need(p.B, p.Hq, p.Hkv, p.d, count * p.page_size));
    if (with_lse) lse = c.empty({B, hq}, at::kFloat), p.lse = lse.data_ptr<float>();
    p.out = c.rows(out, d);
    p.workspace = scratch.data_ptr(), p.ws_bytes = static_cast<uint64_t>(scratch.numel());
    c.call(f_shared, p);
  }
  return c.done() ? give(out, lse) : nullptr;
}

// (k_cache, v_cache, scales, page_table, cu, tokens, bf16, start, k_out, v_out)
PyObject* read_q8(Call& c, PyObject* const* a) {
  rnn_kv_read_q8_args p;
  std::memset(&p, 0, sizeof(p));
  const Coded cache = coded(c, a[0], a[1], a[2]);
  if (!c.ok || !PyLong_CheckExact(a[5]) || !PyBool_Check(a[6])) return nullptr;
  const int64_t T = PyLong_AsLongLong(a[5]);
  if (T < 1 || T > INT32_MAX - 1024) {
    PyErr_Clear();
    return nullptr;
  }
  const at::Tensor* cu = c.tensor(a[4], 1, at::kInt);
  if (!cu || !c.want(channels(cache.d, 256) && cache.heads <= RNN_ATTN_MAX_HEADS) || !c.here())
    return nullptr;
  const int64_t B = cu->size(0) - 1;
  if (B < 1 || B > INT32_MAX - 1024) return nullptr;
  p.cu = c.ints(a[4], B + 1);
  if (a[7] != Py_None) p.start = c.ints(a[7], B);
  p.page_table = c.table(a[3], B, &p.table_stride, &p.max_pages);
  if (!c.ok) return nullptr;
  const at::ScalarType type = a[6] == Py_True ? at::kBFloat16 : at::kHalf;
  at::Tensor k = c.out(a[8], {T, cache.heads, cache.d}, type);
  at::Tensor v = c.out(a[9], {T, cache.heads, cache.d}, type);
  if (!c.ok) return nullptr;
  p.k_cache = cache.k, p.v_cache = cache.v, p.scales = cache.scales;
  p.T = T, p.num_pages = cache.pages;
  p.Hkv = static_cast<int32_t>(cache.heads), p.d = static_cast<int32_t>(cache.d);
  p.dtype = type == at::kBFloat16 ? RNN_BF16 : RNN_F16;
  p.codes = cache.codes, p.page_size = static_cast<int32_t>(cache.size);
  p.B = static_cast<int32_t>(B);
  {
    Unlocked unlocked;
    for (at::Tensor* t : {&k, &v})
      if (!t->defined()) *t = c.empty({T, cache.heads, cache.d}, type);
    p.k = c.rows(k, cache.d), p.v = c.rows(v, cache.d);
    c.call(f_read, p);
  }
  return c.done() ? give(k, v) : nullptr;
}

// (k, v, k_cache, v_cache, scales, page_table, start, cu, q, inv_freq, positions, paired, with_k,
//  q_out, k_out)
PyObject* append_q8(Call& c, PyObject* const* a) {
  at::ScalarType type;
  rnn_kv_append_q8_args p;
  std::memset(&p, 0, sizeof(p));
  p.dtype = c.dtype(a[0], &type);
  const at::Tensor* k = c.ok ? c.tensor(a[0], 3, type) : nullptr;
  const at::Tensor* v = c.ok ? c.tensor(a[1], 3, type) : nullptr;
  const Coded cache = coded(c, a[2], a[3], a[4]);
  if (!c.ok) return nullptr;
  const int64_t T = k->size(0), hkv = k->size(1), d = k->size(2);
  if (!c.want(k->sizes() == v->sizes() && cache.heads == hkv && cache.d == d && channels(d, 256) &&
              hkv <= RNN_ATTN_MAX_HEADS) ||
      T < 1 || T > INT32_MAX - 1024 || !c.here())
    return nullptr;
  const at::Tensor* cu = c.tensor(a[7], 1, at::kInt);
  if (!cu) return nullptr;
  const int64_t B = cu->size(0) - 1;
  if (B < 1 || B > INT32_MAX - 1024) return nullptr;
  p.cu = c.ints(a[7], B + 1);
  p.start = c.ints(a[6], B);
  p.page_table = c.table(a[5], B, &p.table_stride, &p.max_pages);
  p.k = c.rows(*k, d), p.v = c.rows(*v, d);
  const at::Tensor* q = nullptr;
  if (a[8] != Py_None) {
    q = c.tensor(a[8], 3, type);
    if (!q || !c.want(q->size(0) == T && q->size(2) == d && q->size(1) >= 1 &&
                      q->size(1) <= RNN_ATTN_MAX_HEADS && a[9] != Py_None))
      return nullptr;
    p.q = c.rows(*q, d);
    p.Hq = static_cast<int32_t>(q->size(1));
  } else if (a[13] != Py_None) {
    return nullptr;
  }
  if (a[9] != Py_None) {
    const at::Tensor* f = c.tensor(a[9], 1, at::kDouble);
    if (!f || !c.want(f->size(0) >= 1 && f->size(0) <= 128 && f->is_contiguous())) return nullptr;
    p.inv_freq = f->const_data_ptr<double>();
    p.pairs = static_cast<int32_t>(f->size(0));
    p.axes = 1;
  }
  if (a[10] != Py_None) {
    if (!p.axes || !THPVariable_CheckExact(a[10])) return nullptr;
    const int64_t nd = THPVariable_Unpack(a[10]).dim();
    if (nd != 1 && nd != 2) return nullptr;
    const at::Tensor* t = c.tensor(a[10], nd, at::kInt);
    if (!t) return nullptr;
    const int64_t axes = nd == 2 ? t->size(1) : 1;
    if (!c.want(t->size(0) == T && (axes == 1 || (axes == 2 && t->stride(1) == 1)))) return nullptr;
    p.axes = static_cast<int32_t>(axes);
    p.position_stride = T > 1 ? t->stride(0) : axes;
    if (!c.want(p.position_stride >= axes)) return nullptr;
    p.positions = t->const_data_ptr<int32_t>();
  }
  if (!c.want(2 * int64_t{p.pairs} * p.axes <= d)) return nullptr;
  p.paired = c.flag(a[11]);
  const bool with_k = c.flag(a[12]);
  if (!c.ok) return nullptr;
  at::Tensor q_out, k_out = c.out(a[14], k->sizes(), type);
  if (q) q_out = c.out(a[13], q->sizes(), type);
  if (!c.ok) return nullptr;
  p.k_cache = cache.k, p.v_cache = cache.v, p.scales = cache.scales;
  p.T = T, p.num_pages = cache.pages;
  p.Hkv = static_cast<int32_t>(hkv), p.d = static_cast<int32_t>(d);
  p.codes = cache.codes, p.page_size = static_cast<int32_t>(cache.size);
  p.B = static_cast<int32_t>(B);
  {
    Unlocked unlocked;
    if (q && !q_out.defined()) q_out = c.empty({T, p.Hq, d}, type);
    if (with_k && !k_out.defined()) k_out = c.empty({T, hkv, d}, type);
    if (q) p.q_out = c.rows(q_out, d);
    if (k_out.defined()) p.k_out = c.rows(k_out, d);
    c.call(f_append, p);
  }
  if (!c.done()) return nullptr;
  PyObject* qo = q ? THPVariable_Wrap(q_out) : Py_NewRef(Py_None);
  PyObject* ko = k_out.defined() ? THPVariable_Wrap(k_out) : Py_NewRef(Py_None);
  PyObject* both = PyTuple_Pack(2, qo, ko);
  Py_XDECREF(qo);
  Py_XDECREF(ko);
  return both;
}

// A call that could not be served here, by an error of torch's allocator too, is None.
template <PyObject* (*kCall)(Call&, PyObject* const*), Py_ssize_t kArgs>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != kArgs || !f_append) Py_RETURN_NONE;
  Call c;
  try {
    if (PyObject* r = kCall(c, args)) return r;
  } catch (const std::exception& e) {
    if (c.made && !PyErr_Occurred()) PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  if (c.made) {
    if (c.status == RNN_OK) return nullptr;  // its results could not be handed over
    PyErr_Clear();
    return PyLong_FromLong(c.status);
  }
  if (PyErr_Occurred()) PyErr_Clear();
  Py_RETURN_NONE;
}

// The C entry points' addresses, in the order of the pointers above.
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
  void** to[] = {reinterpret_cast<void**>(&f_read),        reinterpret_cast<void**>(&f_decode),
                 reinterpret_cast<void**>(&f_decode_need), reinterpret_cast<void**>(&f_shared),
                 reinterpret_cast<void**>(&f_shared_need), reinterpret_cast<void**>(&f_append)};
  if (n != 6) {
    PyErr_SetString(PyExc_TypeError, "bind takes six addresses");
    return nullptr;
  }
  for (int i = 0; i < 6; ++i) {
    void* at = PyLong_AsVoidPtr(args[i]);
    if (!at) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "an address is null");
      return nullptr;
    }
    *to[i] = at;
  }
  Py_RETURN_NONE;
}

#define FAST(call, args) \
  reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<call, args>)), METH_FASTCALL
PyMethodDef methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&bind)), METH_FASTCALL, nullptr},
    {"attn_decode_q8", FAST(decode_q8, 10), nullptr},
    {"attn_decode_shared", FAST(shared, 11), nullptr},
    {"kv_read_q8", FAST(read_q8, 10), nullptr},
    {"kv_append_q8", FAST(append_q8, 15), nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fast", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fast() { return PyModule_Create(&module); }
