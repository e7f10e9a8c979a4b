// attn_calls.cpp — the Python calls of the paged cache and attention
// operators: torch tensors to the arguments of the C entry points.
//
// A decode step makes these calls for every layer, with kernels of a few
// microseconds.  From Python alone (ctypes, and the tensors' properties read
// one by one) the append of 64 tokens took 16.7 us a call, from here 4.9; the launch
// itself is 2 to 3 of them, a new output tensor 1.5.
// The checks here are those of shapes, types and devices; ranges, alignment and
// the rest are the entry points' own, whose status the package's `check`
// turns into its exception.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <exception>
#include <initializer_list>
#include <string>
#include <type_traits>

#include "mxq.h"

namespace {

decltype(&mxq_rope_append_kv) append_fn;
decltype(&mxq_paged_attention_decode) decode_fn;
decltype(&mxq_paged_attention_decode_workspace_size) decode_size_fn;
decltype(&mxq_attention_varlen) prompt_fn;
decltype(&mxq_attention_varlen_workspace_size) prompt_size_fn;
decltype(&mxq_current_device) device_fn;
decltype(&mxq_paged_attention_decode_ex) decode_ex_fn;
decltype(&mxq_attention_varlen_ex) prompt_ex_fn;
decltype(&mxq_paged_attention_tree) tree_fn;
decltype(&mxq_paged_attention_tree_workspace_size) tree_size_fn;
decltype(&mxq_cache_pages_workspace_size) pages_size_fn;
decltype(&mxq_cache_resize) resize_fn;
decltype(&mxq_cache_fork) fork_fn;
decltype(&mxq_cache_copy_pages) copy_pages_fn;
decltype(&mxq_cache_compact) compact_fn;
PyObject* check_fn;        // raises for a status
PyObject* stream_fn;       // device index -> the current stream's address

struct Raised {};          // a Python exception is set

[[noreturn]] void refuse(PyObject* type, const std::string& what) {
  PyErr_SetString(type, what.c_str());
  throw Raised();
}

// Other Python threads run while torch allocates or copies and while the entry point
// launches (a full queue makes it wait).  Once a call: letting go costs 0.1 us.
template <typename F>
auto unlocked(F f) {
  struct Unlocked {
    PyThreadState* state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
  } u;
  return f();
}

void check(mxq_status status) {
  if (status == MXQ_OK) return;
  PyObject* r = PyObject_CallFunction(check_fn, "i", static_cast<int>(status));
  Py_XDECREF(r);
  if (r != nullptr) refuse(PyExc_RuntimeError, "status " + std::to_string(status));
  throw Raised();
}

// an argument that may be None
const at::Tensor* tensor(const char* name, PyObject* o) {
  if (o == Py_None) return nullptr;
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, std::string(name) + " must be a tensor");
  return &THPVariable_Unpack(o);
}
const at::Tensor& needed(const char* name, PyObject* o) {
  const at::Tensor* t = tensor(name, o);
  if (t == nullptr) refuse(PyExc_TypeError, std::string(name) + " must be a tensor");
  return *t;
}

// The tensors are on one device, and it is the current one: the entry points launch
// there, whatever device the pointers and the stream belong to.
void same_device(std::initializer_list<const at::Tensor*> ts) {
  const at::Tensor& first = **ts.begin();
  for (const at::Tensor* t : ts)
    if (t != nullptr && (!t->is_cuda() || t->device() != first.device()))
      refuse(PyExc_ValueError, "mxq operates on CUDA tensors of one device (got " +
                                   first.device().str() + " and " + t->device().str() + ")");
  int32_t current = 0;
  check(device_fn(&current));
  if (first.device().index() != current)
    refuse(PyExc_ValueError, "the tensors are on " + first.device().str() +
                                 ", the current device is cuda:" + std::to_string(current));
}

std::string shape_of(at::IntArrayRef s) {
  std::string r = "[";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + "]";
}

int32_t narrow(const char* name, int64_t n) {
  if (n < INT32_MIN || n > INT32_MAX)
    refuse(PyExc_ValueError, std::string(name) + " is out of range");
  return static_cast<int32_t>(n);
}
int32_t integer(const char* name, PyObject* o) {
  const long long n = PyLong_AsLongLong(o);
  if (n == -1 && PyErr_Occurred()) throw Raised();
  return narrow(name, n);
}
int32_t truth(PyObject* o) {
  const int n = PyObject_IsTrue(o);
  if (n < 0) throw Raised();
  return n;
}
float scale_of(PyObject* o, int64_t D) {
  if (o == Py_None) return static_cast<float>(1.0 / std::sqrt(static_cast<double>(D)));
  const double s = PyFloat_AsDouble(o);
  if (s == -1.0 && PyErr_Occurred()) throw Raised();
  return static_cast<float>(s);
}

// [n, heads, D] as the kernels read it, with unit inner stride, outer strides
// of 16-byte multiples and at least D (copied only if needed)
struct Heads {
  at::Tensor copy;
  void* p;
  int64_t n, heads, D, s0, s1;
  Heads(const char* name, const at::Tensor& t) {
    if (t.scalar_type() != at::kBFloat16)
      refuse(PyExc_TypeError, std::string(name) + " must be bf16");
    if (t.dim() != 3)
      refuse(PyExc_ValueError, std::string(name) + " must be [tokens, heads, head_dim], got " +
                                   std::to_string(t.dim()) + " dimensions");
    n = t.size(0), heads = t.size(1), D = t.size(2);
    s0 = t.stride(0), s1 = t.stride(1);
    p = t.data_ptr();
    if (t.stride(2) != 1 || (n > 1 && (s0 < D || (s0 & 7))) ||
        (heads > 1 && (s1 < D || (s1 & 7))) || (reinterpret_cast<uintptr_t>(p) & 15)) {
      copy = unlocked([&] { return t.clone(at::MemoryFormat::Contiguous); });
      s0 = copy.stride(0), s1 = copy.stride(1);
      p = copy.data_ptr();
    }
  }
};

struct Caches {
  int32_t dtype, page_size;
  int64_t pages, heads;
  void *k, *v;
  int64_t k0, k1, k2, v0, v1, v2;
  // kv_heads < 0: any
  Caches(const at::Tensor& kc, const at::Tensor& vc, int64_t kv_heads, int64_t D) {
    if (kc.dim() != 4 || kc.size(3) != D || (kv_heads >= 0 && kc.size(2) != kv_heads))
      refuse(PyExc_ValueError,
             "k_cache must be [pages, page_size, " +
                 (kv_heads < 0 ? std::string("kv_heads") : std::to_string(kv_heads)) + ", " +
                 std::to_string(D) + "], got " + shape_of(kc.sizes()));
    const at::ScalarType type = kc.scalar_type();
    if (vc.sizes() != kc.sizes() || vc.scalar_type() != type)
      refuse(PyExc_ValueError, "k_cache and v_cache must have the same shape and dtype");
    if (type != at::kBFloat16 && type != at::kFloat8_e4m3fn)
      refuse(PyExc_TypeError, "k_cache and v_cache must be bf16 or float8_e4m3fn");
    if (kc.stride(3) != 1 || vc.stride(3) != 1)
      refuse(PyExc_ValueError, "k_cache and v_cache need a unit stride along the head dimension");
    dtype = type == at::kBFloat16 ? MXQ_BF16 : MXQ_E4M3;
    pages = kc.size(0), page_size = narrow("the page size", kc.size(1)), heads = kc.size(2);
    k = kc.data_ptr(), v = vc.data_ptr();
    k0 = kc.stride(0), k1 = kc.stride(1), k2 = kc.stride(2);
    v0 = vc.stride(0), v1 = vc.stride(1), v2 = vc.stride(2);
  }
};

// the address of a contiguous vector of n elements (null for none)
template <typename T>
T* vec(const char* name, const at::Tensor* t, at::ScalarType type, int64_t n) {
  if (t == nullptr) return nullptr;
  if (t->scalar_type() != type || t->numel() != n || !t->is_contiguous())
    refuse(PyExc_ValueError, std::string(name) + " must be contiguous " + c10::toString(type) +
                                 " of " + std::to_string(n) + " elements");
  return static_cast<T*>(t->data_ptr());
}

at::Tensor fresh(at::IntArrayRef shape, at::ScalarType type, const at::Tensor& like) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(like.device()));
}

// an output that the caller may have given
at::Tensor output(const char* name, const at::Tensor* given, at::IntArrayRef shape) {
  if (given == nullptr) return at::Tensor();
  if (given->scalar_type() != at::kBFloat16 || given->sizes() != shape || given->stride(2) != 1)
    refuse(PyExc_ValueError, std::string(name) + " must be bf16 " + shape_of(shape) +
                                 " with a unit inner stride");
  return *given;
}

mxq_stream_t stream_of(const at::Tensor& t) {
  PyObject* dev = PyLong_FromLong(t.device().index());
  PyObject* s = dev != nullptr ? PyObject_CallOneArg(stream_fn, dev) : nullptr;
  Py_XDECREF(dev);
  if (s == nullptr) throw Raised();
  void* p = PyLong_AsVoidPtr(s);
  Py_DECREF(s);
  if (p == nullptr && PyErr_Occurred()) throw Raised();
  return static_cast<mxq_stream_t>(p);
}

// a workspace that the caller may have given
at::Tensor workspace(const at::Tensor* given) {
  if (given == nullptr) return at::Tensor();
  // an expanded tensor counts bytes that it does not have
  if (!given->is_contiguous()) refuse(PyExc_ValueError, "workspace must be contiguous");
  return *given;
}

PyObject* result(const at::Tensor& out, const at::Tensor& lse) {
  PyObject* o = THPVariable_Wrap(out);
  if (!lse.defined() || o == nullptr) return o;
  PyObject* l = THPVariable_Wrap(lse);
  PyObject* r = l != nullptr ? PyTuple_Pack(2, o, l) : nullptr;
  Py_DECREF(o);
  Py_XDECREF(l);
  return r;
}

template <typename F>
PyObject* guarded(Py_ssize_t given, Py_ssize_t wanted, F f) {
  try {
    if (given != wanted) refuse(PyExc_TypeError, "wrong number of arguments");
    return f();
  } catch (const Raised&) {
  } catch (const std::exception&) {
    // torch's own, such as its out-of-memory error
    torch::translate_exception_to_python(std::current_exception());
  }
  return nullptr;
}

// (k, v, k_cache, v_cache, slots, cos_sin, positions, q, q_out, k_scale, v_scale,
// interleaved)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  return guarded(nargs, 12, [&]() -> PyObject* {
    const at::Tensor &k = needed("k", a[0]), &v = needed("v", a[1]);
    const at::Tensor &kc = needed("k_cache", a[2]), &vc = needed("v_cache", a[3]);
    const at::Tensor& slots = needed("slots", a[4]);
    const at::Tensor *cs = tensor("cos_sin", a[5]), *pos = tensor("positions", a[6]);
    const at::Tensor *q = tensor("q", a[7]), *q_out = tensor("q_out", a[8]);
    const at::Tensor *ks = tensor("k_scale", a[9]), *vs = tensor("v_scale", a[10]);
    same_device({&k, &v, &kc, &vc, &slots, cs, pos, q, q_out, ks, vs});
    if (k.sizes() != v.sizes()) refuse(PyExc_ValueError, "k and v must have the same shape");
    const Heads hk("k", k), hv("v", v);
    const int64_t T = hk.n, D = hk.D;
    const Caches c(kc, vc, hk.heads, D);
    const float* rotation = nullptr;
    const int32_t* at_pos = nullptr;
    int64_t max_pos = 0, rot = 0;
    if (cs != nullptr) {
      if (cs->dim() != 2 || cs->scalar_type() != at::kFloat || !cs->is_contiguous())
        refuse(PyExc_ValueError, "cos_sin must be contiguous fp32 [max_pos, R]");
      if (pos == nullptr) refuse(PyExc_ValueError, "a rotation needs positions");
      max_pos = cs->size(0), rot = cs->size(1);
      rotation = static_cast<const float*>(cs->data_ptr());
      at_pos = vec<const int32_t>("positions", pos, at::kInt, T);
    }
    at::Tensor out, q_copy;
    void *qp = nullptr, *op = nullptr;
    int64_t Hq = 0, q0 = 0, q1 = 0, o0 = 0, o1 = 0;
    if (q != nullptr) {
      if (q->dim() != 3 || q->size(0) != T || q->size(2) != D)
        refuse(PyExc_ValueError, "q must be [" + std::to_string(T) + ", heads, " +
                                     std::to_string(D) + "]");
      const Heads hq("q", *q);
      q_copy = hq.copy;
      Hq = hq.heads, qp = hq.p, q0 = hq.s0, q1 = hq.s1;
      out = output("q_out", q_out, q->sizes());
    } else if (q_out != nullptr) {
      refuse(PyExc_ValueError, "q_out without q");
    }
    const int32_t nq = narrow("heads", Hq), nkv = narrow("kv_heads", hk.heads);
    const int32_t d = narrow("head_dim", D), r = narrow("the rotation", rot);
    const int32_t interleaved = truth(a[11]);
    const int64_t* at_slot = vec<const int64_t>("slots", &slots, at::kLong, T);
    const float* k_scale = vec<const float>("k_scale", ks, at::kFloat, hk.heads);
    const float* v_scale = vec<const float>("v_scale", vs, at::kFloat, hk.heads);
    const mxq_stream_t stream = stream_of(k);
    check(unlocked([&] {
      if (q != nullptr) {
        if (!out.defined()) out = fresh(q->sizes(), at::kBFloat16, k);
        op = out.data_ptr(), o0 = out.stride(0), o1 = out.stride(1);
      }
      return append_fn(qp, q0, q1, nq, op, o0, o1, hk.p, hk.s0, hk.s1, hv.p, hv.s0, hv.s1, T, nkv,
                       d, rotation, max_pos, r, at_pos, interleaved, at_slot, c.k, c.v, c.dtype,
                       c.pages, c.page_size, c.k0, c.k1, c.k2, c.v0, c.v1, c.v2, k_scale, v_scale,
                       stream);
    }));
    if (q == nullptr) Py_RETURN_NONE;
    if (q_out != nullptr) return Py_NewRef(a[8]);
    return THPVariable_Wrap(out);
  });
}

// (q, k_cache, v_cache, page_table, seq_lens, scale, window, sinks, k_scale, v_scale,
// return_lse, out, workspace[, first])
PyObject* decode(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  return guarded(nargs, nargs == 14 ? 14 : 13, [&]() -> PyObject* {
    const int32_t first = nargs == 14 ? integer("first", a[13]) : 0;
    const at::Tensor &q = needed("q", a[0]), &kc = needed("k_cache", a[1]);
    const at::Tensor &vc = needed("v_cache", a[2]), &table = needed("page_table", a[3]);
    const at::Tensor& lens = needed("seq_lens", a[4]);
    const at::Tensor *sinks = tensor("sinks", a[7]), *ks = tensor("k_scale", a[8]);
    const at::Tensor *vs = tensor("v_scale", a[9]), *given = tensor("out", a[11]);
    const at::Tensor* ws = tensor("workspace", a[12]);
    same_device({&q, &kc, &vc, &table, &lens, sinks, ks, vs, given, ws});
    const Heads hq("q", q);
    const int64_t B = hq.n, D = hq.D;
    const Caches c(kc, vc, -1, D);
    const int32_t Hq = narrow("heads", hq.heads), Hkv = narrow("kv_heads", c.heads);
    if (table.dim() != 2 || table.scalar_type() != at::kInt || table.size(0) != B ||
        (table.size(1) > 1 && table.stride(1) != 1) ||
        (B > 1 && table.stride(0) < table.size(1)))
      refuse(PyExc_ValueError, "page_table must be int32 [" + std::to_string(B) +
                                   ", max_pages] with a unit inner stride");
    const int64_t width = table.size(1);
    at::Tensor out = output("out", given, q.sizes()), space = workspace(ws), lse;
    const bool with_lse = truth(a[10]) != 0;
    const int32_t d = narrow("head_dim", D), window = integer("window", a[6]);
    const int32_t* at_len = vec<const int32_t>("seq_lens", &lens, at::kInt, B);
    const float scale = scale_of(a[5], D);
    const float* sink = vec<const float>("sinks", sinks, at::kFloat, Hq);
    const float* k_scale = vec<const float>("k_scale", ks, at::kFloat, Hkv);
    const float* v_scale = vec<const float>("v_scale", vs, at::kFloat, Hkv);
    const mxq_stream_t stream = stream_of(q);
    check(unlocked([&] {
      if (!space.defined()) {
        size_t n = 0;
        const mxq_status st = decode_size_fn(B, Hq, Hkv, d, &n);
        if (st != MXQ_OK) return st;
        space = fresh({static_cast<int64_t>(n)}, at::kByte, q);
      }
      if (!out.defined()) out = fresh(q.sizes(), at::kBFloat16, q);
      if (with_lse) lse = fresh({B, hq.heads}, at::kFloat, q);
      const int32_t* pages = static_cast<const int32_t*>(table.data_ptr());
      const int64_t ld = B > 1 ? table.stride(0) : width;
      float* sums = with_lse ? static_cast<float*>(lse.data_ptr()) : nullptr;
      if (first != 0)
        return decode_ex_fn(hq.p, hq.s0, hq.s1, B, Hq, Hkv, d, c.k, c.v, c.dtype, c.pages,
                            c.page_size, c.k0, c.k1, c.k2, c.v0, c.v1, c.v2, pages, ld, width,
                            at_len, scale, window, first, sink, k_scale, v_scale, out.data_ptr(),
                            out.stride(0), out.stride(1), sums, space.data_ptr(), space.nbytes(),
                            stream);
      return decode_fn(hq.p, hq.s0, hq.s1, B, Hq, Hkv, d, c.k, c.v, c.dtype, c.pages, c.page_size,
                       c.k0, c.k1, c.k2, c.v0, c.v1, c.v2, pages, ld, width, at_len, scale, window,
                       sink, k_scale, v_scale, out.data_ptr(), out.stride(0), out.stride(1), sums,
                       space.data_ptr(), space.nbytes(), stream);
    }));
    return result(out, lse);
  });
}

// (q, k, v, cu_seqlens_q, cu_seqlens_k, scale, causal, window, sinks, return_lse, out,
// workspace[, first])
PyObject* prompt(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  return guarded(nargs, nargs == 13 ? 13 : 12, [&]() -> PyObject* {
    const int32_t first = nargs == 13 ? integer("first", a[12]) : 0;
    const at::Tensor &q = needed("q", a[0]), &k = needed("k", a[1]), &v = needed("v", a[2]);
    const at::Tensor& cu_q = needed("cu_seqlens_q", a[3]);
    const at::Tensor *cu_k = tensor("cu_seqlens_k", a[4]), *sinks = tensor("sinks", a[8]);
    const at::Tensor *given = tensor("out", a[10]), *ws = tensor("workspace", a[11]);
    same_device({&q, &k, &v, &cu_q, cu_k, sinks, given, ws});
    const Heads hq("q", q), hk("k", k), hv("v", v);
    if (hk.D != hq.D || v.sizes() != k.sizes())
      refuse(PyExc_ValueError,
             "k and v must be [tokens, kv_heads, " + std::to_string(hq.D) + "] alike");
    const int64_t B = cu_q.numel() - 1;
    const int32_t Hq = narrow("heads", hq.heads), Hkv = narrow("kv_heads", hk.heads);
    const int32_t D = narrow("head_dim", hq.D);
    const int32_t* cq = vec<const int32_t>("cu_seqlens_q", &cu_q, at::kInt, B + 1);
    const int32_t* ck =
        cu_k == nullptr ? cq : vec<const int32_t>("cu_seqlens_k", cu_k, at::kInt, B + 1);
    at::Tensor out = output("out", given, q.sizes()), space = workspace(ws), lse;
    const bool with_lse = truth(a[9]) != 0;
    const float scale = scale_of(a[5], D);
    const int32_t causal = truth(a[6]), window = integer("window", a[7]);
    const float* sink = vec<const float>("sinks", sinks, at::kFloat, Hq);
    const mxq_stream_t stream = stream_of(q);
    check(unlocked([&] {
      if (!space.defined()) {
        size_t n = 0;
        const mxq_status st = prompt_size_fn(hq.n, B, Hq, Hkv, D, &n);
        if (st != MXQ_OK) return st;
        space = fresh({static_cast<int64_t>(n)}, at::kByte, q);
      }
      if (!out.defined()) out = fresh(q.sizes(), at::kBFloat16, q);
      if (with_lse) lse = fresh({hq.n, hq.heads}, at::kFloat, q);
      float* sums = with_lse ? static_cast<float*>(lse.data_ptr()) : nullptr;
      if (first != 0)
        return prompt_ex_fn(hq.p, hq.s0, hq.s1, hk.p, hk.s0, hk.s1, hv.p, hv.s0, hv.s1, cq, ck, B,
                            hq.n, hk.n, Hq, Hkv, D, scale, causal, window, first, sink,
                            out.data_ptr(), out.stride(0), out.stride(1), sums, space.data_ptr(),
                            space.nbytes(), stream);
      return prompt_fn(hq.p, hq.s0, hq.s1, hk.p, hk.s0, hk.s1, hv.p, hv.s0, hv.s1, cq, ck, B, hq.n,
                       hk.n, Hq, Hkv, D, scale, causal, window, sink, out.data_ptr(),
                       out.stride(0), out.stride(1), sums, space.data_ptr(), space.nbytes(),
                       stream);
    }));
    return result(out, lse);
  });
}

// int32 [rows, width] with a unit inner stride
struct Table {
  int32_t* p;
  int64_t rows, width, ld;
  // rows < 0: any
  Table(const char* name, const at::Tensor& t, int64_t n) {
    if (t.dim() != 2 || t.scalar_type() != at::kInt || (n >= 0 && t.size(0) != n) ||
        (t.size(1) > 1 && t.stride(1) != 1) || (t.size(0) > 1 && t.stride(0) < t.size(1)))
      refuse(PyExc_ValueError, std::string(name) + " must be int32 [" +
                                   (n < 0 ? std::string("rows") : std::to_string(n)) +
                                   ", width] with a unit inner stride");
    rows = t.size(0), width = t.size(1), ld = rows > 1 ? t.stride(0) : width;
    p = static_cast<int32_t*>(t.data_ptr());
  }
};

// (q, k_cache, v_cache, page_table, seq_lens, cu_seqlens_q, parents, scale, window, first, sinks,
// k_scale, v_scale, return_lse, out, workspace)
PyObject* tree(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  return guarded(nargs, 16, [&]() -> PyObject* {
    const at::Tensor &q = needed("q", a[0]), &kc = needed("k_cache", a[1]);
    const at::Tensor &vc = needed("v_cache", a[2]), &table = needed("page_table", a[3]);
    const at::Tensor &lens = needed("seq_lens", a[4]), &cu = needed("cu_seqlens_q", a[5]);
    const at::Tensor *par = tensor("parents", a[6]), *sinks = tensor("sinks", a[10]);
    const at::Tensor *ks = tensor("k_scale", a[11]), *vs = tensor("v_scale", a[12]);
    const at::Tensor *given = tensor("out", a[14]), *ws = tensor("workspace", a[15]);
    same_device({&q, &kc, &vc, &table, &lens, &cu, par, sinks, ks, vs, given, ws});
    const Heads hq("q", q);
    const Caches c(kc, vc, -1, hq.D);
    const int64_t B = lens.numel();
    const Table t("page_table", table, B);
    const int32_t Hq = narrow("heads", hq.heads), Hkv = narrow("kv_heads", c.heads);
    const int32_t D = narrow("head_dim", hq.D);
    const int32_t* at_len = vec<const int32_t>("seq_lens", &lens, at::kInt, B);
    const int32_t* cq = vec<const int32_t>("cu_seqlens_q", &cu, at::kInt, B + 1);
    const int32_t* parents = vec<const int32_t>("parents", par, at::kInt, hq.n);
    const float scale = scale_of(a[7], hq.D);
    const int32_t window = integer("window", a[8]), first = integer("first", a[9]);
    const float* sink = vec<const float>("sinks", sinks, at::kFloat, Hq);
    const float* k_scale = vec<const float>("k_scale", ks, at::kFloat, Hkv);
    const float* v_scale = vec<const float>("v_scale", vs, at::kFloat, Hkv);
    at::Tensor out = output("out", given, q.sizes()), space = workspace(ws), lse;
    const bool with_lse = truth(a[13]) != 0;
    const mxq_stream_t stream = stream_of(q);
    check(unlocked([&] {
      if (!space.defined()) {
        size_t n = 0;
        const mxq_status st = tree_size_fn(hq.n, B, Hq, Hkv, D, &n);
        if (st != MXQ_OK) return st;
        space = fresh({static_cast<int64_t>(n)}, at::kByte, q);
      }
      if (!out.defined()) out = fresh(q.sizes(), at::kBFloat16, q);
      if (with_lse) lse = fresh({hq.n, hq.heads}, at::kFloat, q);
      return tree_fn(hq.p, hq.s0, hq.s1, hq.n, Hq, Hkv, D, c.k, c.v, c.dtype, c.pages, c.page_size,
                     c.k0, c.k1, c.k2, c.v0, c.v1, c.v2, t.p, t.ld, t.width, at_len, cq, parents,
                     B, scale, window, first, sink, k_scale, v_scale, out.data_ptr(),
                     out.stride(0), out.stride(1),
                     with_lse ? static_cast<float*>(lse.data_ptr()) : nullptr, space.data_ptr(),
                     space.nbytes(), stream);
    }));
    return result(out, lse);
  });
}

// (page_table, seq_lens, new_lens, page_refs, page_size, window, first, workspace)
PyObject* resize(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  return guarded(nargs, 8, [&]() -> PyObject* {
    const at::Tensor &table = needed("page_table", a[0]), &lens = needed("seq_lens", a[1]);
    const at::Tensor &to = needed("new_lens", a[2]), &refs = needed("page_refs", a[3]);
    const at::Tensor* ws = tensor("workspace", a[7]);
    same_device({&table, &lens, &to, &refs, ws});
    const Table t("page_table", table, -1);
    const int32_t* l = vec<const int32_t>("seq_lens", &lens, at::kInt, t.rows);
    const int32_t* n = vec<const int32_t>("new_lens", &to, at::kInt, t.rows);
    int32_t* r = vec<int32_t>("page_refs", &refs, at::kInt, refs.numel());
    const int32_t size = integer("page_size", a[4]), window = integer("window", a[5]);
    const int32_t first = integer("first", a[6]);
    at::Tensor space = workspace(ws);
    const mxq_stream_t stream = stream_of(table);
    check(unlocked([&] {
      if (!space.defined()) {
        size_t bytes = 0;
        const mxq_status st = pages_size_fn(t.rows, refs.numel(), &bytes);
        if (st != MXQ_OK) return st;
        space = fresh({static_cast<int64_t>(bytes)}, at::kByte, table);
      }
      return resize_fn(t.p, t.ld, t.rows, t.width, l, n, r, refs.numel(), size, window, first,
                       space.data_ptr(), space.nbytes(), stream);
    }));
    return Py_NewRef(a[0]);
  });
}

// (page_table, seq_lens, page_refs, parents, page_size, out, workspace)
PyObject* fork_rows(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  return guarded(nargs, 7, [&]() -> PyObject* {
    const at::Tensor &table = needed("page_table", a[0]), &lens = needed("seq_lens", a[1]);
    const at::Tensor &refs = needed("page_refs", a[2]), &parents = needed("parents", a[3]);
    const at::Tensor *given = tensor("out", a[5]), *ws = tensor("workspace", a[6]);
    same_device({&table, &lens, &refs, &parents, given, ws});
    const Table t("page_table", table, -1);
    const int64_t n = parents.numel();
    const int32_t* l = vec<const int32_t>("seq_lens", &lens, at::kInt, t.rows);
    int32_t* r = vec<int32_t>("page_refs", &refs, at::kInt, refs.numel());
    const int32_t* from = vec<const int32_t>("parents", &parents, at::kInt, n);
    const int32_t size = integer("page_size", a[4]);
    at::Tensor out, space = workspace(ws), new_lens, copies;
    if (given != nullptr) {
      const Table o("out", *given, n);
      if (o.width != t.width)
        refuse(PyExc_ValueError, "out must be as wide as page_table, " + std::to_string(t.width));
      out = *given;
    }
    const mxq_stream_t stream = stream_of(table);
    check(unlocked([&] {
      if (!space.defined()) {
        size_t bytes = 0;
        const mxq_status st = pages_size_fn(std::max(t.rows, n), refs.numel(), &bytes);
        if (st != MXQ_OK) return st;
        space = fresh({static_cast<int64_t>(bytes)}, at::kByte, table);
      }
      if (!out.defined()) out = fresh({n, t.width}, at::kInt, table);
      new_lens = fresh({n}, at::kInt, table);
      copies = fresh({n, 3}, at::kInt, table);
      return fork_fn(t.p, t.ld, t.rows, t.width, l, r, refs.numel(), size, from, n,
                     static_cast<int32_t*>(out.data_ptr()), n > 1 ? out.stride(0) : t.width,
                     static_cast<int32_t*>(new_lens.data_ptr()),
                     static_cast<int32_t*>(copies.data_ptr()), space.data_ptr(), space.nbytes(),
                     stream);
    }));
    PyObject* parts[3] = {given != nullptr ? Py_NewRef(a[5]) : THPVariable_Wrap(out),
                          THPVariable_Wrap(new_lens), THPVariable_Wrap(copies)};
    PyObject* all = parts[0] && parts[1] && parts[2]
                        ? PyTuple_Pack(3, parts[0], parts[1], parts[2]) : nullptr;
    for (PyObject* o : parts) Py_XDECREF(o);
    return all;
  });
}

// (k_cache, v_cache, copies)
PyObject* copy_pages(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  return guarded(nargs, 3, [&]() -> PyObject* {
    const at::Tensor &kc = needed("k_cache", a[0]), &vc = needed("v_cache", a[1]);
    const at::Tensor& copies = needed("copies", a[2]);
    same_device({&kc, &vc, &copies});
    const Caches c(kc, vc, -1, kc.dim() == 4 ? kc.size(3) : 0);
    if (copies.dim() != 2 || copies.size(1) != 3)
      refuse(PyExc_ValueError, "copies must be int32 [n, 3]: source page, destination, tokens");
    const int64_t n = copies.size(0);
    const int32_t* list = vec<const int32_t>("copies", &copies, at::kInt, 3 * n);
    const int32_t Hkv = narrow("kv_heads", c.heads), D = narrow("head_dim", kc.size(3));
    const mxq_stream_t stream = stream_of(kc);
    check(unlocked([&] {
      return copy_pages_fn(c.k, c.v, c.dtype, c.pages, c.page_size, Hkv, D, c.k0, c.k1, c.k2,
                           c.v0, c.v1, c.v2, list, n, stream);
    }));
    Py_RETURN_NONE;
  });
}

// (k_cache, v_cache, page_table, starts, kept, counts)
PyObject* compact(PyObject*, PyObject* const* a, Py_ssize_t nargs) {
  return guarded(nargs, 6, [&]() -> PyObject* {
    const at::Tensor &kc = needed("k_cache", a[0]), &vc = needed("v_cache", a[1]);
    const at::Tensor &table = needed("page_table", a[2]), &starts = needed("starts", a[3]);
    const at::Tensor &kept = needed("kept", a[4]), &counts = needed("counts", a[5]);
    same_device({&kc, &vc, &table, &starts, &kept, &counts});
    const Caches c(kc, vc, -1, kc.dim() == 4 ? kc.size(3) : 0);
    const Table t("page_table", table, -1), list("kept", kept, t.rows);
    const int32_t* s = vec<const int32_t>("starts", &starts, at::kInt, t.rows);
    const int32_t* n = vec<const int32_t>("counts", &counts, at::kInt, t.rows);
    const int32_t Hkv = narrow("kv_heads", c.heads), D = narrow("head_dim", kc.size(3));
    const mxq_stream_t stream = stream_of(kc);
    check(unlocked([&] {
      return compact_fn(c.k, c.v, c.dtype, c.pages, c.page_size, Hkv, D, c.k0, c.k1, c.k2, c.v0,
                        c.v1, c.v2, t.p, t.ld, t.rows, t.width, s, list.p, list.ld, list.width, n,
                        stream);
    }));
    Py_RETURN_NONE;
  });
}

// ({name: address}) of the further entry points: once, before their calls
PyObject* connect_more(PyObject*, PyObject* by_name) {
  auto set = [&](const char* name, auto* fn) {
    PyObject* o = PyMapping_GetItemString(by_name, name);
    if (o == nullptr) return false;
    *fn = reinterpret_cast<std::remove_pointer_t<decltype(fn)>>(PyLong_AsVoidPtr(o));
    Py_DECREF(o);
    return !PyErr_Occurred();
  };
  if (!set("mxq_cache_pages_workspace_size", &pages_size_fn) ||
      !set("mxq_cache_resize", &resize_fn) || !set("mxq_cache_fork", &fork_fn) ||
      !set("mxq_paged_attention_decode_ex", &decode_ex_fn) ||
      !set("mxq_attention_varlen_ex", &prompt_ex_fn) ||
      !set("mxq_paged_attention_tree", &tree_fn) ||
      !set("mxq_paged_attention_tree_workspace_size", &tree_size_fn) ||
      !set("mxq_cache_copy_pages", &copy_pages_fn) || !set("mxq_cache_compact", &compact_fn))
    return nullptr;
  Py_RETURN_NONE;
}

// (addresses of the six entry points, check, stream): once, before any call
PyObject* connect(PyObject*, PyObject* args) {
  unsigned long long fn[6];
  PyObject *c, *s;
  if (!PyArg_ParseTuple(args, "KKKKKKOO", &fn[0], &fn[1], &fn[2], &fn[3], &fn[4], &fn[5], &c, &s))
    return nullptr;
  append_fn = reinterpret_cast<decltype(append_fn)>(fn[0]);
  decode_fn = reinterpret_cast<decltype(decode_fn)>(fn[1]);
  decode_size_fn = reinterpret_cast<decltype(decode_size_fn)>(fn[2]);
  prompt_fn = reinterpret_cast<decltype(prompt_fn)>(fn[3]);
  prompt_size_fn = reinterpret_cast<decltype(prompt_size_fn)>(fn[4]);
  device_fn = reinterpret_cast<decltype(device_fn)>(fn[5]);
  Py_XSETREF(check_fn, Py_NewRef(c));
  Py_XSETREF(stream_fn, Py_NewRef(s));
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"connect", connect, METH_VARARGS, nullptr},
    {"append", reinterpret_cast<PyCFunction>(append), METH_FASTCALL, nullptr},
    {"decode", reinterpret_cast<PyCFunction>(decode), METH_FASTCALL, nullptr},
    {"prompt", reinterpret_cast<PyCFunction>(prompt), METH_FASTCALL, nullptr},
    {"tree", reinterpret_cast<PyCFunction>(tree), METH_FASTCALL, nullptr},
    {"resize", reinterpret_cast<PyCFunction>(resize), METH_FASTCALL, nullptr},
    {"fork", reinterpret_cast<PyCFunction>(fork_rows), METH_FASTCALL, nullptr},
    {"copy_pages", reinterpret_cast<PyCFunction>(copy_pages), METH_FASTCALL, nullptr},
    {"compact", reinterpret_cast<PyCFunction>(compact), METH_FASTCALL, nullptr},
    {"connect_more", connect_more, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_attn_calls", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__attn_calls() { return PyModule_Create(&module); }
