// Python binding of the paged-cache operators (module thinned_softmax_attention_b200._paged).
//
// A decode step's calls take a few microseconds on the GPU; reading a call's tensors' properties, checking
// them and allocating its outputs from Python takes several times that (attention of one token: 9 us of checks
// and allocations, 5 us of launches).  This module does what the rest of the binding does in Python, and
// nothing else: checks of arguments, output and workspace tensors from torch's allocator, the current
// stream, one call of the C ABI.  The library's entry points are handed over once as addresses (bind), so
// that there is one place that finds the library.
//
// Functions return their tensors, or the status of the C call when it is not 0; wrong arguments raise
// ValueError.
#include <ATen/ATen.h>
#include <ATen/MemoryOverlap.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>
#include <vector>

#include "thin_attn.h"

namespace {

struct Functions {
  thin_attn_status (*plan)(const thin_attn_paged_plan_args*, void*);
  thin_attn_status (*release)(const thin_attn_paged_release_args*, void*);
  thin_attn_status (*append)(const thin_attn_paged_append_args*, void*);
  thin_attn_status (*workspace)(const thin_attn_paged_attention_args*, size_t*);
  thin_attn_status (*attention)(const thin_attn_paged_attention_args*, void*);
} fns = {};

struct Refused {};   // a Python error is set

[[noreturn]] void refuse(const std::string& what) {
  PyErr_SetString(PyExc_ValueError, what.c_str());
  throw Refused();
}
void need_args(Py_ssize_t got, Py_ssize_t want) {
  if (got != want) {
    PyErr_Format(PyExc_TypeError, "%zd arguments, %zd expected", got, want);
    throw Refused();
  }
  if (!fns.attention) {
    PyErr_SetString(PyExc_RuntimeError, "bind() has not been called");
    throw Refused();
  }
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(std::string(name) + ": expected a tensor, got " + Py_TYPE(o)->tp_name);
  return THPVariable_Unpack(o);
}
int64_t integer(PyObject* o) {
  const int64_t v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused();
  return v;
}
// An argument of the C ABI's int fields.
int int32_of(PyObject* o, const char* name) {
  const int64_t v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX) refuse(std::string(name) + "=" + std::to_string(v) + ": outside 32 bits");
  return (int)v;
}
int fits(int64_t v, const char* name) {
  if (v > INT32_MAX) refuse(std::string(name) + "=" + std::to_string(v) + ": too large");
  return (int)v;
}
bool flag(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Refused();
  return v != 0;
}

bool overlapping(const at::Tensor& x, const at::Tensor& y) {
  const at::MemOverlapStatus s = at::get_overlap_status(x, y);
  return s == at::MemOverlapStatus::Full || s == at::MemOverlapStatus::Partial;
}
// A stride that is used: that of an axis of one may be any number.
int64_t stride_of(const at::Tensor& t, int axis) { return t.size(axis) > 1 ? t.stride(axis) : 0; }

std::string place(const at::Tensor& t) {
  std::string s = std::string(c10::toString(t.scalar_type())) + " (";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + ") on " + t.device().str();
}

// The CUDA device that holds t.
int device_of(const at::Tensor& t, const char* name) {
  if (!t.is_cuda()) refuse(std::string(name) + ": expected a CUDA tensor, got one on " + t.device().str());
  return t.get_device();
}
bool on(const at::Tensor& t, int dev) { return t.is_cuda() && t.get_device() == dev; }

template <typename T>
T* vector(const at::Tensor& t, const char* name, int64_t n, at::ScalarType type, int dev) {
  if (t.scalar_type() != type || !on(t, dev) || t.dim() != 1 || t.size(0) != n || !t.is_contiguous())
    refuse(std::string(name) + ": expected contiguous " + c10::toString(type) + " (" + std::to_string(n) + ") on cuda:" +
           std::to_string(dev) + ", got " + place(t));
  return (T*)t.data_ptr();
}

struct Table {
  int32_t* ids;
  int R, W;
  int64_t row;
};
Table table_of(const at::Tensor& t, int dev) {
  if (t.scalar_type() != at::kInt || !on(t, dev) || t.dim() != 2 || (t.size(1) > 1 && t.stride(1) != 1))
    refuse("table: expected int32 (R, W) with contiguous rows on cuda:" + std::to_string(dev) + ", got " + place(t));
  return {(int32_t*)t.data_ptr(), fits(t.size(0), "R"), fits(t.size(1), "W"), t.stride(0)};
}

struct Pool {
  int n_pages, H, page, E, D;
};
Pool pool_of(const at::Tensor& k, const at::Tensor& v, int dev) {
  if (k.dim() != 4 || v.dim() != 4 || k.size(0) != v.size(0) || k.size(1) != v.size(1) || k.size(2) != v.size(2) ||
      k.scalar_type() != v.scalar_type() || !on(k, dev) || !on(v, dev) || k.stride(3) != 1 || v.stride(3) != 1)
    refuse("k_pages (n_pages, H, page, E) and v_pages (n_pages, H, page, D): expected one type on cuda:" + std::to_string(dev) +
           " and a contiguous last axis, got " + place(k) + " and " + place(v));
  return {fits(k.size(0), "n_pages"), fits(k.size(1), "H"), fits(k.size(2), "page"), fits(k.size(3), "E"), fits(v.size(3), "D")};
}

int type_of(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return THIN_ATTN_FP32;
    case at::kBFloat16: return THIN_ATTN_BF16;
    case at::kHalf: return THIN_ATTN_FP16;
    case at::kFloat8_e4m3fn: return THIN_ATTN_E4M3;
    default: return -1;
  }
}
struct Types {
  int own, cache;
};
Types types_of(const at::Tensor& x, const at::Tensor& pages) {
  const Types t = {type_of(x.scalar_type()), type_of(pages.scalar_type())};
  if (t.own < 0 || t.own == THIN_ATTN_E4M3)
    refuse(std::string("dtype ") + c10::toString(x.scalar_type()) + ": expected float32, bfloat16 or float16");
  if (t.cache != t.own && (t.cache != THIN_ATTN_E4M3 || t.own == THIN_ATTN_FP32))
    refuse(std::string("pages of ") + c10::toString(pages.scalar_type()) + " with " + c10::toString(x.scalar_type()) +
           ": expected the same type, or float8_e4m3fn with bfloat16 or float16");
  return t;
}

// The operators have no gradients: a tensor that is to get one is refused, its gradient not dropped.
void no_gradient(std::initializer_list<const at::Tensor*> ts) {
  if (!c10::GradMode::is_enabled()) return;
  for (const at::Tensor* t : ts)
    if (t->requires_grad()) refuse("a tensor requires a gradient, and the paged operators have none: call them under torch.no_grad()");
}

struct Scales {
  const float *k, *v;
};
Scales scales_of(PyObject* k, PyObject* v, int cache, int H, int dev) {
  if (cache != THIN_ATTN_E4M3) {
    if (k != Py_None || v != Py_None) refuse("k_scale and v_scale belong to float8_e4m3fn pages");
    return {nullptr, nullptr};
  }
  if (k == Py_None || v == Py_None) refuse("float8_e4m3fn pages need k_scale and v_scale");
  no_gradient({&tensor(k, "k_scale"), &tensor(v, "v_scale")});
  return {vector<float>(tensor(k, "k_scale"), "k_scale", H, at::kFloat, dev), vector<float>(tensor(v, "v_scale"), "v_scale", H, at::kFloat, dev)};
}

struct Bounds {
  int8_t *lohi, *exps;
};
Bounds bounds_of(PyObject* lohi, PyObject* exps, const Pool& p, int dev) {
  if (lohi == Py_None && exps == Py_None) return {nullptr, nullptr};
  const at::Tensor &b = tensor(lohi, "bounds[0]"), &x = tensor(exps, "bounds[1]");
  if (b.scalar_type() != at::kChar || !on(b, dev) || !b.sizes().equals({p.n_pages, p.H, 2, p.E}) || !b.is_contiguous())
    refuse("bounds[0]: expected contiguous int8 (n_pages, H, 2, E) of the pool on cuda:" + std::to_string(dev) + ", got " + place(b));
  if (x.scalar_type() != at::kChar || !on(x, dev) || !x.sizes().equals({p.n_pages, p.H}) || !x.is_contiguous())
    refuse("bounds[1]: expected contiguous int8 (n_pages, H) of the pool on cuda:" + std::to_string(dev) + ", got " + place(x));
  return {(int8_t*)b.data_ptr(), (int8_t*)x.data_ptr()};
}

template <typename F, typename A>
thin_attn_status launch(F f, const A& a, int dev) {
  void* stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
  thin_attn_status s;
  Py_BEGIN_ALLOW_THREADS
  s = f(&a, stream);
  Py_END_ALLOW_THREADS
  return s;
}

template <typename F>
PyObject* guarded(F&& f) {
  HANDLE_TH_ERRORS
  try {
    // no tensor here takes part in autograd
    at::AutoDispatchBelowADInplaceOrView below;
    return f();
  } catch (const Refused&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    if (n != 5) refuse("bind takes five addresses");
    void* p[5];
    for (int i = 0; i < 5; ++i) p[i] = (void*)integer(a[i]);
    fns = {(decltype(fns.plan))p[0], (decltype(fns.release))p[1], (decltype(fns.append))p[2], (decltype(fns.workspace))p[3],
           (decltype(fns.attention))p[4]};
    Py_RETURN_NONE;
  });
}

PyObject* tuple_of(std::initializer_list<at::Tensor> ts) {
  PyObject* t = PyTuple_New((Py_ssize_t)ts.size());
  if (!t) return nullptr;
  Py_ssize_t i = 0;
  for (const at::Tensor& x : ts) {
    PyObject* o = x.defined() ? THPVariable_Wrap(x) : Py_NewRef(Py_None);
    if (!o) {
      Py_DECREF(t);
      return nullptr;
    }
    PyTuple_SET_ITEM(t, i++, o);
  }
  return t;
}

// plan(lengths, new, table, free, n_free, page, max_tokens, inplace)
PyObject* plan(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    need_args(n, 8);
    const at::Tensor &lengths = tensor(a[0], "lengths"), &fresh = tensor(a[1], "new"), &free = tensor(a[3], "free"), &n_free = tensor(a[4], "n_free");
    const int dev = device_of(lengths, "lengths");
    const int R = fits(lengths.numel(), "requests");
    thin_attn_paged_plan_args p{};
    p.struct_size = sizeof p;
    p.device = dev;
    p.R = R;
    p.lengths = vector<int32_t>(lengths, "lengths", R, at::kInt, dev);
    p.n_new = vector<int32_t>(fresh, "new", R, at::kInt, dev);
    const Table t = table_of(tensor(a[2], "table"), dev);
    p.table = t.ids;
    p.W = t.W;
    p.table_row = t.row;
    p.n_pages = fits(free.numel(), "free");
    p.free_pages = vector<int32_t>(free, "free", p.n_pages, at::kInt, dev);
    p.n_free = vector<int32_t>(n_free, "n_free", 1, at::kInt, dev);
    p.page = int32_of(a[5], "page");
    p.max_tokens = int32_of(a[6], "max_tokens");
    const bool inplace = flag(a[7]);
    if (t.R != R || p.page < 1 || p.max_tokens < 0)
      refuse("table of " + std::to_string(t.R) + " rows, " + std::to_string(R) + " requests, page=" + std::to_string(p.page) + ", max_tokens=" +
             std::to_string(p.max_tokens) + ": expected a row per request, page >= 1, max_tokens >= 0");
    const int64_t T = p.max_tokens;
    // two allocations, the int32 outputs being parts of one (7.2 us a call; with all in one storage of two types, which
    // torch.save refuses, 5.9)
    const at::Tensor slots = at::empty({T}, lengths.options().dtype(at::kLong));
    std::vector<int64_t> sizes = {T, T, R + 1, R};
    if (!inplace) sizes.insert(sizes.end(), {R, 1});
    const std::vector<at::Tensor> part =
        at::empty({2 * T + 2 * R + 1 + (inplace ? 0 : R + 1)}, lengths.options()).split_with_sizes(sizes);
    const at::Tensor& lengths_out = inplace ? lengths : part[4];
    const at::Tensor& n_free_out = inplace ? n_free : part[5];
    p.slots = (int64_t*)slots.data_ptr();
    p.rows = (int32_t*)part[0].data_ptr();
    p.context = (int32_t*)part[1].data_ptr();
    p.cu = (int32_t*)part[2].data_ptr();
    p.status = (int32_t*)part[3].data_ptr();
    p.lengths_out = (int32_t*)lengths_out.data_ptr();
    p.n_free_out = (int32_t*)n_free_out.data_ptr();
    const thin_attn_status s = launch(fns.plan, p, dev);
    if (s != THIN_ATTN_OK) return PyLong_FromLong(s);
    return tuple_of({lengths_out, n_free_out, part[2], slots, part[0], part[1], part[3]});
  });
}

// release(keep, lengths, table, free, n_free, page)
PyObject* release(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    need_args(n, 6);
    const at::Tensor &lengths = tensor(a[1], "lengths"), &free = tensor(a[3], "free");
    const int dev = device_of(lengths, "lengths");
    thin_attn_paged_release_args p{};
    p.struct_size = sizeof p;
    p.device = dev;
    p.R = fits(lengths.numel(), "requests");
    p.keep = vector<int32_t>(tensor(a[0], "keep"), "keep", p.R, at::kInt, dev);
    p.lengths = vector<int32_t>(lengths, "lengths", p.R, at::kInt, dev);
    const Table t = table_of(tensor(a[2], "table"), dev);
    p.table = t.ids;
    p.W = t.W;
    p.table_row = t.row;
    p.n_pages = fits(free.numel(), "free");
    p.free_pages = vector<int32_t>(free, "free", p.n_pages, at::kInt, dev);
    p.n_free = vector<int32_t>(tensor(a[4], "n_free"), "n_free", 1, at::kInt, dev);
    p.page = int32_of(a[5], "page");
    if (t.R != p.R || p.page < 1)
      refuse("table of " + std::to_string(t.R) + " rows, " + std::to_string(p.R) + " requests, page=" + std::to_string(p.page) +
             ": expected a row per request, page >= 1");
    return PyLong_FromLong(launch(fns.release, p, dev));
  });
}

// append(k, v, slots, k_pages, v_pages, k_scale, v_scale, bounds, exps)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    need_args(n, 9);
    const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v"), &kp = tensor(a[3], "k_pages"), &vp = tensor(a[4], "v_pages");
    no_gradient({&k, &v, &kp, &vp});
    const int dev = device_of(k, "k");
    const Pool pool = pool_of(kp, vp, dev);
    const int64_t N = k.dim() ? k.size(0) : -1;
    if (!k.sizes().equals({N, pool.H, pool.E}) || !v.sizes().equals({N, pool.H, pool.D}) || k.scalar_type() != v.scalar_type() || !on(v, dev) ||
        k.stride(2) != 1 || v.stride(2) != 1)
      refuse("k and v: expected (N, " + std::to_string(pool.H) + ", " + std::to_string(pool.E) + ") and (N, " + std::to_string(pool.H) + ", " +
             std::to_string(pool.D) + ") of one type on cuda:" + std::to_string(dev) + " with a contiguous last axis, got " + place(k) + " and " + place(v));
    thin_attn_paged_append_args p{};
    p.struct_size = sizeof p;
    p.device = dev;
    p.N = fits(N, "N");
    p.slots = vector<int64_t>(tensor(a[2], "slots"), "slots", N, at::kLong, dev);
    if (at::has_internal_overlap(kp) == at::MemOverlap::Yes || at::has_internal_overlap(vp) == at::MemOverlap::Yes || overlapping(kp, vp))
      refuse("k_pages, v_pages: their rows overlap");
    const Types t = types_of(k, kp);
    const Scales s = scales_of(a[5], a[6], t.cache, pool.H, dev);
    const Bounds b = bounds_of(a[7], a[8], pool, dev);
    p.dtype = t.own;
    p.cache_dtype = t.cache;
    p.H = pool.H;
    p.E = pool.E;
    p.D = pool.D;
    p.page = pool.page;
    p.n_pages = pool.n_pages;
    p.k = k.data_ptr();
    p.k_token = stride_of(k, 0);
    p.k_head = stride_of(k, 1);
    p.v = v.data_ptr();
    p.v_token = stride_of(v, 0);
    p.v_head = stride_of(v, 1);
    p.k_pages = kp.data_ptr();
    p.kp_page = stride_of(kp, 0);
    p.kp_head = stride_of(kp, 1);
    p.kp_row = stride_of(kp, 2);
    p.v_pages = vp.data_ptr();
    p.vp_page = stride_of(vp, 0);
    p.vp_head = stride_of(vp, 1);
    p.vp_row = stride_of(vp, 2);
    p.k_scale = s.k;
    p.v_scale = s.v;
    p.bounds = b.lohi;
    p.exps = b.exps;
    return PyLong_FromLong(launch(fns.append, p, dev));
  });
}

// attention(q, k_pages, v_pages, table, lengths, rows, scale, k_scale, v_scale, window, bounds, exps, top, first, last, out, lse,
//           return_lse, return_pages) -> (out, lse, pages), the last two None unless asked for
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    need_args(n, 19);
    const at::Tensor &q = tensor(a[0], "q"), &kp = tensor(a[1], "k_pages"), &vp = tensor(a[2], "v_pages");
    no_gradient({&q, &kp, &vp});
    const int dev = device_of(q, "q");
    const Pool pool = pool_of(kp, vp, dev);
    if (q.dim() != 3 || q.size(2) != pool.E || q.stride(2) != 1 || pool.H == 0 || q.size(1) == 0 || q.size(1) % pool.H)
      refuse("q: expected (N, Hq, " + std::to_string(pool.E) + ") with a contiguous last axis, Hq a multiple of " + std::to_string(pool.H) + ", got " +
             place(q));
    const int64_t N = q.size(0), Hq = q.size(1), D = pool.D;
    thin_attn_paged_attention_args p{};
    p.struct_size = sizeof p;
    p.device = dev;
    const Types t = types_of(q, kp);
    p.dtype = t.own;
    p.cache_dtype = t.cache;
    p.N = fits(N, "N");
    const Table tab = table_of(tensor(a[3], "table"), dev);
    p.table = tab.ids;
    p.R = tab.R;
    p.W = tab.W;
    p.table_row = tab.row;
    p.Hq = fits(Hq, "Hq");
    p.H = pool.H;
    p.E = pool.E;
    p.D = pool.D;
    p.page = pool.page;
    p.n_pages = pool.n_pages;
    p.lengths = vector<int32_t>(tensor(a[4], "lengths"), "lengths", N, at::kInt, dev);
    const bool padded = a[5] != Py_None;
    if (padded) p.rows = vector<int32_t>(tensor(a[5], "rows"), "rows", N, at::kInt, dev);
    if (a[6] != Py_None) {
      p.scale = (float)PyFloat_AsDouble(a[6]);
      if (PyErr_Occurred()) throw Refused();
      if (p.scale == 0.f) refuse("scale=0 (or a number that rounds to 0 in fp32): the C entry would take it for 1/sqrt(E)");
    }
    const Scales s = scales_of(a[7], a[8], t.cache, pool.H, dev);
    p.k_scale = s.k;
    p.v_scale = s.v;
    p.window = int32_of(a[9], "window");
    const Bounds b = bounds_of(a[10], a[11], pool, dev);
    p.bounds = b.lohi;
    p.exps = b.exps;
    p.top = int32_of(a[12], "top");
    p.first = int32_of(a[13], "first");
    p.last = int32_of(a[14], "last");
    p.q = q.data_ptr();
    p.q_token = stride_of(q, 0);
    p.q_head = stride_of(q, 1);
    p.k_pages = kp.data_ptr();
    p.kp_page = stride_of(kp, 0);
    p.kp_head = stride_of(kp, 1);
    p.kp_row = stride_of(kp, 2);
    p.v_pages = vp.data_ptr();
    p.vp_page = stride_of(vp, 0);
    p.vp_head = stride_of(vp, 1);
    p.vp_row = stride_of(vp, 2);
    size_t bytes = 0;
    thin_attn_status status = fns.workspace(&p, &bytes);   // the shapes' refusals, before anything is allocated
    if (status != THIN_ATTN_OK) return PyLong_FromLong(status);
    // rows of padding tokens are not written: zeros there (-1 for pages) where the buffer is made here
    at::Tensor out, lse, pages;
    if (a[15] == Py_None) {
      out = at::empty({N, Hq, D}, q.options());
      if (padded) out.zero_();
    } else {
      out = tensor(a[15], "out");
      no_gradient({&out});
      if (!out.sizes().equals({N, Hq, D}) || out.scalar_type() != q.scalar_type() || !on(out, dev) || out.stride(2) != 1)
        refuse("out: expected (" + std::to_string(N) + ", " + std::to_string(Hq) + ", " + std::to_string(D) +
               ") of q's type with a contiguous last axis on cuda:" + std::to_string(dev) + ", got " + place(out));
      const bool same = out.data_ptr() == q.data_ptr() && out.strides().equals(q.strides()) && pool.E == pool.D;
      if (at::has_internal_overlap(out) == at::MemOverlap::Yes || (!same && overlapping(out, q)))
        refuse("out: its rows overlap one another or those of q");
    }
    if (a[16] != Py_None) {
      lse = tensor(a[16], "lse");
      no_gradient({&lse});
      if (!lse.sizes().equals({N, Hq}) || lse.scalar_type() != at::kFloat || !on(lse, dev) || !lse.is_contiguous())
        refuse("lse: expected contiguous float32 (" + std::to_string(N) + ", " + std::to_string(Hq) + ") on cuda:" + std::to_string(dev) + ", got " + place(lse));
    } else if (flag(a[17])) {
      lse = at::empty({N, Hq}, q.options().dtype(at::kFloat));
      if (padded) lse.zero_();
    }
    if (flag(a[18])) {
      pages = at::empty({N, pool.H, p.top}, q.options().dtype(at::kInt));
      if (padded) pages.fill_(-1);
      p.pages_out = (int32_t*)pages.data_ptr();
    }
    // scratch of this call alone: the caching allocator hands it on in stream order, and a capture
    // gets its own from the graph's pool
    const at::Tensor ws = at::empty({(int64_t)bytes}, q.options().dtype(at::kByte));
    p.workspace = ws.data_ptr();
    p.workspace_bytes = bytes;
    p.out = out.data_ptr();
    p.out_token = stride_of(out, 0);
    p.out_head = stride_of(out, 1);
    p.lse = lse.defined() ? (float*)lse.data_ptr() : nullptr;
    status = launch(fns.attention, p, dev);
    if (status != THIN_ATTN_OK) return PyLong_FromLong(status);
    return tuple_of({out, lse, pages});
  });
}

PyMethodDef methods[] = {
    {"bind", (PyCFunction)(void (*)(void))bind, METH_FASTCALL, nullptr},
    {"plan", (PyCFunction)(void (*)(void))plan, METH_FASTCALL, nullptr},
    {"release", (PyCFunction)(void (*)(void))release, METH_FASTCALL, nullptr},
    {"append", (PyCFunction)(void (*)(void))append, METH_FASTCALL, nullptr},
    {"attention", (PyCFunction)(void (*)(void))attention, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_paged", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__paged() { return PyModule_Create(&module); }
