// The Python module `_torch`: the tensor calls of kv4.py, paged.py and pages.py on the C
// ABI of libmk.so.  Checks of the tensors, the output tensors, the current stream
// of the pool's device, and the call; every computation is libmk.so's.
//
// It is compiled against torch because of the time a call takes on the host: a
// decode step makes these calls for every layer, and the same checks and
// allocations made from Python over ctypes took 16 us for an attention call,
// 14 us for a load (a tensor that Python allocates after a launch costs 4 us).
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cmath>
#include <string>
#include <vector>

#include "mk.h"

namespace {

PyObject* mk_error = nullptr;  // _lib.MKError

// A Python exception is set; leaves the call.
struct Refused {};

[[noreturn]] void refuse(const std::string& what) {
  PyErr_SetString(PyExc_ValueError, what.c_str());
  throw Refused();
}

void check(int code) {
  if (code == MK_OK) return;
  if (PyObject* e = PyObject_CallFunction(mk_error, "is", code, mk_last_error())) {
    PyErr_SetObject(mk_error, e);
    Py_DECREF(e);
  }
  throw Refused();
}

const at::Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) refuse(std::string(what) + " must be a tensor");
  return THPVariable_Unpack(o);
}

int dtype_of(at::ScalarType t) { return t == at::kBFloat16 ? MK_BF16 : t == at::kFloat ? MK_F32 : -1; }

int32_t to_i32(int64_t n, const char* what) {
  if (n > INT_MAX) refuse(std::string(what) + " is too large");
  return (int32_t)n;
}

void* ints(PyObject* o, const char* what, int64_t n, c10::Device dev) {
  const at::Tensor& t = tensor(o, what);
  if (t.scalar_type() != at::kInt || t.device() != dev || t.dim() != 1 || t.size(0) != n || !t.is_contiguous())
    refuse(std::string(what) + " must be a contiguous int32 tensor [" + std::to_string(n) + "] on " + dev.str());
  return t.data_ptr();
}

// pool (n_kv_heads heads of head_dim), table, lengths, n_new, status as the C description.
mk_kv4_cache describe(const at::Tensor& pool, int64_t n_kv_heads, PyObject* table_, PyObject* lengths, PyObject* n_new,
                      PyObject* status, int64_t rows, int64_t head_dim) {
  const at::Tensor& table = tensor(table_, "table");
  if (table.scalar_type() != at::kInt || table.device() != pool.device() || table.dim() != 2 || !table.is_contiguous())
    refuse("table must be a contiguous int32 tensor [n_seqs, max_pages] on " + pool.device().str());
  mk_kv4_cache c;
  c.pool = pool.data_ptr();
  c.table = static_cast<const int32_t*>(table.data_ptr());
  c.lengths = static_cast<const int32_t*>(ints(lengths, "lengths", table.size(0), pool.device()));
  c.n_new = n_new == Py_None ? nullptr : static_cast<const int32_t*>(ints(n_new, "n_new", table.size(0), pool.device()));
  c.status = status == Py_None ? nullptr : static_cast<int32_t*>(ints(status, "status", 1, pool.device()));
  c.n_pages = to_i32(pool.size(0), "n_pages");
  c.n_kv_heads = to_i32(n_kv_heads, "n_kv_heads");
  c.head_dim = to_i32(head_dim, "head_dim");
  c.n_seqs = to_i32(table.size(0), "n_seqs");
  c.max_pages = to_i32(table.size(1), "max_pages");
  c.rows = to_i32(rows, "rows");
  return c;
}

// The 4-bit cache.
mk_kv4_cache cache_of(const at::Tensor& pool, PyObject* table, PyObject* lengths, PyObject* n_new, PyObject* status,
                      int64_t rows, int64_t head_dim) {
  if (!pool.is_cuda() || pool.scalar_type() != at::kByte || pool.dim() != 3 || !pool.is_contiguous())
    refuse("pool must be a contiguous uint8 CUDA tensor [n_pages, n_kv_heads, record]");
  if (pool.size(2) != 136 * head_dim)
    refuse("a record of " + std::to_string(pool.size(2)) + " bytes does not hold heads of " + std::to_string(head_dim));
  return describe(pool, pool.size(1), table, lengths, n_new, status, rows, head_dim);
}

// x [n_seqs, rows, heads, head_dim] of the wanted sizes and dtype on the device.
mk_kv4_rows rows_of(const at::Tensor& x, c10::IntArrayRef sizes, at::ScalarType type, c10::Device dev, const char* what) {
  if (x.sizes() != sizes || x.scalar_type() != type || x.device() != dev) {
    std::string s;
    for (int64_t n : sizes) s += (s.empty() ? "[" : ", ") + std::to_string(n);
    refuse(std::string(what) + " must be " + s + "] of " + c10::toString(type) + " on " + dev.str());
  }
  if (x.stride(3) != 1) refuse(std::string(what) + ": head_dim must be contiguous");
  // a dimension of size 1 may have any stride
  return {x.data_ptr(), x.size(0) > 1 ? x.stride(0) : 0, x.size(1) > 1 ? x.stride(1) : 0, x.size(2) > 1 ? x.stride(2) : 0};
}

const at::Tensor& heads(PyObject* o, const char* what) {
  const at::Tensor& t = tensor(o, what);
  if (t.dim() != 4 || dtype_of(t.scalar_type()) < 0)
    refuse(std::string(what) + " must be bfloat16 or float32 [n_seqs, rows, heads, head_dim]");
  return t;
}

// The calls record nothing for autograd: a tensor that would need it is refused
// rather than its gradient lost.
void no_gradient(const at::Tensor& t, const char* what) {
  if ((t.requires_grad() && c10::GradMode::is_enabled()) || t._fw_grad(0).defined())
    refuse(std::string(what) + " requires a gradient, which this call has none of (torch.no_grad() or detach())");
}

// Whether the spans of two tensors' elements meet.
bool overlap(const at::Tensor& x, const at::Tensor& y) {
  const at::Tensor* t[2] = {&x, &y};
  uintptr_t lo[2], hi[2];
  for (int i = 0; i < 2; ++i) {
    if (!t[i]->numel()) return false;
    int64_t last = 0;
    for (int64_t d = 0; d < t[i]->dim(); ++d) last += (t[i]->size(d) - 1) * t[i]->stride(d);
    lo[i] = reinterpret_cast<uintptr_t>(t[i]->data_ptr());
    hi[i] = lo[i] + (size_t)(last + 1) * t[i]->element_size();
  }
  return lo[0] < hi[1] && lo[1] < hi[0];
}

// The call's device made current, and its current stream there.
struct On {
  c10::cuda::OptionalCUDAGuard guard;
  void* stream;
  explicit On(c10::Device dev) : guard(dev), stream(c10::cuda::getCurrentCUDAStream(dev.index()).stream()) {}
};

// A tensor of the current stream's allocator (without the dispatcher's 0.3 us).
at::Tensor fresh(c10::IntArrayRef sizes, at::ScalarType type, c10::Device dev) {
  return at::Tensor(at::detail::empty_cuda(sizes, type, dev, std::nullopt));
}

#define MK_BEGIN     \
  HANDLE_TH_ERRORS { \
    try {
#define MK_END                  \
    } catch (const Refused&) {  \
      return nullptr;           \
    }                           \
  }                             \
  END_HANDLE_TH_ERRORS

void count(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) refuse("wrong number of arguments");
}

// (pool, table, lengths, k, v, n_new, status)
PyObject* py_store(PyObject*, PyObject* const* a, Py_ssize_t n) {
  MK_BEGIN
  count(n, 7);
  const at::Tensor &pool = tensor(a[0], "pool"), &k = heads(a[3], "k"), &v = heads(a[4], "v");
  no_gradient(k, "k");
  no_gradient(v, "v");
  const mk_kv4_cache c = cache_of(pool, a[1], a[2], a[5], a[6], k.size(1), k.size(3));
  const int64_t sizes[4] = {c.n_seqs, c.rows, c.n_kv_heads, c.head_dim};
  const mk_kv4_rows kr = rows_of(k, sizes, k.scalar_type(), pool.device(), "k");
  const mk_kv4_rows vr = rows_of(v, sizes, k.scalar_type(), pool.device(), "v");
  On on(pool.device());
  check(mk_kv4_store(&c, &kr, &vr, dtype_of(k.scalar_type()), on.stream));
  Py_RETURN_NONE;
  MK_END
}

// (pool, table, lengths, rows, n_new, is_bf16, status) -> (k, v)
PyObject* py_load(PyObject*, PyObject* const* a, Py_ssize_t n) {
  MK_BEGIN
  count(n, 7);
  const at::Tensor& pool = tensor(a[0], "pool");
  const long long rows = PyLong_AsLongLong(a[3]);
  if (rows == -1 && PyErr_Occurred()) return nullptr;
  if (rows < 0) refuse("rows must be >= 0");
  if (pool.dim() != 3) refuse("pool must be a contiguous uint8 CUDA tensor [n_pages, n_kv_heads, record]");
  const mk_kv4_cache c = cache_of(pool, a[1], a[2], a[4], a[6], rows, pool.size(2) / 136);
  const at::ScalarType type = a[5] == Py_True ? at::kBFloat16 : at::kFloat;
  const int64_t sizes[4] = {c.n_seqs, c.rows, c.n_kv_heads, c.head_dim};
  On on(pool.device());
  at::Tensor k = fresh(sizes, type, pool.device()), v = fresh(sizes, type, pool.device());
  const mk_kv4_rows kr = rows_of(k, sizes, type, pool.device(), "k"), vr = rows_of(v, sizes, type, pool.device(), "v");
  check(mk_kv4_load(&c, &kr, &vr, dtype_of(type), on.stream));
  return Py_BuildValue("(NN)", THPVariable_Wrap(std::move(k)), THPVariable_Wrap(std::move(v)));
  MK_END
}

// (q, pool, table, lengths, n_new, scale, out, return_lse, status) -> out or (out, lse)
PyObject* py_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  MK_BEGIN
  count(n, 9);
  const at::Tensor &q = heads(a[0], "q"), &pool = tensor(a[1], "pool");
  no_gradient(q, "q");
  if (a[6] != Py_None) no_gradient(tensor(a[6], "out"), "out");
  const mk_kv4_cache c = cache_of(pool, a[2], a[3], a[4], a[8], q.size(1), q.size(3));
  const int64_t sizes[4] = {c.n_seqs, c.rows, q.size(2), c.head_dim};
  const at::ScalarType type = q.scalar_type();
  const mk_kv4_rows qr = rows_of(q, sizes, type, pool.device(), "q");
  const int32_t n_heads = to_i32(q.size(2), "n_heads");
  double scale = 1.0 / std::sqrt((double)c.head_dim);
  if (a[5] != Py_None) {
    scale = PyFloat_AsDouble(a[5]);
    if (scale == -1.0 && PyErr_Occurred()) return nullptr;
  }
  On on(pool.device());
  at::Tensor out = a[6] == Py_None ? fresh(sizes, type, pool.device()) : tensor(a[6], "out");
  if (!out.is_contiguous()) refuse("out must be contiguous");
  if (a[6] != Py_None && overlap(q, out)) refuse("out must not overlap q");
  if (a[6] != Py_None && overlap(pool, out)) refuse("out must not overlap the pool");
  const mk_kv4_rows outr = rows_of(out, sizes, type, pool.device(), "out");
  const bool want_lse = a[7] == Py_True;
  at::Tensor lse;
  if (want_lse) lse = fresh(c10::IntArrayRef(sizes, 3), at::kFloat, pool.device());
  // The workspace is taken anew for each call from the stream's allocator and
  // given back once the call is enqueued (the stream orders its next use), so
  // that calls on two streams, or two captured graphs, never share one.
  const int dt = dtype_of(type);
  const size_t nws = mk_kv4_attention_bytes(&c, n_heads, dt);
  at::Tensor ws;
  if (nws) ws = fresh({(int64_t)nws}, at::kByte, pool.device());
  check(mk_kv4_attention(&c, n_heads, &qr, dt, (float)scale, &outr, want_lse ? static_cast<float*>(lse.data_ptr()) : nullptr,
                         nws ? ws.data_ptr() : nullptr, nws, on.stream));
  if (!want_lse) {
    if (a[6] != Py_None) {
      Py_INCREF(a[6]);
      return a[6];
    }
    return THPVariable_Wrap(std::move(out));
  }
  PyObject* o = a[6];
  if (o != Py_None) Py_INCREF(o);
  else o = THPVariable_Wrap(std::move(out));
  return Py_BuildValue("(NN)", o, THPVariable_Wrap(std::move(lse)));
  MK_END
}

std::vector<int32_t> page_list(PyObject* o, const char* what) {
  PyObject* f = PySequence_Fast(o, (std::string(what) + " must be a list of page indices").c_str());
  if (!f) throw Refused();
  std::vector<int32_t> out((size_t)PySequence_Fast_GET_SIZE(f));
  for (size_t i = 0; i < out.size(); ++i) {
    const Py_ssize_t v = PyNumber_AsSsize_t(PySequence_Fast_GET_ITEM(f, (Py_ssize_t)i), nullptr);  // held to its range
    if (v == -1 && PyErr_Occurred()) {
      Py_DECREF(f);
      throw Refused();
    }
    out[i] = v < INT_MIN || v > INT_MAX ? -1 : (int32_t)v;  // the library refuses -1
  }
  Py_DECREF(f);
  return out;
}

// (pool, src, dst)
PyObject* py_page_copy(PyObject*, PyObject* const* a, Py_ssize_t n) {
  MK_BEGIN
  count(n, 3);
  const at::Tensor& pool = tensor(a[0], "pool");
  no_gradient(pool, "pool");
  if (!pool.is_cuda() || pool.dim() < 3 || !pool.is_contiguous())
    refuse("pool must be a contiguous CUDA tensor [n_layers, n_pages, ...]");
  if (pool.size(0) == 0 || pool.size(1) == 0) refuse("pool has no page");
  const std::vector<int32_t> src = page_list(a[1], "src"), dst = page_list(a[2], "dst");
  if (src.size() != dst.size()) refuse("src and dst must have the same length");
  On on(pool.device());
  check(mk_page_copy(pool.data_ptr(), to_i32(pool.size(0), "n_layers"), to_i32(pool.size(1), "n_pages"),
                     (size_t)(pool.numel() / (pool.size(0) * pool.size(1))) * pool.element_size(), src.data(), dst.data(),
                     to_i32((int64_t)src.size(), "the list"), on.stream));
  Py_RETURN_NONE;
  MK_END
}

// The 16-bit cache.
mk_paged_cache paged_of(const at::Tensor& pool, PyObject* table, PyObject* lengths, PyObject* n_new, PyObject* status,
                        int64_t rows) {
  if (!pool.is_cuda() || pool.scalar_type() != at::kBFloat16 || pool.dim() != 5 || pool.size(1) != 2 || pool.size(3) != 128 ||
      !pool.is_contiguous())
    refuse("pool must be a contiguous bfloat16 CUDA tensor [n_pages, 2, n_kv_heads, 128, head_dim]");
  no_gradient(pool, "pool");
  return describe(pool, pool.size(2), table, lengths, n_new, status, rows, pool.size(4));
}

mk_paged_mass mass_of(PyObject* o, const mk_paged_cache& c, c10::Device dev, double decay, const char* what) {
  const at::Tensor& m = tensor(o, what);
  no_gradient(m, what);
  if (m.scalar_type() != at::kFloat || m.device() != dev || m.dim() != 3 || m.size(0) != c.n_seqs || m.size(1) != c.n_kv_heads ||
      m.size(2) != (int64_t)c.max_pages * 128 || (m.size(2) > 1 && m.stride(2) != 1))
    refuse(std::string(what) + " must be a float32 tensor [" + std::to_string(c.n_seqs) + ", " + std::to_string(c.n_kv_heads) + ", " +
           std::to_string((int64_t)c.max_pages * 128) + "] on " + dev.str() + ", positions contiguous");
  return {static_cast<float*>(m.data_ptr()), m.size(0) > 1 ? m.stride(0) : 0, m.size(1) > 1 ? m.stride(1) : 0, (float)decay};
}

// (pool, table, lengths, k, v, n_new, status)
PyObject* py_paged_store(PyObject*, PyObject* const* a, Py_ssize_t n) {
  MK_BEGIN
  count(n, 7);
  const at::Tensor &pool = tensor(a[0], "pool"), &k = heads(a[3], "k"), &v = heads(a[4], "v");
  no_gradient(k, "k");
  no_gradient(v, "v");
  const mk_paged_cache c = paged_of(pool, a[1], a[2], a[5], a[6], k.size(1));
  const int64_t sizes[4] = {c.n_seqs, c.rows, c.n_kv_heads, c.head_dim};
  const mk_paged_rows kr = rows_of(k, sizes, k.scalar_type(), pool.device(), "k");
  const mk_paged_rows vr = rows_of(v, sizes, k.scalar_type(), pool.device(), "v");
  if (overlap(pool, k) || overlap(pool, v)) refuse("k and v must not overlap the pool");
  On on(pool.device());
  check(mk_paged_store(&c, &kr, &vr, dtype_of(k.scalar_type()), on.stream));
  Py_RETURN_NONE;
  MK_END
}

// (q, pool, table, lengths, n_new, scale, out, return_lse, mass, decay, status) -> out or (out, lse)
PyObject* py_paged_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  MK_BEGIN
  count(n, 11);
  const at::Tensor &q = heads(a[0], "q"), &pool = tensor(a[1], "pool");
  no_gradient(q, "q");
  if (a[6] != Py_None) no_gradient(tensor(a[6], "out"), "out");
  const mk_paged_cache c = paged_of(pool, a[2], a[3], a[4], a[10], q.size(1));
  const int64_t sizes[4] = {c.n_seqs, c.rows, q.size(2), c.head_dim};
  const at::ScalarType type = q.scalar_type();
  const mk_paged_rows qr = rows_of(q, sizes, type, pool.device(), "q");
  const int32_t n_heads = to_i32(q.size(2), "n_heads");
  double scale = 1.0 / std::sqrt((double)c.head_dim);
  if (a[5] != Py_None) {
    scale = PyFloat_AsDouble(a[5]);
    if (scale == -1.0 && PyErr_Occurred()) return nullptr;
  }
  const double decay = PyFloat_AsDouble(a[9]);
  if (decay == -1.0 && PyErr_Occurred()) return nullptr;
  mk_paged_mass mass;
  const bool weigh = a[8] != Py_None;
  if (weigh) {
    mass = mass_of(a[8], c, pool.device(), decay, "mass");
    const at::Tensor& m = tensor(a[8], "mass");
    if (overlap(q, m) || overlap(pool, m)) refuse("mass must not overlap q or the pool");
  }
  On on(pool.device());
  at::Tensor out = a[6] == Py_None ? fresh(sizes, type, pool.device()) : tensor(a[6], "out");
  if (!out.is_contiguous()) refuse("out must be contiguous");
  if (a[6] != Py_None) {
    if (overlap(q, out)) refuse("out must not overlap q");
    if (overlap(pool, out)) refuse("out must not overlap the pool");
    if (weigh && overlap(tensor(a[8], "mass"), out)) refuse("out must not overlap mass");
  }
  const mk_paged_rows outr = rows_of(out, sizes, type, pool.device(), "out");
  const bool want_lse = a[7] == Py_True;
  at::Tensor lse;
  if (want_lse) lse = fresh(c10::IntArrayRef(sizes, 3), at::kFloat, pool.device());
  // (as for the 4-bit cache: a workspace of the stream's allocator for each call)
  const int dt = dtype_of(type);
  const size_t nws = mk_paged_attention_bytes(&c, n_heads, dt, weigh);
  at::Tensor ws;
  if (nws) ws = fresh({(int64_t)nws}, at::kByte, pool.device());
  check(mk_paged_attention(&c, n_heads, &qr, dt, (float)scale, &outr, want_lse ? static_cast<float*>(lse.data_ptr()) : nullptr,
                           weigh ? &mass : nullptr, nws ? ws.data_ptr() : nullptr, nws, on.stream));
  PyObject* o = a[6];
  if (o != Py_None) Py_INCREF(o);
  else o = THPVariable_Wrap(std::move(out));
  return want_lse ? Py_BuildValue("(NN)", o, THPVariable_Wrap(std::move(lse))) : o;
  MK_END
}

int32_t whole(PyObject* o, const char* what) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused();
  if (v < INT_MIN || v > INT_MAX) refuse(std::string(what) + " is out of range");
  return (int32_t)v;
}

// (pool, table, lengths, mass, keep, recent, new_lengths, new_mass, status) -> (kept, new_lengths, new_mass)
PyObject* py_paged_evict(PyObject*, PyObject* const* a, Py_ssize_t n) {
  MK_BEGIN
  count(n, 9);
  const at::Tensor& pool = tensor(a[0], "pool");
  const c10::Device dev = pool.device();
  const mk_paged_cache c = paged_of(pool, a[1], a[2], Py_None, a[8], 1);
  const int32_t keep = whole(a[4], "keep"), recent = whole(a[5], "recent");
  if (keep < 1 || recent < 0 || recent > keep) refuse("keep must be >= 1 and recent lie in [0, keep]");
  const mk_paged_mass mass = mass_of(a[3], c, dev, 1.0, "mass");
  const at::Tensor &m = tensor(a[3], "mass"), &len = tensor(a[2], "lengths");
  if (overlap(pool, m)) refuse("mass must not overlap the pool");
  On on(dev);
  mk_paged_mass to;
  at::Tensor made, lengths, kept;
  if (a[7] == Py_None) {
    const int64_t sizes[3] = {c.n_seqs, c.n_kv_heads, (int64_t)c.max_pages * 128};
    made = fresh(sizes, at::kFloat, dev);
    to = {static_cast<float*>(made.data_ptr()), sizes[1] * sizes[2], sizes[2], 1.f};
  } else {
    to = mass_of(a[7], c, dev, 1.0, "new_mass");
    const at::Tensor& t = tensor(a[7], "new_mass");
    const bool same = to.data == mass.data && to.seq_stride == mass.seq_stride && to.head_stride == mass.head_stride;
    if (overlap(pool, t) || (!same && overlap(m, t))) refuse("new_mass must be mass or not overlap it, nor the pool");
  }
  if (a[6] == Py_None) {
    lengths = fresh({(int64_t)c.n_seqs}, at::kInt, dev);
  } else {
    ints(a[6], "new_lengths", c.n_seqs, dev);
    lengths = tensor(a[6], "new_lengths");
    if (lengths.data_ptr() != len.data_ptr() && overlap(lengths, len)) refuse("new_lengths must be lengths or not overlap them");
    if (overlap(lengths, tensor(a[1], "table"))) refuse("new_lengths must not overlap table");
  }
  const int64_t sizes[3] = {c.n_seqs, c.n_kv_heads, keep};
  const size_t nws = mk_paged_evict_bytes(&c, keep);
  if (!nws && c.n_seqs)  // a description or keep that the call refuses: before a tensor of its size is made
    check(mk_paged_evict(&c, &mass, keep, recent, nullptr, nullptr, &to, nullptr, 0, on.stream));
  kept = fresh(sizes, at::kInt, dev);
  at::Tensor ws;
  if (nws) ws = fresh({(int64_t)nws}, at::kByte, dev);
  check(mk_paged_evict(&c, &mass, keep, recent, static_cast<int32_t*>(kept.data_ptr()), static_cast<int32_t*>(lengths.data_ptr()),
                       &to, nws ? ws.data_ptr() : nullptr, nws, on.stream));
  PyObject *l = a[6], *t = a[7];
  if (l != Py_None) Py_INCREF(l);
  else l = THPVariable_Wrap(std::move(lengths));
  if (t != Py_None) Py_INCREF(t);
  else t = THPVariable_Wrap(std::move(made));
  return Py_BuildValue("(NNN)", THPVariable_Wrap(std::move(kept)), l, t);
  MK_END
}

PyObject* py_set_error(PyObject*, PyObject* cls) {
  Py_INCREF(cls);
  Py_XDECREF(mk_error);
  mk_error = cls;
  Py_RETURN_NONE;
}

#define FAST(name, f) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FAST("store", py_store), FAST("load", py_load), FAST("attention", py_attention),
                         FAST("page_copy", py_page_copy), FAST("paged_store", py_paged_store),
                         FAST("paged_attention", py_paged_attention), FAST("paged_evict", py_paged_evict),
                         {"set_error", py_set_error, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__torch(void) { return PyModule_Create(&module); }
