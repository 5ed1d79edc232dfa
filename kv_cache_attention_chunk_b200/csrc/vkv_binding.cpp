// Argument marshalling of the paged cache calls: torch tensors -> the C structs of vkv.h.
//
// These calls run once per layer and token, and their checks (type, shape, place, strides of
// a dozen tensors) took 4 to 7 us in Python, more than their kernels.  Nothing is computed
// here: each function checks its tensors, fills the C struct and calls the entry point whose
// address it is given.  A refused argument is a ValueError; the C status is returned.
#include <Python.h>
#include <ATen/MemoryOverlap.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <climits>
#include <cmath>
#include <exception>
#include <string>

#include "vkv.h"

namespace {

struct Refusal {
  std::string text;
};

const at::Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) throw Refusal{std::string(what) + " must be a tensor"};
  return THPVariable_Unpack(o);
}

std::string place(int dev) { return " on cuda:" + std::to_string(dev); }

int device_of(const at::Tensor& x) {
  if (!x.is_cuda()) throw Refusal{"expected CUDA tensors"};
  return x.get_device();
}

int32_t int_of(PyObject* o, const char* what) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    throw Refusal{std::string(what) + " must be an integer"};
  }
  if (v < INT_MIN || v > INT_MAX) throw Refusal{std::string(what) + " is out of range"};
  return (int32_t)v;
}

int32_t size_of(int64_t n, const char* what) {
  if (n > INT_MAX) throw Refusal{std::string(what) + " is out of range"};
  return (int32_t)n;
}

// The address of a contiguous tensor of this type and shape on device `dev`; NULL for None where `optional`.
template <typename T>
T* vec(PyObject* o, const char* what, at::ScalarType type, at::IntArrayRef shape, int dev, bool optional = false) {
  if (optional && o == Py_None) return nullptr;
  const at::Tensor& x = tensor(o, what);
  if (x.scalar_type() != type || !x.is_cuda() || x.get_device() != dev || x.sizes() != shape || !x.is_contiguous())
    throw Refusal{std::string(what) + " must be a contiguous " + c10::toString(type) + " tensor of shape " +
                  c10::str(shape) + place(dev)};
  return static_cast<T*>(x.data_ptr());
}

int32_t* err_word(PyObject* o, int dev) {
  if (o == Py_None) return nullptr;
  const at::Tensor& x = tensor(o, "err");
  if (x.scalar_type() != at::kInt || !x.is_cuda() || x.get_device() != dev || x.numel() < 1)
    throw Refusal{"err must be an int32 tensor" + place(dev)};
  return static_cast<int32_t*>(x.data_ptr());
}

int32_t dtype_of(const at::Tensor& x, const char* what) {
  switch (x.scalar_type()) {
    case at::kBFloat16: return VKV_BF16;
    case at::kHalf: return VKV_FP16;
    case at::kFloat8_e4m3fn: return VKV_E4M3;
    default: throw Refusal{std::string(what) + " is none of bfloat16, float16, float8_e4m3fn"};
  }
}

// The stride of an axis as the entry points check it: that of an axis of one is never used, and
// torch leaves there what it likes.
int64_t step(const at::Tensor& x, int64_t axis) { return x.size(axis) > 1 ? x.stride(axis) : 0; }

// For a tensor that is written: two of its elements must not be one (an expanded tensor).
void no_overlap(const at::Tensor& x, const char* what) {
  if (at::has_internal_overlap(x) == at::MemOverlap::Yes) throw Refusal{std::string(what) + " overlaps itself"};
}

// A tensor and the bytes between its first and behind its last element.
struct Span {
  const at::Tensor& x;
  const char *begin, *end;
  explicit Span(const at::Tensor& t) : x(t) {
    const at::IntArrayRef size = x.sizes(), stride = x.strides();
    int64_t last = 0;
    for (size_t i = 0; i < size.size(); ++i) last += (size[i] - 1) * stride[i];
    begin = static_cast<const char*>(x.const_data_ptr());
    end = begin + (x.numel() ? (last + 1) * (int64_t)x.element_size() : 0);
  }
};

// Whether sum_i x_i stride_i = off has a solution with |x_i| < size_i over the axes from `i` on (largest
// stride first, `reach` the most that the axes behind an axis add up to): two equally strided views meet
// there.  Strides of views into one dense buffer leave two candidates per axis at most; `budget` bounds others.
bool meets(const int64_t* size, const int64_t* stride, const int64_t* reach, int n, int i, int64_t off, int& budget) {
  if (i == n) return off == 0;
  const int64_t s = stride[i], r = reach[i];
  const auto floor_div = [](int64_t a, int64_t b) { return a / b - (a % b < 0); };
  const int64_t lo = std::max(-(size[i] - 1), floor_div(off - r + s - 1, s)), hi = std::min(size[i] - 1, floor_div(off + r, s));
  for (int64_t x = lo; x <= hi && budget > 0; ++x)
    if (--budget, meets(size, stride, reach, n, i + 1, off - x * s, budget)) return true;
  return false;
}

// Whether an element of `a` certainly lies on one of `b`: exact for tensors without gaps and for two of equal
// sizes and strides (two parts of one buffer, side by side or not); others count as apart.
bool share_within(const Span& p, const Span& q) {
  const at::Tensor &a = p.x, &b = q.x;
  if (a.is_non_overlapping_and_dense() && b.is_non_overlapping_and_dense()) return true;
  constexpr int kMost = 4;
  if (a.sizes() != b.sizes() || a.dim() > kMost || a.element_size() != b.element_size()) return false;
  int64_t size[kMost], stride[kMost], reach[kMost], n = 0;
  for (int64_t i = 0; i < a.dim(); ++i) {
    if (a.size(i) == 1) continue;
    if (a.stride(i) != b.stride(i)) return false;
    if (a.stride(i) == 0) continue;
    int64_t at = n++;
    for (; at > 0 && stride[at - 1] < a.stride(i); --at) size[at] = size[at - 1], stride[at] = stride[at - 1];
    size[at] = a.size(i), stride[at] = a.stride(i);
  }
  int64_t sum = 0;
  for (int64_t i = n; i-- > 0; sum += (size[i] - 1) * stride[i]) reach[i] = sum;
  const int64_t e = (int64_t)a.element_size(), bytes = q.begin - p.begin;
  int budget = 64;
  return bytes % e == 0 && meets(size, stride, reach, (int)n, 0, bytes / e, budget);
}
inline bool share(const Span& p, const Span& q) { return p.begin < q.end && q.begin < p.end && share_within(p, q); }

// [.., .., d] with contiguous d: outer and inner stride of a 3-d tensor
vkv_tensor rows3(const at::Tensor& x, const char* what, int dev, bool outer_is_row) {
  if (x.dim() != 3 || !x.is_cuda() || x.get_device() != dev || x.stride(2) != 1)
    throw Refusal{std::string(what) + " must be a 3-d tensor with contiguous last axis" + place(dev)};
  vkv_tensor t;
  t.ptr = x.data_ptr();
  t.sb = outer_is_row ? step(x, 0) : 0;
  t.st = outer_is_row ? 0 : step(x, 0);
  t.sh = step(x, 1);
  return t;
}

struct Table {
  int32_t* ptr;
  int64_t stride;
  int32_t W;
};
Table table_of(PyObject* o, int64_t R, int dev) {
  const at::Tensor& x = tensor(o, "block_table");
  if (x.scalar_type() != at::kInt || x.dim() != 2 || !x.is_cuda() || x.get_device() != dev || x.size(0) != R ||
      (x.size(1) > 1 && x.stride(1) != 1))
    throw Refusal{"block_table must be an int32 tensor [R, W] with contiguous rows" + place(dev)};
  // a single row's stride is never used; a narrower one than W means overlapping rows
  return {static_cast<int32_t*>(x.data_ptr()), R == 1 ? std::max(x.stride(0), x.size(1)) : x.stride(0),
          size_of(x.size(1), "block_table")};
}

struct Cache {
  int32_t n_pages, page, Hkv, d, dtype;
  vkv_tensor k, v;
};
Cache cache_of(PyObject* ko, PyObject* vo, int dev) {
  const at::Tensor &k = tensor(ko, "k_pages"), &v = tensor(vo, "v_pages");
  if (k.dim() != 4 || k.sizes() != v.sizes() || k.scalar_type() != v.scalar_type() || !k.is_cuda() || !v.is_cuda() ||
      k.get_device() != dev || v.get_device() != dev || k.stride(3) != 1 || v.stride(3) != 1)
    throw Refusal{"k_pages and v_pages must be [n_pages, page, Hkv, d] of one type with contiguous d" + place(dev)};
  Cache c;
  c.n_pages = size_of(k.size(0), "n_pages");
  c.page = size_of(k.size(1), "page");
  c.Hkv = size_of(k.size(2), "Hkv");
  c.d = size_of(k.size(3), "d");
  c.dtype = dtype_of(k, "the cache");
  c.k = {k.data_ptr(), step(k, 0), step(k, 1), step(k, 2)};
  c.v = {v.data_ptr(), step(v, 0), step(v, 1), step(v, 2)};
  return c;
}

void scales_of(PyObject* ks, PyObject* vs, const Cache& c, int dev, const float** k, const float** v) {
  *k = *v = nullptr;
  if (ks == Py_None && vs == Py_None) return;
  if (c.dtype != VKV_E4M3) throw Refusal{"k_scale and v_scale belong to a float8_e4m3fn cache"};
  *k = vec<float>(ks, "k_scale", at::kFloat, {c.Hkv}, dev, true);
  *v = vec<float>(vs, "v_scale", at::kFloat, {c.Hkv}, dev, true);
}

void workspace_of(PyObject* o, int dev, void** ptr, size_t* bytes) {
  const at::Tensor& x = tensor(o, "workspace");
  *ptr = nullptr;
  *bytes = 0;
  if (x.numel() == 0) return;  // the entry point says what it needs
  if (!x.is_cuda() || x.get_device() != dev || !x.is_contiguous())
    throw Refusal{"workspace must be a contiguous tensor" + place(dev)};
  *ptr = x.data_ptr();
  *bytes = x.nbytes();
}

// (entry point, stream handle) come first in every call
template <typename A>
PyObject* call(PyObject* fn, PyObject* stream, const A& a) {
  using Fn = vkv_status (*)(const A*, vkv_stream_t);
  Fn f = reinterpret_cast<Fn>(PyLong_AsVoidPtr(fn));
  vkv_stream_t s = reinterpret_cast<vkv_stream_t>(PyLong_AsVoidPtr(stream));
  if (PyErr_Occurred()) return nullptr;
  vkv_status rc;
  Py_BEGIN_ALLOW_THREADS
  rc = f(&a, s);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong((long)rc);
}

template <typename F>
PyObject* guarded(Py_ssize_t have, Py_ssize_t want, F&& body) {
  if (have != want) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, have);
    return nullptr;
  }
  try {
    return body();
  } catch (const Refusal& r) {
    PyErr_SetString(PyExc_ValueError, r.text.c_str());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_ValueError, e.what());
  }
  return nullptr;
}

// The arrays of a map call, in memory: what is written lies in nothing else, but that kv_len and
// ring_pos may be updated in place.
void map_apart(const vkv_page_map_args& a) {
  struct Part {
    const void* begin;
    int64_t bytes;
    const char* name;
  };
  const int64_t R = a.R, n = a.max_tokens;
  const Part part[] = {{a.kv_len_out, 4 * R, "out['kv_len']"}, {a.ring_pos_out, 16, "out['ring']"},
                       {a.slot, 8 * n, "out['slot']"},         {a.row, 4 * n, "out['row']"},
                       {a.pos, 4 * n, "out['pos']"},           {a.cu, 4 * (R + 1), "out['cu']"},
                       {a.ring, 4 * (int64_t)a.n_ring, "ring"}, {a.kv_len, 4 * R, "kv_len"},
                       {a.new_len, 4 * R, "new_len"},          {a.ring_pos, 16, "ring_pos"}};
  constexpr int kWritten = 7, kParts = 10;  // the first are written
  const char* table = reinterpret_cast<const char*>(a.table);
  const int64_t stride = 4 * a.table_stride, row = 4 * (int64_t)a.W;
  for (int i = 0; i < kParts; ++i) {
    const char *x = static_cast<const char*>(part[i].begin), *x_end = x + part[i].bytes;
    if (!x) continue;
    // the table: the first of its rows that ends behind x, if it begins before x_end
    if (x < table + (R - 1) * stride + row && x_end > table) {
      const int64_t off = x - table, r = off < row ? 0 : (off - row) / stride + 1;
      if (r < R && r * stride < x_end - table) throw Refusal{std::string(part[i].name) + " and block_table overlap"};
    }
    for (int j = i + 1; i < kWritten && j < kParts; ++j) {
      const char *y = static_cast<const char*>(part[j].begin), *y_end = y + part[j].bytes;
      if (!y || x_end <= y || y_end <= x) continue;
      if (x == y && ((i == 0 && j == 7) || (i == 1 && j == 9))) continue;
      throw Refusal{std::string(part[i].name) + " and " + part[j].name + " overlap"};
    }
  }
}

// fn, stream, kv_len, new_len, table, ring, ring_pos, page, max_tokens, out_len, out_ring, slot, row, pos, cu, err
PyObject* page_map(PyObject*, PyObject* const* x, Py_ssize_t n) {
  return guarded(n, 16, [&]() -> PyObject* {
    const at::Tensor &len = tensor(x[2], "kv_len"), &ring = tensor(x[5], "ring");
    const int dev = device_of(len);
    const int64_t R = len.dim() == 1 ? len.size(0) : -1, n_ring = ring.dim() == 1 ? ring.size(0) : -1;
    vkv_page_map_args a{};
    a.R = size_of(R, "kv_len");
    a.n_ring = size_of(n_ring, "ring");
    a.page = int_of(x[7], "page_size");
    a.max_tokens = int_of(x[8], "max_tokens");
    const Table t = table_of(x[4], R, dev);
    a.W = t.W;
    a.table = t.ptr;
    a.table_stride = t.stride;
    a.kv_len = vec<int32_t>(x[2], "kv_len", at::kInt, {R}, dev);
    a.new_len = vec<int32_t>(x[3], "new_len", at::kInt, {R}, dev);
    a.ring = vec<int32_t>(x[5], "ring", at::kInt, {n_ring}, dev);
    a.ring_pos = vec<int64_t>(x[6], "ring_pos", at::kLong, {2}, dev);
    a.kv_len_out = vec<int32_t>(x[9], "out['kv_len']", at::kInt, {R}, dev);
    if (a.kv_len_out == a.new_len && R > 0) throw Refusal{"out['kv_len'] must not be new_len"};
    a.ring_pos_out = vec<int64_t>(x[10], "out['ring']", at::kLong, {2}, dev);
    a.slot = vec<int64_t>(x[11], "out['slot']", at::kLong, {a.max_tokens}, dev);
    a.row = vec<int32_t>(x[12], "out['row']", at::kInt, {a.max_tokens}, dev, true);
    a.pos = vec<int32_t>(x[13], "out['pos']", at::kInt, {a.max_tokens}, dev, true);
    a.cu = vec<int32_t>(x[14], "out['cu']", at::kInt, {R + 1}, dev, true);
    a.err_word = err_word(x[15], dev);
    if (R > 0 && a.W > 0 && a.max_tokens > 0) map_apart(a);
    return call(x[0], x[1], a);
  });
}

// fn, stream, k_new, v_new, slot, k_pages, v_pages, k_scale, v_scale, kbar, err
PyObject* page_append(PyObject*, PyObject* const* x, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> PyObject* {
    const at::Tensor &kn = tensor(x[2], "k_new"), &vn = tensor(x[3], "v_new");
    const int dev = device_of(tensor(x[5], "k_pages"));
    const Cache c = cache_of(x[5], x[6], dev);
    if (kn.dim() != 3 || kn.size(1) != c.Hkv || kn.size(2) != c.d || vn.sizes() != kn.sizes() ||
        kn.scalar_type() != vn.scalar_type())
      throw Refusal{"k_new and v_new must be [T, Hkv, d] of one type"};
    vkv_page_append_args a{};
    a.T = size_of(kn.size(0), "k_new");
    a.Hkv = c.Hkv, a.d = c.d, a.page = c.page, a.n_pages = c.n_pages;
    const at::Tensor &k = tensor(x[5], "k_pages"), &v = tensor(x[6], "v_pages");
    no_overlap(k, "k_pages");
    no_overlap(v, "v_pages");
    // one tensor may be both where it gets the same rows as both
    const bool one = c.k.ptr == c.v.ptr && k.strides() == v.strides() && kn.const_data_ptr() == vn.const_data_ptr() &&
                     kn.strides() == vn.strides() && x[7] == x[8];
    const Span ks(k), vs(v);
    if (!one && share(ks, vs)) throw Refusal{"k_pages and v_pages overlap, with unlike rows to store"};
    if (x[9] != Py_None) {
      const Span means(tensor(x[9], "kbar"));
      if (share(means, ks) || share(means, vs)) throw Refusal{"kbar overlaps the cache"};
    }
    a.x_dtype = dtype_of(kn, "k_new");
    a.kv_dtype = c.dtype;
    a.k_new = rows3(kn, "k_new", dev, false);
    a.v_new = rows3(vn, "v_new", dev, false);
    a.k = c.k, a.v = c.v;
    a.slot = vec<int64_t>(x[4], "slot", at::kLong, {a.T}, dev);
    scales_of(x[7], x[8], c, dev, &a.k_scale, &a.v_scale);
    a.kbar = vec<float>(x[9], "kbar", at::kFloat, {c.n_pages, c.Hkv, c.d}, dev, true);
    a.err_word = err_word(x[10], dev);
    return call(x[0], x[1], a);
  });
}

// fn, stream, q, kbar, table, kv_len, page, topk, sink_pages, local_pages, sel, workspace, err
PyObject* page_select(PyObject*, PyObject* const* x, Py_ssize_t n) {
  return guarded(n, 13, [&]() -> PyObject* {
    const at::Tensor &q = tensor(x[2], "q"), &kbar = tensor(x[3], "kbar");
    const int dev = device_of(q);
    if (q.dim() != 3 || kbar.dim() != 3 || q.size(2) != kbar.size(2))
      throw Refusal{"q must be [R, H, d], kbar [n_pages, Hkv, d]"};
    vkv_page_select_args a{};
    const int64_t R = q.size(0), Hkv = kbar.size(1);
    a.R = size_of(R, "q"), a.H = size_of(q.size(1), "q"), a.d = size_of(q.size(2), "q");
    a.n_pages = size_of(kbar.size(0), "kbar"), a.Hkv = size_of(Hkv, "kbar");
    a.page = int_of(x[6], "page_size"), a.topk = int_of(x[7], "topk");
    a.sink_pages = int_of(x[8], "sink_pages"), a.local_pages = int_of(x[9], "local_pages");
    a.q_dtype = dtype_of(q, "q");
    a.q = rows3(q, "q", dev, true);
    a.kbar = vec<float>(x[3], "kbar", at::kFloat, kbar.sizes(), dev);
    const Table t = table_of(x[4], R, dev);
    a.table = t.ptr, a.table_stride = t.stride, a.W = t.W;
    a.kv_len = vec<int32_t>(x[5], "kv_len", at::kInt, {R}, dev);
    a.sel = vec<int32_t>(x[10], "out", at::kInt, {R, Hkv, a.topk}, dev);
    workspace_of(x[11], dev, &a.workspace, &a.workspace_bytes);
    a.err_word = err_word(x[12], dev);
    return call(x[0], x[1], a);
  });
}

// fn, stream, q, k_pages, v_pages, table, kv_len, scale, sink, window, sel, k_scale, v_scale, o, lse, workspace, err
PyObject* page_attn(PyObject*, PyObject* const* x, Py_ssize_t n) {
  return guarded(n, 17, [&]() -> PyObject* {
    const at::Tensor &q = tensor(x[2], "q"), &o = tensor(x[13], "o");
    const int dev = device_of(q);
    const Cache c = cache_of(x[3], x[4], dev);
    if (q.dim() != 3 || q.size(2) != c.d) throw Refusal{"q must be [R, H, d], d as in the cache"};
    if (o.sizes() != q.sizes() || o.scalar_type() != q.scalar_type()) throw Refusal{"o must have the shape and type of q"};
    // a row's queries may be read again after some of its outputs are written
    if (q.numel() && o.data_ptr() == q.data_ptr()) throw Refusal{"o must not be q"};
    no_overlap(o, "o");
    {  // nor may the outputs lie in what other blocks may still read, or in one another
      const Span os(o), ls(tensor(x[14], "lse")), qs(q), ks(tensor(x[3], "k_pages")), vs(tensor(x[4], "v_pages"));
      if (share(os, qs)) throw Refusal{"o overlaps q"};
      if (share(os, ks) || share(os, vs)) throw Refusal{"o overlaps the cache"};
      if (share(ls, os) || share(ls, qs) || share(ls, ks) || share(ls, vs))
        throw Refusal{"lse overlaps o, q or the cache"};
    }
    vkv_page_attn_args a{};
    const int64_t R = q.size(0), H = q.size(1);
    a.R = size_of(R, "q"), a.H = size_of(H, "q");
    a.Hkv = c.Hkv, a.d = c.d, a.page = c.page, a.n_pages = c.n_pages;
    a.q_dtype = dtype_of(q, "q");
    a.kv_dtype = c.dtype;
    double scale = 1.0 / std::sqrt((double)std::max(c.d, 1));
    if (x[7] != Py_None) {
      scale = PyFloat_AsDouble(x[7]);
      if (PyErr_Occurred()) return nullptr;
    }
    a.scale = (float)scale;
    a.sink = int_of(x[8], "sink"), a.window = int_of(x[9], "window");
    a.q = rows3(q, "q", dev, true);
    a.o = rows3(o, "o", dev, true);
    a.k = c.k, a.v = c.v;
    const Table t = table_of(x[5], R, dev);
    a.table = t.ptr, a.table_stride = t.stride, a.W = t.W;
    a.kv_len = vec<int32_t>(x[6], "kv_len", at::kInt, {R}, dev);
    if (x[10] != Py_None) {
      const at::Tensor& sel = tensor(x[10], "sel");
      a.topk = size_of(sel.dim() == 3 ? sel.size(2) : -1, "sel");
      // an empty tensor has no address, which the entry point would take for no selection
      if (a.topk == 0) throw Refusal{"sel must have at least one entry per row and key head"};
      a.sel = vec<int32_t>(x[10], "sel", at::kInt, {R, c.Hkv, a.topk}, dev);
    }
    scales_of(x[11], x[12], c, dev, &a.k_scale, &a.v_scale);
    a.lse = vec<float>(x[14], "lse", at::kFloat, {R, H}, dev);
    workspace_of(x[15], dev, &a.workspace, &a.workspace_bytes);
    a.err_word = err_word(x[16], dev);
    return call(x[0], x[1], a);
  });
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}
PyMethodDef methods[] = {method<page_map>("page_map"), method<page_append>("page_append"),
                         method<page_select>("page_select"), method<page_attn>("page_attn"), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

// The torch and the Python that this file was built for: the build and the import look for it in the library.
extern "C" __attribute__((used, visibility("default"))) const char vkv_binding_tag[] = VKV_BINDING_TAG;

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
