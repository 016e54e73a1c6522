// Python binding of the serving operators: tensors to rope_tensor_t descriptors, and the call.
//
// The operators run in the C library, which is found by the path given to init(); this module
// only marshals.  A decoding step calls them with about ten tensors each, which cost 15 to 20
// us to describe through ctypes and about 1 us here.
//
// Every call returns the library's status; a tensor that cannot be described (not on a CUDA
// device, another device than the first one's, not contiguous, of another type) raises
// ValueError before anything is enqueued.
#include <Python.h>
#include <dlfcn.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ops/empty.h>

#include <vector>

#include "rope_gb300.h"

namespace {

decltype(&rope_scaled_frequencies) g_frequencies;
decltype(&rope_scaled_cos_sin_cache) g_cos_sin_cache;
decltype(&rope_scaled_cos_sin) g_cos_sin;
decltype(&rope_append_paged_kv) g_append;
decltype(&rope_paged_attention) g_attend;
decltype(&rope_paged_attention_workspace) g_workspace;
decltype(&rope_append_paged_kv_8bit) g_append_8bit;
decltype(&rope_paged_attention_8bit) g_attend_8bit;
decltype(&rope_paged_attention_8bit_workspace) g_workspace_8bit;
decltype(&rope_rearrange_sequences) g_rearrange;
decltype(&rope_compact_pages) g_compact;
decltype(&rope_copy_pages) g_copy_pages;

struct Failed {};  // a Python error is set

[[noreturn]] void fail(PyObject* type, const char* text) {
  PyErr_SetString(type, text);
  throw Failed();
}

const at::Tensor& tensor(PyObject* o) {
  if (!THPVariable_Check(o)) fail(PyExc_TypeError, "expected a torch.Tensor");
  return THPVariable_Unpack(o);
}

// `more`: with the types of the operators on codes and on pages, which the others do not take.
int32_t type_of(const at::Tensor& t, bool more) {
  switch (t.scalar_type()) {
    case at::kFloat:
      return ROPE_F32;
    case at::kHalf:
      return ROPE_F16;
    case at::kBFloat16:
      return ROPE_BF16;
    case at::kLong:
      return ROPE_I64;
    case at::kFloat8_e4m3fn:
      if (more) return ROPE_F8E4M3;
      break;
    case at::kFloat8_e8m0fnu:
      if (more) return ROPE_E8M0;
      break;
    case at::kInt:
      if (more) return ROPE_I32;
      break;
    default:
      break;
  }
  fail(PyExc_ValueError, "unsupported dtype");
}

// Descriptors of one call; all tensors on the device of the first.  What the call writes says so
// (kWrites): a tensor that shares its memory until one is written gets its own first.
enum Use { kReads, kWrites };

class Call {
 public:
  explicit Call(bool more = false) : more_(more) {}

  const rope_tensor_t* whole(PyObject* o, Use use = kReads) {  // NULL for None
    if (o == Py_None) return nullptr;
    const at::Tensor& t = tensor(o);
    if (!t.is_contiguous()) fail(PyExc_ValueError, "expected a contiguous tensor");
    return add(t, use);
  }

  // Pages of a tensor of any type and number of dimensions, as bytes.
  rope_tensor_t pages(PyObject* o) {
    const at::Tensor& t = tensor(o);
    if (!t.is_contiguous()) fail(PyExc_ValueError, "expected a contiguous tensor");
    check(t);
    if (t.dim() < 1) fail(PyExc_ValueError, "expected a tensor with a dimension of pages");
    rope_tensor_t d;
    d.data = t.mutable_data_ptr();
    d.dtype = ROPE_U8;
    d.ndim = 2;
    d.shape[0] = t.size(0);
    d.shape[1] = t.size(0) ? (int64_t)t.nbytes() / t.size(0) : 0;
    return d;
  }

  // Rows of a 2-D tensor that may be strided; rows must not overlap.
  const rope_tensor_t* rows(PyObject* o, int64_t* stride, Use use = kReads) {
    *stride = 0;
    if (o == Py_None) return nullptr;
    const at::Tensor& t = tensor(o);
    if (t.dim() != 2 || (t.size(1) > 1 && t.stride(1) != 1))
      fail(PyExc_ValueError, "expected a 2-D tensor with contiguous rows");
    *stride = t.size(0) > 1 ? t.stride(0) : t.size(1);
    if (*stride < t.size(1)) fail(PyExc_ValueError, "rows overlap: the row stride is below the row width");
    return add(t, use);
  }

 private:
  void check(const at::Tensor& t) {
    if (!t.is_cuda()) fail(PyExc_ValueError, "expected a CUDA tensor");
    if (device_ < 0) device_ = t.get_device();
    if (t.get_device() != device_) fail(PyExc_ValueError, "tensors on different devices");
  }

  const rope_tensor_t* add(const at::Tensor& t, Use use) {
    check(t);
    if (t.dim() < 1 || t.dim() > 4) fail(PyExc_ValueError, "expected 1 to 4 dimensions");
    rope_tensor_t& d = descs_[n_++];
    d.data = use == kWrites ? t.mutable_data_ptr() : const_cast<void*>(t.const_data_ptr());
    d.dtype = type_of(t, more_);
    d.ndim = (int32_t)t.dim();
    for (int i = 0; i < d.ndim; ++i) d.shape[i] = t.size(i);
    return &d;
  }

  const bool more_;
  rope_tensor_t descs_[14];
  int n_ = 0;
  int64_t device_ = -1;
};

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Failed();
  return v;
}

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Failed();
  return v;
}

// Frequencies: a contiguous float64 tensor on the host.
const at::Tensor& host_doubles(PyObject* o, int64_t* n) {
  const at::Tensor& t = tensor(o);
  if (t.is_cuda()) fail(PyExc_ValueError, "expected frequencies on the host, got a CUDA tensor");
  if (t.scalar_type() != at::kDouble || !t.is_contiguous())
    fail(PyExc_ValueError, "expected contiguous float64 frequencies");
  *n = t.numel();
  return t;
}

const double* frequencies_of(PyObject* o, int64_t* n) {
  return static_cast<const double*>(host_doubles(o, n).const_data_ptr());
}

template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F&& f) {
  if (n != want) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    return f();
  } catch (const Failed&) {
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

template <typename F>
PyObject* status_of(F&& f) {
  int st;
  Py_BEGIN_ALLOW_THREADS st = f();
  Py_END_ALLOW_THREADS return PyLong_FromLong(st);
}

PyObject* init(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 1, [&]() -> PyObject* {
    const char* path = PyUnicode_AsUTF8(a[0]);
    if (!path) throw Failed();
    void* lib = dlopen(path, RTLD_NOW | RTLD_LOCAL);
    if (!lib) fail(PyExc_RuntimeError, dlerror());
    auto find = [&](auto& fn, const char* name) {
      fn = reinterpret_cast<std::decay_t<decltype(fn)>>(dlsym(lib, name));
      if (!fn) fail(PyExc_RuntimeError, name);
    };
    find(g_frequencies, "rope_scaled_frequencies");
    find(g_cos_sin_cache, "rope_scaled_cos_sin_cache");
    find(g_cos_sin, "rope_scaled_cos_sin");
    find(g_append, "rope_append_paged_kv");
    find(g_attend, "rope_paged_attention");
    find(g_workspace, "rope_paged_attention_workspace");
    find(g_append_8bit, "rope_append_paged_kv_8bit");
    find(g_attend_8bit, "rope_paged_attention_8bit");
    find(g_workspace_8bit, "rope_paged_attention_8bit_workspace");
    find(g_rearrange, "rope_rearrange_sequences");
    find(g_compact, "rope_compact_pages");
    find(g_copy_pages, "rope_copy_pages");
    Py_RETURN_NONE;
  });
}

// (rotary_dim, base, kind or -1, factor, original_length, low, high, attention, factors or None, out)
// -> (status, scale)
PyObject* frequencies(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject* {
    rope_scaling_t s = {};
    s.kind = (int32_t)integer(a[2]);
    s.factor = number(a[3]);
    s.original_length = number(a[4]);
    s.low = number(a[5]);
    s.high = number(a[6]);
    s.attention = number(a[7]);
    int64_t count = 0, size = 0;
    const int64_t dim = integer(a[0]);
    s.factors = a[8] == Py_None ? nullptr : frequencies_of(a[8], &count);
    double scale = 0;
    double* out = static_cast<double*>(host_doubles(a[9], &size).mutable_data_ptr());
    int st = ROPE_ERR_PARAM_INVALID;
    if (size >= dim / 2 && (!s.factors || count == dim / 2))
      st = g_frequencies(dim, number(a[1]), s.kind < 0 ? nullptr : &s, out, &scale);
    return Py_BuildValue("(id)", st, scale);
  });
}

// (inv_freq, scale, positions or None, first_position, cache, stream) -> status
PyObject* scaled_cos_sin_cache(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 6, [&]() -> PyObject* {
    Call c;
    int64_t F = 0;
    const double* f = frequencies_of(a[0], &F);
    const double scale = number(a[1]);
    const rope_tensor_t *cache = c.whole(a[4], kWrites), *positions = c.whole(a[2]);
    const int64_t first = integer(a[3]), stream = integer(a[5]);
    return status_of([&] { return g_cos_sin_cache(f, F, scale, positions, first, cache, (void*)stream); });
  });
}

// (inv_freq, scale, positions or None, first_position, rotary_mode, cos, sin, stream) -> status
PyObject* scaled_cos_sin(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> PyObject* {
    Call c;
    int64_t F = 0;
    const double* f = frequencies_of(a[0], &F);
    const double scale = number(a[1]);
    const rope_tensor_t *cos = c.whole(a[5], kWrites), *sin = c.whole(a[6], kWrites);
    const rope_tensor_t* positions = c.whole(a[2]);
    const int64_t first = integer(a[3]), mode = integer(a[4]), stream = integer(a[7]);
    return status_of([&] { return g_cos_sin(f, F, scale, positions, first, mode, cos, sin, (void*)stream); });
  });
}

// The arguments of an append: a[0 .. caches) tensors up to the caches (and scales), then
// (head_size, rotary_dim or None, is_neox, mrope_section or None, cache_mode, stream).
PyObject* append(PyObject* const* a, bool coded) {
  Call c(coded);
  int64_t ks, qs, vs;
  // (written ones first: a query that is its own output, or the fused buffer of an in-place query's key, has
  // the address that it is written at)
  const rope_tensor_t* out = c.whole(a[6], kWrites);
  const rope_tensor_t *kc = c.whole(a[7], kWrites), *vc = c.whole(a[8], kWrites);
  const rope_tensor_t *kz = coded ? c.whole(a[9], kWrites) : nullptr, *vz = coded ? c.whole(a[10], kWrites) : nullptr;
  const rope_tensor_t* query = c.rows(a[1], &qs, out ? kReads : kWrites);
  const rope_tensor_t *key = c.rows(a[2], &ks), *value = c.rows(a[3], &vs);
  const rope_tensor_t *positions = c.whole(a[0]), *table = c.whole(a[4]), *slots = c.whole(a[5]);
  a += coded ? 11 : 9;
  const int64_t head = integer(a[0]);
  const int64_t rotary = a[1] != Py_None ? integer(a[1]) : table && table->ndim == 2 ? table->shape[1] : 0;
  const int neox = PyObject_IsTrue(a[2]);
  if (neox < 0) throw Failed();
  int64_t section[4] = {0, 0, 0, 0}, sections = 0;
  const bool mrope = a[3] != Py_None;
  if (mrope) {
    sections = PySequence_Size(a[3]);
    if (sections < 0) throw Failed();
    for (int64_t i = 0; i < sections && i < 4; ++i) {
      PyObject* v = PySequence_GetItem(a[3], i);
      if (!v) throw Failed();
      section[i] = PyLong_AsLongLong(v);
      Py_DECREF(v);
      if (section[i] == -1 && PyErr_Occurred()) throw Failed();
    }
  }
  const int32_t mode = (int32_t)integer(a[4]);
  const int64_t stream = integer(a[5]);
  return status_of([&] {
    if (coded)
      return g_append_8bit(positions, query, key, value, table, slots, out, kc, vc, kz, vz, head, rotary, neox,
                           mrope ? section : nullptr, sections, mode, qs, ks, vs, (void*)stream);
    return g_append(positions, query, key, value, table, slots, out, kc, vc, head, rotary, neox,
                    mrope ? section : nullptr, sections, mode, qs, ks, vs, (void*)stream);
  });
}

// (positions, query or None, key, value, table, slots, query_out or None, k_cache, v_cache, head_size,
//  rotary_dim or None, is_neox, mrope_section or None, cache_mode, stream) -> status
PyObject* append_paged_kv(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 15, [&]() -> PyObject* { return append(a, false); });
}

// The same with k_scale and v_scale behind v_cache.
PyObject* append_paged_kv_8bit(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 17, [&]() -> PyObject* { return append(a, true); });
}

int64_t workspace_bytes(const at::Tensor& q, const at::Tensor& k, int64_t prefix_len) {
  int64_t bytes = 0;
  if (q.dim() != 2 || k.dim() != 4 || k.size(3) < 1) return -1;
  const bool coded = k.scalar_type() == at::kFloat8_e4m3fn;
  const int st = (coded ? g_workspace_8bit : g_workspace)(q.size(0), q.size(1) / k.size(3), k.size(1), k.size(3),
                                                          type_of(q, coded), prefix_len, &bytes);
  return st == ROPE_OK ? bytes : -1;
}

// (query, k_cache, prefix_len) -> bytes, or -1 for sizes that the operator refuses
PyObject* attention_workspace(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 3, [&]() -> PyObject* {
    return PyLong_FromLongLong(workspace_bytes(tensor(a[0]), tensor(a[1]), integer(a[2])));
  });
}

// (query, k_cache, v_cache, [k_scale, v_scale,] block_table, seq_lens, query_start_loc, prefix_blocks or None,
//  prefix_len, scale, out, lse or None, workspace or None, stream) -> status.  Without a workspace one is taken from
// the allocator for the current stream, which then has to be the stream of the call.
PyObject* attention(PyObject* const* a, bool coded) {
  Call c(coded);
  int64_t qs;
  PyObject* const* b = a + (coded ? 5 : 3);  // from block_table on
  const rope_tensor_t *query = c.rows(a[0], &qs), *kc = c.whole(a[1]), *vc = c.whole(a[2]);
  const rope_tensor_t *kz = coded ? c.whole(a[3]) : nullptr, *vz = coded ? c.whole(a[4]) : nullptr;
  const rope_tensor_t *bt = c.whole(b[0]), *lens = c.whole(b[1]), *starts = c.whole(b[2]), *prefix = c.whole(b[3]);
  const rope_tensor_t *out = c.whole(b[6], kWrites), *lse = c.whole(b[7], kWrites);
  const int64_t prefix_len = integer(b[4]), stream = integer(b[9]);
  const float scale = (float)number(b[5]);
  at::Tensor ws;
  if (b[8] != Py_None) {
    ws = tensor(b[8]);
    if (!ws.is_cuda() || !ws.is_contiguous() || ws.get_device() != tensor(a[0]).get_device())
      fail(PyExc_ValueError, "expected a contiguous workspace on the tensors' device");
  } else {
    const int64_t bytes = workspace_bytes(tensor(a[0]), tensor(a[1]), prefix_len);
    if (bytes < 0) return PyLong_FromLong(ROPE_ERR_PARAM_INVALID);
    ws = at::empty({bytes}, tensor(a[0]).options().dtype(at::kByte));
  }
  void* const at = ws.mutable_data_ptr();
  const int64_t bytes = (int64_t)ws.nbytes();
  return status_of([&] {
    if (coded)
      return g_attend_8bit(query, qs, kc, vc, kz, vz, bt, lens, starts, prefix, prefix_len, scale, out, lse, at, bytes,
                           (void*)stream);
    return g_attend(query, qs, kc, vc, bt, lens, starts, prefix, prefix_len, scale, out, lse, at, bytes,
                    (void*)stream);
  });
}

PyObject* paged_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&]() -> PyObject* { return attention(a, false); });
}

PyObject* paged_attention_8bit(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 15, [&]() -> PyObject* { return attention(a, true); });
}

// (block_table, seq_lens, ref_counts, parents, room or None, new_block_table, new_seq_lens, new_ref_counts, copy_src,
//  copy_dst, counts, block_size, prefix_len, stream) -> status
PyObject* rearrange_sequences(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 14, [&]() -> PyObject* {
    Call c(true);
    const rope_tensor_t* t[11];
    for (int i = 10; i >= 0; --i) t[i] = c.whole(a[i], i >= 5 ? kWrites : kReads);  // (written ones first, as above)
    const int64_t block = integer(a[11]), prefix = integer(a[12]), stream = integer(a[13]);
    return status_of([&] {
      return g_rearrange(t[0], t[1], t[2], t[3], t[4], t[5], t[6], t[7], t[8], t[9], t[10], block, prefix,
                         (void*)stream);
    });
  });
}

// (block_table, seq_lens, ref_counts, prefix_blocks or None, new_block_table, new_ref_counts, new_prefix_blocks or
//  None, copy_src, copy_dst, counts, block_size, prefix_len, stream) -> status
PyObject* compact_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&]() -> PyObject* {
    Call c(true);
    const rope_tensor_t* t[10];
    for (int i = 9; i >= 0; --i) t[i] = c.whole(a[i], i >= 4 ? kWrites : kReads);
    const int64_t block = integer(a[10]), prefix = integer(a[11]), stream = integer(a[12]);
    return status_of([&] {
      return g_compact(t[0], t[1], t[2], t[3], t[4], t[5], t[6], t[7], t[8], t[9], block, prefix, (void*)stream);
    });
  });
}

// (src, dst, count or None, a tuple or list of tensors, stream) -> status
PyObject* copy_pages(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 5, [&]() -> PyObject* {
    Call c(true);
    if (!PyList_Check(a[3]) && !PyTuple_Check(a[3])) fail(PyExc_TypeError, "expected a list or tuple of tensors");
    const Py_ssize_t count = PySequence_Fast_GET_SIZE(a[3]);
    std::vector<rope_tensor_t> list;
    list.reserve(count);
    const rope_tensor_t *src = c.whole(a[0]), *dst = c.whole(a[1]), *pairs = c.whole(a[2]);
    for (Py_ssize_t i = 0; i < count; ++i) list.push_back(c.pages(PySequence_Fast_GET_ITEM(a[3], i)));
    const int64_t stream = integer(a[4]);
    return status_of([&] { return g_copy_pages(src, dst, pairs, list.data(), (int64_t)count, (void*)stream); });
  });
}

#define ROPE_METHOD(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {ROPE_METHOD(init),
                         ROPE_METHOD(frequencies),
                         ROPE_METHOD(scaled_cos_sin_cache),
                         ROPE_METHOD(scaled_cos_sin),
                         ROPE_METHOD(append_paged_kv),
                         ROPE_METHOD(attention_workspace),
                         ROPE_METHOD(paged_attention),
                         ROPE_METHOD(append_paged_kv_8bit),
                         ROPE_METHOD(paged_attention_8bit),
                         ROPE_METHOD(rearrange_sequences),
                         ROPE_METHOD(compact_pages),
                         ROPE_METHOD(copy_pages),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "rope_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_rope_binding() { return PyModule_Create(&module); }
