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

#include "rope_gb300.h"

namespace {

decltype(&rope_scaled_frequencies) g_frequencies;
decltype(&rope_scaled_cos_sin_cache) g_cos_sin_cache;
decltype(&rope_scaled_cos_sin) g_cos_sin;
decltype(&rope_append_paged_kv) g_append;
decltype(&rope_paged_attention) g_attend;
decltype(&rope_paged_attention_workspace) g_workspace;

struct Failed {};  // a Python error is set

[[noreturn]] void fail(PyObject* type, const char* text) {
  PyErr_SetString(type, text);
  throw Failed();
}

const at::Tensor& tensor(PyObject* o) {
  if (!THPVariable_Check(o)) fail(PyExc_TypeError, "expected a torch.Tensor");
  return THPVariable_Unpack(o);
}

int32_t type_of(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kFloat:
      return ROPE_F32;
    case at::kHalf:
      return ROPE_F16;
    case at::kBFloat16:
      return ROPE_BF16;
    case at::kLong:
      return ROPE_I64;
    default:
      fail(PyExc_ValueError, "unsupported dtype");
  }
}

// Descriptors of one call; all tensors on the device of the first.  What the call writes says so
// (kWrites): a tensor that shares its memory until one is written gets its own first.
enum Use { kReads, kWrites };

class Call {
 public:
  const rope_tensor_t* whole(PyObject* o, Use use = kReads) {  // NULL for None
    if (o == Py_None) return nullptr;
    const at::Tensor& t = tensor(o);
    if (!t.is_contiguous()) fail(PyExc_ValueError, "expected a contiguous tensor");
    return add(t, use);
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
  const rope_tensor_t* add(const at::Tensor& t, Use use) {
    if (!t.is_cuda()) fail(PyExc_ValueError, "expected a CUDA tensor");
    if (device_ < 0) device_ = t.get_device();
    if (t.get_device() != device_) fail(PyExc_ValueError, "tensors on different devices");
    if (t.dim() < 1 || t.dim() > 4) fail(PyExc_ValueError, "expected 1 to 4 dimensions");
    rope_tensor_t& d = descs_[n_++];
    d.data = use == kWrites ? t.mutable_data_ptr() : const_cast<void*>(t.const_data_ptr());
    d.dtype = type_of(t);
    d.ndim = (int32_t)t.dim();
    for (int i = 0; i < d.ndim; ++i) d.shape[i] = t.size(i);
    return &d;
  }

  rope_tensor_t descs_[12];
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

// (positions, query or None, key, value, table, slots, query_out or None, k_cache, v_cache, head_size,
//  rotary_dim or None, is_neox, mrope_section or None, cache_mode, stream) -> status
PyObject* append_paged_kv(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 15, [&]() -> PyObject* {
    Call c;
    int64_t ks, qs, vs;
    // (written ones first: a query that is its own output, or the fused buffer of an in-place query's key, has
    // the address that it is written at)
    const rope_tensor_t* out = c.whole(a[6], kWrites);
    const rope_tensor_t *kc = c.whole(a[7], kWrites), *vc = c.whole(a[8], kWrites);
    const rope_tensor_t* query = c.rows(a[1], &qs, out ? kReads : kWrites);
    const rope_tensor_t *key = c.rows(a[2], &ks), *value = c.rows(a[3], &vs);
    const rope_tensor_t *positions = c.whole(a[0]), *table = c.whole(a[4]), *slots = c.whole(a[5]);
    const int64_t head = integer(a[9]);
    const int64_t rotary = a[10] != Py_None ? integer(a[10]) : table && table->ndim == 2 ? table->shape[1] : 0;
    const int neox = PyObject_IsTrue(a[11]);
    if (neox < 0) throw Failed();
    int64_t section[4] = {0, 0, 0, 0}, sections = 0;
    const bool mrope = a[12] != Py_None;
    if (mrope) {
      sections = PySequence_Size(a[12]);
      if (sections < 0) throw Failed();
      for (int64_t i = 0; i < sections && i < 4; ++i) {
        PyObject* v = PySequence_GetItem(a[12], i);
        if (!v) throw Failed();
        section[i] = PyLong_AsLongLong(v);
        Py_DECREF(v);
        if (section[i] == -1 && PyErr_Occurred()) throw Failed();
      }
    }
    const int32_t mode = (int32_t)integer(a[13]);
    const int64_t stream = integer(a[14]);
    return status_of([&] {
      return g_append(positions, query, key, value, table, slots, out, kc, vc, head, rotary, neox,
                      mrope ? section : nullptr, sections, mode, qs, ks, vs, (void*)stream);
    });
  });
}

int64_t workspace_bytes(const at::Tensor& q, const at::Tensor& k, int64_t prefix_len) {
  int64_t bytes = 0;
  if (q.dim() != 2 || k.dim() != 4 || k.size(3) < 1) return -1;
  const int st = g_workspace(q.size(0), q.size(1) / k.size(3), k.size(1), k.size(3), type_of(q), prefix_len, &bytes);
  return st == ROPE_OK ? bytes : -1;
}

// (query, k_cache, prefix_len) -> bytes, or -1 for sizes that the operator refuses
PyObject* attention_workspace(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 3, [&]() -> PyObject* {
    return PyLong_FromLongLong(workspace_bytes(tensor(a[0]), tensor(a[1]), integer(a[2])));
  });
}

// (query, k_cache, v_cache, block_table, seq_lens, query_start_loc, prefix_blocks or None, prefix_len, scale, out,
//  lse or None, workspace or None, stream) -> status.  Without a workspace one is taken from the allocator for the
// current stream, which then has to be the stream of the call.
PyObject* paged_attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 13, [&]() -> PyObject* {
    Call c;
    int64_t qs;
    const rope_tensor_t *query = c.rows(a[0], &qs), *kc = c.whole(a[1]), *vc = c.whole(a[2]), *bt = c.whole(a[3]);
    const rope_tensor_t *lens = c.whole(a[4]), *starts = c.whole(a[5]), *prefix = c.whole(a[6]);
    const rope_tensor_t *out = c.whole(a[9], kWrites), *lse = c.whole(a[10], kWrites);
    const int64_t prefix_len = integer(a[7]), stream = integer(a[12]);
    const float scale = (float)number(a[8]);
    at::Tensor ws;
    if (a[11] != Py_None) {
      ws = tensor(a[11]);
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
      return g_attend(query, qs, kc, vc, bt, lens, starts, prefix, prefix_len, scale, out, lse, at, bytes,
                      (void*)stream);
    });
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
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "rope_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_rope_binding() { return PyModule_Create(&module); }
