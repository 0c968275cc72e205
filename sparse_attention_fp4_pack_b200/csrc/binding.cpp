// The paged 8-bit cache's calls from Python without its per-argument cost (module _native).
//
// These calls take 10 to 13 tensors and are made for every layer of a step, where reading the
// tensors' properties from Python costs more than the kernels take (11.5 us against 4.5 for a
// plan of 256 requests; 5 from here).  Every function checks types, shapes, devices and layout as
// csa2.py does, calls the C entry point on the current stream, and returns its status; it returns
// -1 without having called anything when an argument is not as it should be, and csa2.py's own
// checks then name the argument.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "csa2.h"

namespace {

constexpr long kExplain = -1;

// Arguments read in order; ok turns false at the first that is not as it should be.
struct Args {
  PyObject* const* arg;
  Py_ssize_t n, at = 0;
  int dev = -1;
  bool ok = true;

  PyObject* next() {
    if (at >= n) ok = false;
    return ok ? arg[at++] : nullptr;
  }
  const at::Tensor* tensor() {
    PyObject* o = next();
    if (!ok || !THPVariable_Check(o)) {
      ok = false;
      return nullptr;
    }
    return &THPVariable_Unpack(o);
  }
  // A contiguous tensor of the given type and shape on the call's device (the first one's).
  bool fits(const at::Tensor* t, at::ScalarType type, at::IntArrayRef shape) {
    if (!ok || t->scalar_type() != type || t->sizes() != shape || !t->is_cuda() || !t->is_contiguous()) return ok = false;
    if (dev < 0) dev = t->get_device();
    return ok = t->get_device() == dev;
  }
  template <typename T>
  T* data(at::ScalarType type, at::IntArrayRef shape) {
    const at::Tensor* t = tensor();
    return ok && fits(t, type, shape) ? static_cast<T*>(t->data_ptr()) : nullptr;
  }
  // The same for a [T, heads, hd] view whose tokens are each contiguous.
  const void* tokens(const at::Tensor* t, at::ScalarType type, int64_t T, int64_t heads, int64_t hd, int64_t* stride) {
    if (!ok || t->scalar_type() != type || t->sizes() != at::IntArrayRef({T, heads, hd}) || !t->is_cuda()) {
      ok = false;
      return nullptr;
    }
    if (dev < 0) dev = t->get_device();
    const auto s = t->strides();
    *stride = T > 1 ? s[0] : heads * hd;
    ok = t->get_device() == dev && (T == 0 || (s[2] == 1 && (s[1] == hd || heads == 1))) && *stride >= heads * hd &&
         *stride % 8 == 0;
    return ok ? t->data_ptr() : nullptr;
  }
  int64_t integer(int64_t least, int64_t most) {
    PyObject* o = next();
    if (!ok || !PyLong_Check(o)) return ok = false;
    int overflow = 0;
    const long long v = PyLong_AsLongLongAndOverflow(o, &overflow);
    ok = overflow == 0 && v >= least && v <= most;
    return ok ? v : 0;
  }
  int number() { return (int)integer(INT32_MIN, INT32_MAX); }
  float real() {
    PyObject* o = next();
    if (!ok || !(PyFloat_Check(o) || PyLong_Check(o))) return ok = false;
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) {
      PyErr_Clear();
      ok = false;
    }
    return (float)v;
  }
  uint32_t* status() {
    PyObject* o = next();
    if (!ok || o == Py_None) return nullptr;
    if (!THPVariable_Check(o)) return ok = false, nullptr;
    const at::Tensor& t = THPVariable_Unpack(o);
    ok = t.scalar_type() == at::kInt && t.numel() > 0 && t.is_cuda() && t.get_device() == dev;
    return ok ? static_cast<uint32_t*>(t.data_ptr()) : nullptr;
  }
  bool done() { return ok = ok && at == n; }
};

PyObject* result(long v) { return PyLong_FromLong(v); }

// f(stream) with the call's device current.
template <class F>
PyObject* on_device(int dev, F f) {
  const c10::cuda::OptionalCUDAGuard guard(c10::Device(c10::kCUDA, (c10::DeviceIndex)dev));
  return result(f(c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream()));
}

// One layer's cache: [n_pages][Hk][page][hd] and [n_pages][Hk].
struct Cache {
  int64_t pages = 0, Hk = 0, page = 0, hd = 0;
  uint8_t *k = nullptr, *v = nullptr;
  float *ks = nullptr, *vs = nullptr;
};
bool read_cache(Args& a, Cache& c) {
  const at::Tensor* k = a.tensor();
  if (!a.ok || k->dim() != 4) return a.ok = false;
  c.pages = k->size(0);
  c.Hk = k->size(1);
  c.page = k->size(2);
  c.hd = k->size(3);
  if (c.Hk > INT32_MAX || c.page > INT32_MAX || c.hd > INT32_MAX || !a.fits(k, at::kByte, k->sizes())) return a.ok = false;
  c.k = static_cast<uint8_t*>(k->data_ptr());
  c.v = a.data<uint8_t>(at::kByte, {c.pages, c.Hk, c.page, c.hd});
  c.ks = a.data<float>(at::kFloat, {c.pages, c.Hk});
  c.vs = a.data<float>(at::kFloat, {c.pages, c.Hk});
  return a.ok;
}
int kind_of(at::ScalarType t) { return t == at::kBFloat16 ? CSA2_BF16 : t == at::kHalf ? CSA2_F16 : -1; }
const int32_t* read_table(Args& a, int64_t R, int* cols, int32_t** out = nullptr) {
  const at::Tensor* t = a.tensor();
  if (!a.ok || t->dim() != 2 || t->size(1) > INT32_MAX || !a.fits(t, at::kInt, {R, t->size(1)})) {
    a.ok = false;
    return nullptr;
  }
  *cols = (int)t->size(1);
  int32_t* p = static_cast<int32_t*>(t->data_ptr());
  if (out) *out = p;
  return p;
}
// A 1-D tensor of any length, at most INT32_MAX when it counts requests.
template <typename T>
T* read_vector(Args& a, at::ScalarType type, int64_t* n) {
  const at::Tensor* t = a.tensor();
  if (!a.ok || t->dim() != 1 || !a.fits(t, type, t->sizes())) {
    a.ok = false;
    return nullptr;
  }
  *n = t->size(0);
  return static_cast<T*>(t->data_ptr());
}

PyObject* paged_plan(PyObject* const* argv, Py_ssize_t argc) {
  Args a{argv, argc};
  int64_t R = 0, F = 0, T = 0;
  int cols = 0;
  int32_t* table = nullptr;
  const int32_t* ctx = read_vector<int32_t>(a, at::kInt, &R);
  const int32_t* fresh = a.data<int32_t>(at::kInt, {R});
  read_table(a, R, &cols, &table);
  const int32_t* free_pages = read_vector<int32_t>(a, at::kInt, &F);
  const int32_t* n_free = a.data<int32_t>(at::kInt, {1});
  const int page = a.number();
  const int64_t n_pages = a.integer(INT64_MIN, INT64_MAX);
  int32_t* seq = a.data<int32_t>(at::kInt, {R});
  int32_t* n_out = a.data<int32_t>(at::kInt, {1});
  int32_t* q_start = a.data<int32_t>(at::kInt, {R + 1});
  int64_t* slot = read_vector<int64_t>(a, at::kLong, &T);
  int64_t* pos = a.data<int64_t>(at::kLong, {T});
  uint32_t* status = a.status();
  if (!a.done() || R > INT32_MAX) return result(kExplain);
  return on_device(a.dev, [&](cudaStream_t stream) {
    return (long)csa2_paged_plan(ctx, fresh, (int)R, page, table, cols, free_pages, F, n_free, n_pages, seq, n_out, q_start,
                                 slot, pos, T, status, stream);
  });
}

PyObject* paged_release(PyObject* const* argv, Py_ssize_t argc) {
  Args a{argv, argc};
  int64_t R = 0, F = 0;
  int cols = 0;
  const int32_t* seq = read_vector<int32_t>(a, at::kInt, &R);
  const int32_t* table = read_table(a, R, &cols);
  const uint8_t* gone = a.data<uint8_t>(at::kByte, {R});
  int32_t* free_pages = read_vector<int32_t>(a, at::kInt, &F);
  const int32_t* n_free = a.data<int32_t>(at::kInt, {1});
  const int page = a.number();
  const int64_t n_pages = a.integer(INT64_MIN, INT64_MAX);
  int32_t* seq_out = a.data<int32_t>(at::kInt, {R});
  int32_t* n_out = a.data<int32_t>(at::kInt, {1});
  uint32_t* status = a.status();
  if (!a.done() || R > INT32_MAX) return result(kExplain);
  return on_device(a.dev, [&](cudaStream_t stream) {
    return (long)csa2_paged_release(seq, table, gone, (int)R, page, cols, free_pages, F, n_free, n_pages, seq_out, n_out,
                                    status, stream);
  });
}

PyObject* kv8_append(PyObject* const* argv, Py_ssize_t argc) {
  Args a{argv, argc};
  int64_t T = 0, k_stride = 0, v_stride = 0;
  const at::Tensor *k = a.tensor(), *v = a.tensor();
  const int64_t* slot = read_vector<int64_t>(a, at::kLong, &T);
  Cache c;
  if (!read_cache(a, c)) return result(kExplain);
  const at::ScalarType type = k->scalar_type();
  const int kind = kind_of(type);
  const void* kp = a.tokens(k, type, T, c.Hk, c.hd, &k_stride);
  const void* vp = a.tokens(v, type, T, c.Hk, c.hd, &v_stride);
  uint32_t* status = a.status();
  if (!a.done() || kind < 0) return result(kExplain);
  return on_device(a.dev, [&](cudaStream_t stream) {
    return (long)csa2_kv8_append(kp, vp, k_stride, v_stride, kind, T, (int)c.Hk, (int)c.hd, slot, c.k, c.v, c.ks, c.vs,
                                 c.pages, (int)c.page, status, stream);
  });
}

PyObject* kv8_attn(PyObject* const* argv, Py_ssize_t argc) {
  Args a{argv, argc};
  const at::Tensor* q = a.tensor();
  Cache c;
  if (!read_cache(a, c) || q->dim() != 3) return result(kExplain);
  const int64_t T = q->size(0), Hq = q->size(1);
  const at::ScalarType type = q->scalar_type();
  const int kind = kind_of(type);
  int64_t R = 0, q_stride = 0;
  int cols = 0;
  const void* qp = a.tokens(q, type, T, Hq, c.hd, &q_stride);
  // block_table, q_start, seq_len: the last one's length counts
  if (a.ok && a.n - a.at >= 3 && THPVariable_Check(a.arg[a.at + 2])) {
    const at::Tensor& s = THPVariable_Unpack(a.arg[a.at + 2]);
    if (s.dim() == 1) R = s.size(0);
  }
  const int32_t* table = read_table(a, R, &cols);
  const int32_t* q_start = a.data<int32_t>(at::kInt, {R + 1});
  const int32_t* seq = a.data<int32_t>(at::kInt, {R});
  const float scale = a.real();
  void* out = a.data<void>(type, {T, Hq, c.hd});
  float* lse = nullptr;
  if (a.ok && a.at < a.n && a.arg[a.at] == Py_None) ++a.at;
  else lse = a.data<float>(at::kFloat, {T, Hq});
  const int max_q = a.number(), window = a.number();
  const float softcap = a.real();
  at::Tensor ws;
  if (a.ok && a.at < a.n && a.arg[a.at] == Py_None) {
    ++a.at;
  } else if (const at::Tensor* t = a.tensor()) {
    if (t->scalar_type() != at::kByte || !t->is_cuda() || t->get_device() != a.dev || !t->is_contiguous()) a.ok = false;
    else ws = *t;
  }
  uint32_t* status = a.status();
  if (!a.done() || kind < 0 || R > INT32_MAX || Hq > INT32_MAX) return result(kExplain);
  return on_device(a.dev, [&](cudaStream_t stream) {
    if (!ws.defined()) {  // from the current stream's pool, so it is not handed out before the kernels are done
      const size_t need = csa2_kv8_attn_workspace_size((int)Hq, (int)c.Hk, (int)c.hd, max_q, kind);
      ws = at::empty({(int64_t)(need > 0 ? need : 1)}, q->options().dtype(at::kByte));
    }
    return (long)csa2_kv8_attn(qp, q_stride, kind, T, (int)Hq, (int)c.Hk, (int)c.hd, c.k, c.v, c.ks, c.vs, c.pages,
                               (int)c.page, table, cols, q_start, seq, (int)R, max_q, scale, window, softcap, out, lse,
                               ws.data_ptr(), (size_t)ws.numel(), status, stream);
  });
}

// What torch throws (a tensor without storage or strides, no memory) is asked again, and
// reported, by csa2.py.
template <PyObject* (*F)(PyObject* const*, Py_ssize_t)>
PyObject* guarded(PyObject*, PyObject* const* argv, Py_ssize_t argc) {
  try {
    return F(argv, argc);
  } catch (...) {
    return result(kExplain);
  }
}

PyMethodDef methods[] = {
    {"paged_plan", (PyCFunction)(void (*)(void))guarded<paged_plan>, METH_FASTCALL, nullptr},
    {"paged_release", (PyCFunction)(void (*)(void))guarded<paged_release>, METH_FASTCALL, nullptr},
    {"kv8_append", (PyCFunction)(void (*)(void))guarded<kv8_append>, METH_FASTCALL, nullptr},
    {"kv8_attn", (PyCFunction)(void (*)(void))guarded<kv8_attn>, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native(void) { return PyModule_Create(&module); }
