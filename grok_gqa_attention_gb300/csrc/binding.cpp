// The checks and the call of the functions over parts of a paged cache, for the Python
// binding (sparse.py), whose own checks cost as much time as a decode step's short
// kernels: 0.6 us a tensor, 3.7 us for the bounds of a step's blocks, which the GPU makes
// in 3.5 us. Python.h only: a tensor is asked for its type, shape, device, layout and
// address by the same names as in Python.
//
// Each function returns the library's status, or None where something is not as it should
// be (another type, shape or device, not contiguous, not the current device): the caller
// then goes through its own checks, which say what.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <climits>

#include "grok_attn.h"

namespace {

PyObject *s_dtype, *s_shape, *s_get_device, *s_is_contiguous, *s_data_ptr, *s_cuda_stream, *s_device, *s_index;
PyObject *t_bf16, *t_f32, *t_i32, *t_i8, *t_u8;      // torch's types
PyObject *f_device, *f_stream;                       // the current device; a device's current stream
decltype(&grok_kv_bounds_paged) c_bounds;
decltype(&grok_attn_select_paged) c_select;
decltype(&grok_attn_decode_sparse_paged) c_sparse;
decltype(&grok_attn_decode_shared_paged) c_shared;

// The value of a Python integer, which is released; false for anything else.
bool take_int(PyObject* o, long long* v) {
  if (!o) return PyErr_Clear(), false;
  *v = PyLong_Check(o) ? PyLong_AsLongLong(o) : (PyErr_SetNone(PyExc_TypeError), -1);
  Py_DECREF(o);
  if (*v == -1 && PyErr_Occurred()) return PyErr_Clear(), false;
  return true;
}
bool to_int(PyObject* o, int* v) {
  long long x;
  Py_INCREF(o);
  if (!take_int(o, &x) || x < INT_MIN || x > INT_MAX) return false;
  *v = int(x);
  return true;
}

struct Call {
  long long at = -1;  // the device of the tensors so far
  // A contiguous CUDA tensor of this type and shape, on the same device as those before it. An extent of -1 is set.
  bool tensor(PyObject* t, PyObject* dtype, int nd, long long* shape, void** ptr) {
    PyObject* o = PyObject_GetAttr(t, s_dtype);
    if (!o) return PyErr_Clear(), false;
    const bool type = o == dtype;
    Py_DECREF(o);
    if (!type) return false;
    if (!(o = PyObject_GetAttr(t, s_shape))) return PyErr_Clear(), false;
    bool fits = PyTuple_Check(o) && PyTuple_GET_SIZE(o) == nd;
    for (int i = 0; fits && i < nd; ++i) {
      const long long n = PyLong_AsLongLong(PyTuple_GET_ITEM(o, i));
      if (n < 0) PyErr_Clear();
      if (shape[i] < 0) shape[i] = n;
      fits = n >= 0 && shape[i] == n;
    }
    Py_DECREF(o);
    if (!fits) return false;
    long long dev, address;
    if (!take_int(PyObject_CallMethodNoArgs(t, s_get_device), &dev) || dev < 0 || (at >= 0 && dev != at)) return false;
    at = dev;
    if (!(o = PyObject_CallMethodNoArgs(t, s_is_contiguous))) return PyErr_Clear(), false;
    const bool packed = o == Py_True;
    Py_DECREF(o);
    if (!packed || !take_int(PyObject_CallMethodNoArgs(t, s_data_ptr), &address)) return false;
    *ptr = reinterpret_cast<void*>(address);
    return true;
  }
  bool optional(PyObject* t, PyObject* dtype, int nd, long long* shape, void** ptr) {
    *ptr = nullptr;
    return t == Py_None || tensor(t, dtype, nd, shape, ptr);
  }
  bool vector(PyObject* t, PyObject* dtype, long long n, void** ptr) { return tensor(t, dtype, 1, &n, ptr); }
  bool status(PyObject* t, int32_t** ptr) {
    long long one = 1;
    return optional(t, t_i32, 1, &one, reinterpret_cast<void**>(ptr));
  }
  bool table(PyObject* t, long long B, long long* max_pages, void** ptr) {
    long long shape[2] = {B, -1};
    const bool ok = tensor(t, t_i32, 2, shape, ptr);
    *max_pages = shape[1];
    return ok && *max_pages <= INT_MAX;
  }
  bool pool(PyObject* t, long long* n, void** ptr) {
    long long shape[4] = {*n, GROK_PAGE_TOKENS, GROK_N_KV_HEADS, GROK_HEAD_DIM};
    const bool ok = tensor(t, t_bf16, 4, shape, ptr);
    *n = shape[0];
    return ok && *n <= INT_MAX;
  }
  bool heads(PyObject* t, long long* B, void** ptr) {
    long long shape[3] = {*B, GROK_N_Q_HEADS, GROK_HEAD_DIM};
    const bool ok = tensor(t, t_bf16, 3, shape, ptr);
    *B = shape[0];
    return ok && *B <= INT_MAX;
  }
  bool bounds(PyObject* codes, PyObject* scale, long long* n, void** c, void** s) {
    long long cs[5] = {*n, GROK_PAGE_TOKENS / GROK_SPARSE_BLOCK, GROK_N_KV_HEADS, 2, GROK_HEAD_DIM};
    const bool ok = tensor(codes, t_i8, 5, cs, c);
    *n = cs[0];
    long long ss[3] = {*n, GROK_PAGE_TOKENS / GROK_SPARSE_BLOCK, GROK_N_KV_HEADS};
    return ok && *n <= INT_MAX && tensor(scale, t_f32, 3, ss, s);
  }
  // The stream to launch on: `given`, or the device's current one; the device has to be the current one.
  bool stream(PyObject* given, void** out) {
    long long dev, s;
    if (!take_int(PyObject_CallNoArgs(f_device), &dev) || dev != at) return false;
    if (given == Py_None) {
      PyObject* index = PyLong_FromLongLong(at);
      if (!index) return PyErr_Clear(), false;
      const bool ok = take_int(PyObject_CallOneArg(f_stream, index), &s);
      Py_DECREF(index);
      if (!ok) return false;
    } else {
      PyObject* d = PyObject_GetAttr(given, s_device);
      if (!d) return PyErr_Clear(), false;
      const bool here = take_int(PyObject_GetAttr(d, s_index), &dev) && dev == at;
      Py_DECREF(d);
      if (!here || !take_int(PyObject_GetAttr(given, s_cuda_stream), &s)) return false;
    }
    *out = reinterpret_cast<void*>(s);
    return true;
  }
};

#define RUN(call)        \
  grok_status st;        \
  Py_BEGIN_ALLOW_THREADS \
  st = call;             \
  Py_END_ALLOW_THREADS   \
  return PyLong_FromLong(st)

// (k_pool, block_table, start_pos, valid_len, T, codes, scale, dev_status, stream)
PyObject* bounds(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  Call c;
  long long n = -1, B = -1, mp, m;
  void *k, *table, *start, *valid, *codes, *scale, *stream;
  int32_t* status;
  int T;
  if (n_args != 9 || !c.pool(a[0], &n, &k) || !c.tensor(a[2], t_i32, 1, &B, &start) || B > INT_MAX ||
      !c.table(a[1], B, &mp, &table) || !c.optional(a[3], t_i32, 1, &B, &valid) || !to_int(a[4], &T) ||
      (m = n, !c.bounds(a[5], a[6], &m, &codes, &scale)) || !c.status(a[7], &status) || !c.stream(a[8], &stream))
    Py_RETURN_NONE;
  RUN(c_bounds(static_cast<grok_bf16*>(k), int(n), static_cast<int32_t*>(table), int(mp), static_cast<int32_t*>(start),
               static_cast<int32_t*>(valid), int(B), T, static_cast<int8_t*>(codes), static_cast<float*>(scale), status,
               stream));
}

// (q_rot, codes, scale, block_table, kv_len, sink, recent, score, sel, dev_status, stream)
PyObject* select(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  Call c;
  long long n = -1, B = -1, mp;
  void *q, *codes, *scale, *table, *len, *score, *sel, *stream;
  int32_t* status;
  int sink, recent;
  if (n_args != 11 || !c.heads(a[0], &B, &q) || !c.bounds(a[1], a[2], &n, &codes, &scale) ||
      !c.table(a[3], B, &mp, &table) || !c.vector(a[4], t_i32, B, &len) || !to_int(a[5], &sink) || !to_int(a[6], &recent))
    Py_RETURN_NONE;
  long long blocks[3] = {B, GROK_N_KV_HEADS, mp * (GROK_PAGE_TOKENS / GROK_SPARSE_BLOCK)};
  long long lists[3] = {B, GROK_N_KV_HEADS, -1};
  if (!c.tensor(a[7], t_f32, 3, blocks, &score) || !c.tensor(a[8], t_i32, 3, lists, &sel) || lists[2] > INT_MAX ||
      !c.status(a[9], &status) || !c.stream(a[10], &stream))
    Py_RETURN_NONE;
  RUN(c_select(static_cast<grok_bf16*>(q), static_cast<int8_t*>(codes), static_cast<float*>(scale), int(n),
               static_cast<int32_t*>(table), int(mp), static_cast<int32_t*>(len), int(B), int(lists[2]), sink, recent,
               static_cast<float*>(score), static_cast<int32_t*>(sel), status, stream));
}

// (q_rot, k_pool, v_pool, block_table, kv_len, sel, workspace, out, dev_status, stream)
PyObject* sparse(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  Call c;
  long long n = -1, B = -1, mp, bytes = -1;
  void *q, *k, *v, *table, *len, *sel, *ws, *out, *stream;
  int32_t* status;
  if (n_args != 10 || !c.heads(a[0], &B, &q) || !c.pool(a[1], &n, &k) || !c.pool(a[2], &n, &v) ||
      !c.table(a[3], B, &mp, &table) || !c.vector(a[4], t_i32, B, &len))
    Py_RETURN_NONE;
  long long lists[3] = {B, GROK_N_KV_HEADS, -1};
  if (!c.tensor(a[5], t_i32, 3, lists, &sel) || lists[2] > INT_MAX || !c.tensor(a[6], t_u8, 1, &bytes, &ws) ||
      !c.heads(a[7], &B, &out) || !c.status(a[8], &status) || !c.stream(a[9], &stream))
    Py_RETURN_NONE;
  RUN(c_sparse(static_cast<grok_bf16*>(q), static_cast<grok_bf16*>(k), static_cast<grok_bf16*>(v), int(n),
               static_cast<int32_t*>(table), int(mp), static_cast<int32_t*>(len), static_cast<int32_t*>(sel),
               int(lists[2]), int(B), ws, size_t(bytes), static_cast<grok_bf16*>(out), status, stream));
}

// (q_rot, k_pool, v_pool, block_table, kv_len, group_start, shared_pages, workspace, out, dev_status, stream)
PyObject* shared(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  Call c;
  long long n = -1, B = -1, mp, bytes = -1, groups = -1;
  void *q, *k, *v, *table, *len, *start, *pages, *ws, *out, *stream;
  int32_t* status;
  if (n_args != 11 || !c.heads(a[0], &B, &q) || !c.pool(a[1], &n, &k) || !c.pool(a[2], &n, &v) ||
      !c.table(a[3], B, &mp, &table) || !c.vector(a[4], t_i32, B, &len) || !c.tensor(a[6], t_i32, 1, &groups, &pages) ||
      groups > INT_MAX - 1 || !c.vector(a[5], t_i32, groups + 1, &start) || !c.tensor(a[7], t_u8, 1, &bytes, &ws) ||
      !c.heads(a[8], &B, &out) || !c.status(a[9], &status) || !c.stream(a[10], &stream))
    Py_RETURN_NONE;
  RUN(c_shared(static_cast<grok_bf16*>(q), static_cast<grok_bf16*>(k), static_cast<grok_bf16*>(v), int(n),
               static_cast<int32_t*>(table), int(mp), static_cast<int32_t*>(len), int(B), static_cast<int32_t*>(start),
               static_cast<int32_t*>(pages), int(groups), ws, size_t(bytes), static_cast<grok_bf16*>(out), status,
               stream));
}

// bind(bounds, select, sparse, shared, bf16, f32, i32, i8, u8, current device, current stream): the library's functions by
// address, torch's types and functions; before any other call.
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t n_args) {
  if (n_args != 11) return PyErr_Format(PyExc_TypeError, "bind takes 11 arguments, got %zd", n_args);
  void* f[4];
  for (int i = 0; i < 4; ++i)
    if (!(f[i] = PyLong_AsVoidPtr(a[i]))) return PyErr_Occurred() ? nullptr : PyErr_Format(PyExc_ValueError, "null function");
  c_bounds = reinterpret_cast<decltype(c_bounds)>(f[0]);
  c_select = reinterpret_cast<decltype(c_select)>(f[1]);
  c_sparse = reinterpret_cast<decltype(c_sparse)>(f[2]);
  c_shared = reinterpret_cast<decltype(c_shared)>(f[3]);
  PyObject** to[] = {&t_bf16, &t_f32, &t_i32, &t_i8, &t_u8, &f_device, &f_stream};
  for (int i = 0; i < 7; ++i) {
    Py_INCREF(a[4 + i]);
    Py_XDECREF(*to[i]);
    *to[i] = a[4 + i];
  }
  Py_RETURN_NONE;
}

template <typename F>
constexpr PyCFunction as_function(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f));
}

PyMethodDef methods[] = {{"bind", as_function(bind), METH_FASTCALL, nullptr},
                         {"kv_bounds_paged", as_function(bounds), METH_FASTCALL, nullptr},
                         {"select_blocks_paged", as_function(select), METH_FASTCALL, nullptr},
                         {"decode_sparse_paged", as_function(sparse), METH_FASTCALL, nullptr},
                         {"decode_shared_paged", as_function(shared), METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() {
  struct {
    PyObject** to;
    const char* name;
  } names[] = {{&s_dtype, "dtype"},       {&s_shape, "shape"},         {&s_get_device, "get_device"},
               {&s_data_ptr, "data_ptr"}, {&s_is_contiguous, "is_contiguous"}, {&s_cuda_stream, "cuda_stream"},
               {&s_device, "device"},     {&s_index, "index"}};
  for (auto& n : names)
    if (!(*n.to = PyUnicode_InternFromString(n.name))) return nullptr;
  return PyModule_Create(&module);
}
