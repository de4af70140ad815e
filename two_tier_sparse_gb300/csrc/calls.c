/* The plain case of a serving call from Python: dsa_plan_step, dsa_norm_rope, dsa_kv_write and
 * dsa_kv_read on the current stream with contiguous tensors of the right types, shapes
 * and device. Each function checks that in C, makes the call and returns its status; for
 * anything else it returns None, and the binding's own code then refuses the arguments or makes the
 * call. (A small call's kernel takes 2 - 5 us. Checked in Python and passed by ctypes the calls took
 * 4.2 - 4.9 us of the host, 1.7 of them the launch; this way 2.9 - 3.6.) */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "dsa.h"

typedef dsa_status_t (*plan_fn)(const dsa_config_t*, int, const int32_t*, const int32_t*,
                                const dsa_page_pool_t*, const dsa_step_plan_t*, void*, size_t,
                                dsa_stream_t);
typedef dsa_status_t (*norm_fn)(int, const int32_t*, const int32_t*, dsa_dtype_t,
                                const dsa_heads_t*, int, const dsa_rope_t*, dsa_stream_t);
typedef dsa_status_t (*write_fn)(const dsa_config_t*, int, const int32_t*, const void*, int64_t,
                                 const int32_t*, void*, int64_t, void*, size_t, dsa_stream_t);
typedef dsa_status_t (*read_fn)(const dsa_config_t*, int, const int32_t*, const void*, int64_t,
                                const int32_t*, void*, int64_t, void*, size_t, dsa_stream_t);

static plan_fn f_plan;
static norm_fn f_norm;
static write_fn f_write;
static read_fn f_read;
/* torch's dtypes, its current device and a device's current stream */
static PyObject *t_int32, *t_bf16, *t_int16, *get_device_fn, *raw_stream_fn;
static PyObject *n_shape, *n_dtype, *n_contiguous, *n_device, *n_ptr, *n_nbytes, *n_itemsize;

/* A number from a method or attribute; -1 if there is none (the error is dropped). */
static int64_t number(PyObject* r) {
  int64_t v = -1;
  if (r != NULL) {
    v = PyLong_AsLongLong(r);
    Py_DECREF(r);
  }
  if (PyErr_Occurred()) {
    PyErr_Clear();
    v = -1;
  }
  return v;
}
static int64_t method(PyObject* t, PyObject* name) {
  PyObject* args[2] = {NULL, t}; /* (a vectorcall may use the slot before its arguments) */
  return number(
      PyObject_VectorcallMethod(name, args + 1, 1 | PY_VECTORCALL_ARGUMENTS_OFFSET, NULL));
}

/* What a call needs of a contiguous tensor of a device; 0 if it is not one. */
typedef struct {
  PyObject* dtype; /* borrowed: torch's dtypes live on */
  int dim;
  int64_t size[2]; /* first and last */
  void* ptr;
} tensor_t;
static int tensor(PyObject* t, int64_t dev, tensor_t* out) {
  PyObject* args[2] = {NULL, t};
  PyObject* r = PyObject_VectorcallMethod(n_contiguous, args + 1,
                                          1 | PY_VECTORCALL_ARGUMENTS_OFFSET, NULL);
  const int contiguous = r == Py_True;
  Py_XDECREF(r);
  PyObject* dtype = contiguous ? PyObject_GetAttr(t, n_dtype) : NULL;
  PyObject* shape = dtype ? PyObject_GetAttr(t, n_shape) : NULL;
  int ok = 0;
  if (shape != NULL && PyTuple_Check(shape) && PyTuple_GET_SIZE(shape) >= 1) {
    out->dim = (int)PyTuple_GET_SIZE(shape);
    out->size[0] = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, 0));
    out->size[1] = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, out->dim - 1));
    out->dtype = dtype;
    ok = 1;
  }
  Py_XDECREF(dtype);
  Py_XDECREF(shape);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    return 0;
  }
  if (!ok) return 0;
  if (method(t, n_device) != dev) return 0;
  const int64_t p = method(t, n_ptr);
  out->ptr = (void*)(intptr_t)p;
  return p >= 0;
}
/* An int32 tensor of n elements in one dimension. */
static int int32s(PyObject* t, int64_t dev, int64_t n, const int32_t** p) {
  tensor_t x;
  if (!tensor(t, dev, &x) || x.dtype != t_int32 || x.dim != 1 || x.size[0] != n) return 0;
  *p = (const int32_t*)x.ptr;
  return 1;
}

/* The current stream of the tensor's device, which has to be the current device. */
static int current(PyObject* t, int64_t* dev, dsa_stream_t* stream) {
  *dev = method(t, n_device);
  if (*dev < 0 || number(PyObject_CallNoArgs(get_device_fn)) != *dev) return 0;
  PyObject* d = PyLong_FromLongLong(*dev);
  if (d == NULL) {
    PyErr_Clear();
    return 0;
  }
  PyObject* r = PyObject_CallOneArg(raw_stream_fn, d);
  Py_DECREF(d);
  if (r == NULL) {
    PyErr_Clear();
    return 0;
  }
  *stream = PyLong_AsVoidPtr(r);
  Py_DECREF(r);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    return 0;
  }
  return 1;
}

/* A workspace's address and bytes. */
static int workspace(PyObject* ws, int64_t dev, void** p, size_t* bytes) {
  if (method(ws, n_device) != dev) return 0;
  const int64_t b = number(PyObject_GetAttr(ws, n_nbytes)), at = method(ws, n_ptr);
  *p = (void*)(intptr_t)at;
  *bytes = (size_t)b;
  return b >= 0 && at >= 0;
}
/* The dsa_config_t that a ctypes structure holds. */
static int config(PyObject* o, const dsa_config_t** c) {
  Py_buffer b;
  if (PyObject_GetBuffer(o, &b, PyBUF_SIMPLE) != 0) {
    PyErr_Clear();
    return 0;
  }
  const int ok = b.len == (Py_ssize_t)sizeof(dsa_config_t);
  *c = (const dsa_config_t*)b.buf;
  PyBuffer_Release(&b); /* (the structure lives as long as the call's argument) */
  return ok;
}

/* rows(write, cfg, rows, slots, cache, ws, n_valid) */
static PyObject* rows_call(PyObject* self, PyObject* const* a, Py_ssize_t n_args) {
  (void)self;
  if (n_args != 7) Py_RETURN_NONE;
  int64_t dev;
  dsa_stream_t stream;
  const dsa_config_t* c;
  tensor_t rows, cache;
  const int32_t *slots, *valid = NULL;
  void* ws;
  size_t ws_bytes;
  if (!current(a[2], &dev, &stream) || !config(a[1], &c) || !tensor(a[2], dev, &rows) ||
      rows.dim != 2 || rows.size[1] != 512 || (rows.dtype != t_bf16 && rows.dtype != t_int16) ||
      !int32s(a[3], dev, rows.size[0], &slots) || !tensor(a[4], dev, &cache) ||
      !workspace(a[5], dev, &ws, &ws_bytes) ||
      (a[6] != Py_None && !int32s(a[6], dev, 1, &valid))) {
    Py_RETURN_NONE;
  }
  const int64_t row = c->kv_fmt == DSA_KV_BF16       ? 1024
                      : c->kv_fmt == DSA_KV_FP8_E4M3 ? 512
                      : c->kv_fmt == DSA_KV_MXFP4    ? 272
                                                     : 0;
  const int64_t item = number(PyObject_GetAttr(a[4], n_itemsize));
  const int64_t bytes = number(PyObject_GetAttr(a[4], n_nbytes));
  if (row == 0 || item < 1 || bytes < 0 || cache.size[1] * item != row ||
      rows.size[0] > INT32_MAX) {
    Py_RETURN_NONE;
  }
  const int n = (int)rows.size[0];
  const int write = a[0] == Py_True;
  dsa_status_t code;
  Py_BEGIN_ALLOW_THREADS;
  code = write ? f_write(c, n, valid, rows.ptr, 512, slots, cache.ptr, bytes / row, ws, ws_bytes,
                         stream)
               : f_read(c, n, valid, cache.ptr, bytes / row, slots, rows.ptr, 512, ws, ws_bytes,
                        stream);
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong((long)code);
}

/* The integers of a tuple that a handle keeps. */
static int key(PyObject* t, int n, int64_t* out) {
  if (!PyTuple_Check(t) || PyTuple_GET_SIZE(t) != n) return 0;
  for (int i = 0; i < n; ++i) out[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(t, i));
  if (PyErr_Occurred()) {
    PyErr_Clear();
    return 0;
  }
  return 1;
}

/* plan(cfg, n_tokens, n_new, pool key, plan key, ws); a key: (address, requests, device) */
static PyObject* plan_call(PyObject* self, PyObject* const* a, Py_ssize_t n_args) {
  (void)self;
  if (n_args != 6) Py_RETURN_NONE;
  int64_t dev, pool[3], plan[3];
  dsa_stream_t stream;
  const dsa_config_t* c;
  const int32_t *n_tokens, *n_new;
  void* ws;
  size_t ws_bytes;
  if (!current(a[1], &dev, &stream) || !config(a[0], &c) || !key(a[3], 3, pool) ||
      !key(a[4], 3, plan) || pool[2] != dev || plan[2] != dev || pool[1] != plan[1] ||
      !int32s(a[1], dev, plan[1], &n_tokens) || !int32s(a[2], dev, plan[1], &n_new) ||
      !workspace(a[5], dev, &ws, &ws_bytes)) {
    Py_RETURN_NONE;
  }
  dsa_status_t code;
  Py_BEGIN_ALLOW_THREADS;
  code = f_plan(c, (int)plan[1], n_tokens, n_new, (const dsa_page_pool_t*)(intptr_t)pool[0],
                (const dsa_step_plan_t*)(intptr_t)plan[0], ws, ws_bytes, stream);
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong((long)code);
}

/* norm(positions, x of the first group, heads key, rope key or None, n_valid); heads key:
 * (address, groups, tokens, element type, device), rope key: (address, device) */
static PyObject* norm_call(PyObject* self, PyObject* const* a, Py_ssize_t n_args) {
  (void)self;
  if (n_args != 5) Py_RETURN_NONE;
  int64_t dev, heads[5], rope[2] = {0, 0};
  dsa_stream_t stream;
  const int32_t *positions = NULL, *valid = NULL;
  if (!current(a[1], &dev, &stream) || !key(a[2], 5, heads) || heads[4] != dev ||
      (a[3] != Py_None && (!key(a[3], 2, rope) || rope[1] != dev)) ||
      ((a[3] != Py_None || a[0] != Py_None) && !int32s(a[0], dev, heads[2], &positions)) ||
      (a[4] != Py_None && !int32s(a[4], dev, 1, &valid)) || heads[2] > INT32_MAX) {
    Py_RETURN_NONE;
  }
  dsa_status_t code;
  Py_BEGIN_ALLOW_THREADS;
  code = f_norm((int)heads[2], valid, positions, (dsa_dtype_t)heads[3],
                (const dsa_heads_t*)(intptr_t)heads[0], (int)heads[1],
                (const dsa_rope_t*)(intptr_t)rope[0], stream);
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong((long)code);
}

/* init(addresses of the four functions, (int32, bfloat16, int16), current device, raw stream) */
static PyObject* init(PyObject* self, PyObject* const* a, Py_ssize_t n_args) {
  (void)self;
  int64_t fn[4];
  if (n_args != 4 || !key(a[0], 4, fn) || !PyTuple_Check(a[1]) || PyTuple_GET_SIZE(a[1]) != 3) {
    PyErr_SetString(PyExc_ValueError, "init(functions, dtypes, current device, raw stream)");
    return NULL;
  }
  f_plan = (plan_fn)(intptr_t)fn[0];
  f_norm = (norm_fn)(intptr_t)fn[1];
  f_write = (write_fn)(intptr_t)fn[2];
  f_read = (read_fn)(intptr_t)fn[3];
  t_int32 = Py_NewRef(PyTuple_GET_ITEM(a[1], 0));
  t_bf16 = Py_NewRef(PyTuple_GET_ITEM(a[1], 1));
  t_int16 = Py_NewRef(PyTuple_GET_ITEM(a[1], 2));
  get_device_fn = Py_NewRef(a[2]);
  raw_stream_fn = Py_NewRef(a[3]);
  Py_RETURN_NONE;
}

static PyMethodDef methods[] = {
    {"init", (PyCFunction)(void (*)(void))init, METH_FASTCALL, NULL},
    {"rows", (PyCFunction)(void (*)(void))rows_call, METH_FASTCALL, NULL},
    {"plan", (PyCFunction)(void (*)(void))plan_call, METH_FASTCALL, NULL},
    {"norm", (PyCFunction)(void (*)(void))norm_call, METH_FASTCALL, NULL},
    {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", NULL, -1, methods,
                                    NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__calls(void) {
  n_shape = PyUnicode_InternFromString("shape");
  n_dtype = PyUnicode_InternFromString("dtype");
  n_contiguous = PyUnicode_InternFromString("is_contiguous");
  n_device = PyUnicode_InternFromString("get_device");
  n_ptr = PyUnicode_InternFromString("data_ptr");
  n_nbytes = PyUnicode_InternFromString("nbytes");
  n_itemsize = PyUnicode_InternFromString("itemsize");
  if (PyErr_Occurred()) return NULL;
  return PyModule_Create(&module);
}
