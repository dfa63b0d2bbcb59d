/*
 * CPython side of the binding for the calls of a decode step that follow one
 * another too quickly for ctypes: it turns torch tensors into kda_tensor
 * descriptors and calls the library.  Describing a tensor takes 0.3 us here
 * and 1.1 us through ctypes on the Grace host, of 7 to 11 a call, where the
 * kernels of a small step run for 2 to 8 us.
 *
 * It knows torch only through the attributes every tensor has (data_ptr,
 * dtype, shape, stride) and the library only through the addresses that
 * bind() is given, so it links against neither.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <string.h>

#include "../../include/kda.h"

static PyObject *s_shape, *s_stride, *s_dtype, *s_data_ptr, *s_get_device;
static PyObject* dtypes[3]; /* torch.float32, torch.bfloat16, torch.int32, in kda_dtype order */

static int64_t as_int(PyObject* o, int* bad) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) *bad = 1;
  return (int64_t)v;
}

/* Fills *d from tensor t of CUDA device `device`; 0, or -1 with an exception set.  A tensor of the host or of another
 * device is refused: its address would mean something else, or nothing, to the kernels. */
static int describe(PyObject* t, kda_tensor* d, long device) {
  int bad = 0, i;
  long where;
  Py_ssize_t n;
  PyObject *dtype, *shape = NULL, *stride = NULL, *ptr = NULL, *at;
  memset(d, 0, sizeof(*d));
  at = PyObject_CallMethodNoArgs(t, s_get_device);
  if (at == NULL) return -1;
  where = PyLong_AsLong(at);
  Py_DECREF(at);
  if (where == -1 && PyErr_Occurred()) return -1;
  if (where != device) {
    if (where < 0)
      PyErr_Format(PyExc_ValueError, "expected every tensor on cuda:%ld, got one of the host", device);
    else
      PyErr_Format(PyExc_ValueError, "expected every tensor on cuda:%ld, got one on cuda:%ld", device, where);
    return -1;
  }
  dtype = PyObject_GetAttr(t, s_dtype);
  if (dtype == NULL) return -1;
  d->dtype = -1;
  for (i = 0; i < 3; ++i)
    if (dtype == dtypes[i]) d->dtype = i;
  if (d->dtype < 0) {
    PyErr_Format(PyExc_TypeError, "unsupported dtype %S", dtype);
    Py_DECREF(dtype);
    return -1;
  }
  Py_DECREF(dtype);
  shape = PyObject_GetAttr(t, s_shape);
  stride = shape != NULL ? PyObject_CallMethodNoArgs(t, s_stride) : NULL;
  ptr = stride != NULL ? PyObject_CallMethodNoArgs(t, s_data_ptr) : NULL;
  if (ptr == NULL) {
    bad = 1;
  } else if (!PyTuple_Check(shape) || !PyTuple_Check(stride) || PyTuple_GET_SIZE(shape) != PyTuple_GET_SIZE(stride)) {
    PyErr_SetString(PyExc_TypeError, "expected a strided tensor");
    bad = 1;
  } else if ((n = PyTuple_GET_SIZE(shape)) < 1 || n > 4) {
    PyErr_Format(PyExc_ValueError, "rank %zd not in 1..4", n);
    bad = 1;
  } else {
    int64_t numel = 1;
    d->ndim = (int32_t)n;
    for (i = 0; i < (int)n; ++i) {
      d->shape[i] = as_int(PyTuple_GET_ITEM(shape, i), &bad);
      d->stride[i] = as_int(PyTuple_GET_ITEM(stride, i), &bad);
      if (d->shape[i] == 0) numel = 0;
    }
    if (numel != 0) {
      d->data = PyLong_AsVoidPtr(ptr);
      if (d->data == NULL && PyErr_Occurred()) bad = 1;
    }
  }
  Py_XDECREF(shape);
  Py_XDECREF(stride);
  Py_XDECREF(ptr);
  return bad ? -1 : 0;
}

/* Describes the first n arguments into d; p[i] is NULL for None. */
static int describe_all(PyObject* const* args, Py_ssize_t n, kda_tensor* d, const kda_tensor** p, long device) {
  Py_ssize_t i;
  for (i = 0; i < n; ++i) {
    p[i] = NULL;
    if (args[i] == Py_None) continue;
    if (describe(args[i], &d[i], device) != 0) return -1;
    p[i] = &d[i];
  }
  return 0;
}

static int int32_of(PyObject* o, int32_t* out) {
  int overflow = 0;
  const long v = PyLong_AsLongAndOverflow(o, &overflow);
  if (v == -1 && PyErr_Occurred()) return -1;
  if (overflow != 0 || v > INT32_MAX || v < INT32_MIN) {
    PyErr_SetString(PyExc_OverflowError, "argument does not fit 32 bits");
    return -1;
  }
  *out = (int32_t)v;
  return 0;
}

static int float_of(PyObject* o, float* out) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) return -1;
  *out = (float)v;
  return 0;
}

static int device_of(PyObject* o, long* out) {
  *out = PyLong_AsLong(o);
  return *out == -1 && PyErr_Occurred() ? -1 : 0;
}

static int stream_of(PyObject* o, void** out) {
  *out = PyLong_AsVoidPtr(o); /* 0: the legacy default stream */
  return *out == NULL && PyErr_Occurred() ? -1 : 0;
}

static int arity(const char* name, Py_ssize_t got, Py_ssize_t want) {
  if (got == want) return 0;
  PyErr_Format(PyExc_TypeError, "%s takes %zd arguments, not %zd", name, want, got);
  return -1;
}

static struct {
  kda_status (*rope_append)(const kda_tensor*, const kda_tensor*, const kda_tensor*, const kda_tensor*, const kda_tensor*,
                            const kda_tensor*, const kda_tensor*, const kda_tensor*, const kda_tensor*,
                            const kda_tensor*, int32_t, float, void*);
  kda_status (*attention)(const kda_tensor*, const kda_tensor*, const kda_tensor*, const kda_tensor*, const kda_tensor*,
                          const kda_tensor*, int32_t, float, const kda_tensor*, const kda_tensor*, void*);
  kda_status (*beam)(const kda_tensor*, const kda_tensor*, const kda_tensor*, int32_t, const kda_tensor*,
                     const kda_tensor*, const kda_tensor*, const kda_tensor*, void*);
  kda_status (*move)(const kda_tensor* const*, int32_t, const kda_tensor*, const kda_tensor*, const kda_tensor*, void*);
} fn;

/* rope_append(q, k, v, phase_steps, cu_seqlens, seq_lens, page_table, k_pages, v_pages, q_out, interleaved, amplitude, stream, device) */
static PyObject* rope_append(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  kda_tensor d[10];
  const kda_tensor* p[10];
  int32_t interleaved;
  float amplitude;
  long device;
  void* stream;
  kda_status st;
  (void)self;
  if (arity("rope_append", n, 14) != 0 || device_of(args[13], &device) != 0 || describe_all(args, 10, d, p, device) != 0 ||
      int32_of(args[10], &interleaved) != 0 ||
      float_of(args[11], &amplitude) != 0 || stream_of(args[12], &stream) != 0)
    return NULL;
  Py_BEGIN_ALLOW_THREADS
  st = fn.rope_append(p[0], p[1], p[2], p[3], p[4], p[5], p[6], p[7], p[8], p[9], interleaved, amplitude, stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong((long)st);
}

/* attention(q, k_pages, v_pages, page_table, seq_lens, workspace, out, lse, window, scale, stream, device) */
static PyObject* attention(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  kda_tensor d[8];
  const kda_tensor* p[8];
  int32_t window;
  float scale;
  long device;
  void* stream;
  kda_status st;
  (void)self;
  if (arity("attention", n, 12) != 0 || device_of(args[11], &device) != 0 || describe_all(args, 8, d, p, device) != 0 ||
      int32_of(args[8], &window) != 0 ||
      float_of(args[9], &scale) != 0 || stream_of(args[10], &stream) != 0)
    return NULL;
  Py_BEGIN_ALLOW_THREADS
  st = fn.attention(p[0], p[1], p[2], p[3], p[4], p[5], window, scale, p[6], p[7], stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong((long)st);
}

/* beam(logits, scores, finished, workspace, out_scores, out_parents, out_tokens, eos_token, stream, device) */
static PyObject* beam(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  kda_tensor d[7];
  const kda_tensor* p[7];
  int32_t eos;
  long device;
  void* stream;
  kda_status st;
  (void)self;
  if (arity("beam", n, 10) != 0 || device_of(args[9], &device) != 0 || describe_all(args, 7, d, p, device) != 0 ||
      int32_of(args[7], &eos) != 0 ||
      stream_of(args[8], &stream) != 0)
    return NULL;
  Py_BEGIN_ALLOW_THREADS
  st = fn.beam(p[0], p[1], p[2], eos, p[3], p[4], p[5], p[6], stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong((long)st);
}

/* move(pools, src_slots, dst_slots, parents, stream, device); pools a list or tuple of at most 256 tensors (more are refused
 * by the library, from the count alone) */
static PyObject* move(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  enum { MOST = 256 };
  kda_tensor d[3], pool[MOST];
  const kda_tensor *p[3], *pools[MOST];
  PyObject* list;
  Py_ssize_t count, i;
  long device;
  void* stream;
  kda_status st;
  (void)self;
  if (arity("move", n, 6) != 0 || device_of(args[5], &device) != 0) return NULL;
  list = args[0];
  if (!PyList_Check(list) && !PyTuple_Check(list)) { /* a tensor would pass for the sequence of its rows */
    PyErr_SetString(PyExc_TypeError, "pools must be a list or tuple of tensors");
    return NULL;
  }
  count = PySequence_Fast_GET_SIZE(list);
  for (i = 0; i < count && i < MOST; ++i) {
    if (describe(PySequence_Fast_GET_ITEM(list, i), &pool[i], device) != 0) return NULL;
    pools[i] = &pool[i];
  }
  if (describe_all(args + 1, 3, d, p, device) != 0 || stream_of(args[4], &stream) != 0) return NULL;
  Py_BEGIN_ALLOW_THREADS
  st = fn.move(pools, count > MOST ? MOST + 1 : (int32_t)count, p[0], p[1], p[2], stream);
  Py_END_ALLOW_THREADS
  return PyLong_FromLong((long)st);
}

/* bind((rope_append, attention, beam, move) addresses, (float32, bfloat16, int32)) */
static PyObject* bind(PyObject* self, PyObject* const* args, Py_ssize_t n) {
  int i;
  void* address[4];
  (void)self;
  if (arity("bind", n, 2) != 0) return NULL;
  if (!PyTuple_Check(args[0]) || PyTuple_GET_SIZE(args[0]) != 4 || !PyTuple_Check(args[1]) ||
      PyTuple_GET_SIZE(args[1]) != 3) {
    PyErr_SetString(PyExc_TypeError, "bind takes four addresses and three dtypes");
    return NULL;
  }
  for (i = 0; i < 4; ++i) {
    address[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(args[0], i));
    if (address[i] == NULL) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null address");
      return NULL;
    }
  }
  memcpy(&fn.rope_append, &address[0], sizeof(void*));
  memcpy(&fn.attention, &address[1], sizeof(void*));
  memcpy(&fn.beam, &address[2], sizeof(void*));
  memcpy(&fn.move, &address[3], sizeof(void*));
  for (i = 0; i < 3; ++i) {
    Py_INCREF(PyTuple_GET_ITEM(args[1], i));
    Py_XSETREF(dtypes[i], PyTuple_GET_ITEM(args[1], i));
  }
  Py_RETURN_NONE;
}

#define METHOD(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {METHOD(rope_append), METHOD(attention), METHOD(beam), METHOD(move), METHOD(bind),
                                {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_kda_python", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__kda_python(void) {
  s_shape = PyUnicode_InternFromString("shape");
  s_stride = PyUnicode_InternFromString("stride");
  s_dtype = PyUnicode_InternFromString("dtype");
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  s_get_device = PyUnicode_InternFromString("get_device");
  if (s_shape == NULL || s_stride == NULL || s_dtype == NULL || s_data_ptr == NULL || s_get_device == NULL) return NULL;
  return PyModule_Create(&module);
}
