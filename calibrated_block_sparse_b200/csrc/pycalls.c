/* Calls of the streaming entry points from Python without ctypes' conversion
 * of some twenty arguments: 0.3 us instead of 2.2 us of a call that takes 10.
 * The functions are those of the loaded libcalibatt, given by address; the
 * binding uses ctypes where this module was not built. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "calibatt.h"

typedef int (*rope_fn)(const calibatt_rope_plan*, const calibatt_bf16*, int64_t, int64_t, int, const calibatt_bf16*,
                       int64_t, int64_t, int, int64_t, int, const int32_t*, int, int, const int32_t*, calibatt_bf16*,
                       int64_t, int64_t, calibatt_bf16*, int64_t, int64_t, calibatt_stream_t);
typedef int (*write_fn)(const calibatt_bf16*, int64_t, int64_t, const calibatt_bf16*, int64_t, int64_t, int, int, int,
                        const int32_t*, const int32_t*, int, int, const int32_t*, int, int, uint8_t*, uint8_t*, float*,
                        float*, calibatt_stream_t);
typedef int (*attn_fn)(const calibatt_bf16*, int, int, int, int, float, int, const int32_t*, const int32_t*, int, int,
                       int, const int32_t*, int, int, const uint8_t*, const uint8_t*, const float*, const float*,
                       calibatt_bf16*, float*, void*, size_t, calibatt_stream_t);

/* Integers and addresses (None: 0) of a call, but for argument `other`; 0 with an exception set on failure. */
static int take(PyObject* const* args, Py_ssize_t n, Py_ssize_t want, long long* v, Py_ssize_t other) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "%zd arguments, %zd expected", n, want);
    return 0;
  }
  for (Py_ssize_t i = 0; i < n; ++i) {
    v[i] = 0;
    if (args[i] == Py_None || i == other) continue;
    v[i] = PyLong_AsLongLong(args[i]);
    if (v[i] == -1 && PyErr_Occurred()) return 0;
  }
  return 1;
}

/* An int argument of the C call: what does not fit becomes one that is refused. */
static int small(long long x) { return x > INT32_MAX || x < INT32_MIN ? INT32_MIN : (int)x; }

#define PTR(T, x) ((T*)(intptr_t)(x))

static PyObject* rope(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  long long v[24];
  (void)self;
  if (!take(a, n, 24, v, -1)) return NULL;
  for (int i = 14; i < 17; ++i)
    if (v[i] != small(v[i])) {
      PyErr_SetString(PyExc_OverflowError, "a start that does not fit 32 bits");
      return NULL;
    }
  const int32_t start[3] = {small(v[14]), small(v[15]), small(v[16])};
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = ((rope_fn)(intptr_t)v[0])(PTR(const calibatt_rope_plan, v[1]), PTR(const calibatt_bf16, v[2]), v[3], v[4],
                                 small(v[5]), PTR(const calibatt_bf16, v[6]), v[7], v[8], small(v[9]), v[10],
                                 CALIBATT_HEAD_DIM, PTR(const int32_t, v[11]), small(v[12]), small(v[13]), start,
                                 PTR(calibatt_bf16, v[17]), v[18], v[19], PTR(calibatt_bf16, v[20]), v[21], v[22],
                                 PTR(struct CUstream_st, v[23]));
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(rc);
}

static PyObject* cache_write(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  long long v[21];
  (void)self;
  if (!take(a, n, 21, v, -1)) return NULL;
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = ((write_fn)(intptr_t)v[0])(PTR(const calibatt_bf16, v[1]), v[2], v[3], PTR(const calibatt_bf16, v[4]), v[5],
                                  v[6], small(v[7]), small(v[8]), CALIBATT_HEAD_DIM, PTR(const int32_t, v[9]),
                                  PTR(const int32_t, v[10]), small(v[11]), small(v[12]), PTR(const int32_t, v[13]),
                                  small(v[14]), small(v[15]), PTR(uint8_t, v[16]), PTR(uint8_t, v[17]),
                                  PTR(float, v[18]), PTR(float, v[19]), PTR(struct CUstream_st, v[20]));
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(rc);
}

static PyObject* cache_attn(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  long long v[24];
  (void)self;
  if (!take(a, n, 24, v, 5)) return NULL;
  const double scale = PyFloat_AsDouble(a[5]);
  if (scale == -1.0 && PyErr_Occurred()) return NULL;
  int rc;
  Py_BEGIN_ALLOW_THREADS;
  rc = ((attn_fn)(intptr_t)v[0])(PTR(const calibatt_bf16, v[1]), small(v[2]), small(v[3]), small(v[4]),
                                 CALIBATT_HEAD_DIM, (float)scale, small(v[6]), PTR(const int32_t, v[7]),
                                 PTR(const int32_t, v[8]), small(v[9]), small(v[10]), small(v[11]),
                                 PTR(const int32_t, v[12]), small(v[13]), small(v[14]), PTR(const uint8_t, v[15]),
                                 PTR(const uint8_t, v[16]), PTR(const float, v[17]), PTR(const float, v[18]),
                                 PTR(calibatt_bf16, v[19]), PTR(float, v[20]), PTR(void, v[21]), (size_t)v[22],
                                 PTR(struct CUstream_st, v[23]));
  Py_END_ALLOW_THREADS;
  return PyLong_FromLong(rc);
}

static PyMethodDef methods[] = {
    {"rope", (PyCFunction)(void (*)(void))rope, METH_FASTCALL, "calibatt_rope_fwd or _bwd, by address"},
    {"cache_write", (PyCFunction)(void (*)(void))cache_write, METH_FASTCALL, "calibatt_cache_write, by address"},
    {"cache_attn", (PyCFunction)(void (*)(void))cache_attn, METH_FASTCALL, "calibatt_cache_attn_fwd, by address"},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pycalls", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__pycalls(void) { return PyModule_Create(&module); }
