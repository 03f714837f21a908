/*
 * mx_calls.c -- the host side of small calls of the microscaled operators: a CPython
 * module that looks at the tensors of a call (type, device, layout, sizes), through their
 * public methods, and calls the C ABI with their addresses on the current stream.
 *
 * A decode step's launches follow one another every few microseconds, and what the
 * interpreter and ctypes take for a call (2 to 4 us on the GB300's host) is more than
 * the launch itself (1.4 us).  Every function returns the status of the C call, or None where
 * something does not fit: the binding then finds out what, and says so.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

typedef int (*quantize_fn)(int, const void *, int, int, void *, void *, void *);
typedef int (*dequantize_fn)(int, const void *, const void *, int, int, void *, void *);
typedef int (*norm_fn)(const void *, const void *, const void *, float, int, int, void *, void *, void *, void *);
typedef int (*matvec_fn)(const void *, const void *, const void *, void *, int, int, int, const void *, void *);
typedef int (*gemm_fn)(const void *, const void *, const void *, const void *, void *, int, int, int, const void *, void *);
typedef int (*gated_fn)(const void *, const void *, const void *, const void *, const void *, const void *, int, int, int,
                        void *, void *, void *, void *);

static quantize_fn quantize_c;
static dequantize_fn dequantize_c;
static norm_fn norm_c;
static matvec_fn matvec_c;
static gemm_fn gemm_c;
static gated_fn gated_c;

/* torch.float16, uint8, float8_e4m3fn, int32, uint32; the current device and a device's stream */
static PyObject *half_, *u8_, *e4m3_, *i32_, *u32_, *get_device_, *get_stream_;
static PyObject *s_dtype, *s_device, *s_contiguous, *s_numel, *s_size, *s_ptr, *minus_one;

/* A method's whole number; -1 with *ok = 0 where there is none (the exception is dropped: the
 * caller finds out by itself). */
static long long number(PyObject *r, int *ok) {
  long long v = -1;
  if (r == NULL) {
    PyErr_Clear();
    *ok = 0;
    return -1;
  }
  v = PyLong_AsLongLong(r);
  Py_DECREF(r);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    *ok = 0;
  }
  return v;
}

static long long ask(PyObject *t, PyObject *method, int *ok) {
  return number(PyObject_CallMethodNoArgs(t, method), ok);
}

static long long last_axis(PyObject *t, int *ok) {
  return number(PyObject_CallMethodOneArg(t, s_size, minus_one), ok);
}

/* Whether t is of type a or b, contiguous, on GPU `index`, with `count` values. */
static int fits(PyObject *t, PyObject *a, PyObject *b, long long index, long long count) {
  int ok = 1;
  PyObject *r = PyObject_GetAttr(t, s_dtype);
  if (r == NULL) {
    PyErr_Clear();
    return 0;
  }
  Py_DECREF(r); /* (types are kept by their module) */
  if (r != a && r != b) return 0;
  r = PyObject_CallMethodNoArgs(t, s_contiguous);
  if (r == NULL) {
    PyErr_Clear();
    return 0;
  }
  Py_DECREF(r);
  if (r != Py_True) return 0;
  return ask(t, s_device, &ok) == index && ask(t, s_numel, &ok) == count && ok;
}

static void *address(PyObject *t, int *ok) { return (void *)(intptr_t)ask(t, s_ptr, ok); }

/* The device of t where it is the current one, else -1. */
static long long here(PyObject *t, int *ok) {
  const long long index = ask(t, s_device, ok);
  if (!*ok || index < 0 || number(PyObject_CallNoArgs(get_device_), ok) != index) return -1;
  return index;
}

static void *stream_of(long long index, int *ok) {
  PyObject *n = PyLong_FromLongLong(index), *r;
  if (n == NULL) {
    PyErr_Clear();
    *ok = 0;
    return NULL;
  }
  r = PyObject_CallOneArg(get_stream_, n);
  Py_DECREF(n);
  return (void *)(intptr_t)number(r, ok);
}

/* The C call without the interpreter's lock: a launch can wait for room in the queue. */
#define CALL(rc, what)      \
  Py_BEGIN_ALLOW_THREADS    \
  rc = what;                \
  Py_END_ALLOW_THREADS

/* Rows and columns as the C ABI takes them. */
static int small(long long a, long long b) { return a >= 0 && b >= 0 && a <= INT32_MAX && b <= INT32_MAX; }

/* x, bits, codes, scales */
static PyObject *quantize(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  int ok = 1, bits, rc;
  long long index, count, k, m;
  void *x, *codes, *scales, *st;
  if (n != 4) Py_RETURN_NONE;
  index = here(a[0], &ok);
  if (index < 0) Py_RETURN_NONE;
  count = ask(a[0], s_numel, &ok);
  k = last_axis(a[0], &ok);
  bits = (int)PyLong_AsLong(a[1]);
  if (PyErr_Occurred()) PyErr_Clear();
  if (!ok || k <= 0 || k % 32 != 0 || (bits != 4 && bits != 8)) Py_RETURN_NONE;
  m = count / k;
  if (!fits(a[0], half_, half_, index, count)) Py_RETURN_NONE;
  if (bits == 8 ? !fits(a[2], u8_, e4m3_, index, count) : !fits(a[2], i32_, u32_, index, count / 8)) Py_RETURN_NONE;
  if (!fits(a[3], u8_, u8_, index, count / 32) || last_axis(a[2], &ok) != (bits == 8 ? k : k / 8)) Py_RETURN_NONE;
  x = address(a[0], &ok), codes = address(a[2], &ok), scales = address(a[3], &ok), st = stream_of(index, &ok);
  if (!ok || !small(m, k)) Py_RETURN_NONE;
  CALL(rc, quantize_c(bits, x, (int)m, (int)k, codes, scales, st))
  return PyLong_FromLong(rc);
}

/* codes, scales, out */
static PyObject *dequantize(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  int ok = 1, bits = 8, rc;
  long long index, count, k, m;
  void *codes, *scales, *out, *st;
  if (n != 3) Py_RETURN_NONE;
  index = here(a[0], &ok);
  if (index < 0) Py_RETURN_NONE;
  count = ask(a[0], s_numel, &ok);
  k = last_axis(a[0], &ok);
  if (!ok) Py_RETURN_NONE;
  if (!fits(a[0], u8_, e4m3_, index, count)) {
    if (!fits(a[0], i32_, u32_, index, count)) Py_RETURN_NONE;
    bits = 4;
    count *= 8;
    k *= 8;
  }
  if (k <= 0 || k % 32 != 0) Py_RETURN_NONE;
  m = count / k;
  if (!fits(a[1], u8_, u8_, index, count / 32) || !fits(a[2], half_, half_, index, count) ||
      last_axis(a[2], &ok) != k)
    Py_RETURN_NONE;
  codes = address(a[0], &ok), scales = address(a[1], &ok), out = address(a[2], &ok), st = stream_of(index, &ok);
  if (!ok || !small(m, k)) Py_RETURN_NONE;
  CALL(rc, dequantize_c(bits, codes, scales, (int)m, (int)k, out, st))
  return PyLong_FromLong(rc);
}

/* x, gamma, residual or None, eps, h (anything without a residual), codes, scales */
static PyObject *norm(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  int ok = 1, rc;
  long long index, count, k, m;
  double eps;
  void *x, *gamma, *res = NULL, *h = NULL, *codes, *scales, *st;
  if (n != 7) Py_RETURN_NONE;
  index = here(a[0], &ok);
  if (index < 0) Py_RETURN_NONE;
  count = ask(a[0], s_numel, &ok);
  k = last_axis(a[0], &ok);
  eps = PyFloat_AsDouble(a[3]);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
  if (!ok || k <= 0 || k % 32 != 0) Py_RETURN_NONE;
  m = count / k;
  if (!fits(a[0], half_, half_, index, count) || !fits(a[1], half_, half_, index, k) ||
      !fits(a[5], u8_, e4m3_, index, count) || !fits(a[6], u8_, u8_, index, count / 32) ||
      last_axis(a[5], &ok) != k)
    Py_RETURN_NONE;
  if (a[2] != Py_None) {
    if (!fits(a[2], half_, half_, index, count) || !fits(a[4], half_, half_, index, count) ||
        last_axis(a[2], &ok) != k || last_axis(a[4], &ok) != k)
      Py_RETURN_NONE;
    res = address(a[2], &ok), h = address(a[4], &ok);
  }
  x = address(a[0], &ok), gamma = address(a[1], &ok), codes = address(a[5], &ok), scales = address(a[6], &ok);
  st = stream_of(index, &ok);
  if (!ok || !small(m, k)) Py_RETURN_NONE;
  CALL(rc, norm_c(x, res, gamma, (float)eps, (int)m, (int)k, h, codes, scales, st))
  return PyLong_FromLong(rc);
}

/* An MXFP4 weight, codes [n][k / 8] and scales: its rows and columns. */
static int weight(PyObject *codes, PyObject *scales, long long index, long long *n, long long *k) {
  int ok = 1;
  const long long count = ask(codes, s_numel, &ok), words = last_axis(codes, &ok);
  if (!ok || words <= 0 || words % 4 != 0) return 0;
  *n = count / words;
  *k = 8 * words;
  return fits(codes, i32_, u32_, index, count) && fits(scales, u8_, u8_, index, count / 4);
}

/* codes, scales, x, y, residual or None */
static PyObject *matvec(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  int ok = 1, rc;
  long long index, rows, k, count, m;
  void *w, *s, *x, *y, *res = NULL, *st;
  if (n != 5) Py_RETURN_NONE;
  index = here(a[2], &ok);
  if (index < 0 || !weight(a[0], a[1], index, &rows, &k)) Py_RETURN_NONE;
  count = ask(a[2], s_numel, &ok);
  m = count / k;
  if (!ok || !fits(a[2], half_, half_, index, count) || last_axis(a[2], &ok) != k ||
      !fits(a[3], half_, half_, index, m * rows) || last_axis(a[3], &ok) != rows)
    Py_RETURN_NONE;
  if (a[4] != Py_None) {
    if (!fits(a[4], half_, half_, index, m * rows) || last_axis(a[4], &ok) != rows) Py_RETURN_NONE;
    res = address(a[4], &ok);
  }
  w = address(a[0], &ok), s = address(a[1], &ok), x = address(a[2], &ok), y = address(a[3], &ok);
  st = stream_of(index, &ok);
  if (!ok || !small(m, rows) || !small(k, k)) Py_RETURN_NONE;
  CALL(rc, matvec_c(w, s, x, y, (int)m, (int)rows, (int)k, res, st))
  return PyLong_FromLong(rc);
}

/* MXFP8 rows of k columns: how many. */
static int activations(PyObject *codes, PyObject *scales, long long index, long long k, long long *m) {
  int ok = 1;
  const long long count = ask(codes, s_numel, &ok);
  *m = count / k;
  return ok && fits(codes, u8_, e4m3_, index, count) && fits(scales, u8_, u8_, index, count / 32) &&
         last_axis(codes, &ok) == k && ok;
}

/* codes, scales, x codes, x scales, y, residual or None */
static PyObject *gemm(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  int ok = 1, rc;
  long long index, rows, k, m;
  void *w, *s, *x, *xs, *y, *res = NULL, *st;
  if (n != 6) Py_RETURN_NONE;
  index = here(a[2], &ok);
  if (index < 0 || !weight(a[0], a[1], index, &rows, &k) || !activations(a[2], a[3], index, k, &m)) Py_RETURN_NONE;
  if (!fits(a[4], half_, half_, index, m * rows) || last_axis(a[4], &ok) != rows) Py_RETURN_NONE;
  if (a[5] != Py_None) {
    if (!fits(a[5], half_, half_, index, m * rows) || last_axis(a[5], &ok) != rows) Py_RETURN_NONE;
    res = address(a[5], &ok);
  }
  w = address(a[0], &ok), s = address(a[1], &ok), x = address(a[2], &ok), xs = address(a[3], &ok);
  y = address(a[4], &ok), st = stream_of(index, &ok);
  if (!ok || !small(m, rows) || !small(k, k)) Py_RETURN_NONE;
  CALL(rc, gemm_c(w, s, x, xs, y, (int)m, (int)rows, (int)k, res, st))
  return PyLong_FromLong(rc);
}

/* gate codes, gate scales, up codes, up scales, x codes, x scales, h or None, codes or None, scales or None */
static PyObject *gated(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  int ok = 1, i, rc;
  long long index, rows, k, rows2, k2, m;
  void *p[9] = {NULL}, *st;
  if (n != 9) Py_RETURN_NONE;
  index = here(a[4], &ok);
  if (index < 0 || !weight(a[0], a[1], index, &rows, &k) || !weight(a[2], a[3], index, &rows2, &k2) || rows != rows2 ||
      k != k2 || !activations(a[4], a[5], index, k, &m))
    Py_RETURN_NONE;
  if (a[6] != Py_None && (!fits(a[6], half_, half_, index, m * rows) || last_axis(a[6], &ok) != rows)) Py_RETURN_NONE;
  if ((a[7] == Py_None) != (a[8] == Py_None)) Py_RETURN_NONE;
  if (a[7] != Py_None && (rows % 32 != 0 || !fits(a[7], u8_, e4m3_, index, m * rows) || last_axis(a[7], &ok) != rows ||
                          !fits(a[8], u8_, u8_, index, m * (rows / 32))))
    Py_RETURN_NONE;
  for (i = 0; i < 9; ++i)
    if (a[i] != Py_None) p[i] = address(a[i], &ok);
  st = stream_of(index, &ok);
  if (!ok || !small(m, rows) || !small(k, k)) Py_RETURN_NONE;
  CALL(rc, gated_c(p[0], p[1], p[2], p[3], p[4], p[5], (int)m, (int)rows, (int)k, p[6], p[7], p[8], st))
  return PyLong_FromLong(rc);
}

/* bind(addresses of the six C functions, types and functions of torch): once, by the binding */
static PyObject *bind(PyObject *self, PyObject *args) {
  unsigned long long f[6];
  PyObject *o[7];
  int i;
  PyObject **to[7] = {&half_, &u8_, &e4m3_, &i32_, &u32_, &get_device_, &get_stream_};
  if (!PyArg_ParseTuple(args, "KKKKKKOOOOOOO", &f[0], &f[1], &f[2], &f[3], &f[4], &f[5], &o[0], &o[1], &o[2], &o[3],
                        &o[4], &o[5], &o[6]))
    return NULL;
  quantize_c = (quantize_fn)(uintptr_t)f[0];
  dequantize_c = (dequantize_fn)(uintptr_t)f[1];
  norm_c = (norm_fn)(uintptr_t)f[2];
  matvec_c = (matvec_fn)(uintptr_t)f[3];
  gemm_c = (gemm_fn)(uintptr_t)f[4];
  gated_c = (gated_fn)(uintptr_t)f[5];
  for (i = 0; i < 7; ++i) {
    Py_INCREF(o[i]);
    Py_XDECREF(*to[i]);
    *to[i] = o[i];
  }
  Py_RETURN_NONE;
}

#define FAST(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {FAST(quantize), FAST(dequantize), FAST(norm), FAST(matvec), FAST(gemm), FAST(gated),
                                {"bind", bind, METH_VARARGS, NULL}, {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_mx_calls", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__mx_calls(void) {
  s_dtype = PyUnicode_InternFromString("dtype");
  s_device = PyUnicode_InternFromString("get_device");
  s_contiguous = PyUnicode_InternFromString("is_contiguous");
  s_numel = PyUnicode_InternFromString("numel");
  s_size = PyUnicode_InternFromString("size");
  s_ptr = PyUnicode_InternFromString("data_ptr");
  minus_one = PyLong_FromLong(-1);
  return PyModule_Create(&module);
}
