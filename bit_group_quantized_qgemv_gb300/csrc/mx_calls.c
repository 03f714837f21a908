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
static PyObject *s_dtype, *s_device, *s_contiguous, *s_shape, *s_ptr;

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

/* A tensor's number of values, first and last axis; one without axes fits nothing. */
typedef struct {
  long long count, first, last;
} Shape;

static Shape shape_of(PyObject *t, int *ok) {
  Shape s = {1, -1, -1};
  PyObject *r = PyObject_GetAttr(t, s_shape);
  Py_ssize_t i, n;
  if (r == NULL || !PyTuple_Check(r) || PyTuple_GET_SIZE(r) == 0) {
    Py_XDECREF(r);
    PyErr_Clear();
    *ok = 0;
    return s;
  }
  n = PyTuple_GET_SIZE(r);
  for (i = 0; i < n && *ok; ++i) {
    s.last = PyLong_AsLongLong(PyTuple_GET_ITEM(r, i));
    if (s.last < 0 || __builtin_mul_overflow(s.count, s.last, &s.count)) {
      PyErr_Clear();
      *ok = 0;
    }
    if (i == 0) s.first = s.last;
  }
  Py_DECREF(r);
  return s;
}

/* Whether t is of type a or b, contiguous and on GPU `index`. */
static int is_on(PyObject *t, PyObject *a, PyObject *b, long long index) {
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
  return r == Py_True && ask(t, s_device, &ok) == index && ok;
}

/* And has `count` values in rows of `last`.  (Rows of scales are looked at as those of values
 * are: the scales of a transposed matrix are as many.) */
static int fits(PyObject *t, PyObject *a, PyObject *b, long long index, long long count, long long last) {
  int ok = 1;
  const Shape s = shape_of(t, &ok);
  return ok && s.count == count && s.last == last && is_on(t, a, b, index);
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
  long long index;
  Shape s;
  void *x, *codes, *scales, *st;
  if (n != 4) Py_RETURN_NONE;
  index = here(a[0], &ok);
  if (index < 0) Py_RETURN_NONE;
  s = shape_of(a[0], &ok);
  bits = (int)PyLong_AsLong(a[1]);
  if (PyErr_Occurred()) PyErr_Clear();
  if (!ok || s.last <= 0 || s.last % 32 != 0 || (bits != 4 && bits != 8)) Py_RETURN_NONE;
  if (!is_on(a[0], half_, half_, index) || !fits(a[3], u8_, u8_, index, s.count / 32, s.last / 32)) Py_RETURN_NONE;
  if (bits == 8 ? !fits(a[2], u8_, e4m3_, index, s.count, s.last) : !fits(a[2], i32_, u32_, index, s.count / 8, s.last / 8))
    Py_RETURN_NONE;
  x = address(a[0], &ok), codes = address(a[2], &ok), scales = address(a[3], &ok), st = stream_of(index, &ok);
  if (!ok || !small(s.count / s.last, s.last)) Py_RETURN_NONE;
  CALL(rc, quantize_c(bits, x, (int)(s.count / s.last), (int)s.last, codes, scales, st))
  return PyLong_FromLong(rc);
}

/* codes, scales, out */
static PyObject *dequantize(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  int ok = 1, bits = 8, rc;
  long long index;
  Shape s;
  void *codes, *scales, *out, *st;
  if (n != 3) Py_RETURN_NONE;
  index = here(a[0], &ok);
  if (index < 0) Py_RETURN_NONE;
  s = shape_of(a[0], &ok);
  if (!ok) Py_RETURN_NONE;
  if (!is_on(a[0], u8_, e4m3_, index)) {
    if (!is_on(a[0], i32_, u32_, index)) Py_RETURN_NONE;
    bits = 4;
    s.count *= 8;
    s.last *= 8;
  }
  if (s.last <= 0 || s.last % 32 != 0) Py_RETURN_NONE;
  if (!fits(a[1], u8_, u8_, index, s.count / 32, s.last / 32) || !fits(a[2], half_, half_, index, s.count, s.last))
    Py_RETURN_NONE;
  codes = address(a[0], &ok), scales = address(a[1], &ok), out = address(a[2], &ok), st = stream_of(index, &ok);
  if (!ok || !small(s.count / s.last, s.last)) Py_RETURN_NONE;
  CALL(rc, dequantize_c(bits, codes, scales, (int)(s.count / s.last), (int)s.last, out, st))
  return PyLong_FromLong(rc);
}

/* x, gamma, residual or None, eps, h (anything without a residual), codes, scales */
static PyObject *norm(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  int ok = 1, rc;
  long long index, count, k;
  Shape s, g;
  double eps;
  void *x, *gamma, *res = NULL, *h = NULL, *codes, *scales, *st;
  if (n != 7) Py_RETURN_NONE;
  index = here(a[0], &ok);
  if (index < 0) Py_RETURN_NONE;
  s = shape_of(a[0], &ok), g = shape_of(a[1], &ok);
  count = s.count, k = s.last;
  eps = PyFloat_AsDouble(a[3]);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
  if (!ok || k <= 0 || k % 32 != 0 || g.count != k) Py_RETURN_NONE;
  if (!is_on(a[0], half_, half_, index) || !is_on(a[1], half_, half_, index) ||
      !fits(a[5], u8_, e4m3_, index, count, k) || !fits(a[6], u8_, u8_, index, count / 32, k / 32))
    Py_RETURN_NONE;
  if (a[2] != Py_None) {
    if (!fits(a[2], half_, half_, index, count, k) || !fits(a[4], half_, half_, index, count, k)) Py_RETURN_NONE;
    res = address(a[2], &ok), h = address(a[4], &ok);
  }
  x = address(a[0], &ok), gamma = address(a[1], &ok), codes = address(a[5], &ok), scales = address(a[6], &ok);
  st = stream_of(index, &ok);
  if (!ok || !small(count / k, k)) Py_RETURN_NONE;
  CALL(rc, norm_c(x, res, gamma, (float)eps, (int)(count / k), (int)k, h, codes, scales, st))
  return PyLong_FromLong(rc);
}

/* An MXFP4 weight, codes [n][k / 8] and scales [n][k / 32]: its rows and columns. */
static int weight(PyObject *codes, PyObject *scales, long long index, long long *n, long long *k) {
  int ok = 1;
  const Shape s = shape_of(codes, &ok);
  if (!ok || s.last <= 0 || s.last % 4 != 0 || s.first != s.count / s.last) return 0;
  *n = s.first;
  *k = 8 * s.last;
  return is_on(codes, i32_, u32_, index) && fits(scales, u8_, u8_, index, s.count / 4, s.last / 4);
}

/* codes, scales, x, y, residual or None */
static PyObject *matvec(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  int ok = 1, rc;
  long long index, rows, k, m;
  Shape x_shape;
  void *w, *s, *x, *y, *res = NULL, *st;
  if (n != 5) Py_RETURN_NONE;
  index = here(a[2], &ok);
  if (index < 0 || !weight(a[0], a[1], index, &rows, &k)) Py_RETURN_NONE;
  x_shape = shape_of(a[2], &ok);
  m = x_shape.count / k;
  if (!ok || x_shape.last != k || !is_on(a[2], half_, half_, index) || !fits(a[3], half_, half_, index, m * rows, rows))
    Py_RETURN_NONE;
  if (a[4] != Py_None) {
    if (!fits(a[4], half_, half_, index, m * rows, rows)) Py_RETURN_NONE;
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
  const Shape s = shape_of(codes, &ok);
  *m = s.count / k;
  return ok && s.last == k && is_on(codes, u8_, e4m3_, index) && fits(scales, u8_, u8_, index, s.count / 32, k / 32);
}

/* codes, scales, x codes, x scales, y, residual or None */
static PyObject *gemm(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  int ok = 1, rc;
  long long index, rows, k, m;
  void *w, *s, *x, *xs, *y, *res = NULL, *st;
  if (n != 6) Py_RETURN_NONE;
  index = here(a[2], &ok);
  if (index < 0 || !weight(a[0], a[1], index, &rows, &k) || !activations(a[2], a[3], index, k, &m)) Py_RETURN_NONE;
  if (!fits(a[4], half_, half_, index, m * rows, rows)) Py_RETURN_NONE;
  if (a[5] != Py_None) {
    if (!fits(a[5], half_, half_, index, m * rows, rows)) Py_RETURN_NONE;
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
  if (a[6] != Py_None && !fits(a[6], half_, half_, index, m * rows, rows)) Py_RETURN_NONE;
  if ((a[7] == Py_None) != (a[8] == Py_None)) Py_RETURN_NONE;
  if (a[7] != Py_None && (rows % 32 != 0 || !fits(a[7], u8_, e4m3_, index, m * rows, rows) ||
                          !fits(a[8], u8_, u8_, index, m * (rows / 32), rows / 32)))
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
  s_shape = PyUnicode_InternFromString("shape");
  s_ptr = PyUnicode_InternFromString("data_ptr");
  return PyModule_Create(&module);
}
