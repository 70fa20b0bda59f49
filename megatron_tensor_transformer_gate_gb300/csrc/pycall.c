/* pycall.c — CPython module _tpcall: the block-scaled E4M3 calls of binding.py
 * for arguments in their ordinary form.
 *
 * A generated token's calls are as long as what the host does before their
 * launch, and reading eight tensors' types, shapes, strides, devices and
 * addresses from Python takes longer than the launch itself (4.7 µs of 7.8
 * for tp_add_rmsnorm_fp8_fwd).  Each function here reads them once, checks
 * what binding.py's functions check, and calls the C entry with the GIL
 * released; where anything is not as it should be it returns None without a
 * call, and the Python function goes through its own checks and says what is
 * wrong.  It returns the tp_status else.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

enum { DT_OTHER, DT_BF16, DT_F32, DT_CODE };
enum { GROUP_ROW = 0, GROUP_BLOCK = 1 };

static PyObject *n_dtype, *n_shape, *n_stride, *n_device, *n_ptr, *n_stream;
/* set by bind(): torch's dtypes, device and stream lookups, the C entries */
static PyObject *t_bf16, *t_f32, *t_e4m3, *t_u8, *f_device, *f_stream;

typedef int32_t (*quantize_fn)(int32_t, int32_t, int64_t, int64_t,
                               const void*, int64_t, void*, int64_t, float*,
                               int64_t, void*, int64_t, float*, int64_t,
                               void*);
typedef int32_t (*swiglu_fn)(int64_t, int64_t, const void*, int64_t, void*,
                             int64_t, float*, int64_t, void*, int64_t, float*,
                             int64_t, void*);
typedef int32_t (*swiglu_bwd_fn)(int64_t, int64_t, const void*, int64_t,
                                 const void*, int64_t, void*, int64_t, float*,
                                 int64_t, void*, int64_t, float*, int64_t,
                                 void*);
typedef int32_t (*norm_fn)(int64_t, int64_t, float, const void*, const void*,
                           const void*, void*, void*, float*, void*, int64_t,
                           float*, int64_t, void*);
typedef int32_t (*gemm_fn)(int64_t, int64_t, int64_t, const void*, int64_t,
                           const float*, int64_t, int32_t, const void*,
                           int64_t, const float*, int64_t, int32_t, int32_t,
                           void*, int64_t, void*);
static quantize_fn c_quantize;
static swiglu_fn c_swiglu;
static swiglu_bwd_fn c_swiglu_bwd;
static norm_fn c_norm;
static gemm_fn c_gemm;

typedef struct {
  int64_t rows, cols, ld; /* a vector: rows elements, cols = 1 */
  int dtype, unit;        /* unit: adjacent elements of a row */
  long dev;
  void* p;
} view;

static int64_t item(PyObject* tuple, Py_ssize_t i) {
  return PyLong_AsLongLong(PyTuple_GET_ITEM(tuple, i));
}

/* The tensor as a matrix (dims 2) or a vector (dims 1); 0 if it is none. */
static int look(PyObject* t, Py_ssize_t dims, view* v) {
  PyObject *dt = NULL, *shape = NULL, *stride = NULL, *dev = NULL, *p = NULL;
  int ok = 0;
  if ((dt = PyObject_GetAttr(t, n_dtype)) == NULL ||
      (shape = PyObject_GetAttr(t, n_shape)) == NULL ||
      (stride = PyObject_CallMethodNoArgs(t, n_stride)) == NULL ||
      (dev = PyObject_CallMethodNoArgs(t, n_device)) == NULL ||
      (p = PyObject_CallMethodNoArgs(t, n_ptr)) == NULL)
    goto out;
  if (!PyTuple_Check(shape) || !PyTuple_Check(stride) ||
      PyTuple_GET_SIZE(shape) != dims || PyTuple_GET_SIZE(stride) != dims)
    goto out;
  v->dtype = dt == t_bf16 ? DT_BF16
             : dt == t_f32 ? DT_F32
             : dt == t_e4m3 || dt == t_u8 ? DT_CODE : DT_OTHER;
  v->rows = item(shape, 0);
  if (dims == 2) {
    v->cols = item(shape, 1);
    v->ld = v->rows > 1 ? item(stride, 0) : v->cols;
    v->unit = v->cols == 1 || item(stride, 1) == 1;
  } else {
    v->cols = v->ld = 1;
    v->unit = v->rows == 1 || item(stride, 0) == 1;
  }
  v->dev = PyLong_AsLong(dev);
  v->p = PyLong_AsVoidPtr(p);
  ok = !PyErr_Occurred();
out:
  Py_XDECREF(dt);
  Py_XDECREF(shape);
  Py_XDECREF(stride);
  Py_XDECREF(dev);
  Py_XDECREF(p);
  return ok;
}

/* A matrix with adjacent columns. */
static int matrix(PyObject* t, view* v) {
  return t != Py_None && look(t, 2, v) && v->unit;
}

typedef struct {
  void* q;
  int64_t ldq;
  float* s;
  int64_t lds;
  int group, either; /* either: one row, where both groups are the same */
} pair;

static int codes(PyObject* q, PyObject* s, int64_t rows, int64_t cols,
                 long dev, pair* o) {
  view a, b;
  if (!matrix(q, &a) || !matrix(s, &b)) return 0;
  if (a.dtype != DT_CODE || b.dtype != DT_F32 || a.rows != rows ||
      a.cols != cols || a.dev != dev || b.dev != dev)
    return 0;
  if (b.rows != (cols + 127) / 128 ||
      (b.cols != rows && b.cols != (rows + 127) / 128))
    return 0;
  o->q = a.p;
  o->ldq = rows > 1 ? a.ld : (cols + 15) / 16 * 16;
  o->s = (float*)b.p;
  o->lds = b.ld;
  o->group = b.cols == rows ? GROUP_ROW : GROUP_BLOCK;
  o->either = rows == 1;
  return 1;
}

/* The codes of a matrix and of its transpose, of one group. */
static int outputs(PyObject* const* x, int64_t rows, int64_t cols, long dev,
                   pair* q, pair* t, int* group) {
  memset(q, 0, sizeof(*q));
  memset(t, 0, sizeof(*t));
  q->either = t->either = 1;
  if (x[0] == Py_None && x[2] == Py_None) return 0;
  if (x[0] != Py_None && !codes(x[0], x[1], rows, cols, dev, q)) return 0;
  if (x[2] != Py_None && !codes(x[2], x[3], cols, rows, dev, t)) return 0;
  if (!q->either && !t->either && q->group != t->group) return 0;
  *group = !q->either ? q->group : t->group;
  if (q->either && t->either) *group = GROUP_ROW;
  return 1;
}

/* The stream to launch on; 0 unless dev is the current device. */
static int stream_of(PyObject* s, long dev, void** out) {
  PyObject* r = PyObject_CallNoArgs(f_device);
  if (r == NULL) return 0;
  const long cur = PyLong_AsLong(r);
  if (cur != dev || dev < 0) {
    Py_DECREF(r);
    return 0;
  }
  PyObject* h = s == Py_None ? PyObject_CallOneArg(f_stream, r)
                             : PyObject_GetAttr(s, n_stream);
  Py_DECREF(r);
  if (h == NULL) return 0;
  *out = PyLong_AsVoidPtr(h);
  Py_DECREF(h);
  return !PyErr_Occurred();
}

static PyObject* not_handled(void) {
  PyErr_Clear();
  Py_RETURN_NONE;
}

#define CALL(expr)              \
  int32_t rc;                   \
  Py_BEGIN_ALLOW_THREADS        \
  rc = (expr);                  \
  Py_END_ALLOW_THREADS          \
  return PyLong_FromLong(rc)

/* x, q, s, qt, st, stream */
static PyObject* quantize(PyObject* self, PyObject* const* x, Py_ssize_t n) {
  view v;
  pair q, t;
  void* st;
  int group;
  (void)self;
  if (n != 6 || !matrix(x[0], &v) ||
      (v.dtype != DT_BF16 && v.dtype != DT_F32) ||
      !outputs(x + 1, v.rows, v.cols, v.dev, &q, &t, &group) ||
      !stream_of(x[5], v.dev, &st))
    return not_handled();
  CALL(c_quantize(v.dtype == DT_BF16, group, v.rows, v.cols, v.p, v.ld, q.q,
                  q.ldq, q.s, q.lds, t.q, t.ldq, t.s, t.lds, st));
}

/* gu, q, s, qt, st, stream */
static PyObject* swiglu(PyObject* self, PyObject* const* x, Py_ssize_t n) {
  view v;
  pair q, t;
  void* st;
  int group;
  (void)self;
  if (n != 6 || !matrix(x[0], &v) || v.dtype != DT_BF16 || v.cols % 2 ||
      !outputs(x + 1, v.rows, v.cols / 2, v.dev, &q, &t, &group) ||
      (group != GROUP_ROW && v.rows > 1) || !stream_of(x[5], v.dev, &st))
    return not_handled();
  CALL(c_swiglu(v.rows, v.cols / 2, v.p, v.ld, q.q, q.ldq, q.s, q.lds, t.q,
                t.ldq, t.s, t.lds, st));
}

/* dA, gu, q, s, qt, st, stream */
static PyObject* swiglu_bwd(PyObject* self, PyObject* const* x, Py_ssize_t n) {
  view a, v;
  pair q, t;
  void* st;
  int group;
  (void)self;
  if (n != 7 || !matrix(x[1], &v) || v.dtype != DT_BF16 || v.cols % 2 ||
      !matrix(x[0], &a) || a.dtype != DT_BF16 || a.rows != v.rows ||
      a.cols != v.cols / 2 || a.dev != v.dev ||
      !outputs(x + 2, v.rows, v.cols, v.dev, &q, &t, &group) ||
      (group != GROUP_ROW && v.rows > 1) || !stream_of(x[6], v.dev, &st))
    return not_handled();
  CALL(c_swiglu_bwd(v.rows, v.cols / 2, a.p, a.ld, v.p, v.ld, q.q, q.ldq, q.s,
                    q.lds, t.q, t.ldq, t.s, t.lds, st));
}

/* A dense bf16 matrix like `as`, or None (p NULL). */
static int like(PyObject* t, const view* as, void** p) {
  view v;
  *p = NULL;
  if (t == Py_None) return 1;
  if (!matrix(t, &v) || v.dtype != DT_BF16 || v.rows != as->rows ||
      v.cols != as->cols || v.ld != v.cols || v.dev != as->dev)
    return 0;
  *p = v.p;
  return 1;
}

/* x, r, gamma, x1, q, s, rstd, y, eps, stream */
static PyObject* norm(PyObject* self, PyObject* const* x, Py_ssize_t n) {
  view v, g, rs;
  pair q;
  void *r, *x1, *y, *st;
  (void)self;
  if (n != 10 || !matrix(x[0], &v) || v.dtype != DT_BF16 || v.ld != v.cols ||
      !like(x[1], &v, &r) || !like(x[3], &v, &x1) || !like(x[7], &v, &y) ||
      (r != NULL && x1 == NULL) || !look(x[2], 1, &g) ||
      g.dtype != DT_BF16 || g.rows != v.cols || !g.unit || g.dev != v.dev ||
      !look(x[6], 1, &rs) || rs.dtype != DT_F32 || rs.rows != v.rows ||
      !rs.unit || rs.dev != v.dev ||
      !codes(x[4], x[5], v.rows, v.cols, v.dev, &q) ||
      (q.group != GROUP_ROW && !q.either) || !stream_of(x[9], v.dev, &st))
    return not_handled();
  const double eps = PyFloat_AsDouble(x[8]);
  if (PyErr_Occurred()) return not_handled();
  CALL(c_norm(v.rows, v.cols, (float)eps, v.p, r, g.p, x1, y, (float*)rs.p,
              q.q, q.ldq, q.s, q.lds, st));
}

/* qa, sa, qb, sb, C, stream */
static PyObject* gemm(PyObject* self, PyObject* const* x, Py_ssize_t n) {
  view c, a;
  pair pa, pb;
  void* st;
  (void)self;
  if (n != 6 || !matrix(x[4], &c) ||
      (c.dtype != DT_BF16 && c.dtype != DT_F32) || !matrix(x[0], &a) ||
      !codes(x[0], x[1], c.rows, a.cols, c.dev, &pa) ||
      !codes(x[2], x[3], c.cols, a.cols, c.dev, &pb) ||
      !stream_of(x[5], c.dev, &st))
    return not_handled();
  CALL(c_gemm(c.rows, c.cols, a.cols, pa.q, pa.ldq, pa.s, pa.lds, pa.group,
              pb.q, pb.ldq, pb.s, pb.lds, pb.group, c.dtype == DT_BF16, c.p,
              c.ld, st));
}

/* bind(bf16, f32, e4m3, u8, device, stream, five addresses) */
static PyObject* bind(PyObject* self, PyObject* const* x, Py_ssize_t n) {
  PyObject** keep[6] = {&t_bf16, &t_f32, &t_e4m3, &t_u8, &f_device, &f_stream};
  void* fn[5];
  (void)self;
  if (n != 11) {
    PyErr_SetString(PyExc_TypeError, "bind takes 11 arguments");
    return NULL;
  }
  for (int i = 0; i < 5; ++i) {
    fn[i] = PyLong_AsVoidPtr(x[6 + i]);
    if (PyErr_Occurred()) return NULL;
  }
  for (int i = 0; i < 6; ++i) {
    Py_INCREF(x[i]);
    Py_XSETREF(*keep[i], x[i]);
  }
  c_quantize = (quantize_fn)fn[0];
  c_swiglu = (swiglu_fn)fn[1];
  c_swiglu_bwd = (swiglu_bwd_fn)fn[2];
  c_norm = (norm_fn)fn[3];
  c_gemm = (gemm_fn)fn[4];
  Py_RETURN_NONE;
}

#define METHOD(name) \
  { #name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, NULL }
static PyMethodDef methods[] = {METHOD(bind),       METHOD(quantize),
                                METHOD(swiglu),     METHOD(swiglu_bwd),
                                METHOD(norm),       METHOD(gemm),
                                {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tpcall", NULL, -1,
                                    methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__tpcall(void) {
  n_dtype = PyUnicode_InternFromString("dtype");
  n_shape = PyUnicode_InternFromString("shape");
  n_stride = PyUnicode_InternFromString("stride");
  n_device = PyUnicode_InternFromString("get_device");
  n_ptr = PyUnicode_InternFromString("data_ptr");
  n_stream = PyUnicode_InternFromString("cuda_stream");
  if (PyErr_Occurred()) return NULL;
  return PyModule_Create(&module);
}
