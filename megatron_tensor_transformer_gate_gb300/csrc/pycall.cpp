// pycall.cpp — CPython module _tpcall: the block-scaled E4M3 calls of binding.py
// for arguments in their ordinary form.
//
// A generated token's calls are as long as what the host does before their
// launch, and reading eight tensors' types, shapes, strides, devices and
// addresses through Python takes longer than the launch itself (4.7 µs of 7.8
// for tp_add_rmsnorm_fp8_fwd; 2.7 in all this way).  Each function here reads
// them from the tensors behind the Python objects, checks what binding.py's
// functions check, and calls the C entry with the GIL released; where anything
// is not as it should be it returns None without a call, and the Python
// function goes through its own checks and says what is wrong.  It returns the
// tp_status else.
#define PY_SSIZE_T_CLEAN
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>

namespace {

enum { DT_OTHER, DT_BF16, DT_F32, DT_CODE };
enum { GROUP_ROW = 0, GROUP_BLOCK = 1 };

PyObject* n_stream;

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
quantize_fn c_quantize;
swiglu_fn c_swiglu;
swiglu_bwd_fn c_swiglu_bwd;
norm_fn c_norm;
gemm_fn c_gemm;

struct view {
  int64_t rows, cols, ld;  // a vector: rows elements, cols = 1
  int dtype;
  bool unit;               // adjacent elements of a row
  long dev;
  void* p;
};

// The tensor as a matrix (dims 2) or a vector (dims 1); false if it is none.
bool look(PyObject* o, int64_t dims, view* v) {
  if (!THPVariable_Check(o)) return false;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda() || t.layout() != at::kStrided || t.dim() != dims)
    return false;
  switch (t.scalar_type()) {
    case at::kBFloat16: v->dtype = DT_BF16; break;
    case at::kFloat: v->dtype = DT_F32; break;
    case at::kFloat8_e4m3fn:
    case at::kByte: v->dtype = DT_CODE; break;
    default: v->dtype = DT_OTHER;
  }
  v->rows = t.size(0);
  if (dims == 2) {
    v->cols = t.size(1);
    v->ld = v->rows > 1 ? t.stride(0) : v->cols;
    v->unit = v->cols == 1 || t.stride(1) == 1;
  } else {
    v->cols = v->ld = 1;
    v->unit = v->rows == 1 || t.stride(0) == 1;
  }
  v->dev = t.get_device();
  v->p = t.data_ptr();
  return true;
}

// A matrix with adjacent columns.
bool matrix(PyObject* t, view* v) {
  return t != Py_None && look(t, 2, v) && v->unit;
}

struct pair {
  void* q = nullptr;
  int64_t ldq = 0;
  float* s = nullptr;
  int64_t lds = 0;
  int group = GROUP_ROW;
  bool either = true;   // one row, where both groups are the same
};

bool codes(PyObject* q, PyObject* s, int64_t rows, int64_t cols, long dev,
           pair* o) {
  view a, b;
  if (!matrix(q, &a) || !matrix(s, &b)) return false;
  if (a.dtype != DT_CODE || b.dtype != DT_F32 || a.rows != rows ||
      a.cols != cols || a.dev != dev || b.dev != dev)
    return false;
  if (b.rows != (cols + 127) / 128 ||
      (b.cols != rows && b.cols != (rows + 127) / 128))
    return false;
  o->q = a.p;
  o->ldq = rows > 1 ? a.ld : (cols + 15) / 16 * 16;
  o->s = (float*)b.p;
  o->lds = b.ld;
  o->group = b.cols == rows ? GROUP_ROW : GROUP_BLOCK;
  o->either = rows == 1;
  return true;
}

// The codes of a matrix and of its transpose, of one group.
bool outputs(PyObject* const* x, int64_t rows, int64_t cols, long dev,
             pair* q, pair* t, int* group) {
  if (x[0] == Py_None && x[2] == Py_None) return false;
  if (x[0] != Py_None && !codes(x[0], x[1], rows, cols, dev, q)) return false;
  if (x[2] != Py_None && !codes(x[2], x[3], cols, rows, dev, t)) return false;
  if (!q->either && !t->either && q->group != t->group) return false;
  *group = !q->either ? q->group : t->group;
  if (q->either && t->either) *group = GROUP_ROW;
  return true;
}

// The stream to launch on; false unless dev is the current device.
bool stream_of(PyObject* s, long dev, void** out) {
  if (c10::cuda::current_device() != dev) return false;
  if (s == Py_None) {
    *out = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream();
    return true;
  }
  PyObject* h = PyObject_GetAttr(s, n_stream);
  if (h == nullptr) return false;
  *out = PyLong_AsVoidPtr(h);
  Py_DECREF(h);
  return !PyErr_Occurred();
}

PyObject* not_handled() {
  PyErr_Clear();
  Py_RETURN_NONE;
}

#define CALL(expr)              \
  int32_t rc;                   \
  Py_BEGIN_ALLOW_THREADS        \
  rc = (expr);                  \
  Py_END_ALLOW_THREADS          \
  return PyLong_FromLong(rc)

// x, q, s, qt, st, stream
PyObject* quantize(PyObject*, PyObject* const* x, Py_ssize_t n) {
  view v;
  pair q, t;
  void* st;
  int group;
  if (n != 6 || !matrix(x[0], &v) ||
      (v.dtype != DT_BF16 && v.dtype != DT_F32) ||
      !outputs(x + 1, v.rows, v.cols, v.dev, &q, &t, &group) ||
      !stream_of(x[5], v.dev, &st))
    return not_handled();
  CALL(c_quantize(v.dtype == DT_BF16, group, v.rows, v.cols, v.p, v.ld, q.q,
                  q.ldq, q.s, q.lds, t.q, t.ldq, t.s, t.lds, st));
}

// gu, q, s, qt, st, stream
PyObject* swiglu(PyObject*, PyObject* const* x, Py_ssize_t n) {
  view v;
  pair q, t;
  void* st;
  int group;
  if (n != 6 || !matrix(x[0], &v) || v.dtype != DT_BF16 || v.cols % 2 ||
      !outputs(x + 1, v.rows, v.cols / 2, v.dev, &q, &t, &group) ||
      (group != GROUP_ROW && v.rows > 1) || !stream_of(x[5], v.dev, &st))
    return not_handled();
  CALL(c_swiglu(v.rows, v.cols / 2, v.p, v.ld, q.q, q.ldq, q.s, q.lds, t.q,
                t.ldq, t.s, t.lds, st));
}

// dA, gu, q, s, qt, st, stream
PyObject* swiglu_bwd(PyObject*, PyObject* const* x, Py_ssize_t n) {
  view a, v;
  pair q, t;
  void* st;
  int group;
  if (n != 7 || !matrix(x[1], &v) || v.dtype != DT_BF16 || v.cols % 2 ||
      !matrix(x[0], &a) || a.dtype != DT_BF16 || a.rows != v.rows ||
      a.cols != v.cols / 2 || a.dev != v.dev ||
      !outputs(x + 2, v.rows, v.cols, v.dev, &q, &t, &group) ||
      (group != GROUP_ROW && v.rows > 1) || !stream_of(x[6], v.dev, &st))
    return not_handled();
  CALL(c_swiglu_bwd(v.rows, v.cols / 2, a.p, a.ld, v.p, v.ld, q.q, q.ldq, q.s,
                    q.lds, t.q, t.ldq, t.s, t.lds, st));
}

// A dense bf16 matrix like `as`, or None (p null).
bool like(PyObject* t, const view* as, void** p) {
  view v;
  *p = nullptr;
  if (t == Py_None) return true;
  if (!matrix(t, &v) || v.dtype != DT_BF16 || v.rows != as->rows ||
      v.cols != as->cols || v.ld != v.cols || v.dev != as->dev)
    return false;
  *p = v.p;
  return true;
}

// x, r, gamma, x1, q, s, rstd, y, eps, stream
PyObject* norm(PyObject*, PyObject* const* x, Py_ssize_t n) {
  view v, g, rs;
  pair q;
  void *r, *x1, *y, *st;
  if (n != 10 || !matrix(x[0], &v) || v.dtype != DT_BF16 || v.ld != v.cols ||
      !like(x[1], &v, &r) || !like(x[3], &v, &x1) || !like(x[7], &v, &y) ||
      (r != nullptr && x1 == nullptr) || !look(x[2], 1, &g) ||
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

// qa, sa, qb, sb, C, stream
PyObject* gemm(PyObject*, PyObject* const* x, Py_ssize_t n) {
  view c, a;
  pair pa, pb;
  void* st;
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

// bind(five addresses): the C entries
PyObject* bind(PyObject*, PyObject* const* x, Py_ssize_t n) {
  void* fn[5];
  if (n != 5) {
    PyErr_SetString(PyExc_TypeError, "bind takes 5 arguments");
    return nullptr;
  }
  for (int i = 0; i < 5; ++i) {
    fn[i] = PyLong_AsVoidPtr(x[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  c_quantize = (quantize_fn)fn[0];
  c_swiglu = (swiglu_fn)fn[1];
  c_swiglu_bwd = (swiglu_bwd_fn)fn[2];
  c_norm = (norm_fn)fn[3];
  c_gemm = (gemm_fn)fn[4];
  Py_RETURN_NONE;
}

// What throws (a tensor without storage or with symbolic sizes) is for
// binding.py to name.
using function = PyObject* (*)(PyObject*, PyObject* const*, Py_ssize_t);
template <function F>
PyObject* caught(PyObject* m, PyObject* const* x, Py_ssize_t n) {
  try {
    return F(m, x, n);
  } catch (...) {
    return not_handled();
  }
}

template <function F>
PyMethodDef method(const char* name) {
  return {name, (PyCFunction)(void (*)(void))F, METH_FASTCALL, nullptr};
}
PyMethodDef methods[] = {method<bind>("bind"),
                         method<caught<quantize>>("quantize"),
                         method<caught<swiglu>>("swiglu"),
                         method<caught<swiglu_bwd>>("swiglu_bwd"),
                         method<caught<norm>>("norm"),
                         method<caught<gemm>>("gemm"),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tpcall", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tpcall(void) {
  n_stream = PyUnicode_InternFromString("cuda_stream");
  if (n_stream == nullptr) return nullptr;
  return PyModule_Create(&module);
}
