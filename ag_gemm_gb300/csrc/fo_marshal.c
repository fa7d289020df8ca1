/* Argument marshalling of the operators between the residual stream and the
 * attention, for Python callers: checks the tensors and hands their addresses to the C
 * ABI. The same checks exist in binding.py, which explains what is
 * wrong with an argument; this module only recognises calls that are right and
 * returns -1 for all others, having done nothing. A decode step's norm has
 * seven tensors: 5 us of its 11 us call were spent on them in Python. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "flashoverlap.h"

#define MAX_R 16

static PyObject *s_dtype, *s_numel, *s_is_contiguous, *s_is_cuda, *s_data_ptr, *s_shape, *s_stride;
static PyObject *t_bf16, *t_f32, *t_e4m3, *t_u8, *t_i32, *t_i64;

enum { KIND_BF16 = 0, KIND_F32 = 1, KIND_8BIT = 2 };

/* 1 when the attribute is the very object `a` or `b`, 0 when not, -1 on error. */
static int is_dtype(PyObject *x, PyObject *a, PyObject *b) {
  PyObject *d = PyObject_GetAttr(x, s_dtype);
  if (!d) return -1;
  const int yes = d == a || d == b;
  Py_DECREF(d);
  return yes;
}
static int of_kind(PyObject *x, int kind) {
  return kind == KIND_BF16 ? is_dtype(x, t_bf16, t_bf16) : kind == KIND_F32 ? is_dtype(x, t_f32, t_f32)
                                                                            : is_dtype(x, t_e4m3, t_u8);
}
static long long number(PyObject *x, PyObject *method) {
  PyObject *v = PyObject_CallMethodNoArgs(x, method);
  if (!v) return -1;
  const long long n = PyLong_AsLongLong(v);
  Py_DECREF(v);
  return n;
}
static int truth(PyObject *v) {
  if (!v) return -1;
  const int t = v == Py_True;
  Py_DECREF(v);
  return t;
}
static void *address(PyObject *x) {
  PyObject *v = PyObject_CallMethodNoArgs(x, s_data_ptr);
  if (!v) return NULL;
  void *p = PyLong_AsVoidPtr(v);
  Py_DECREF(v);
  return p;
}

/* A dense CUDA tensor of n values: 1 and its address, else 0 (errors are cleared by the caller). */
static int dense(PyObject *x, long long n, int kind, void **out) {
  if (of_kind(x, kind) != 1 || number(x, s_numel) != n ||
      truth(PyObject_CallMethodNoArgs(x, s_is_contiguous)) != 1 || truth(PyObject_GetAttr(x, s_is_cuda)) != 1)
    return 0;
  *out = address(x);
  return *out != NULL;
}

typedef struct {
  void *at[MAX_R];
  void **p; /* at, or NULL for None */
} array;

/* R tensors in a list, or None where that is allowed. */
static int arrays(PyObject *xs, int R, long long n, int kind, int optional, array *a) {
  a->p = NULL;
  if (xs == Py_None) return optional;
  if (!PyList_CheckExact(xs) || PyList_GET_SIZE(xs) != R) return 0;
  PyObject *last = NULL;
  for (int r = 0; r < R; ++r) {
    PyObject *x = PyList_GET_ITEM(xs, r);
    if (x == last) a->at[r] = a->at[r - 1];
    else if (!dense(x, n, kind, &a->at[r])) return 0;
    last = x;
  }
  a->p = a->at;
  return 1;
}

/* The R matrices [rows x width] of a list, their rows dense and one stride apart. */
static int row_arrays(PyObject *xs, int R, long long rows, long long width, int kind, array *a, int64_t *ld) {
  a->p = NULL;
  if (!PyList_CheckExact(xs) && !PyTuple_CheckExact(xs)) return 0;
  if (PySequence_Fast_GET_SIZE(xs) != R) return 0;
  *ld = -1;
  for (int r = 0; r < R; ++r) {
    PyObject *x = PySequence_Fast_GET_ITEM(xs, r);
    if (x == Py_None || of_kind(x, kind) != 1) return 0;
    PyObject *shape = PyObject_GetAttr(x, s_shape);
    if (!shape) return 0;
    int ok = PyTuple_Check(shape) && PyTuple_GET_SIZE(shape) == 2 &&
             PyLong_AsLongLong(PyTuple_GET_ITEM(shape, 0)) == rows && PyLong_AsLongLong(PyTuple_GET_ITEM(shape, 1)) == width;
    Py_DECREF(shape);
    if (!ok) return 0;
    PyObject *stride = PyObject_CallMethodNoArgs(x, s_stride);
    if (!stride) return 0;
    ok = PyTuple_Check(stride) && PyTuple_GET_SIZE(stride) == 2;
    const long long up = ok ? PyLong_AsLongLong(PyTuple_GET_ITEM(stride, 0)) : 0;
    const long long across = ok ? PyLong_AsLongLong(PyTuple_GET_ITEM(stride, 1)) : 0;
    Py_DECREF(stride);
    if (!ok || (width > 1 && across != 1)) return 0;
    const long long step = rows > 1 ? up : width;
    if (*ld >= 0 && step != *ld) return 0;
    *ld = step;
    if (truth(PyObject_GetAttr(x, s_is_cuda)) != 1 || !(a->at[r] = address(x))) return 0;
  }
  a->p = a->at;
  return 1;
}

/* A description (a ctypes structure) of the wanted size. */
static void *description(PyObject *o, Py_buffer *view, Py_ssize_t size) {
  if (PyObject_GetBuffer(o, view, PyBUF_SIMPLE)) return NULL;
  if (view->len == size) return view->buf;
  PyBuffer_Release(view);
  return NULL;
}

static PyObject *unknown(void) {
  PyErr_Clear();
  return PyLong_FromLong(-1);
}

static int in_range(int R) { return R >= 1 && R <= MAX_R; }

/* (desc, rows, x, residual, weight, h, y, q, scale, rstd, stream) */
static PyObject *m_rmsnorm(PyObject *self, PyObject *const *v, Py_ssize_t n) {
  Py_buffer b;
  fo_norm_desc *d = n == 11 ? description(v[0], &b, sizeof(*d)) : NULL;
  if (!d) return unknown();
  const long long rows = PyLong_AsLongLong(v[1]);
  long code = -1;
  if (in_range(d->R) && rows > 0 && d->H > 0) {
    const long long all = rows * d->H, groups = rows * ((d->H + FO_FP8_BLOCK - 1) / FO_FP8_BLOCK);
    array x, res, h, y, q, scale, rstd;
    void *w;
    if (arrays(v[2], d->R, all, d->dtype, 0, &x) && arrays(v[3], d->R, all, d->dtype, 1, &res) &&
        dense(v[4], d->H, d->w_dtype, &w) && arrays(v[5], d->R, all, d->dtype, 1, &h) &&
        arrays(v[6], d->R, all, d->dtype, 1, &y) && arrays(v[7], d->R, all, KIND_8BIT, 1, &q) &&
        arrays(v[8], d->R, groups, KIND_F32, 1, &scale) && arrays(v[9], d->R, rows, KIND_F32, 1, &rstd)) {
      fo_stream_t s = (fo_stream_t)PyLong_AsVoidPtr(v[10]);
      if (!PyErr_Occurred()) {
        Py_BEGIN_ALLOW_THREADS
        code = fo_rmsnorm(d, rows, (const void *const *)x.p, (const void *const *)res.p, w, h.p, y.p, q.p,
                          (float *const *)scale.p, (float *const *)rstd.p, s);
        Py_END_ALLOW_THREADS
      }
    }
  }
  PyBuffer_Release(&b);
  return code < 0 ? unknown() : PyLong_FromLong(code);
}

/* (desc, rows, dy, dh, h, weight, rstd, dx, dweight, ws, stream) */
static PyObject *m_rmsnorm_bwd(PyObject *self, PyObject *const *v, Py_ssize_t n) {
  Py_buffer b;
  fo_norm_desc *d = n == 11 ? description(v[0], &b, sizeof(*d)) : NULL;
  if (!d) return unknown();
  const long long rows = PyLong_AsLongLong(v[1]);
  long code = -1;
  if (in_range(d->R) && rows > 0 && d->H > 0) {
    const long long all = rows * d->H;
    array dy, dh, h, rstd, dx;
    void *w, *dw = NULL, *ws = NULL;
    size_t need;
    if (arrays(v[2], d->R, all, d->dtype, 0, &dy) && arrays(v[3], d->R, all, d->dtype, 1, &dh) &&
        arrays(v[4], d->R, all, d->dtype, 0, &h) && dense(v[5], d->H, d->w_dtype, &w) &&
        arrays(v[6], d->R, rows, KIND_F32, 0, &rstd) && arrays(v[7], d->R, all, d->dtype, 0, &dx) &&
        (v[8] == Py_None || dense(v[8], d->H, KIND_F32, &dw)) && fo_rmsnorm_bwd_workspace(d, rows, &need) == FO_OK &&
        (v[9] == Py_None || (is_dtype(v[9], t_u8, t_u8) == 1 && number(v[9], s_numel) >= (long long)need &&
                             dense(v[9], number(v[9], s_numel), KIND_8BIT, &ws)))) {
      fo_stream_t s = (fo_stream_t)PyLong_AsVoidPtr(v[10]);
      if (!PyErr_Occurred()) {
        Py_BEGIN_ALLOW_THREADS
        code = fo_rmsnorm_bwd(d, rows, (const void *const *)dy.p, (const void *const *)dh.p, (const void *const *)h.p, w,
                              (const float *const *)rstd.p, dx.p, (float *)dw, ws, s);
        Py_END_ALLOW_THREADS
      }
    }
  }
  PyBuffer_Release(&b);
  return code < 0 ? unknown() : PyLong_FromLong(code);
}

/* (rows, cols, dtype, block_rows, x, q, scale, qt, scale_t, stream) */
static PyObject *m_quant_fp8(PyObject *self, PyObject *const *v, Py_ssize_t n) {
  if (n != 10 || !PyList_CheckExact(v[4])) return unknown();
  const long long rows = PyLong_AsLongLong(v[0]), cols = PyLong_AsLongLong(v[1]);
  const long dtype = PyLong_AsLong(v[2]), block = PyLong_AsLong(v[3]);
  const Py_ssize_t R = PyList_GET_SIZE(v[4]);
  long code = -1;
  if (R >= 1 && R <= MAX_R && rows > 0 && cols > 0 && (block == 1 || block == FO_FP8_BLOCK) && (dtype == 0 || dtype == 1)) {
    const long long all = rows * cols;
    const long long blocks = ((rows + block - 1) / block) * ((cols + FO_FP8_BLOCK - 1) / FO_FP8_BLOCK);
    array x, q, scale, qt, st;
    if (arrays(v[4], (int)R, all, (int)dtype, 0, &x) && arrays(v[5], (int)R, all, KIND_8BIT, 0, &q) &&
        arrays(v[6], (int)R, blocks, KIND_F32, 0, &scale) && arrays(v[7], (int)R, all, KIND_8BIT, 1, &qt) &&
        arrays(v[8], (int)R, blocks, KIND_F32, 1, &st)) {
      fo_stream_t s = (fo_stream_t)PyLong_AsVoidPtr(v[9]);
      if (!PyErr_Occurred()) {
        Py_BEGIN_ALLOW_THREADS
        code = fo_quant_fp8((int32_t)R, rows, cols, (int32_t)dtype, (int32_t)block, (const void *const *)x.p, q.p,
                            (float *const *)scale.p, qt.p, (float *const *)st.p, s);
        Py_END_ALLOW_THREADS
      }
    }
  }
  return code < 0 ? unknown() : PyLong_FromLong(code);
}

/* (desc, M, A, sA, W, sW, Y, ws, stream) */
static PyObject *m_gemm_fp8(PyObject *self, PyObject *const *v, Py_ssize_t n) {
  Py_buffer b;
  fo_gemm_fp8_desc *d = n == 9 ? description(v[0], &b, sizeof(*d)) : NULL;
  if (!d) return unknown();
  const long long M = PyLong_AsLongLong(v[1]);
  long code = -1;
  if (in_range(d->R) && M > 0 && d->N > 0 && d->K > 0) {
    const long long k = (d->K + FO_FP8_BLOCK - 1) / FO_FP8_BLOCK, nb = (d->N + FO_FP8_BLOCK - 1) / FO_FP8_BLOCK;
    array A, sA, W, sW, Y;
    void *ws;
    size_t need;
    if (arrays(v[2], d->R, M * d->K, KIND_8BIT, 0, &A) && arrays(v[3], d->R, M * k, KIND_F32, 0, &sA) &&
        arrays(v[4], d->R, d->N * d->K, KIND_8BIT, 0, &W) && arrays(v[5], d->R, nb * k, KIND_F32, 0, &sW) &&
        arrays(v[6], d->R, M * d->N, d->out_dtype, 0, &Y) && fo_gemm_fp8_workspace(d, M, &need) == FO_OK &&
        is_dtype(v[7], t_u8, t_u8) == 1 && number(v[7], s_numel) >= (long long)need &&
        dense(v[7], number(v[7], s_numel), KIND_8BIT, &ws)) {
      fo_stream_t s = (fo_stream_t)PyLong_AsVoidPtr(v[8]);
      if (!PyErr_Occurred()) {
        Py_BEGIN_ALLOW_THREADS
        code = fo_gemm_fp8(d, M, (const void *const *)A.p, (const float *const *)sA.p, (const void *const *)W.p,
                           (const float *const *)sW.p, Y.p, ws, s);
        Py_END_ALLOW_THREADS
      }
    }
  }
  PyBuffer_Release(&b);
  return code < 0 ? unknown() : PyLong_FromLong(code);
}

/* (desc, rows, positions, q_in, k_in, v_in, q_out, k_out, v_out, inverse, stream) */
static PyObject *m_rope(PyObject *self, PyObject *const *v, Py_ssize_t n) {
  Py_buffer b;
  fo_rope_desc *d = n == 11 ? description(v[0], &b, sizeof(*d)) : NULL;
  if (!d) return unknown();
  const long long rows = PyLong_AsLongLong(v[1]);
  long code = -1;
  int ok = in_range(d->R) && rows > 0;
  void *pos = NULL;
  int32_t bytes = 8;
  if (ok && v[2] != Py_None) {
    const int wide = is_dtype(v[2], t_i64, t_i64);
    ok = (wide == 1 || is_dtype(v[2], t_i32, t_i32) == 1) && number(v[2], s_numel) == rows &&
         truth(PyObject_CallMethodNoArgs(v[2], s_is_contiguous)) == 1 && truth(PyObject_GetAttr(v[2], s_is_cuda)) == 1 &&
         (pos = address(v[2])) != NULL;
    bytes = wide == 1 ? 8 : 4;
  }
  const int32_t heads[3] = {d->heads_q, d->heads_k, d->heads_v};
  array in[3], out[3];
  int64_t ld_in[3] = {0, 0, 0}, ld_out[3] = {0, 0, 0};
  for (int j = 0; j < 3; ++j) {
    in[j].p = out[j].p = NULL;
    if (!ok || heads[j] == 0) continue;
    const long long width = (long long)heads[j] * d->head_dim;
    ok = heads[j] > 0 && row_arrays(v[3 + j], d->R, rows, width, d->dtype, &in[j], &ld_in[j]) &&
         row_arrays(v[6 + j], d->R, rows, width, d->dtype, &out[j], &ld_out[j]);
  }
  if (ok) {
    const int inverse = PyObject_IsTrue(v[9]);
    fo_stream_t s = (fo_stream_t)PyLong_AsVoidPtr(v[10]);
    if (!PyErr_Occurred() && inverse >= 0) {
      Py_BEGIN_ALLOW_THREADS
      code = fo_rope(d, rows, pos, bytes, (const void *const *)in[0].p, (const void *const *)in[1].p,
                     (const void *const *)in[2].p, ld_in, out[0].p, out[1].p, out[2].p, ld_out, inverse, s);
      Py_END_ALLOW_THREADS
    }
  }
  PyBuffer_Release(&b);
  return code < 0 ? unknown() : PyLong_FromLong(code);
}

/* (bfloat16, float32, float8_e4m3fn, uint8, int32, int64): torch's types. */
static PyObject *m_setup(PyObject *self, PyObject *const *v, Py_ssize_t n) {
  PyObject **to[6] = {&t_bf16, &t_f32, &t_e4m3, &t_u8, &t_i32, &t_i64};
  if (n != 6) {
    PyErr_SetString(PyExc_TypeError, "setup takes six types");
    return NULL;
  }
  for (int i = 0; i < 6; ++i) {
    Py_INCREF(v[i]);
    Py_XSETREF(*to[i], v[i]);
  }
  Py_RETURN_NONE;
}

#define FAST(name) {#name, (PyCFunction)(void (*)(void))m_##name, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {FAST(setup), FAST(rmsnorm), FAST(rmsnorm_bwd), FAST(quant_fp8), FAST(gemm_fp8), FAST(rope),
                                {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fo_marshal", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__fo_marshal(void) {
  s_dtype = PyUnicode_InternFromString("dtype");
  s_numel = PyUnicode_InternFromString("numel");
  s_is_contiguous = PyUnicode_InternFromString("is_contiguous");
  s_is_cuda = PyUnicode_InternFromString("is_cuda");
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  s_shape = PyUnicode_InternFromString("shape");
  s_stride = PyUnicode_InternFromString("stride");
  return PyModule_Create(&module);
}
