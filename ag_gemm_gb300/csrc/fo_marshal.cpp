/* Argument marshalling of the operators between the residual stream and the
 * attention, for Python callers: checks the tensors and hands their addresses to the C
 * ABI. The same checks exist in binding.py, which explains what is
 * wrong with an argument; this module only recognises calls that are right and
 * returns -1 for all others, having done nothing. A decode step's norm (8 x
 * 4096, seven tensors) takes 4.9 us of host time this way, with its caller's
 * lists, and 15.4 us marshalled in Python; of both, the driver's look at the
 * seven addresses is 1.1 us. */
#define PY_SSIZE_T_CLEAN
#include <torch/csrc/autograd/python_variable.h>
#include <c10/cuda/CUDAStream.h>

#include "flashoverlap.h"

#define MAX_R 16

namespace {

enum { KIND_BF16 = 0, KIND_F32 = 1, KIND_8BIT = 2 };

/* The tensor in x (a plain one: other classes may compute what they hold), or NULL. */
const at::Tensor *tensor(PyObject *x) { return THPVariable_CheckExact(x) ? &THPVariable_Unpack(x) : NULL; }

bool of_kind(const at::Tensor &t, int kind) {
  const at::ScalarType s = t.scalar_type();
  return kind == KIND_BF16  ? s == at::kBFloat16
         : kind == KIND_F32 ? s == at::kFloat
                            : s == at::kFloat8_e4m3fn || s == at::kByte;
}

/* A dense CUDA tensor of n values: true and its address. */
bool dense(PyObject *x, long long n, int kind, void **out) {
  const at::Tensor *t = tensor(x);
  if (!t || !t->is_cuda() || !of_kind(*t, kind) || t->numel() != n || !t->is_contiguous()) return false;
  *out = t->data_ptr();
  return *out != NULL;
}
/* A workspace of at least `need` bytes. */
bool workspace(PyObject *x, size_t need, void **out) {
  const at::Tensor *t = tensor(x);
  return t && t->scalar_type() == at::kByte && (unsigned long long)t->numel() >= need && dense(x, t->numel(), KIND_8BIT, out);
}

struct array {
  void *at[MAX_R];
  void **p; /* at, or NULL for None */
};

/* R tensors in a list, or None where that is allowed. */
bool arrays(PyObject *xs, int R, long long n, int kind, bool optional, array *a) {
  a->p = NULL;
  if (xs == Py_None) return optional;
  if (!PyList_CheckExact(xs) || PyList_GET_SIZE(xs) != R) return false;
  PyObject *last = NULL;
  for (int r = 0; r < R; ++r) {
    PyObject *x = PyList_GET_ITEM(xs, r);
    if (x == last) a->at[r] = a->at[r - 1];
    else if (!dense(x, n, kind, &a->at[r])) return false;
    last = x;
  }
  a->p = a->at;
  return true;
}

/* The R matrices [rows x width] of a list, their rows dense and one stride apart. */
bool row_arrays(PyObject *xs, int R, long long rows, long long width, int kind, array *a, int64_t *ld) {
  a->p = NULL;
  if (!PyList_CheckExact(xs) && !PyTuple_CheckExact(xs)) return false;
  if (PySequence_Fast_GET_SIZE(xs) != R) return false;
  *ld = -1;
  for (int r = 0; r < R; ++r) {
    const at::Tensor *t = tensor(PySequence_Fast_GET_ITEM(xs, r));
    if (!t || !t->is_cuda() || !of_kind(*t, kind) || t->dim() != 2 || t->size(0) != rows || t->size(1) != width) return false;
    if (width > 1 && t->stride(1) != 1) return false;
    const long long step = rows > 1 ? t->stride(0) : width;
    if (*ld >= 0 && step != *ld) return false;
    *ld = step;
    if (!(a->at[r] = t->data_ptr())) return false;
  }
  a->p = a->at;
  return true;
}

/* The stream's address: an int, None for torch's current one, or a torch stream. */
bool stream_of(PyObject *o, fo_stream_t *s) {
  if (o == Py_None) {
    *s = (fo_stream_t)c10::cuda::getCurrentCUDAStream().stream();
    return true;
  }
  if (PyLong_Check(o)) {
    *s = (fo_stream_t)PyLong_AsVoidPtr(o);
    return !PyErr_Occurred();
  }
  PyObject *at = PyObject_GetAttrString(o, "cuda_stream");
  if (!at) return false;
  *s = (fo_stream_t)PyLong_AsVoidPtr(at);
  Py_DECREF(at);
  return !PyErr_Occurred();
}

/* A description (a ctypes structure of that size), held until the call ends. */
template <typename T>
struct Description {
  Py_buffer view;
  bool held;
  explicit Description(PyObject *o) : held(o && PyObject_GetBuffer(o, &view, PyBUF_SIMPLE) == 0) {}
  ~Description() {
    if (held) PyBuffer_Release(&view);
  }
  const T *get() const { return held && view.len == (Py_ssize_t)sizeof(T) ? (const T *)view.buf : NULL; }
};

PyObject *unknown(void) {
  PyErr_Clear();
  return PyLong_FromLong(-1);
}

bool in_range(int R) { return R >= 1 && R <= MAX_R; }

/* (desc, rows, x, residual, weight, h, y, q, scale, rstd, stream) */
PyObject *m_rmsnorm(PyObject *self, PyObject *const *v, Py_ssize_t n) {
  const Description<fo_norm_desc> held(n == 11 ? v[0] : NULL);
  const fo_norm_desc *d = held.get();
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
      fo_stream_t s;
      if (stream_of(v[10], &s)) {
        Py_BEGIN_ALLOW_THREADS
        code = fo_rmsnorm(d, rows, (const void *const *)x.p, (const void *const *)res.p, w, h.p, y.p, q.p,
                          (float *const *)scale.p, (float *const *)rstd.p, s);
        Py_END_ALLOW_THREADS
      }
    }
  }
  return code < 0 ? unknown() : PyLong_FromLong(code);
}

/* (desc, rows, dy, dh, h, weight, rstd, dx, dweight, ws, stream) */
PyObject *m_rmsnorm_bwd(PyObject *self, PyObject *const *v, Py_ssize_t n) {
  const Description<fo_norm_desc> held(n == 11 ? v[0] : NULL);
  const fo_norm_desc *d = held.get();
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
        (v[9] == Py_None || workspace(v[9], need, &ws))) {
      fo_stream_t s;
      if (stream_of(v[10], &s)) {
        Py_BEGIN_ALLOW_THREADS
        code = fo_rmsnorm_bwd(d, rows, (const void *const *)dy.p, (const void *const *)dh.p, (const void *const *)h.p, w,
                              (const float *const *)rstd.p, dx.p, (float *)dw, ws, s);
        Py_END_ALLOW_THREADS
      }
    }
  }
  return code < 0 ? unknown() : PyLong_FromLong(code);
}

/* (rows, cols, dtype, block_rows, x, q, scale, qt, scale_t, stream) */
PyObject *m_quant_fp8(PyObject *self, PyObject *const *v, Py_ssize_t n) {
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
      fo_stream_t s;
      if (stream_of(v[9], &s)) {
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
PyObject *m_gemm_fp8(PyObject *self, PyObject *const *v, Py_ssize_t n) {
  const Description<fo_gemm_fp8_desc> held(n == 9 ? v[0] : NULL);
  const fo_gemm_fp8_desc *d = held.get();
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
        workspace(v[7], need, &ws)) {
      fo_stream_t s;
      if (stream_of(v[8], &s)) {
        Py_BEGIN_ALLOW_THREADS
        code = fo_gemm_fp8(d, M, (const void *const *)A.p, (const float *const *)sA.p, (const void *const *)W.p,
                           (const float *const *)sW.p, Y.p, ws, s);
        Py_END_ALLOW_THREADS
      }
    }
  }
  return code < 0 ? unknown() : PyLong_FromLong(code);
}

/* (desc, rows, positions, q_in, k_in, v_in, q_out, k_out, v_out, inverse, stream) */
PyObject *m_rope(PyObject *self, PyObject *const *v, Py_ssize_t n) {
  const Description<fo_rope_desc> held(n == 11 ? v[0] : NULL);
  const fo_rope_desc *d = held.get();
  if (!d) return unknown();
  const long long rows = PyLong_AsLongLong(v[1]);
  long code = -1;
  bool ok = in_range(d->R) && rows > 0;
  void *pos = NULL;
  int32_t bytes = 8;
  if (ok && v[2] != Py_None) {
    const at::Tensor *t = tensor(v[2]);
    ok = t && t->is_cuda() && (t->scalar_type() == at::kLong || t->scalar_type() == at::kInt) && t->numel() == rows &&
         t->is_contiguous() && (pos = t->data_ptr()) != NULL;
    if (ok) bytes = (int32_t)t->element_size();
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
    fo_stream_t s;
    if (inverse >= 0 && stream_of(v[10], &s)) {
      Py_BEGIN_ALLOW_THREADS
      code = fo_rope(d, rows, pos, bytes, (const void *const *)in[0].p, (const void *const *)in[1].p,
                     (const void *const *)in[2].p, ld_in, out[0].p, out[1].p, out[2].p, ld_out, inverse, s);
      Py_END_ALLOW_THREADS
    }
  }
  return code < 0 ? unknown() : PyLong_FromLong(code);
}

/* No C++ exception leaves the module: a call that meets one is for binding.py too. */
template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyObject *guarded(PyObject *self, PyObject *const *v, Py_ssize_t n) {
  try {
    return F(self, v, n);
  } catch (...) {
    return unknown();
  }
}

#define FAST(name) {#name, (PyCFunction)(void (*)(void))guarded<m_##name>, METH_FASTCALL, NULL}
PyMethodDef methods[] = {FAST(rmsnorm), FAST(rmsnorm_bwd), FAST(quant_fp8), FAST(gemm_fp8), FAST(rope),
                         {NULL, NULL, 0, NULL}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fo_marshal", NULL, -1, methods, NULL, NULL, NULL, NULL};

}  // namespace

PyMODINIT_FUNC PyInit__fo_marshal(void) { return PyModule_Create(&module); }
