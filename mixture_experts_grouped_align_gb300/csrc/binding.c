/* Argument marshalling of the training and dense calls for CPython.
 *
 * The small calls of these operators take less time on the GPU than their Python side: through
 * ctypes a call of nine tensors spent 4 us on checking and converting its arguments.  Each
 * function here takes the arguments of its C call in order -- tensors (torch tensors, raw device
 * pointers as ints, or None), numbers, and the address of the moe_ctx -- checks every tensor's
 * type, density, place and size, and calls the library.  It returns the status; a tensor that
 * fails the checks is handed to the error function, which raises.
 *
 * setup(error, f32, i32, bf16, u8, addresses): the error function (tensor, name, type, elements),
 * the torch types and the addresses of the library's functions, in the order of `enum`.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

#include "moe_gb300.h"

enum { F_ROUTER, F_ACT_FWD, F_ACT_BWD, F_DENSE, F_BIAS, F_PAIRS, F_COUNT };
enum { T_F32, T_I32, T_BF16, T_U8, T_COUNT };

static void* g_fn[F_COUNT];
static PyObject* g_type[T_COUNT];
static PyObject* g_error;
static PyObject *s_dtype, *s_is_contiguous, *s_is_cuda, *s_numel, *s_data_ptr;

/* The device pointer of a tensor argument; 0 and an exception if it is not what the call reads. */
static int tensor_arg(PyObject* t, const char* what, int type, int64_t need, void** out) {
  if (t == Py_None) {
    *out = NULL;
    return 1;
  }
  if (PyLong_Check(t)) {
    *out = PyLong_AsVoidPtr(t);
    return *out != NULL || !PyErr_Occurred();
  }
  int ok = 0;
  PyObject* v = PyObject_GetAttr(t, s_dtype);
  if (v == NULL) return 0;
  ok = v == g_type[type];
  Py_DECREF(v);
  if (ok) {
    if ((v = PyObject_CallMethodNoArgs(t, s_is_contiguous)) == NULL) return 0;
    ok = v == Py_True;
    Py_DECREF(v);
  }
  if (ok) {
    if ((v = PyObject_GetAttr(t, s_is_cuda)) == NULL) return 0;
    ok = v == Py_True;
    Py_DECREF(v);
  }
  if (ok) {
    if ((v = PyObject_CallMethodNoArgs(t, s_numel)) == NULL) return 0;
    const long long n = PyLong_AsLongLong(v);
    Py_DECREF(v);
    if (n == -1 && PyErr_Occurred()) return 0;
    ok = n >= need;
  }
  if (ok) {
    if ((v = PyObject_CallMethodNoArgs(t, s_data_ptr)) == NULL) return 0;
    *out = PyLong_AsVoidPtr(v);
    Py_DECREF(v);
    return *out != NULL || !PyErr_Occurred();
  }
  PyObject* r = PyObject_CallFunction(g_error, "OsOL", t, what, g_type[type], (long long)need);
  Py_XDECREF(r);
  if (r != NULL) PyErr_Format(PyExc_RuntimeError, "%s: refused", what);
  return 0;
}

/* The error function's path for numbers: 0 and an exception if `o` does not fit. */
static int int_arg(PyObject* o, long long lo, long long hi, long long* out) {
  *out = PyLong_AsLongLong(o);
  if (*out == -1 && PyErr_Occurred()) return 0;
  if (*out < lo || *out > hi) {
    PyErr_SetString(PyExc_OverflowError, "an argument does not fit the C call's type");
    return 0;
  }
  return 1;
}
static int float_arg(PyObject* o, float* out) {
  const double d = PyFloat_AsDouble(o);
  if (d == -1.0 && PyErr_Occurred()) return 0;
  *out = (float)d;
  return 1;
}

/* Elements of a product of sizes for the check (negative sizes are the C call's to refuse). */
static int64_t elems(int64_t a, int64_t b) {
  int64_t r;
  if (a <= 0 || b <= 0) return 0;
  return __builtin_mul_overflow(a, b, &r) ? INT64_MAX : r;
}

static int count(Py_ssize_t got, Py_ssize_t want) {
  if (got == want) return 1;
  PyErr_Format(PyExc_TypeError, "%zd arguments, need %zd", got, want);
  return 0;
}

#define I64(o, v) int_arg(o, INT64_MIN, INT64_MAX, &v)
#define I32(o, v) int_arg(o, INT32_MIN, INT32_MAX, &v)
/* Calls the library without the interpreter lock, as a launch may wait for room in its queue. */
#define CALL(name, index, ...)                                     \
  moe_status status;                                               \
  Py_BEGIN_ALLOW_THREADS;                                          \
  status = ((__typeof__(&name))g_fn[index])(__VA_ARGS__);          \
  Py_END_ALLOW_THREADS;                                            \
  return PyLong_FromLong(status)
#define CTX(o, v) tensor_arg(o, "ctx", T_U8, 0, &v)

static PyObject* router_loss(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  long long T, k, E;
  float bal, z;
  void *lg, *ids, *w, *dw, *mask, *counts, *mean, *loss, *d, *ctx;
  if (!count(n, 15) || !I64(a[5], T) || !I32(a[6], k) || !I32(a[7], E) || !float_arg(a[8], &bal) || !float_arg(a[9], &z))
    return NULL;
  const int64_t te = elems(T, E), tk = elems(T, k);
  if (!tensor_arg(a[0], "logits", T_F32, te, &lg) || !tensor_arg(a[1], "topk_ids", T_I32, tk, &ids) ||
      !tensor_arg(a[2], "topk_w", T_F32, tk, &w) || !tensor_arg(a[3], "d_topk_w", T_F32, tk, &dw) ||
      !tensor_arg(a[4], "token_mask", T_U8, T, &mask) || !tensor_arg(a[10], "counts", T_I32, E, &counts) ||
      !tensor_arg(a[11], "prob_mean", T_F32, E, &mean) || !tensor_arg(a[12], "loss", T_F32, 3, &loss) ||
      !tensor_arg(a[13], "d_logits", T_F32, te, &d) || !CTX(a[14], ctx))
    return NULL;
  CALL(moe_router_loss, F_ROUTER, lg, ids, w, dw, mask, T, (int32_t)k, (int32_t)E, bal, z, counts, mean, loss, d, ctx);
}

static PyObject* act_checkpoint(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  long long rows, I, act;
  void *gu, *w, *h, *codes, *scales, *ctx;
  if (!count(n, 9) || !I64(a[2], rows) || !I32(a[3], I) || !I32(a[4], act)) return NULL;
  const int64_t n1 = act == MOE_ACT_RELU2 ? I : 2 * I;
  if (!tensor_arg(a[0], "gu", T_BF16, elems(rows, n1), &gu) || !tensor_arg(a[1], "row_w", T_F32, rows, &w) ||
      !tensor_arg(a[5], "h", T_BF16, elems(rows, I), &h) || !tensor_arg(a[6], "codes", T_U8, elems(rows, n1), &codes) ||
      !tensor_arg(a[7], "scales", T_U8, elems(rows, n1 / 32), &scales) || !CTX(a[8], ctx))
    return NULL;
  CALL(moe_act_checkpoint, F_ACT_FWD, gu, w, rows, (int32_t)I, (int32_t)act, h, codes, scales, ctx);
}

static PyObject* act_backward(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  long long rows, I, act;
  void *codes, *scales, *dh, *w, *dgu, *h, *dw, *ctx;
  if (!count(n, 11) || !I64(a[4], rows) || !I32(a[5], I) || !I32(a[6], act)) return NULL;
  const int64_t n1 = act == MOE_ACT_RELU2 ? I : 2 * I;
  if (!tensor_arg(a[0], "codes", T_U8, elems(rows, n1), &codes) ||
      !tensor_arg(a[1], "scales", T_U8, elems(rows, n1 / 32), &scales) ||
      !tensor_arg(a[2], "dh", T_BF16, elems(rows, I), &dh) || !tensor_arg(a[3], "row_w", T_F32, rows, &w) ||
      !tensor_arg(a[7], "d_gu", T_BF16, elems(rows, n1), &dgu) || !tensor_arg(a[8], "h", T_BF16, elems(rows, I), &h) ||
      !tensor_arg(a[9], "d_row_w", T_F32, rows, &dw) || !CTX(a[10], ctx))
    return NULL;
  CALL(moe_act_backward, F_ACT_BWD, codes, scales, dh, w, rows, (int32_t)I, (int32_t)act, dgu, h, dw, ctx);
}

static PyObject* dense_gemm(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  long long layout, M, N, K, act, f32;
  float scale;
  void *x, *w, *bias, *res, *out, *ctx;
  if (!count(n, 13) || !I32(a[2], layout) || !float_arg(a[5], &scale) || !I64(a[6], M) || !I32(a[7], N) || !I32(a[8], K) ||
      !I32(a[9], act) || !I32(a[11], f32))
    return NULL;
  const int64_t n1 = act == MOE_ACT_SWIGLU ? 2 * N : N;
  const int ot = f32 ? T_F32 : T_BF16;
  if (!tensor_arg(a[0], "x", T_BF16, elems(M, K), &x) || !tensor_arg(a[1], "w", T_BF16, elems(n1, K), &w) ||
      !tensor_arg(a[3], "bias", T_BF16, n1, &bias) || !tensor_arg(a[4], "residual", ot, elems(M, N), &res) ||
      !tensor_arg(a[10], "out", ot, elems(M, N), &out) || !CTX(a[12], ctx))
    return NULL;
  CALL(moe_dense_gemm, F_DENSE, x, w, (int32_t)layout, bias, res, scale, M, (int32_t)N, (int32_t)K, (int32_t)act, out, (int32_t)f32, ctx);
}

static PyObject* dense_bias_grad(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  long long M, N;
  void *dz, *db, *ctx;
  if (!count(n, 5) || !I64(a[1], M) || !I32(a[2], N) || !tensor_arg(a[0], "dz", T_BF16, elems(M, N), &dz) ||
      !tensor_arg(a[3], "d_bias", T_F32, N, &db) || !CTX(a[4], ctx))
    return NULL;
  CALL(moe_dense_bias_grad, F_BIAS, dz, M, (int32_t)N, db, ctx);
}

static PyObject* pair_sum(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  long long T, k, K;
  void *o, *res, *y, *ctx;
  if (!count(n, 7) || !I64(a[2], T) || !I32(a[3], k) || !I32(a[4], K) ||
      !tensor_arg(a[0], "o", T_BF16, elems(elems(T, k), K), &o) || !tensor_arg(a[1], "residual", T_BF16, elems(T, K), &res) ||
      !tensor_arg(a[5], "y", T_BF16, elems(T, K), &y) || !CTX(a[6], ctx))
    return NULL;
  CALL(moe_pair_sum, F_PAIRS, o, res, T, (int32_t)k, (int32_t)K, y, ctx);
}

static PyObject* setup(PyObject* self, PyObject* args) {
  (void)self;
  PyObject *error, *type[T_COUNT], *fns;
  if (!PyArg_ParseTuple(args, "OOOOOO!", &error, &type[0], &type[1], &type[2], &type[3], &PyTuple_Type, &fns)) return NULL;
  if (PyTuple_GET_SIZE(fns) != F_COUNT) {
    PyErr_Format(PyExc_ValueError, "need %d addresses", (int)F_COUNT);
    return NULL;
  }
  for (int i = 0; i < F_COUNT; ++i)
    if ((g_fn[i] = PyLong_AsVoidPtr(PyTuple_GET_ITEM(fns, i))) == NULL) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null address");
      return NULL;
    }
  Py_INCREF(error);
  Py_XSETREF(g_error, error);
  for (int i = 0; i < T_COUNT; ++i) {
    Py_INCREF(type[i]);
    Py_XSETREF(g_type[i], type[i]);
  }
  Py_RETURN_NONE;
}

#define FAST(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {{"setup", setup, METH_VARARGS, NULL}, FAST(router_loss), FAST(act_checkpoint), FAST(act_backward),
                                FAST(dense_gemm), FAST(dense_bias_grad), FAST(pair_sum), {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__binding(void) {
  if (!(s_dtype = PyUnicode_InternFromString("dtype")) || !(s_is_contiguous = PyUnicode_InternFromString("is_contiguous")) ||
      !(s_is_cuda = PyUnicode_InternFromString("is_cuda")) || !(s_numel = PyUnicode_InternFromString("numel")) ||
      !(s_data_ptr = PyUnicode_InternFromString("data_ptr")))
    return NULL;
  return PyModule_Create(&module);
}
