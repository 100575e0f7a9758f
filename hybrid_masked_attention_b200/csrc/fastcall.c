/* Argument marshalling of the 8-bit operators for CPython.
 *
 * One function for each operator: it reads the tensors' attributes, and where every check of
 * the Python wrapper holds and the tensors' device is the current one, calls the C entry point
 * and returns its status.  In any other case it returns None without having called anything,
 * and the wrapper in __init__.py goes through its own checks, which name the fault (or switch
 * the device).  A wrapper alone spends 5 to 9 microseconds a call on attribute reads and
 * ctypes, more than the kernels of one-token calls; this takes about 2.
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "../../include/mtfm.h"

#define FN(name) static __typeof__(&name) p_##name
FN(mtfm_add_rmsnorm_fp8);
FN(mtfm_rmsnorm_bwd);
FN(mtfm_gate_fwd_fp8);
FN(mtfm_fp8_quant);
FN(mtfm_fp8_gemm);

static PyObject *s_dtype, *s_shape, *s_stride, *s_data_ptr, *s_get_device;
static PyObject *d_f32, *d_bf16, *d_f8, *d_u8, *d_i32; /* torch dtypes */
static PyObject *f_device, *f_stream;                  /* current device, raw stream of a device */

typedef struct {
  void* p;
  int64_t ld;
  int type;
} Mat;

/* Integer result of a method without arguments; -1 with `*ok` 0 on any error. */
static long long call_int(PyObject* t, PyObject* name, int* ok) {
  PyObject* r = PyObject_CallMethodNoArgs(t, name);
  if (!r) { *ok = 0; return -1; }
  long long v = PyLong_Check(r) ? (long long)PyLong_AsUnsignedLongLongMask(r) : -1;
  if (!PyLong_Check(r)) *ok = 0;
  Py_DECREF(r);
  return v;
}

/* shape (attribute) or stride (method) as up to two integers; returns their number, -1 on error. */
static int two(PyObject* r, int64_t* a, int64_t* b) {
  int n = -1;
  if (r && PyTuple_Check(r)) {
    n = (int)PyTuple_GET_SIZE(r);
    if (n >= 1) *a = PyLong_AsLongLong(PyTuple_GET_ITEM(r, 0));
    if (n >= 2) *b = PyLong_AsLongLong(PyTuple_GET_ITEM(r, 1));
    if (PyErr_Occurred()) n = -1;
  }
  Py_XDECREF(r);
  return n;
}

/* The device of a CUDA matrix and its shape; -1 where t is none. */
static long matrix(PyObject* t, int64_t* rows, int64_t* cols) {
  int ok = 1;
  long dev = (long)call_int(t, s_get_device, &ok);
  if (!ok || dev < 0) return -1;
  return two(PyObject_GetAttr(t, s_shape), rows, cols) == 2 ? dev : -1;
}

/* A [rows, cols] matrix with unit column stride on device dev; dtype NULL: fp32 or bf16. */
static int mat(PyObject* t, long dev, PyObject* dtype, int64_t rows, int64_t cols, Mat* m) {
  int64_t r = -1, c = -1, inner = 0;
  int ok = 1;
  PyObject* d = PyObject_GetAttr(t, s_dtype);
  if (!d) return 0;
  Py_DECREF(d); /* dtypes live as long as torch */
  if (dtype ? d != dtype : (d != d_f32 && d != d_bf16)) return 0;
  m->type = d == d_bf16;
  if (matrix(t, &r, &c) != dev || r != rows || c != cols) return 0;
  if (two(PyObject_CallMethodNoArgs(t, s_stride), &m->ld, &inner) != 2) return 0;
  if ((inner != 1 && cols > 1) || (m->ld < cols && rows > 1)) return 0;
  m->p = (void*)(uintptr_t)call_int(t, s_data_ptr, &ok);
  return ok;
}
static int opt_mat(PyObject* t, long dev, PyObject* dtype, int64_t rows, int64_t cols, Mat* m) {
  m->p = NULL;
  m->ld = m->type = 0;
  return t == Py_None || mat(t, dev, dtype, rows, cols, m);
}
/* A contiguous matrix, or None. */
static int opt_packed(PyObject* t, long dev, PyObject* dtype, int64_t rows, int64_t cols, void** p) {
  Mat m;
  int ok = opt_mat(t, dev, dtype, rows, cols, &m) && (t == Py_None || rows <= 1 || m.ld == cols);
  *p = ok ? m.p : NULL;
  return ok;
}
/* A contiguous vector; n < 0: of any length, returned there. */
static int vec(PyObject* t, long dev, PyObject* dtype, int64_t* n, void** p) {
  int64_t len = -1, x = 0, stride = 0;
  int ok = 1;
  PyObject* d = PyObject_GetAttr(t, s_dtype);
  if (!d) return 0;
  Py_DECREF(d);
  if (d != dtype || (long)call_int(t, s_get_device, &ok) != dev || !ok) return 0;
  if (two(PyObject_GetAttr(t, s_shape), &len, &x) != 1 || (*n >= 0 && len != *n)) return 0;
  if (two(PyObject_CallMethodNoArgs(t, s_stride), &stride, &x) != 1 || (stride != 1 && len > 1)) return 0;
  *n = len;
  *p = (void*)(uintptr_t)call_int(t, s_data_ptr, &ok);
  return ok;
}
static int vec_n(PyObject* t, long dev, PyObject* dtype, int64_t n, void** p) { return vec(t, dev, dtype, &n, p); }

/* The current stream of `dev`, if that is the current device. */
static int stream_of(long dev, void** st) {
  PyObject* r = PyObject_CallNoArgs(f_device);
  if (!r) return 0;
  long cur = PyLong_AsLong(r);
  Py_DECREF(r);
  if (cur != dev) return 0;
  PyObject* arg = PyLong_FromLong(dev);
  r = arg ? PyObject_CallOneArg(f_stream, arg) : NULL;
  Py_XDECREF(arg);
  if (!r) return 0;
  *st = (void*)(uintptr_t)PyLong_AsUnsignedLongLongMask(r);
  Py_DECREF(r);
  return 1;
}
static int64_t groups(int64_t n) { return (n + 127) / 128; }
static int fits(int64_t n) { return n >= 0 && n <= INT32_MAX; }
/* Returns the status of a call made without the interpreter's lock: a launch that waits for room
 * in its queue must not stop the other threads, one of which the queue may be waiting for. */
#define CALL(expr)             \
  do {                         \
    mtfm_status s_;            \
    Py_BEGIN_ALLOW_THREADS     \
    s_ = (expr);               \
    Py_END_ALLOW_THREADS       \
    return PyLong_FromLong(s_); \
  } while (0)
static PyObject* not_taken(void) {
  PyErr_Clear();
  Py_RETURN_NONE;
}

#define ARGS(n) \
  (void)self;   \
  if (nargs != (n)) return not_taken()

/* x, delta, weight, x_out, out, scale, rstd, eps */
static PyObject* add_rmsnorm_fp8(PyObject* self, PyObject* const* a, Py_ssize_t nargs) {
  ARGS(8);
  int64_t rows, dim;
  Mat x, d, xo, q, s;
  void *w, *r = NULL, *st;
  long dev = matrix(a[0], &rows, &dim);
  if (dev < 0 || !fits(rows) || !fits(dim) || !mat(a[0], dev, NULL, rows, dim, &x) ||
      !opt_mat(a[1], dev, NULL, rows, dim, &d) || !vec_n(a[2], dev, d_f32, dim, &w) ||
      !opt_mat(a[3], dev, x.type ? d_bf16 : d_f32, rows, dim, &xo) || !mat(a[4], dev, d_f8, rows, dim, &q) ||
      !mat(a[5], dev, d_f32, rows, groups(dim), &s) || (a[6] != Py_None && !vec_n(a[6], dev, d_f32, rows, &r)) ||
      !PyFloat_Check(a[7]) || !stream_of(dev, &st))
    return not_taken();
  CALL(p_mtfm_add_rmsnorm_fp8((int32_t)rows, (int32_t)dim, x.p, x.type, x.ld, d.p, d.type, d.ld, w,
                              (float)PyFloat_AS_DOUBLE(a[7]), xo.p, xo.ld, q.p, q.ld, s.p, s.ld, r, st));
}

/* x, weight, rstd, dy, dres, dx, dw, ws */
static PyObject* rmsnorm_bwd(PyObject* self, PyObject* const* a, Py_ssize_t nargs) {
  ARGS(8);
  int64_t rows, dim, ws_bytes = -1;
  Mat x, y, dr, dx;
  void *w, *r, *dw, *ws, *st;
  long dev = matrix(a[0], &rows, &dim);
  if (dev < 0 || !fits(rows) || !fits(dim) || !mat(a[0], dev, NULL, rows, dim, &x) || !vec_n(a[1], dev, d_f32, dim, &w) ||
      !vec_n(a[2], dev, d_f32, rows, &r) || !mat(a[3], dev, NULL, rows, dim, &y) ||
      !opt_mat(a[4], dev, NULL, rows, dim, &dr) || !mat(a[5], dev, x.type ? d_bf16 : d_f32, rows, dim, &dx) ||
      !vec_n(a[6], dev, d_f32, dim, &dw) || !vec(a[7], dev, d_u8, &ws_bytes, &ws) || !stream_of(dev, &st))
    return not_taken();
  CALL(p_mtfm_rmsnorm_bwd((int32_t)rows, (int32_t)dim, x.p, x.type, x.ld, w, r, y.p, y.type, y.ld, dr.p, dr.type,
                          dr.ld, dx.p, dx.ld, dw, ws, (size_t)ws_bytes, st));
}

/* cfg (address of an mtfm_cfg), meta, target, a, u, gamma, beta, out, scale, stats */
static PyObject* gate_fwd_fp8(PyObject* self, PyObject* const* a, Py_ssize_t nargs) {
  ARGS(10);
  const mtfm_cfg* cfg = (const mtfm_cfg*)PyLong_AsVoidPtr(a[0]);
  int target = PyObject_IsTrue(a[2]);
  if (!cfg || target < 0) return not_taken();
  const int64_t rows = target ? cfg->total_t : cfg->total_tokens, D = (int64_t)cfg->hq * cfg->head_dim;
  int64_t r, c, meta_bytes = -1;
  void *pa, *pu, *pg, *pb, *ps, *meta, *st;
  Mat q, s;
  long dev = matrix(a[3], &r, &c);
  if (dev < 0 || !vec(a[1], dev, d_u8, &meta_bytes, &meta) || a[3] == Py_None || a[4] == Py_None ||
      !opt_packed(a[3], dev, d_f32, rows, D, &pa) || !opt_packed(a[4], dev, d_bf16, rows, D, &pu) ||
      !opt_packed(a[5], dev, d_f32, 3, D, &pg) || !opt_packed(a[6], dev, d_f32, 3, D, &pb) ||
      !mat(a[7], dev, d_f8, rows, D, &q) || !mat(a[8], dev, d_f32, rows, groups(D), &s) ||
      !opt_packed(a[9], dev, d_f32, rows, 2, &ps) || !stream_of(dev, &st))
    return not_taken();
  CALL(p_mtfm_gate_fwd_fp8(cfg, meta, target, pa, pu, pg, pb, q.p, q.ld, s.p, s.ld, ps, st));
}

/* x, out, scale, block_rows */
static PyObject* fp8_quant(PyObject* self, PyObject* const* a, Py_ssize_t nargs) {
  ARGS(4);
  int64_t rows, cols;
  Mat x, q, s;
  void* st;
  const long br = PyLong_Check(a[3]) ? PyLong_AsLong(a[3]) : 0;
  long dev = matrix(a[0], &rows, &cols);
  if ((br != 1 && br != 128) || dev < 0 || !fits(rows) || !fits(cols) || !mat(a[0], dev, NULL, rows, cols, &x) ||
      !mat(a[1], dev, d_f8, rows, cols, &q) || !mat(a[2], dev, d_f32, (rows + br - 1) / br, groups(cols), &s) ||
      !stream_of(dev, &st))
    return not_taken();
  CALL(p_mtfm_fp8_quant((int32_t)rows, (int32_t)cols, x.p, x.type, x.ld, (int32_t)br, q.p, q.ld, s.p, s.ld, st));
}

/* a, a_scale, b, b_scale, out, status, act (an mtfm_act), residual */
static PyObject* fp8_gemm(PyObject* self, PyObject* const* a, Py_ssize_t nargs) {
  ARGS(8);
  int64_t m, k, n, kb;
  Mat qa, sa, qb, sb, out, res;
  void *status, *st;
  const long act = PyLong_Check(a[6]) ? PyLong_AsLong(a[6]) : -1;
  long dev = matrix(a[0], &m, &k);
  if (dev < 0 || act < 0 || matrix(a[2], &n, &kb) != dev || !fits(m) || !fits(n) || !fits(k) ||
      !mat(a[0], dev, d_f8, m, k, &qa) || !mat(a[1], dev, d_f32, m, groups(k), &sa) || !mat(a[2], dev, d_f8, n, k, &qb) ||
      !mat(a[3], dev, d_f32, groups(n), groups(k), &sb) || !mat(a[4], dev, NULL, m, n, &out) ||
      !vec_n(a[5], dev, d_i32, 1, &status) || !opt_mat(a[7], dev, out.type ? d_bf16 : d_f32, m, n, &res) ||
      !stream_of(dev, &st))
    return not_taken();
  CALL(p_mtfm_fp8_gemm((int32_t)m, (int32_t)n, (int32_t)k, qa.p, qa.ld, sa.p, sa.ld, qb.p, qb.ld, sb.p, sb.ld,
                       (int32_t)act, res.p, res.ld, out.p, out.type, out.ld, status, st));
}

/* (fp32, bf16, e4m3, uint8, int32) dtypes, current device, raw current stream, entry addresses */
static PyObject* setup(PyObject* self, PyObject* args) {
  unsigned long long f[5];
  (void)self;
  if (!PyArg_ParseTuple(args, "OOOOOOOKKKKK", &d_f32, &d_bf16, &d_f8, &d_u8, &d_i32, &f_device, &f_stream, f, f + 1, f + 2,
                        f + 3, f + 4))
    return NULL;
  Py_INCREF(d_f32);
  Py_INCREF(d_bf16);
  Py_INCREF(d_f8);
  Py_INCREF(d_u8);
  Py_INCREF(d_i32);
  Py_INCREF(f_device);
  Py_INCREF(f_stream);
  p_mtfm_add_rmsnorm_fp8 = (__typeof__(p_mtfm_add_rmsnorm_fp8))(uintptr_t)f[0];
  p_mtfm_rmsnorm_bwd = (__typeof__(p_mtfm_rmsnorm_bwd))(uintptr_t)f[1];
  p_mtfm_gate_fwd_fp8 = (__typeof__(p_mtfm_gate_fwd_fp8))(uintptr_t)f[2];
  p_mtfm_fp8_quant = (__typeof__(p_mtfm_fp8_quant))(uintptr_t)f[3];
  p_mtfm_fp8_gemm = (__typeof__(p_mtfm_fp8_gemm))(uintptr_t)f[4];
  Py_RETURN_NONE;
}

#define FAST(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {FAST(add_rmsnorm_fp8), FAST(rmsnorm_bwd), FAST(gate_fwd_fp8), FAST(fp8_quant), FAST(fp8_gemm),
                                {"setup", setup, METH_VARARGS, NULL}, {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fastcall", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__fastcall(void) {
  s_dtype = PyUnicode_InternFromString("dtype");
  s_shape = PyUnicode_InternFromString("shape");
  s_stride = PyUnicode_InternFromString("stride");
  s_data_ptr = PyUnicode_InternFromString("data_ptr");
  s_get_device = PyUnicode_InternFromString("get_device");
  return PyModule_Create(&module);
}
