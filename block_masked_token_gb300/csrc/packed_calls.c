/* The packed-sequence calls of packed.py, from Python objects to the C ABI in one C function
 * each. A step's smallest calls take 3 to 8 us on the GPU; checking ten tensors in Python takes
 * 6 us and ctypes 1.6 us more, these take about 3 together.
 *
 * Each function checks what packed.py checks and, where all is well, makes the call and returns
 * its code. Anything else returns None with nothing called, and packed.py, which then goes
 * through its own checks, raises the error that fits. The stream is the current one. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <limits.h>
#include <stdint.h>

#include "mars.h"

static PyObject *n_device, *n_dtype, *n_shape, *n_stride, *n_contiguous, *n_ptr;
static PyObject *t_tensor, *d_bf16, *d_i32, *d_f32, *d_u8, *f_device, *f_stream;
static __typeof__(&mars_attn_packed) p_packed;
static __typeof__(&mars_attn_packed_grad) p_grad;
static __typeof__(&mars_attn_chunk) p_chunk;
static __typeof__(&mars_kv_append) p_append;
static PyObject* d_e4m3;
static __typeof__(&mars_rotary) p_rotary;
static __typeof__(&mars_kv_append_q8) p_append_q8;
static __typeof__(&mars_attn_chunk_q8) p_chunk_q8;

static PyObject* method(PyObject* t, PyObject* name) {
  PyObject* args[2] = {NULL, t};
  return PyObject_VectorcallMethod(name, args + 1, 1 | PY_VECTORCALL_ARGUMENTS_OFFSET, NULL);
}

/* A Python integer that is not negative, or -1. */
static long long take_int(PyObject* o) {
  if (!o) return -1;
  const long long v = PyLong_AsLongLong(o);
  Py_DECREF(o);
  return v;
}

static int same_device(PyObject* t, long long dev) {
  return PyObject_TypeCheck(t, (PyTypeObject*)t_tensor) && take_int(method(t, n_device)) == dev;
}

/* `nd` numbers of a tuple; 0 if it has not just these, or any is negative or beyond 31 bits. */
static int numbers(PyObject* o, int nd, int* out) {
  int good = o && PyTuple_Check(o) && PyTuple_GET_SIZE(o) == nd;
  for (int i = 0; good && i < nd; ++i) {
    const long long v = PyLong_AsLongLong(PyTuple_GET_ITEM(o, i));
    good = v >= 0 && v <= INT_MAX;
    if (good) out[i] = (int)v;
  }
  Py_XDECREF(o);
  return good;
}

static int shape_of(PyObject* t, int nd, int* out) {
  return numbers(PyObject_GetAttr(t, n_shape), nd, out);
}

static int is_dtype(PyObject* t, PyObject* dtype) {
  PyObject* d = PyObject_GetAttr(t, n_dtype);
  const int good = d == dtype;
  Py_XDECREF(d);
  return good;
}

static int address(PyObject* t, void** p) {
  PyObject* o = method(t, n_ptr);
  if (!o) return 0;
  *p = PyLong_AsVoidPtr(o);
  Py_DECREF(o);
  return !PyErr_Occurred();
}

/* A contiguous tensor of the type, on dev, of shape want[0 .. nd) (-1: any, stored there). */
static int flat(PyObject* t, PyObject* dtype, long long dev, int nd, int* want, void** p) {
  int s[4];
  if (!same_device(t, dev) || !is_dtype(t, dtype) || !shape_of(t, nd, s)) return 0;
  for (int i = 0; i < nd; ++i) {
    if (want[i] < 0) want[i] = s[i];
    if (want[i] != s[i]) return 0;
  }
  PyObject* c = method(t, n_contiguous);
  const int good = c == Py_True;
  Py_XDECREF(c);
  return good && address(t, p);
}

static int flat_or_none(PyObject* t, PyObject* dtype, long long dev, int nd, int* want, void** p) {
  *p = NULL;
  return t == Py_None || flat(t, dtype, dev, nd, want, p);
}

/* A bf16 [total, heads, d] tensor (-1: any) whose rows may be slices of a wider one. */
static int rows(PyObject* t, long long dev, int* total, int* heads, int* d, void** p, int* pitch) {
  int s[3], st[3];
  if (!same_device(t, dev) || !is_dtype(t, d_bf16) || !shape_of(t, 3, s)) return 0;
  if (*total < 0) *total = s[0];
  if (*heads < 0) *heads = s[1];
  if (*d < 0) *d = s[2];
  if (s[0] != *total || s[1] != *heads || s[2] != *d || !numbers(method(t, n_stride), 3, st))
    return 0;
  const long long row = (long long)s[1] * s[2];
  if (row > INT_MAX) return 0;
  *pitch = (int)row;
  if (s[0] && s[1] && s[2]) {
    if ((st[2] != 1 && s[2] > 1) || (st[1] != s[2] && s[1] > 1)) return 0;
    if (s[0] > 1) {
      if (st[0] < row || st[0] % 8) return 0;
      *pitch = st[0];
    }
  }
  return address(t, p);
}

/* The device of the first tensor, which has to be the current one, and its current stream. */
static int target(PyObject* first, long long* dev, void** stream) {
  if (!PyObject_TypeCheck(first, (PyTypeObject*)t_tensor)) return 0;
  *dev = take_int(method(first, n_device));
  if (*dev < 0 || take_int(PyObject_CallNoArgs(f_device)) != *dev) return 0;
  PyObject* number = PyLong_FromLongLong(*dev);
  PyObject* s = number ? PyObject_CallOneArg(f_stream, number) : NULL;
  Py_XDECREF(number);
  if (!s) return 0;
  *stream = PyLong_AsVoidPtr(s);
  Py_DECREF(s);
  return !PyErr_Occurred();
}

/* cu_seqlens [batch + 1] */
static int boundaries(PyObject* t, long long dev, int* batch, void** p) {
  int n = -1;
  if (!flat(t, d_i32, dev, 1, &n, p) || n < 1) return 0;
  *batch = n - 1;
  return 1;
}

static int scratch(PyObject* t, long long dev, int* bytes, void** p) {
  *bytes = -1;
  return flat(t, d_u8, dev, 1, bytes, p);
}

static PyObject* decline(void) {
  PyErr_Clear();
  Py_RETURN_NONE;
}

#define CALL(expr)                                   \
  int rc;                                            \
  Py_BEGIN_ALLOW_THREADS rc = (expr);                \
  Py_END_ALLOW_THREADS return PyLong_FromLong(rc)

/* q, k, v, cu_seqlens, o, workspace, lse, scale, status */
static PyObject* attn_packed(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  long long dev;
  void *stream, *q, *k, *v, *cu, *o, *ws, *lse, *status;
  int total = -1, hq = -1, hkv = -1, d = -1, batch, qs, ks, vs, bytes, one = 1;
  if (n != 9 || !target(a[0], &dev, &stream) || !rows(a[0], dev, &total, &hq, &d, &q, &qs) ||
      !rows(a[1], dev, &total, &hkv, &d, &k, &ks) || !rows(a[2], dev, &total, &hkv, &d, &v, &vs) ||
      !boundaries(a[3], dev, &batch, &cu))
    return decline();
  int os[3] = {total, hq, d}, ls[2] = {hq, total};
  if (!flat(a[4], d_bf16, dev, 3, os, &o) || !scratch(a[5], dev, &bytes, &ws) ||
      !flat_or_none(a[6], d_f32, dev, 2, ls, &lse) || !PyFloat_Check(a[7]) ||
      !flat_or_none(a[8], d_i32, dev, 1, &one, &status))
    return decline();
  const float scale = (float)PyFloat_AS_DOUBLE(a[7]);
  CALL(p_packed(q, k, v, cu, o, lse, batch, total, hq, hkv, d, qs, ks, vs, scale, ws,
                (size_t)bytes, status, stream));
}

/* q, k, v, o, d_o, lse, cu_seqlens, dq, dk, dv, workspace, scale, status */
static PyObject* attn_packed_grad(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  long long dev;
  void *stream, *q, *k, *v, *o, *d_o, *lse, *cu, *dq, *dk, *dv, *ws, *status;
  int total = -1, hq = -1, hkv = -1, d = -1, batch, qs, ks, vs, dqs, dks, dvs, bytes, one = 1;
  if (n != 13 || !target(a[0], &dev, &stream) || !rows(a[0], dev, &total, &hq, &d, &q, &qs) ||
      !rows(a[1], dev, &total, &hkv, &d, &k, &ks) || !rows(a[2], dev, &total, &hkv, &d, &v, &vs) ||
      !rows(a[7], dev, &total, &hq, &d, &dq, &dqs) ||
      !rows(a[8], dev, &total, &hkv, &d, &dk, &dks) ||
      !rows(a[9], dev, &total, &hkv, &d, &dv, &dvs) || !boundaries(a[6], dev, &batch, &cu))
    return decline();
  int os[3] = {total, hq, d}, ls[2] = {hq, total};
  if (!flat(a[3], d_bf16, dev, 3, os, &o) || !flat(a[4], d_bf16, dev, 3, os, &d_o) ||
      !flat(a[5], d_f32, dev, 2, ls, &lse) || !scratch(a[10], dev, &bytes, &ws) ||
      !PyFloat_Check(a[11]) || !flat_or_none(a[12], d_i32, dev, 1, &one, &status))
    return decline();
  const float scale = (float)PyFloat_AS_DOUBLE(a[11]);
  CALL(p_grad(q, k, v, o, d_o, lse, cu, dq, dk, dv, batch, total, hq, hkv, d, qs, ks, vs, dqs, dks,
              dvs, scale, ws, (size_t)bytes, status, stream));
}

/* k_pool and v_pool [pages, hkv, page, d], block_table [batch, width], seq_lens [batch] */
static int cache(PyObject* const* a, long long dev, int batch, int hkv, int page, int d, int* pages,
                 int* width, void** kp, void** vp, void** table, void** lens) {
  int ps[4] = {-1, hkv, page, d}, ts[2] = {batch, -1};
  if (!flat(a[0], d_bf16, dev, 4, ps, kp) || !flat(a[1], d_bf16, dev, 4, ps, vp) ||
      !flat(a[2], d_i32, dev, 2, ts, table) || !flat(a[3], d_i32, dev, 1, &batch, lens))
    return 0;
  *pages = ps[0];
  *width = ts[1];
  return 1;
}

/* q, k, v, cu_seqlens, k_pool, v_pool, block_table, seq_lens, max_len_hint, o, workspace,
 * status, scale, page */
static PyObject* attn_chunk(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  long long dev;
  void *stream, *q, *k, *v, *cu, *kp, *vp, *table, *lens, *o, *ws, *status;
  int total = -1, hq = -1, hkv = -1, d = -1, batch, qs, ks, vs, pages, width, bytes, one = 1;
  if (n != 14 || !PyLong_Check(a[8]) || !PyFloat_Check(a[12])) return decline();
  const long long hint = PyLong_AsLongLong(a[8]), page = PyLong_AsLongLong(a[13]);
  if (hint < 0 || hint > INT_MAX || page <= 0 || page > INT_MAX || !target(a[0], &dev, &stream) ||
      !rows(a[0], dev, &total, &hq, &d, &q, &qs) || !rows(a[1], dev, &total, &hkv, &d, &k, &ks) ||
      !rows(a[2], dev, &total, &hkv, &d, &v, &vs) || !boundaries(a[3], dev, &batch, &cu) ||
      !cache(a + 4, dev, batch, hkv, (int)page, d, &pages, &width, &kp, &vp, &table, &lens))
    return decline();
  int os[3] = {total, hq, d};
  if (!flat(a[9], d_bf16, dev, 3, os, &o) || !scratch(a[10], dev, &bytes, &ws) ||
      !flat_or_none(a[11], d_i32, dev, 1, &one, &status))
    return decline();
  const float scale = (float)PyFloat_AS_DOUBLE(a[12]);
  CALL(p_chunk(q, k, v, cu, kp, vp, pages, table, width, lens, (int)hint, o, batch, total, hq, hkv,
               d, (int)page, qs, ks, vs, scale, ws, (size_t)bytes, status, stream));
}

/* k, v, cu_seqlens, k_pool, v_pool, block_table, seq_lens, new_lens, slots, status, page */
static PyObject* kv_append(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  long long dev;
  void *stream, *k, *v, *cu, *kp, *vp, *table, *lens, *new_lens, *slots, *status;
  int total = -1, hkv = -1, d = -1, batch, ks, vs, pages, width, one = 1;
  if (n != 11) return decline();
  const long long page = PyLong_AsLongLong(a[10]);
  if (page <= 0 || page > INT_MAX || !target(a[0], &dev, &stream) ||
      !rows(a[0], dev, &total, &hkv, &d, &k, &ks) ||
      !rows(a[1], dev, &total, &hkv, &d, &v, &vs) || !boundaries(a[2], dev, &batch, &cu) ||
      !cache(a + 3, dev, batch, hkv, (int)page, d, &pages, &width, &kp, &vp, &table, &lens) ||
      !flat_or_none(a[7], d_i32, dev, 1, &batch, &new_lens) ||
      !flat_or_none(a[8], d_i32, dev, 1, &total, &slots) ||
      !flat_or_none(a[9], d_i32, dev, 1, &one, &status))
    return decline();
  CALL(p_append(k, v, cu, lens, new_lens, table, width, kp, vp, pages, slots, batch, total, hkv, d,
                (int)page, ks, vs, status, stream));
}

/* q, k, cu_seqlens, inv_freq, q_out, k_out, seq_lens, interleaved, factor, inverse, status */
static PyObject* rotary(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  long long dev;
  void *stream, *q, *k, *cu, *freq, *qo, *ko, *lens, *status;
  int total = -1, hq = -1, hkv = -1, d = -1, batch, qs, ks, qos, kos, half = -1, one = 1;
  if (n != 11 || !p_rotary || !PyBool_Check(a[7]) || !PyFloat_Check(a[8]) || !PyBool_Check(a[9]) ||
      !target(a[0], &dev, &stream) || !rows(a[0], dev, &total, &hq, &d, &q, &qs) ||
      !rows(a[1], dev, &total, &hkv, &d, &k, &ks) || !boundaries(a[2], dev, &batch, &cu) ||
      !flat(a[3], d_f32, dev, 1, &half, &freq) || half > d / 2 ||
      !rows(a[4], dev, &total, &hq, &d, &qo, &qos) ||
      !rows(a[5], dev, &total, &hkv, &d, &ko, &kos) ||
      !flat_or_none(a[6], d_i32, dev, 1, &batch, &lens) ||
      !flat_or_none(a[10], d_i32, dev, 1, &one, &status))
    return decline();
  const float factor = (float)PyFloat_AS_DOUBLE(a[8]);
  CALL(p_rotary(q, k, cu, lens, freq, qo, ko, batch, total, hq, hkv, d, 2 * half, a[7] == Py_True,
                a[9] == Py_True, factor, qs, ks, qos, kos, status, stream));
}

/* k_pool, v_pool [pages, hkv, page, d] codes, k_scale, v_scale [pages, hkv], block_table
 * [batch, width], seq_lens [batch] */
static int cache_q8(PyObject* const* a, long long dev, int batch, int hkv, int page, int d,
                    int* pages, int* width, void** kp, void** vp, void** ks, void** vs,
                    void** table, void** lens) {
  int ps[4] = {-1, hkv, page, d}, ss[2], ts[2] = {batch, -1};
  if (!flat(a[0], d_e4m3, dev, 4, ps, kp) || !flat(a[1], d_e4m3, dev, 4, ps, vp)) return 0;
  ss[0] = *pages = ps[0];
  ss[1] = hkv;
  if (!flat(a[2], d_u8, dev, 2, ss, ks) || !flat(a[3], d_u8, dev, 2, ss, vs) ||
      !flat(a[4], d_i32, dev, 2, ts, table) || !flat(a[5], d_i32, dev, 1, &batch, lens))
    return 0;
  *width = ts[1];
  return 1;
}

/* k, v, cu_seqlens, k_pool, v_pool, k_scale, v_scale, block_table, seq_lens, counts, new_lens,
 * slots, status, page */
static PyObject* kv_append_q8(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  long long dev;
  void *stream, *k, *v, *cu, *kp, *vp, *kc, *vc, *table, *lens, *counts, *new_lens, *slots, *status;
  int total = -1, hkv = -1, d = -1, batch, ks, vs, pages, width, one = 1;
  if (n != 14 || !p_append_q8) return decline();
  const long long page = PyLong_AsLongLong(a[13]);
  if (page <= 0 || page > INT_MAX || !target(a[0], &dev, &stream) ||
      !rows(a[0], dev, &total, &hkv, &d, &k, &ks) ||
      !rows(a[1], dev, &total, &hkv, &d, &v, &vs) || !boundaries(a[2], dev, &batch, &cu) ||
      !cache_q8(a + 3, dev, batch, hkv, (int)page, d, &pages, &width, &kp, &vp, &kc, &vc, &table,
                &lens) ||
      !flat_or_none(a[9], d_i32, dev, 1, &batch, &counts) ||
      !flat_or_none(a[10], d_i32, dev, 1, &batch, &new_lens) ||
      !flat_or_none(a[11], d_i32, dev, 1, &total, &slots) ||
      !flat_or_none(a[12], d_i32, dev, 1, &one, &status))
    return decline();
  CALL(p_append_q8(k, v, cu, lens, counts, new_lens, table, width, kp, vp, kc, vc, pages, slots,
                   batch, total, hkv, d, (int)page, ks, vs, status, stream));
}

/* q, k, v, cu_seqlens, k_pool, v_pool, k_scale, v_scale, block_table, seq_lens, max_len_hint, o,
 * workspace, status, scale, page */
static PyObject* attn_chunk_q8(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  long long dev;
  void *stream, *q, *k, *v, *cu, *kp, *vp, *kc, *vc, *table, *lens, *o, *ws, *status;
  int total = -1, hq = -1, hkv = -1, d = -1, batch, qs, ks, vs, pages, width, bytes, one = 1;
  if (n != 16 || !p_chunk_q8 || !PyLong_Check(a[10]) || !PyFloat_Check(a[14])) return decline();
  const long long hint = PyLong_AsLongLong(a[10]), page = PyLong_AsLongLong(a[15]);
  if (hint < 0 || hint > INT_MAX || page <= 0 || page > INT_MAX || !target(a[0], &dev, &stream) ||
      !rows(a[0], dev, &total, &hq, &d, &q, &qs) || !rows(a[1], dev, &total, &hkv, &d, &k, &ks) ||
      !rows(a[2], dev, &total, &hkv, &d, &v, &vs) || !boundaries(a[3], dev, &batch, &cu) ||
      !cache_q8(a + 4, dev, batch, hkv, (int)page, d, &pages, &width, &kp, &vp, &kc, &vc, &table,
                &lens))
    return decline();
  int os[3] = {total, hq, d};
  if (!flat(a[11], d_bf16, dev, 3, os, &o) || !scratch(a[12], dev, &bytes, &ws) ||
      !flat_or_none(a[13], d_i32, dev, 1, &one, &status))
    return decline();
  const float scale = (float)PyFloat_AS_DOUBLE(a[14]);
  CALL(p_chunk_q8(q, k, v, cu, kp, vp, kc, vc, pages, table, width, lens, (int)hint, o, batch,
                  total, hq, hkv, d, (int)page, qs, ks, vs, scale, ws, (size_t)bytes, status,
                  stream));
}

/* What the calls above need beside setup's: the dtype of the codes, and the addresses of the
 * three entry points. */
static PyObject* setup_q8(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  void* p[3];
  if (n != 4) {
    PyErr_SetString(PyExc_TypeError, "setup_q8: four arguments");
    return NULL;
  }
  for (int i = 0; i < 3; ++i) {
    p[i] = PyLong_AsVoidPtr(a[1 + i]);
    if (PyErr_Occurred()) return NULL;
  }
  Py_INCREF(a[0]);
  Py_XSETREF(d_e4m3, a[0]);
  p_rotary = (__typeof__(p_rotary))p[0];
  p_append_q8 = (__typeof__(p_append_q8))p[1];
  p_chunk_q8 = (__typeof__(p_chunk_q8))p[2];
  Py_RETURN_NONE;
}

/* Tensor type, the dtypes bf16, int32, float32, uint8, the functions giving the current device
 * and a device's raw current stream, and the addresses of the four entry points. */
static PyObject* setup(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  PyObject** keep[7] = {&t_tensor, &d_bf16, &d_i32, &d_f32, &d_u8, &f_device, &f_stream};
  if (n != 11 || !PyType_Check(a[0])) {
    PyErr_SetString(PyExc_TypeError, "setup: eleven arguments, a type first");
    return NULL;
  }
  void* p[4];
  for (int i = 0; i < 4; ++i) {
    p[i] = PyLong_AsVoidPtr(a[7 + i]);
    if (PyErr_Occurred()) return NULL;
  }
  for (int i = 0; i < 7; ++i) {
    Py_INCREF(a[i]);
    Py_XSETREF(*keep[i], a[i]);
  }
  p_packed = (__typeof__(p_packed))p[0];
  p_grad = (__typeof__(p_grad))p[1];
  p_chunk = (__typeof__(p_chunk))p[2];
  p_append = (__typeof__(p_append))p[3];
  Py_RETURN_NONE;
}

#define METHOD(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {METHOD(setup),      METHOD(attn_packed), METHOD(attn_packed_grad),
                                METHOD(attn_chunk), METHOD(kv_append),   METHOD(setup_q8),
                                METHOD(rotary),     METHOD(kv_append_q8), METHOD(attn_chunk_q8),
                                {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_packed_calls", NULL, -1, methods,
                                    NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__packed_calls(void) {
  PyObject** names[6] = {&n_device, &n_dtype, &n_shape, &n_stride, &n_contiguous, &n_ptr};
  const char* text[6] = {"get_device", "dtype", "shape", "stride", "is_contiguous", "data_ptr"};
  for (int i = 0; i < 6; ++i)
    if (!(*names[i] = PyUnicode_InternFromString(text[i]))) return NULL;
  return PyModule_Create(&module);
}
