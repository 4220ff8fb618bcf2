/* CPython side of the 8-bit expert calls: checks the tensors of a call, makes the outputs that are not given, and calls
 * the library. In C because a call on a few rows is bound by its host time: the same checks in Python with ctypes took
 * 8.6 us for moe_combine, here 4.1. Tensors are read through their Python attributes, so that torch's own headers are not
 * needed. Two names are private to torch: _C._cuda_getDevice and _C._cuda_getCurrentRawStream, which give the current
 * device and its stream without making objects. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>

#include "../../include/moe_gb300.h"

static PyObject *g_torch, *g_torch_c, *g_tensor, *g_error, *g_rows_class, *g_weights_class;
static PyObject *g_int16, *g_int32, *g_float32, *g_uint8;
static PyObject *s_dtype, *s_device, *s_get_device, *s_shape, *s_stride, *s_data_ptr, *s_is_contiguous, *s_empty, *s_q, *s_scale,
    *s_cuda_device, *s_cuda_stream, *g_empty_names;

/* ---------------------------------------------------------------------------------- tensors */
typedef struct {
  int64_t size[3], stride[3];
  int dims;
  int64_t device; /* -1: the host */
  void* data;
} tensor;

static int64_t to_int(PyObject* o) { /* takes the reference; -1 with no error set where it is none */
  int64_t v = -1;
  if (o) {
    v = PyLong_AsLongLong(o);
    Py_DECREF(o);
  }
  if (PyErr_Occurred()) PyErr_Clear();
  return v;
}

static int read_sizes(PyObject* o, int64_t* to, int* n) { /* takes the reference of a tuple of ints */
  int ok = o && PyTuple_Check(o) && PyTuple_GET_SIZE(o) <= 3;
  if (ok) {
    *n = (int)PyTuple_GET_SIZE(o);
    for (int i = 0; i < *n; ++i) to[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(o, i));
  }
  Py_XDECREF(o);
  if (PyErr_Occurred()) {
    PyErr_Clear();
    return 0;
  }
  return ok;
}

/* A tensor of the dtype with at most three axes; `strided`: with its strides, else contiguous. No exception is set where
 * it is something else. */
static int read_tensor(PyObject* o, PyObject* dtype, int strided, tensor* t) {
  if (!PyObject_TypeCheck(o, (PyTypeObject*)g_tensor)) return 0;
  PyObject* d = PyObject_GetAttr(o, s_dtype);
  Py_XDECREF(d);
  if (d != dtype) {
    PyErr_Clear();
    return 0;
  }
  t->device = to_int(PyObject_CallMethodNoArgs(o, s_get_device));
  if (!read_sizes(PyObject_GetAttr(o, s_shape), t->size, &t->dims)) return 0;
  if (strided) {
    int n;
    if (!read_sizes(PyObject_CallMethodNoArgs(o, s_stride), t->stride, &n)) return 0;
  } else {
    PyObject* c = PyObject_CallMethodNoArgs(o, s_is_contiguous);
    Py_XDECREF(c);
    if (c != Py_True) {
      PyErr_Clear();
      return 0;
    }
  }
  PyObject* p = PyObject_CallMethodNoArgs(o, s_data_ptr);
  if (!p) {
    PyErr_Clear();
    return 0;
  }
  t->data = (void*)(uintptr_t)PyLong_AsUnsignedLongLong(p);
  Py_DECREF(p);
  return 1;
}

#define MANY ((int64_t)1 << 31) /* sizes from here on do not fit the library's integers; it refuses smaller ones itself */
#define ANY ((int64_t)-1)

static int64_t blocks(int64_t n) { return (n + 127) / 128; }

static const char* size_text(int64_t n, const char* any, char* buf, size_t len) {
  if (n == ANY) return any;
  PyOS_snprintf(buf, len, "%lld", (long long)n);
  return buf;
}

/* The current device, on which the call's tensors have to lie; `device` is the first one's. */
static int current_device(int64_t device, const char* name, int64_t* dev) {
  if (device >= 0) {
    PyObject* d = PyObject_CallMethodNoArgs(g_torch_c, s_cuda_device);
    if (!d) return 0;
    *dev = to_int(d);
    if (*dev == device) return 1;
  }
  PyErr_Format(PyExc_ValueError, "%s must be on the current CUDA device", name);
  return 0;
}

/* A tensor's device, or -1 if it is none. */
static int64_t device_of(PyObject* o) {
  if (!PyObject_TypeCheck(o, (PyTypeObject*)g_tensor)) return -1;
  return to_int(PyObject_CallMethodNoArgs(o, s_get_device));
}

static int stream_of(int64_t dev, moe_stream_t* stream) {
  PyObject* d = PyLong_FromLongLong(dev);
  if (!d) return 0;
  PyObject* s = PyObject_CallMethodOneArg(g_torch_c, s_cuda_stream, d);
  Py_DECREF(d);
  if (!s) return 0;
  *stream = (moe_stream_t)(uintptr_t)PyLong_AsUnsignedLongLong(s);
  Py_DECREF(s);
  return !PyErr_Occurred();
}

/* ---------------------------------------------------------------------------------- arguments */
typedef struct {
  moe_rows r;
  int64_t rows, cols, device;
} rows_t;

/* bf16 rows: an int16 tensor [rows, cols] whose rows are runs of memory; ANY: of any number. */
static int bf16_rows(PyObject* o, const char* name, int64_t rows, int64_t cols, int64_t dev, rows_t* r) {
  tensor t;
  if (read_tensor(o, g_int16, 1, &t) && t.device == dev && t.dims == 2 && (rows == ANY || t.size[0] == rows) &&
      (cols == ANY || t.size[1] == cols) && t.size[0] < MANY && t.size[1] < MANY &&
      (t.stride[1] == 1 || t.size[0] == 0 || t.size[1] == 0)) {
    r->rows = t.size[0];
    r->cols = t.size[1];
    r->device = dev;
    r->r.format = MOE_ROWS_BF16;
    r->r.p = t.data;
    /* the stride of an axis of length one is never used, and torch may give any */
    r->r.stride = t.size[0] > 1 ? t.stride[0] : (t.size[1] + 7) / 8 * 8;
    r->r.scale = NULL;
    r->r.scale_stride = 0;
    return 1;
  }
  char a[24], b[24];
  PyErr_Format(PyExc_ValueError,
               "%s must be an int16 tensor [%s, %s] on the current CUDA device, the values of a row contiguous", name,
               size_text(rows, "rows", a, sizeof a), size_text(cols, "columns", b, sizeof b));
  return 0;
}

/* An object that carries two tensors, q and scale. They are read at every call and nothing is kept of them: they may have been
 * exchanged, moved or copied with the object since the call before. New references; 0 without an exception if the object is
 * not of the class. */
static int carried(PyObject* o, PyObject* class, PyObject** q, PyObject** scale) {
  *q = *scale = NULL;
  if (PyObject_IsInstance(o, class) == 1 && (*q = PyObject_GetAttr(o, s_q)) && (*scale = PyObject_GetAttr(o, s_scale))) return 1;
  PyErr_Clear();
  Py_CLEAR(*q);
  return 0;
}

/* The tensors of E4m3Rows; `of`: the object's name and a dot, for messages. */
static int read_rows(PyObject* q_obj, PyObject* scale_obj, const char* of, rows_t* r) {
  tensor q, s;
  if (!read_tensor(q_obj, g_uint8, 1, &q) || q.device < 0 || q.dims != 2 || q.size[0] >= MANY || q.size[1] >= MANY ||
      (q.stride[1] != 1 && q.size[0] && q.size[1])) {
    PyErr_Format(PyExc_ValueError, "%sq must be a CUDA tensor of uint8 [rows, columns], the values of a row contiguous", of);
    return 0;
  }
  const int64_t nb = blocks(q.size[1]);
  if (!read_tensor(scale_obj, g_float32, 1, &s) || s.device != q.device || s.dims != 2 || s.size[0] != q.size[0] || s.size[1] != nb ||
      (s.stride[1] != 1 && nb > 1 && q.size[0])) {
    PyErr_Format(PyExc_ValueError,
                 "%sscale must be a float32 tensor [%lld, %lld] on q's device, the values of a row contiguous", of,
                 (long long)q.size[0], (long long)nb);
    return 0;
  }
  r->rows = q.size[0];
  r->cols = q.size[1];
  r->device = q.device;
  r->r.format = MOE_ROWS_E4M3;
  r->r.p = q.data;
  r->r.stride = q.size[0] > 1 ? q.stride[0] : nb * 128;
  r->r.scale = s.data;
  r->r.scale_stride = q.size[0] > 1 ? s.stride[0] : nb;
  return 1;
}

typedef struct {
  moe_e4m3_weights w;
  int64_t device;
} weights_t;

/* The same for E4m3Weights. */
static int read_weights(PyObject* q_obj, PyObject* scale_obj, const char* of, weights_t* w) {
  tensor q, s;
  if (!read_tensor(q_obj, g_uint8, 0, &q) || q.device < 0 || q.dims != 3 || q.size[0] >= MANY || q.size[1] >= MANY || q.size[2] >= MANY) {
    PyErr_Format(PyExc_ValueError, "%sq must be a contiguous CUDA tensor of uint8 [n_experts, n, k]", of);
    return 0;
  }
  if (!read_tensor(scale_obj, g_float32, 0, &s) || s.device != q.device || s.dims != 3 || s.size[0] != q.size[0] ||
      s.size[1] != blocks(q.size[1]) || s.size[2] != blocks(q.size[2])) {
    PyErr_Format(PyExc_ValueError, "%sscale must be a contiguous float32 tensor [%lld, %lld, %lld] on q's device", of,
                 (long long)q.size[0], (long long)blocks(q.size[1]), (long long)blocks(q.size[2]));
    return 0;
  }
  w->w.q = q.data;
  w->w.scale = s.data;
  w->w.n_experts = (int32_t)q.size[0];
  w->w.n = (int32_t)q.size[1];
  w->w.k = (int32_t)q.size[2];
  w->device = q.device;
  return 1;
}

/* E4m3Rows as they are now, on any device. */
static int carried_rows(PyObject* o, const char* name, rows_t* r) {
  PyObject *q, *scale;
  char of[16];
  if (!carried(o, g_rows_class, &q, &scale)) {
    PyErr_Format(PyExc_ValueError, "%s must be E4m3Rows", name);
    return 0;
  }
  PyOS_snprintf(of, sizeof of, "%s.", name);
  const int ok = read_rows(q, scale, of, r);
  Py_DECREF(q);
  Py_DECREF(scale);
  return ok;
}

static int carried_weights(PyObject* o, const char* name, weights_t* w) {
  PyObject *q, *scale;
  char of[16];
  if (!carried(o, g_weights_class, &q, &scale)) {
    PyErr_Format(PyExc_ValueError, "%s must be E4m3Weights", name);
    return 0;
  }
  PyOS_snprintf(of, sizeof of, "%s.", name);
  const int ok = read_weights(q, scale, of, w);
  Py_DECREF(q);
  Py_DECREF(scale);
  return ok;
}

/* Whether E4m3Rows that were read are of the size, and on the device, that the call takes. */
static int rows_fit(const rows_t* r, const char* name, int64_t rows, int64_t cols, int64_t dev) {
  if (r->device == dev && (rows == ANY || r->rows == rows) && (cols == ANY || r->cols == cols)) return 1;
  char a[24], b[24];
  PyErr_Format(PyExc_ValueError, "%s must be E4m3Rows [%s, %s] on the current CUDA device", name,
               size_text(rows, "rows", a, sizeof a), size_text(cols, "columns", b, sizeof b));
  return 0;
}

/* A contiguous int32 tensor, of n values (ANY: of any number). */
static int ints(PyObject* o, const char* name, int64_t n, int64_t dev, tensor* t) {
  if (read_tensor(o, g_int32, 0, t) && t->device == dev) {
    int64_t m = 1;
    for (int i = 0; i < t->dims; ++i) m *= t->size[i];
    if ((n == ANY || m == n) && m < MANY) return 1;
  }
  if (n == ANY)
    PyErr_Format(PyExc_ValueError, "%s must be a contiguous int32 tensor on the current CUDA device", name);
  else
    PyErr_Format(PyExc_ValueError, "%s must be a contiguous int32 tensor of %lld on the current CUDA device", name, (long long)n);
  return 0;
}

/* inv int32 [T, top_k]; T ANY: as many as there are. */
static int places(PyObject* o, int64_t T, int64_t dev, tensor* t) {
  if (!ints(o, "inv", ANY, dev, t)) return 0;
  if (t->dims == 2 && (T == ANY || t->size[0] == T)) return 1;
  char a[24];
  PyErr_Format(PyExc_ValueError, "inv must be [%s, top_k]", size_text(T, "tokens", a, sizeof a));
  return 0;
}

static int floats(PyObject* o, const char* name, int64_t T, int64_t k, int64_t dev, float** p) {
  tensor t;
  if (read_tensor(o, g_float32, 0, &t) && t.device == dev && t.dims == 2 && t.size[0] == T && t.size[1] == k) {
    *p = t.data;
    return 1;
  }
  PyErr_Format(PyExc_ValueError, "%s must be a contiguous float32 tensor [%lld, %lld] on the current CUDA device", name,
               (long long)T, (long long)k);
  return 0;
}

typedef struct {
  void* p;
  size_t bytes;
  moe_stream_t stream;
} space_t;

/* The workspace, and the stream that the call runs on. */
static int space(PyObject* o, int64_t dev, space_t* s) {
  tensor t;
  if (read_tensor(o, g_uint8, 0, &t) && t.device == dev && t.dims == 1) {
    s->p = t.data;
    s->bytes = (size_t)t.size[0];
    return stream_of(dev, &s->stream);
  }
  PyErr_SetString(PyExc_ValueError,
                  "ws must be a contiguous uint8 tensor on the current CUDA device (expert_workspace)");
  return 0;
}

/* ---------------------------------------------------------------------------------- outputs and status */
/* torch.empty of up to two axes on the device of `like`. */
static PyObject* new_tensor(PyObject* like, PyObject* dtype, int dims, int64_t a, int64_t b) {
  PyObject* device = PyObject_GetAttr(like, s_device);
  PyObject* shape = dims == 2 ? Py_BuildValue("(LL)", (long long)a, (long long)b) : Py_BuildValue("(L)", (long long)a);
  PyObject *empty = PyObject_GetAttr(g_torch, s_empty), *out = NULL;
  if (device && shape && empty) {
    PyObject* args[3] = {shape, dtype, device};
    out = PyObject_Vectorcall(empty, args, 1, g_empty_names);
  }
  Py_XDECREF(device);
  Py_XDECREF(shape);
  Py_XDECREF(empty);
  return out;
}

/* The output rows, a new reference: those given, or `rows` new ones of the kind asked for. */
static PyObject* rows_out(PyObject* out, PyObject* e4m3, PyObject* like, int64_t rows, int64_t made, int64_t cols, int64_t dev, rows_t* r) {
  const int as_codes = out == Py_None ? PyObject_IsTrue(e4m3) : 0;
  if (as_codes < 0) return NULL;
  if (out != Py_None) {
    Py_INCREF(out);
  } else if (as_codes) {
    PyObject* device = PyObject_GetAttr(like, s_device);
    out = device ? PyObject_CallMethod(g_rows_class, "empty", "LLO", (long long)made, (long long)cols, device) : NULL;
    Py_XDECREF(device);
  } else {
    out = new_tensor(like, g_int16, 2, made, cols);
  }
  if (!out) return NULL;
  const int ok = PyObject_TypeCheck(out, (PyTypeObject*)g_tensor)
                     ? bf16_rows(out, "out", rows, cols, dev, r)
                     : carried_rows(out, "out", r) && rows_fit(r, "out", rows, cols, dev);
  if (ok) return out;
  Py_DECREF(out);
  return NULL;
}

/* MoeError for a status that is not MOE_OK. */
static int status_ok(int status, const char* what) {
  if (status == MOE_OK) return 1;
  PyObject* e = PyObject_CallFunction(g_error, "is", status, what);
  if (e) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  return 0;
}

#define CALL(status, call)  \
  do {                      \
    Py_BEGIN_ALLOW_THREADS; \
    status = call;          \
    Py_END_ALLOW_THREADS;   \
  } while (0)

static int arity(Py_ssize_t n, Py_ssize_t want, const char* name) {
  if (n == want) return 1;
  PyErr_Format(PyExc_TypeError, "%s takes %zd arguments", name, want);
  return 0;
}

/* ---------------------------------------------------------------------------------- the calls */
/* check_rows(q, scale), check_weights(q, scale): whether the classes can carry these tensors. */
static PyObject* check_rows(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  rows_t r;
  if (!arity(n, 2, "check_rows") || !read_rows(a[0], a[1], "", &r)) return NULL;
  Py_RETURN_NONE;
}

static PyObject* check_weights(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  weights_t w;
  if (!arity(n, 2, "check_weights") || !read_weights(a[0], a[1], "", &w)) return NULL;
  Py_RETURN_NONE;
}

/* workspace_bytes(n_experts) */
static PyObject* workspace_bytes(PyObject* self, PyObject* arg) {
  (void)self;
  const long n = PyLong_AsLong(arg);
  if (n == -1 && PyErr_Occurred()) return NULL;
  return PyLong_FromSize_t(n < 0 || n >= MANY ? 0 : moe_expert_workspace_bytes((int32_t)n));
}

/* sort_tokens(ids, n_experts, ws) -> offsets, perm, inv */
static PyObject* sort_tokens(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  int64_t dev;
  tensor ids, t;
  space_t ws;
  if (!arity(n, 3, "sort_tokens") || !current_device(device_of(a[0]), "ids", &dev) || !ints(a[0], "ids", ANY, dev, &ids) ||
      !space(a[2], dev, &ws))
    return NULL;
  const long experts = PyLong_AsLong(a[1]);
  if (experts == -1 && PyErr_Occurred()) return NULL;
  if (experts < 0 || experts >= MANY) return status_ok(MOE_ERR_UNSUPPORTED_SHAPE, "moe_sort_tokens"), NULL;
  int64_t m = 1;
  for (int i = 0; i < ids.dims; ++i) m *= ids.size[i];
  PyObject *offsets = new_tensor(a[0], g_int32, 1, experts + 1, 0), *perm = new_tensor(a[0], g_int32, 1, m, 0), *inv = NULL;
  int32_t *po = NULL, *pp = NULL, *pi = NULL;
  if (offsets && perm) inv = PyObject_CallMethod(g_torch, "empty_like", "O", a[0]);
  if (inv && ints(offsets, "offsets", experts + 1, dev, &t)) po = t.data;
  if (po && ints(perm, "perm", m, dev, &t)) pp = t.data;
  PyObject* out = NULL;
  if (po && !PyErr_Occurred() && ints(inv, "inv", m, dev, &t)) {
    pi = t.data;
    int st;
    CALL(st, moe_sort_tokens(ids.data, (int32_t)m, (int32_t)experts, po, pp, pi, ws.p, ws.bytes, ws.stream));
    if (status_ok(st, "moe_sort_tokens")) out = PyTuple_Pack(3, offsets, perm, inv);
  }
  Py_XDECREF(offsets);
  Py_XDECREF(perm);
  Py_XDECREF(inv);
  return out;
}

/* dispatch(x, inv or None, ws, e4m3, out or None) -> out */
static PyObject* dispatch(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  int64_t dev;
  rows_t x, o;
  tensor inv = {0};
  space_t ws;
  if (!arity(n, 5, "dispatch") || !current_device(device_of(a[0]), "x", &dev) || !bf16_rows(a[0], "x", ANY, ANY, dev, &x) ||
      (a[1] != Py_None && !places(a[1], x.rows, dev, &inv)) || !space(a[2], dev, &ws))
    return NULL;
  const int64_t k = a[1] != Py_None ? inv.size[1] : 1;
  PyObject* out = rows_out(a[4], a[3], a[0], ANY, x.rows * k, x.cols, dev, &o);
  if (!out) return NULL;
  int st;
  CALL(st, moe_dispatch(&x.r, a[1] != Py_None ? inv.data : NULL, (int32_t)x.rows, (int32_t)k, (int32_t)x.cols, &o.r,
                        (int32_t)o.rows, ws.p, ws.bytes, ws.stream));
  if (status_ok(st, "moe_dispatch")) return out;
  Py_DECREF(out);
  return NULL;
}

/* combine(ys, inv, w or None, ws, add or None, y or None) -> y */
static PyObject* combine(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  int64_t dev;
  rows_t ys, add, y;
  tensor inv;
  float* w = NULL;
  space_t ws;
  if (!arity(n, 6, "combine") || !current_device(device_of(a[0]), "ys", &dev) || !bf16_rows(a[0], "ys", ANY, ANY, dev, &ys) ||
      !places(a[1], ANY, dev, &inv) || (a[2] != Py_None && !floats(a[2], "w", inv.size[0], inv.size[1], dev, &w)) ||
      !space(a[3], dev, &ws) || (a[4] != Py_None && !bf16_rows(a[4], "add", inv.size[0], ys.cols, dev, &add)))
    return NULL;
  PyObject* out = a[5];
  if (out == Py_None) {
    if (!(out = new_tensor(a[0], g_int16, 2, inv.size[0], ys.cols))) return NULL;
  } else {
    Py_INCREF(out);
  }
  int st = MOE_OK;
  if (bf16_rows(out, "y", inv.size[0], ys.cols, dev, &y)) {
    CALL(st, moe_combine(&ys.r, (int32_t)ys.rows, inv.data, w, (int32_t)inv.size[0], (int32_t)inv.size[1], (int32_t)ys.cols,
                         a[4] != Py_None ? &add.r : NULL, &y.r, ws.p, ws.bytes, ws.stream));
    if (status_ok(st, "moe_combine")) return out;
  }
  Py_DECREF(out);
  return NULL;
}

/* combine_grad(dy, ys, inv, w, ws, e4m3, out or None, dw or None) -> dys, dw */
static PyObject* combine_grad(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  int64_t dev;
  rows_t dy, ys, o;
  tensor inv;
  float *w, *dw;
  space_t ws;
  if (!arity(n, 8, "combine_grad") || !current_device(device_of(a[0]), "dy", &dev) ||
      !bf16_rows(a[0], "dy", ANY, ANY, dev, &dy) || !bf16_rows(a[1], "ys", ANY, dy.cols, dev, &ys) ||
      !places(a[2], dy.rows, dev, &inv) || !floats(a[3], "w", dy.rows, inv.size[1], dev, &w) || !space(a[4], dev, &ws))
    return NULL;
  PyObject *dw_out = a[7], *result = NULL;
  PyObject* out = rows_out(a[6], a[5], a[0], ys.rows, ys.rows, dy.cols, dev, &o);
  if (!out) return NULL;
  if (dw_out == Py_None)
    dw_out = new_tensor(a[0], g_float32, 2, dy.rows, inv.size[1]);
  else
    Py_INCREF(dw_out);
  if (dw_out && floats(dw_out, "dw", dy.rows, inv.size[1], dev, &dw)) {
    int st;
    CALL(st, moe_combine_grad(&dy.r, &ys.r, (int32_t)ys.rows, inv.data, w, (int32_t)dy.rows, (int32_t)inv.size[1], (int32_t)dy.cols,
                              &o.r, dw, ws.p, ws.bytes, ws.stream));
    if (status_ok(st, "moe_combine_grad")) result = PyTuple_Pack(2, out, dw_out);
  }
  Py_DECREF(out);
  Py_XDECREF(dw_out);
  return result;
}

/* quant_weights(w, q, scale): int16 [E, n, k] into q and scale of E4m3Weights' shapes. */
static PyObject* quant_weights(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  int64_t dev;
  tensor w, q, s;
  moe_stream_t stream;
  if (!arity(n, 3, "quant_weights") || !current_device(device_of(a[0]), "w", &dev)) return NULL;
  if (!read_tensor(a[0], g_int16, 0, &w) || w.dims != 3 || w.size[0] >= MANY || w.size[1] >= MANY || w.size[2] >= MANY) {
    PyErr_SetString(PyExc_ValueError, "w must be a contiguous int16 tensor [n_experts, n, k]");
    return NULL;
  }
  if (!read_tensor(a[1], g_uint8, 0, &q) || !read_tensor(a[2], g_float32, 0, &s) || q.device != dev || s.device != dev) {
    PyErr_SetString(PyExc_ValueError, "q and scale must be on the current CUDA device");
    return NULL;
  }
  int st;
  if (!stream_of(dev, &stream)) return NULL;
  CALL(st, moe_quant_weights(w.data, (int32_t)w.size[0], (int32_t)w.size[1], (int32_t)w.size[2], q.data, s.data, stream));
  if (!status_ok(st, "moe_quant_weights")) return NULL;
  Py_RETURN_NONE;
}

/* gemm_e4m3(a, w, offsets or None, ws, transposed, out or None) -> out */
static PyObject* gemm_e4m3(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  int64_t dev;
  rows_t x, o;
  tensor offsets = {0};
  space_t ws;
  if (!arity(n, 6, "gemm_e4m3")) return NULL;
  weights_t w;
  if (!carried_rows(a[0], "a", &x) || !carried_weights(a[1], "w", &w)) return NULL;
  const int transposed = PyObject_IsTrue(a[4]);
  if (transposed < 0 || !current_device(x.device, "a", &dev)) return NULL;
  if (w.device != dev) {
    PyErr_SetString(PyExc_ValueError, "w must be on the current CUDA device");
    return NULL;
  }
  if (!rows_fit(&x, "a", ANY, transposed ? w.w.n : w.w.k, dev) ||
      (a[2] != Py_None && !ints(a[2], "offsets", (int64_t)w.w.n_experts + 1, dev, &offsets)) || !space(a[3], dev, &ws))
    return NULL;
  PyObject* out = a[5];
  const int64_t cols = transposed ? w.w.k : w.w.n;
  if (out == Py_None) {
    PyObject* q = PyObject_GetAttr(a[0], s_q);
    if (!q) return NULL;
    out = new_tensor(q, g_int16, 2, x.rows, cols);
    Py_DECREF(q);
    if (!out) return NULL;
  } else {
    Py_INCREF(out);
  }
  if (bf16_rows(out, "out", x.rows, cols, dev, &o)) {
    int st;
    CALL(st, moe_gemm_e4m3(&x.r, (int32_t)x.rows, &w.w, a[2] != Py_None ? offsets.data : NULL, transposed, &o.r, ws.p, ws.bytes,
                           ws.stream));
    if (status_ok(st, "moe_gemm_e4m3")) return out;
  }
  Py_DECREF(out);
  return NULL;
}

/* gu's rows and half their columns, and the number of rows that count. */
static int gate_up(PyObject* gu, PyObject* total, int64_t* dev, rows_t* r, tensor* t) {
  if (!current_device(device_of(gu), "gu", dev) || !bf16_rows(gu, "gu", ANY, ANY, *dev, r)) return 0;
  if (r->cols % 2) {
    PyErr_SetString(PyExc_ValueError, "gu must have an even number of columns");
    return 0;
  }
  return total == Py_None || ints(total, "total", 1, *dev, t);
}

/* swiglu(gu, ws, total or None, e4m3, out or None) -> out */
static PyObject* swiglu(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  int64_t dev;
  rows_t gu, o;
  tensor total = {0};
  space_t ws;
  if (!arity(n, 5, "swiglu") || !gate_up(a[0], a[2], &dev, &gu, &total) || !space(a[1], dev, &ws)) return NULL;
  PyObject* out = rows_out(a[4], a[3], a[0], gu.rows, gu.rows, gu.cols / 2, dev, &o);
  if (!out) return NULL;
  int st;
  CALL(st, moe_swiglu(&gu.r, (int32_t)gu.rows, (int32_t)(gu.cols / 2), a[2] != Py_None ? total.data : NULL, &o.r, ws.p, ws.bytes,
                      ws.stream));
  if (status_ok(st, "moe_swiglu")) return out;
  Py_DECREF(out);
  return NULL;
}

/* swiglu_grad(gu, dh, ws, total or None, e4m3, out or None) -> out */
static PyObject* swiglu_grad(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  int64_t dev;
  rows_t gu, dh, o;
  tensor total = {0};
  space_t ws;
  if (!arity(n, 6, "swiglu_grad") || !gate_up(a[0], a[3], &dev, &gu, &total) ||
      !bf16_rows(a[1], "dh", gu.rows, gu.cols / 2, dev, &dh) || !space(a[2], dev, &ws))
    return NULL;
  PyObject* out = rows_out(a[5], a[4], a[0], gu.rows, gu.rows, gu.cols, dev, &o);
  if (!out) return NULL;
  int st;
  CALL(st, moe_swiglu_grad(&gu.r, &dh.r, (int32_t)gu.rows, (int32_t)(gu.cols / 2), a[3] != Py_None ? total.data : NULL, &o.r, ws.p,
                           ws.bytes, ws.stream));
  if (status_ok(st, "moe_swiglu_grad")) return out;
  Py_DECREF(out);
  return NULL;
}

/* setup(MoeError, E4m3Rows, E4m3Weights): the package's classes. */
static PyObject* setup(PyObject* self, PyObject* const* a, Py_ssize_t n) {
  (void)self;
  if (!arity(n, 3, "setup")) return NULL;
  Py_INCREF(a[0]);
  Py_XSETREF(g_error, a[0]);
  Py_INCREF(a[1]);
  Py_XSETREF(g_rows_class, a[1]);
  Py_INCREF(a[2]);
  Py_XSETREF(g_weights_class, a[2]);
  Py_RETURN_NONE;
}

#define FAST(name) {#name, (PyCFunction)(void (*)(void))name, METH_FASTCALL, NULL}
static PyMethodDef methods[] = {FAST(setup), FAST(check_rows), FAST(check_weights), {"workspace_bytes", workspace_bytes, METH_O, NULL},
                                FAST(sort_tokens), FAST(dispatch), FAST(combine), FAST(combine_grad), FAST(quant_weights),
                                FAST(gemm_e4m3), FAST(swiglu), FAST(swiglu_grad), {NULL, NULL, 0, NULL}};
static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_experts", NULL, -1, methods, NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__experts(void) {
  if (!(g_torch = PyImport_ImportModule("torch"))) return NULL;
  struct {
    PyObject** to;
    const char* name;
  } const attrs[] = {{&g_torch_c, "_C"},         {&g_tensor, "Tensor"},     {&g_int16, "int16"},
                     {&g_int32, "int32"},        {&g_float32, "float32"},   {&g_uint8, "uint8"}};
  for (size_t i = 0; i < sizeof attrs / sizeof *attrs; ++i)
    if (!(*attrs[i].to = PyObject_GetAttrString(g_torch, attrs[i].name))) return NULL;
  struct {
    PyObject** to;
    const char* text;
  } const names[] = {{&s_dtype, "dtype"},
                     {&s_device, "device"},
                     {&s_get_device, "get_device"},
                     {&s_shape, "shape"},
                     {&s_stride, "stride"},
                     {&s_data_ptr, "data_ptr"},
                     {&s_is_contiguous, "is_contiguous"},
                     {&s_empty, "empty"},
                     {&s_q, "q"},
                     {&s_scale, "scale"},
                     {&s_cuda_device, "_cuda_getDevice"},
                     {&s_cuda_stream, "_cuda_getCurrentRawStream"}};
  for (size_t i = 0; i < sizeof names / sizeof *names; ++i)
    if (!(*names[i].to = PyUnicode_InternFromString(names[i].text))) return NULL;
  if (!(g_empty_names = Py_BuildValue("(OO)", s_dtype, s_device))) return NULL;
  return PyModule_Create(&module);
}
