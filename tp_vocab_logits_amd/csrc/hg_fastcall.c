/*
 * _hgcall: fast-call Python wrappers of the per-call entry points of
 * libhg.so (hg_gather, hg_push, hg_collect, hg_stock_gather, hg_embed,
 * hg_embed_grad, hg_xent, hg_xent_grad, hg_xent_step), for loops where the ctypes conversion of the arguments
 * (about 0.5 us a call, 2 us with a dozen of them) is a sizeable part of a
 * call of a few microseconds.
 * Argument marshalling only: every argument is an integer (a handle, a
 * host-array address, a row count, a device address, a stream), a float or a
 * tuple of device addresses, passed on unchanged; the return value is the
 * library's status code.
 *
 * The module does not link against libhg.so: bind() receives the addresses of
 * the nine entry points from the already loaded library (see _lib.fast()).
 */
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include "hg.h"

typedef int (*gather_fn)(void *h, const void *const *shards, int m, void *out, void *stream);
typedef int (*push_fn)(void *h, const void *const *shards, int m, void *stream);
typedef int (*collect_fn)(void *h, int m, void *out, void *stream);
typedef int (*stock_fn)(int tp, int shard, const void *const *shards, int m, void *out,
                        int vocab, void *stream);

typedef int (*embed_fn)(int tp, int shard, int hidden, int dtype, const void *const *w,
                        const void *tokens, int token_bytes, int n, float scale, void *out,
                        void *stream);
typedef int (*embed_grad_fn)(int tp, int shard, int hidden, int dtype, const void *tokens,
                             int token_bytes, int n, const void *dy, float scale, void *dw,
                             int dw_wide, int accumulate, void *ws, size_t ws_bytes, void *stream);

static gather_fn g_gather;
static push_fn g_push;
static collect_fn g_collect;
static stock_fn g_stock;
static embed_fn g_embed;
static embed_grad_fn g_embed_grad;

typedef int (*xent_fn)(const hg_xent_shape *s, const void *x, const void *const *w,
                       const void *labels, float *loss, float *lse, void *ws, size_t ws_bytes,
                       void *stream);
typedef int (*xent_grad_fn)(const hg_xent_shape *s, const void *x, const void *const *w,
                            const void *labels, const float *lse, const float *grad, void *dx,
                            void *dw, int dw_wide, int accumulate, void *ws, size_t ws_bytes,
                            void *stream);
typedef int (*xent_step_fn)(const hg_xent_shape *s, const void *x, const void *const *w,
                            const void *labels, const float *grad, float *loss, float *lse,
                            void *dx, void *dw, int dw_wide, int accumulate, void *ws,
                            size_t ws_bytes, void *stream);
static xent_fn g_xent;
static xent_grad_fn g_xent_grad;
static xent_step_fn g_xent_step;

#define MAX_BLOCKS HG_MAX_TP

static int as_ptr(PyObject *o, void **p) {
  *p = PyLong_AsVoidPtr(o);
  return !(*p == NULL && PyErr_Occurred());
}

static int as_int(PyObject *o, int *v) {
  long x = PyLong_AsLong(o);
  if (x == -1 && PyErr_Occurred()) return 0;
  if (x < INT_MIN || x > INT_MAX) {
    PyErr_SetString(PyExc_OverflowError, "integer argument out of range");
    return 0;
  }
  *v = (int)x;
  return 1;
}

static int check_bound(void *fn, Py_ssize_t nargs, Py_ssize_t want) {
  if (!fn) {
    PyErr_SetString(PyExc_RuntimeError, "_hgcall: bind() has not been called");
    return 0;
  }
  if (nargs != want) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, nargs);
    return 0;
  }
  return 1;
}

static int as_float(PyObject *o, float *v) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) return 0;
  *v = (float)x;
  return 1;
}

/* bind(gather, push, collect, stock, embed, embed_grad, xent, xent_grad, xent_step): their
 * addresses */
static PyObject *py_bind(PyObject *self, PyObject *const *args, Py_ssize_t nargs) {
  void *fn[9];
  (void)self;
  if (nargs != 9) {
    PyErr_SetString(PyExc_TypeError, "bind expects nine function addresses");
    return NULL;
  }
  for (int k = 0; k < 9; ++k) {
    if (!as_ptr(args[k], &fn[k])) return NULL;
    if (!fn[k]) {
      PyErr_SetString(PyExc_ValueError, "bind: null function address");
      return NULL;
    }
  }
  g_gather = (gather_fn)fn[0];
  g_push = (push_fn)fn[1];
  g_collect = (collect_fn)fn[2];
  g_stock = (stock_fn)fn[3];
  g_embed = (embed_fn)fn[4];
  g_embed_grad = (embed_grad_fn)fn[5];
  g_xent = (xent_fn)fn[6];
  g_xent_grad = (xent_grad_fn)fn[7];
  g_xent_step = (xent_step_fn)fn[8];
  Py_RETURN_NONE;
}

/* gather(handle, shards_array_addr, m, out_addr, stream) -> status */
static PyObject *py_gather(PyObject *self, PyObject *const *args, Py_ssize_t nargs) {
  void *h, *shards, *out, *stream;
  int m;
  (void)self;
  if (!check_bound((void *)g_gather, nargs, 5)) return NULL;
  if (!as_ptr(args[0], &h) || !as_ptr(args[1], &shards) || !as_int(args[2], &m) ||
      !as_ptr(args[3], &out) || !as_ptr(args[4], &stream))
    return NULL;
  return PyLong_FromLong(g_gather(h, (const void *const *)shards, m, out, stream));
}

/* push(handle, shards_array_addr, m, stream) -> status */
static PyObject *py_push(PyObject *self, PyObject *const *args, Py_ssize_t nargs) {
  void *h, *shards, *stream;
  int m;
  (void)self;
  if (!check_bound((void *)g_push, nargs, 4)) return NULL;
  if (!as_ptr(args[0], &h) || !as_ptr(args[1], &shards) || !as_int(args[2], &m) ||
      !as_ptr(args[3], &stream))
    return NULL;
  return PyLong_FromLong(g_push(h, (const void *const *)shards, m, stream));
}

/* collect(handle, m, out_addr, stream) -> status */
static PyObject *py_collect(PyObject *self, PyObject *const *args, Py_ssize_t nargs) {
  void *h, *out, *stream;
  int m;
  (void)self;
  if (!check_bound((void *)g_collect, nargs, 4)) return NULL;
  if (!as_ptr(args[0], &h) || !as_int(args[1], &m) || !as_ptr(args[2], &out) ||
      !as_ptr(args[3], &stream))
    return NULL;
  return PyLong_FromLong(g_collect(h, m, out, stream));
}

/* stock(tp, shard, shards_array_addr, m, out_addr, vocab, stream) -> status */
static PyObject *py_stock(PyObject *self, PyObject *const *args, Py_ssize_t nargs) {
  void *shards, *out, *stream;
  int tp, shard, m, vocab;
  (void)self;
  if (!check_bound((void *)g_stock, nargs, 7)) return NULL;
  if (!as_int(args[0], &tp) || !as_int(args[1], &shard) || !as_ptr(args[2], &shards) ||
      !as_int(args[3], &m) || !as_ptr(args[4], &out) || !as_int(args[5], &vocab) ||
      !as_ptr(args[6], &stream))
    return NULL;
  return PyLong_FromLong(g_stock(tp, shard, (const void *const *)shards, m, out, vocab, stream));
}

/* embed(tp, shard, hidden, dtype, blocks, tokens, token_bytes, n, scale, out, stream) -> status;
 * blocks: a tuple of tp device addresses */
static PyObject *py_embed(PyObject *self, PyObject *const *args, Py_ssize_t nargs) {
  const void *w[MAX_BLOCKS];
  void *tokens, *out, *stream;
  int tp, shard, hidden, dtype, bytes, n;
  float scale;
  (void)self;
  if (!check_bound((void *)g_embed, nargs, 11)) return NULL;
  if (!as_int(args[0], &tp) || !as_int(args[1], &shard) || !as_int(args[2], &hidden) ||
      !as_int(args[3], &dtype) || !as_ptr(args[5], &tokens) || !as_int(args[6], &bytes) ||
      !as_int(args[7], &n) || !as_float(args[8], &scale) || !as_ptr(args[9], &out) ||
      !as_ptr(args[10], &stream))
    return NULL;
  if (!PyTuple_Check(args[4]) || tp < 0 || tp > MAX_BLOCKS || PyTuple_GET_SIZE(args[4]) != tp) {
    PyErr_SetString(PyExc_TypeError, "blocks must be a tuple of tp addresses");
    return NULL;
  }
  for (int r = 0; r < tp; ++r) {
    void *p;
    if (!as_ptr(PyTuple_GET_ITEM(args[4], r), &p)) return NULL;
    w[r] = p;
  }
  return PyLong_FromLong(
      g_embed(tp, shard, hidden, dtype, w, tokens, bytes, n, scale, out, stream));
}

/* embed_grad(tp, shard, hidden, dtype, tokens, token_bytes, n, dy, scale, dw, dw_wide, accumulate,
 * ws, ws_bytes, stream) -> status */
static PyObject *py_embed_grad(PyObject *self, PyObject *const *args, Py_ssize_t nargs) {
  void *tokens, *dy, *dw, *ws, *stream;
  int tp, shard, hidden, dtype, bytes, n, wide, accumulate;
  float scale;
  size_t ws_bytes;
  (void)self;
  if (!check_bound((void *)g_embed_grad, nargs, 15)) return NULL;
  if (!as_int(args[0], &tp) || !as_int(args[1], &shard) || !as_int(args[2], &hidden) ||
      !as_int(args[3], &dtype) || !as_ptr(args[4], &tokens) || !as_int(args[5], &bytes) ||
      !as_int(args[6], &n) || !as_ptr(args[7], &dy) || !as_float(args[8], &scale) ||
      !as_ptr(args[9], &dw) || !as_int(args[10], &wide) || !as_int(args[11], &accumulate) ||
      !as_ptr(args[12], &ws))
    return NULL;
  ws_bytes = PyLong_AsSize_t(args[13]);
  if (ws_bytes == (size_t)-1 && PyErr_Occurred()) return NULL;
  if (!as_ptr(args[14], &stream)) return NULL;
  return PyLong_FromLong(g_embed_grad(tp, shard, hidden, dtype, tokens, bytes, n, dy, scale, dw,
                                      wide, accumulate, ws, ws_bytes, stream));
}

/* xent(kind, (tp, shard, hidden, m, vocab, dtype, label_bytes), ignore, scale, z_weight, x, blocks,
 * labels, grad, loss, lse, dx, dw, dw_wide, accumulate, ws, ws_bytes, stream) -> status;
 * kind: HG_XENT_*; blocks: a tuple of tp addresses, or of one where the blocks follow one another;
 * addresses that the kind has no use for are 0 (HG_XENT_GRAD reads lse, the others write it) */
static PyObject *py_xent(PyObject *self, PyObject *const *args, Py_ssize_t nargs) {
  const void *w[MAX_BLOCKS];
  hg_xent_shape s;
  void *x, *labels, *grad, *loss, *lse, *dx, *dw, *ws, *stream;
  int kind, wide, accumulate;
  size_t ws_bytes;
  Py_ssize_t blocks;
  (void)self;
  if (!check_bound((void *)g_xent, nargs, 18)) return NULL;
  if (!PyTuple_Check(args[1]) || PyTuple_GET_SIZE(args[1]) != 7 || !PyTuple_Check(args[6])) {
    PyErr_SetString(PyExc_TypeError, "the shape must be a tuple of seven integers, blocks a tuple");
    return NULL;
  }
  memset(&s, 0, sizeof s);
  int *const dims[7] = {&s.tp, &s.shard, &s.hidden, &s.m, &s.vocab, &s.dtype, &s.label_bytes};
  for (int k = 0; k < 7; ++k)
    if (!as_int(PyTuple_GET_ITEM(args[1], k), dims[k])) return NULL;
  s.ignore = PyLong_AsLongLong(args[2]);
  if (s.ignore == -1 && PyErr_Occurred()) return NULL;
  if (!as_int(args[0], &kind) || !as_float(args[3], &s.scale) || !as_float(args[4], &s.z_weight) ||
      !as_ptr(args[5], &x) || !as_ptr(args[7], &labels) || !as_ptr(args[8], &grad) ||
      !as_ptr(args[9], &loss) || !as_ptr(args[10], &lse) || !as_ptr(args[11], &dx) ||
      !as_ptr(args[12], &dw) || !as_int(args[13], &wide) || !as_int(args[14], &accumulate) ||
      !as_ptr(args[15], &ws))
    return NULL;
  ws_bytes = PyLong_AsSize_t(args[16]);
  if (ws_bytes == (size_t)-1 && PyErr_Occurred()) return NULL;
  if (!as_ptr(args[17], &stream)) return NULL;
  blocks = PyTuple_GET_SIZE(args[6]);
  if (s.tp < 1 || s.tp > MAX_BLOCKS) return PyLong_FromLong(HG_EINVAL);
  if (blocks != 1 && blocks != s.tp) {
    PyErr_SetString(PyExc_TypeError, "blocks must hold one or tp addresses");
    return NULL;
  }
  for (int r = 0; r < s.tp; ++r) {
    if (r < blocks) {
      void *p;
      if (!as_ptr(PyTuple_GET_ITEM(args[6], r), &p)) return NULL;
      w[r] = p;
    } else {
      w[r] = (const char *)w[r - 1] + (size_t)s.shard * (size_t)s.hidden * 2;
    }
  }
  switch (kind) {
    case HG_XENT_SCORE:
      return PyLong_FromLong(g_xent(&s, x, w, labels, loss, lse, ws, ws_bytes, stream));
    case HG_XENT_GRAD:
      return PyLong_FromLong(g_xent_grad(&s, x, w, labels, lse, grad, dx, dw, wide, accumulate, ws,
                                         ws_bytes, stream));
    case HG_XENT_STEP:
      return PyLong_FromLong(g_xent_step(&s, x, w, labels, grad, loss, lse, dx, dw, wide,
                                         accumulate, ws, ws_bytes, stream));
    default: return PyLong_FromLong(HG_EINVAL);
  }
}

static PyMethodDef methods[] = {
    {"bind", (PyCFunction)(void (*)(void))py_bind, METH_FASTCALL,
     "bind(gather, push, collect, stock, embed, embed_grad, xent, xent_grad, xent_step)"},
    {"gather", (PyCFunction)(void (*)(void))py_gather, METH_FASTCALL,
     "gather(handle, shards_addr, m, out_addr, stream) -> status"},
    {"push", (PyCFunction)(void (*)(void))py_push, METH_FASTCALL,
     "push(handle, shards_addr, m, stream) -> status"},
    {"collect", (PyCFunction)(void (*)(void))py_collect, METH_FASTCALL,
     "collect(handle, m, out_addr, stream) -> status"},
    {"stock", (PyCFunction)(void (*)(void))py_stock, METH_FASTCALL,
     "stock(tp, shard, shards_addr, m, out_addr, vocab, stream) -> status"},
    {"embed", (PyCFunction)(void (*)(void))py_embed, METH_FASTCALL,
     "embed(tp, shard, hidden, dtype, blocks, tokens, token_bytes, n, scale, out, stream) -> status"},
    {"embed_grad", (PyCFunction)(void (*)(void))py_embed_grad, METH_FASTCALL,
     "embed_grad(tp, shard, hidden, dtype, tokens, token_bytes, n, dy, scale, dw, dw_wide, "
     "accumulate, ws, ws_bytes, stream) -> status"},
    {"xent", (PyCFunction)(void (*)(void))py_xent, METH_FASTCALL,
     "xent(kind, shape, ignore, scale, z_weight, x, blocks, labels, grad, loss, lse, dx, dw, "
     "dw_wide, accumulate, ws, ws_bytes, stream) -> status"},
    {NULL, NULL, 0, NULL},
};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_hgcall",
                                    "Fast-call wrappers of libhg.so's per-call entry points.",
                                    -1, methods};

PyMODINIT_FUNC PyInit__hgcall(void) { return PyModule_Create(&module); }
