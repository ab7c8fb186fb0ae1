/* CPython fast path for the per-step calls of the Python binding:
 * pkd_plan, pkd_plan_shared and pkd_plan_cascade with the page tables passed as int32 arrays
 * through the buffer protocol, and pkd_run_scaled with its pointers as
 * integers (no per-argument ctypes conversion).  It only marshals arguments:
 * the entry points are the C ABI's own, whose addresses the binding hands
 * over once (init), so this module does not link libpkd.
 *
 * plan(ctx, indptr, indices, last, stream) -> (status, epoch)
 * plan_shared(ctx, group_indptr, indptr, indices, last, stream) -> (status, epoch)
 * plan_cascade(ctx, group_indptr, p_indptr, p_indices, p_last, s_indptr, s_indices, s_last,
 *              stream) -> (status, epoch)
 * run(ctx, q, kv, out, lse, k_scale, v_scale, expect_epoch, stream) -> status
 *
 * accumulate, append_latent, evict: pkd_accumulate_weights, pkd_append_latent and
 * pkd_evict_kv with their addresses as integers (evict: one sequence of them per
 * layer array), after init_ops; an integer that does not fit its C type raises
 * OverflowError.
 *
 * plan_tree, run_tree, rotate_append, accept_kv: pkd_plan_tree (arrays as plan's),
 * pkd_run_tree_scaled, pkd_rotate_append_kv and pkd_accept_kv (a list of addresses), after
 * init_step.
 *
 * status is the C ABI's return value, or NOT_HANDLED (1000) when an argument
 * is not a 1-D C-contiguous int32 buffer: the caller then takes its general
 * path, which converts or rejects the input with a proper message. */
#define PY_SSIZE_T_CLEAN
#include <Python.h>
#include <stdint.h>
#include <string.h>

typedef int (*plan_fn)(void *ctx, const int32_t *indptr, const int32_t *indices,
                       const int32_t *last, int32_t batch, void *stream, uint64_t *epoch);
typedef int (*plan_shared_fn)(void *ctx, const int32_t *group_indptr, int32_t num_groups,
                              const int32_t *indptr, const int32_t *indices,
                              const int32_t *last, void *stream, uint64_t *epoch);

typedef int (*plan_cascade_fn)(void *ctx, const int32_t *group_indptr, int32_t num_groups,
                               const int32_t *p_indptr, const int32_t *p_indices,
                               const int32_t *p_last, const int32_t *s_indptr,
                               const int32_t *s_indices, const int32_t *s_last, void *stream,
                               uint64_t *epoch);

typedef int (*run_fn)(void *ctx, const void *q, const void *kv, void *out, float *lse,
                      float k_scale, float v_scale, uint64_t expect_epoch, void *stream);

static plan_fn g_plan = NULL;
static plan_shared_fn g_plan_shared = NULL;
static plan_cascade_fn g_plan_cascade = NULL;
static run_fn g_run = NULL;

#define NOT_HANDLED 1000
#define BAD_TABLE (-2)

static PyObject *init(PyObject *self, PyObject *args) {
  unsigned long long p, ps, pc = 0, pr = 0;
  (void)self;
  if (!PyArg_ParseTuple(args, "KK|KK", &p, &ps, &pc, &pr)) return NULL;
  g_plan = (plan_fn)(uintptr_t)p;
  g_plan_shared = (plan_shared_fn)(uintptr_t)ps;
  g_plan_cascade = (plan_cascade_fn)(uintptr_t)pc;
  g_run = (run_fn)(uintptr_t)pr;
  Py_RETURN_NONE;
}

/* The caller (the binding) has checked the tensors behind the pointers. */
static PyObject *run(PyObject *self, PyObject *args) {
  unsigned long long ctx, q, kv, out, lse, epoch, stream;
  float ks, vs;
  (void)self;
  if (!PyArg_ParseTuple(args, "KKKKKffKK", &ctx, &q, &kv, &out, &lse, &ks, &vs, &epoch, &stream))
    return NULL;
  if (g_run == NULL) return PyLong_FromLong(NOT_HANDLED);
  return PyLong_FromLong(g_run((void *)(uintptr_t)ctx, (const void *)(uintptr_t)q,
                               (const void *)(uintptr_t)kv, (void *)(uintptr_t)out,
                               (float *)(uintptr_t)lse, ks, vs, (uint64_t)epoch,
                               (void *)(uintptr_t)stream));
}

/* A 1-D C-contiguous buffer of 4-byte signed integers, or 0. */
static int get_i32(PyObject *obj, Py_buffer *view) {
  if (PyObject_GetBuffer(obj, view, PyBUF_C_CONTIGUOUS | PyBUF_FORMAT) != 0) {
    PyErr_Clear();
    return 0;
  }
  const char *f = view->format ? view->format : "B";
  if (f[0] == '<' || f[0] == '=' || f[0] == '@') ++f;
  if (view->ndim != 1 || view->itemsize != 4 || (strcmp(f, "i") != 0 && strcmp(f, "l") != 0)) {
    PyBuffer_Release(view);
    return 0;
  }
  return 1;
}

static PyObject *plan(PyObject *self, PyObject *args) {
  unsigned long long ctx, stream;
  PyObject *o_ip, *o_ix, *o_la;
  Py_buffer ip, ix, la;
  (void)self;
  if (!PyArg_ParseTuple(args, "KOOOK", &ctx, &o_ip, &o_ix, &o_la, &stream)) return NULL;
  if (g_plan == NULL) return Py_BuildValue("iK", NOT_HANDLED, 0ULL);
  if (!get_i32(o_ip, &ip)) return Py_BuildValue("iK", NOT_HANDLED, 0ULL);
  if (!get_i32(o_ix, &ix)) {
    PyBuffer_Release(&ip);
    return Py_BuildValue("iK", NOT_HANDLED, 0ULL);
  }
  if (!get_i32(o_la, &la)) {
    PyBuffer_Release(&ip);
    PyBuffer_Release(&ix);
    return Py_BuildValue("iK", NOT_HANDLED, 0ULL);
  }
  const Py_ssize_t batch = la.shape[0];
  int st;
  uint64_t epoch = 0;
  if (ip.shape[0] != batch + 1 || batch > INT32_MAX) {
    st = NOT_HANDLED;   /* the general path reports the shape error */
  } else if (batch > 0 && ix.shape[0] < ((const int32_t *)ip.buf)[batch]) {
    st = NOT_HANDLED;
  } else {
    st = g_plan((void *)(uintptr_t)ctx, (const int32_t *)ip.buf,
                ix.shape[0] ? (const int32_t *)ix.buf : NULL, (const int32_t *)la.buf,
                (int32_t)batch, (void *)(uintptr_t)stream, &epoch);
  }
  PyBuffer_Release(&ip);
  PyBuffer_Release(&ix);
  PyBuffer_Release(&la);
  return Py_BuildValue("iK", st, (unsigned long long)epoch);
}

static PyObject *plan_shared(PyObject *self, PyObject *args) {
  unsigned long long ctx, stream;
  PyObject *o_gi, *o_ip, *o_ix, *o_la;
  Py_buffer gi, ip, ix, la;
  (void)self;
  if (!PyArg_ParseTuple(args, "KOOOOK", &ctx, &o_gi, &o_ip, &o_ix, &o_la, &stream)) return NULL;
  if (g_plan_shared == NULL) return Py_BuildValue("iK", NOT_HANDLED, 0ULL);
  PyObject *objs[4] = {o_gi, o_ip, o_ix, o_la};
  Py_buffer *views[4] = {&gi, &ip, &ix, &la};
  for (int k = 0; k < 4; ++k) {
    if (!get_i32(objs[k], views[k])) {
      for (int j = 0; j < k; ++j) PyBuffer_Release(views[j]);
      return Py_BuildValue("iK", NOT_HANDLED, 0ULL);
    }
  }
  const Py_ssize_t groups = la.shape[0];
  int st;
  uint64_t epoch = 0;
  if (gi.shape[0] != groups + 1 || ip.shape[0] != groups + 1 || groups > INT32_MAX) {
    st = NOT_HANDLED;
  } else {
    st = g_plan_shared((void *)(uintptr_t)ctx, (const int32_t *)gi.buf, (int32_t)groups,
                       (const int32_t *)ip.buf, ix.shape[0] ? (const int32_t *)ix.buf : NULL,
                       (const int32_t *)la.buf, (void *)(uintptr_t)stream, &epoch);
  }
  for (int k = 0; k < 4; ++k) PyBuffer_Release(views[k]);
  return Py_BuildValue("iK", st, (unsigned long long)epoch);
}

static PyObject *plan_cascade(PyObject *self, PyObject *args) {
  unsigned long long ctx, stream;
  PyObject *objs[7];
  Py_buffer v[7];   /* group_indptr, prefix (indptr, indices, last), suffix (same) */
  (void)self;
  if (!PyArg_ParseTuple(args, "KOOOOOOOK", &ctx, &objs[0], &objs[1], &objs[2], &objs[3],
                        &objs[4], &objs[5], &objs[6], &stream))
    return NULL;
  if (g_plan_cascade == NULL) return Py_BuildValue("iK", NOT_HANDLED, 0ULL);
  for (int k = 0; k < 7; ++k) {
    if (!get_i32(objs[k], &v[k])) {
      for (int j = 0; j < k; ++j) PyBuffer_Release(&v[j]);
      return Py_BuildValue("iK", NOT_HANDLED, 0ULL);
    }
  }
  const Py_ssize_t groups = v[3].shape[0], batch = v[6].shape[0];
  const int32_t *gi = (const int32_t *)v[0].buf;
  int st;
  uint64_t epoch = 0;
  if (v[0].shape[0] != groups + 1 || v[1].shape[0] != groups + 1 || v[4].shape[0] != batch + 1 ||
      groups > INT32_MAX || (groups > 0 && gi[groups] != batch) ||
      (groups > 0 && v[2].shape[0] < ((const int32_t *)v[1].buf)[groups]) ||
      (batch > 0 && v[5].shape[0] < ((const int32_t *)v[4].buf)[batch])) {
    st = NOT_HANDLED;
  } else {
    st = g_plan_cascade((void *)(uintptr_t)ctx, gi, (int32_t)groups, (const int32_t *)v[1].buf,
                        v[2].shape[0] ? (const int32_t *)v[2].buf : NULL,
                        (const int32_t *)v[3].buf, (const int32_t *)v[4].buf,
                        v[5].shape[0] ? (const int32_t *)v[5].buf : NULL,
                        (const int32_t *)v[6].buf, (void *)(uintptr_t)stream, &epoch);
  }
  for (int k = 0; k < 7; ++k) PyBuffer_Release(&v[k]);
  return Py_BuildValue("iK", st, (unsigned long long)epoch);
}

typedef int (*accumulate_fn)(void *ctx, const void *q, const void *kv, const float *lse,
                             float *weights, int32_t *positions, const int32_t *new_tokens,
                             const int32_t *seen, float k_scale, uint64_t expect_epoch,
                             void *stream);
typedef int (*append_latent_fn)(const void *latent, int64_t latent_stride, const void *rope,
                                int64_t rope_stride, const int32_t *batch_indices,
                                const int32_t *positions, int32_t n, const int32_t *indptr,
                                const int32_t *indices, int32_t num_indices, const int32_t *last,
                                int32_t batch, void *cache, int32_t num_pages, int32_t page_size, int32_t *err,
                                void *stream);
typedef int (*evict_fn)(int32_t layers, void *const *kv, float *const *weights,
                        int32_t *const *positions, const int32_t *indptr, const int32_t *indices,
                        int32_t num_indices, const int32_t *last, const int32_t *seen, int32_t batch, int32_t max_len,
                        int32_t budget, int32_t sinks, int32_t recent, int32_t per_head,
                        int32_t num_pages, int32_t page_size, int32_t num_kv_heads,
                        int32_t head_dim, uint32_t flags, void *workspace, size_t workspace_bytes,
                        int32_t *err, void *stream);
typedef size_t (*evict_bytes_fn)(int32_t layers, int32_t batch, int32_t max_len, int32_t budget,
                                 int32_t per_head, int32_t num_kv_heads);
static evict_bytes_fn g_evict_bytes = NULL;
static accumulate_fn g_accumulate = NULL;
static append_latent_fn g_append_latent = NULL;
static evict_fn g_evict = NULL;

static PyObject *init_ops(PyObject *self, PyObject *args) {
  unsigned long long a, b, c, d;
  (void)self;
  if (!PyArg_ParseTuple(args, "KKKK", &a, &b, &c, &d)) return NULL;
  g_evict_bytes = (evict_bytes_fn)(uintptr_t)d;
  g_accumulate = (accumulate_fn)(uintptr_t)a;
  g_append_latent = (append_latent_fn)(uintptr_t)b;
  g_evict = (evict_fn)(uintptr_t)c;
  Py_RETURN_NONE;
}

#define ADDR(x) ((void *)(uintptr_t)(x))

static PyObject *accumulate(PyObject *self, PyObject *args) {
  unsigned long long ctx, q, kv, lse, w, pos, nt, seen, epoch, stream;
  float ks;
  (void)self;
  if (!PyArg_ParseTuple(args, "KKKKKKKKfKK", &ctx, &q, &kv, &lse, &w, &pos, &nt, &seen, &ks, &epoch,
                        &stream))
    return NULL;
  if (g_accumulate == NULL) return PyLong_FromLong(NOT_HANDLED);
  return PyLong_FromLong(g_accumulate(ADDR(ctx), ADDR(q), ADDR(kv), (const float *)ADDR(lse),
                                      (float *)ADDR(w), (int32_t *)ADDR(pos),
                                      (const int32_t *)ADDR(nt), (const int32_t *)ADDR(seen), ks,
                                      (uint64_t)epoch, ADDR(stream)));
}

static PyObject *append_latent(PyObject *self, PyObject *args) {
  unsigned long long lat, rope, bi, pos, ip, ix, la, cache, err, stream;
  long long ls, rs;
  int n, nnz, batch, pages, page;
  (void)self;
  if (!PyArg_ParseTuple(args, "KLKLKKiKKiKiKiiKK", &lat, &ls, &rope, &rs, &bi, &pos, &n, &ip, &ix,
                        &nnz, &la, &batch, &cache, &pages, &page, &err, &stream))
    return NULL;
  if (g_append_latent == NULL) return PyLong_FromLong(NOT_HANDLED);
  return PyLong_FromLong(g_append_latent(
      ADDR(lat), (int64_t)ls, ADDR(rope), (int64_t)rs, (const int32_t *)ADDR(bi),
      (const int32_t *)ADDR(pos), n, (const int32_t *)ADDR(ip), (const int32_t *)ADDR(ix), nnz,
      (const int32_t *)ADDR(la), batch, ADDR(cache), pages, page, (int32_t *)ADDR(err),
      ADDR(stream)));
}

static PyObject *evict_bytes(PyObject *self, PyObject *args) {
  int layers, batch, max_len, budget, per_head, hkv;
  (void)self;
  if (!PyArg_ParseTuple(args, "iiiiii", &layers, &batch, &max_len, &budget, &per_head, &hkv))
    return NULL;
  if (g_evict_bytes == NULL) return PyLong_FromLong(0);
  return PyLong_FromSize_t(g_evict_bytes(layers, batch, max_len, budget, per_head, hkv));
}

#define MAX_LAYERS 128
/* n addresses of a sequence into out; 0 when it is not a list of n integers */
static int addresses(PyObject *list, Py_ssize_t n, void **out) {
  if (!PyList_Check(list) || PyList_GET_SIZE(list) != n) return 0;
  for (Py_ssize_t i = 0; i < n; ++i) {
    const unsigned long long v = PyLong_AsUnsignedLongLong(PyList_GET_ITEM(list, i));
    if (v == (unsigned long long)-1 && PyErr_Occurred()) {
      PyErr_Clear();
      return 0;
    }
    out[i] = ADDR(v);
  }
  return 1;
}

static PyObject *evict(PyObject *self, PyObject *args) {
  PyObject *kv, *w, *p;
  unsigned long long ip, ix, la, seen, ws, err, stream, ws_bytes;
  int nnz, batch, max_len, budget, sinks, recent, per_head, pages, page, hkv, dim;
  unsigned int flags;
  void *kvs[MAX_LAYERS], *ws_[MAX_LAYERS], *ps[MAX_LAYERS];
  (void)self;
  if (!PyArg_ParseTuple(args, "OOOKKiKKiiiiiiiiiiIKKKK", &kv, &w, &p, &ip, &ix, &nnz, &la, &seen, &batch,
                        &max_len, &budget, &sinks, &recent, &per_head, &pages, &page, &hkv, &dim,
                        &flags, &ws, &ws_bytes, &err, &stream))
    return NULL;
  const Py_ssize_t layers = PyList_Check(kv) ? PyList_GET_SIZE(kv) : 0;
  if (g_evict == NULL || layers < 1 || layers > MAX_LAYERS || !addresses(kv, layers, kvs) ||
      !addresses(w, layers, ws_) || !addresses(p, layers, ps))
    return PyLong_FromLong(NOT_HANDLED);
  return PyLong_FromLong(g_evict(
      (int32_t)layers, kvs, (float *const *)ws_, (int32_t *const *)ps, (const int32_t *)ADDR(ip),
      (const int32_t *)ADDR(ix), nnz, (const int32_t *)ADDR(la), (const int32_t *)ADDR(seen), batch,
      max_len, budget, sinks, recent, per_head, pages, page, hkv, dim, (uint32_t)flags, ADDR(ws),
      (size_t)ws_bytes, (int32_t *)ADDR(err), ADDR(stream)));
}

typedef int (*plan_tree_fn)(void *ctx, const int32_t *q_indptr, const int32_t *indptr,
                            const int32_t *indices, const int32_t *last, int32_t batch,
                            int32_t causal, int32_t window, void *stream, uint64_t *epoch);
typedef int (*run_tree_fn)(void *ctx, const void *q, int32_t rows, const void *kv, void *out,
                           float *lse, const uint32_t *mask, int32_t mask_words,
                           const int32_t *depths, const float *slopes, float scale,
                           float score_cap, float k_scale, float v_scale, uint64_t expect_epoch,
                           void *stream);
typedef int (*rotate_fn)(const void *q, int64_t q_token, int64_t q_head, void *q_out,
                         int64_t out_token, int64_t out_head, const void *k, int64_t k_token,
                         int64_t k_head, const void *v, int64_t v_token, int64_t v_head,
                         const void *q_norm, const void *k_norm, int32_t norms_f32, float eps,
                         const uint64_t *turns, const int32_t *axes, int32_t rotary_dim,
                         int32_t interleaved, float rope_scale, const int32_t *rope_positions,
                         int32_t num_axes, const int32_t *batch_indices,
                         const int32_t *positions, int32_t n, const int32_t *indptr,
                         const int32_t *indices, int32_t num_indices, const int32_t *last,
                         int32_t batch, void *kv, int32_t num_pages, int32_t page_size,
                         int32_t hq, int32_t hkv, int32_t head_dim, float k_scale, float v_scale,
                         uint32_t flags, int32_t *err, void *stream);
typedef int (*accept_fn)(int32_t layers, void *const *kv, const int32_t *accepted, int32_t width,
                         const int32_t *drafted, const int32_t *indptr, const int32_t *indices,
                         int32_t num_indices, const int32_t *last, int32_t batch,
                         int32_t num_pages, int32_t page_size, int32_t hkv, int32_t head_dim,
                         uint32_t flags, int32_t *err, void *stream);
static plan_tree_fn g_plan_tree = NULL;
static run_tree_fn g_run_tree = NULL;
static rotate_fn g_rotate = NULL;
static accept_fn g_accept = NULL;

static PyObject *init_step(PyObject *self, PyObject *args) {
  unsigned long long a, b, c, d;
  (void)self;
  if (!PyArg_ParseTuple(args, "KKKK", &a, &b, &c, &d)) return NULL;
  g_plan_tree = (plan_tree_fn)(uintptr_t)a;
  g_run_tree = (run_tree_fn)(uintptr_t)b;
  g_rotate = (rotate_fn)(uintptr_t)c;
  g_accept = (accept_fn)(uintptr_t)d;
  Py_RETURN_NONE;
}

static PyObject *plan_tree(PyObject *self, PyObject *args) {
  unsigned long long ctx, stream;
  int causal, window;
  PyObject *objs[4];
  Py_buffer v[4];   /* q_indptr, indptr, indices, last */
  (void)self;
  if (!PyArg_ParseTuple(args, "KOOOOiiK", &ctx, &objs[0], &objs[1], &objs[2], &objs[3], &causal,
                        &window, &stream))
    return NULL;
  if (g_plan_tree == NULL) return Py_BuildValue("iK", NOT_HANDLED, 0ULL);
  for (int k = 0; k < 4; ++k) {
    if (!get_i32(objs[k], &v[k])) {
      for (int j = 0; j < k; ++j) PyBuffer_Release(&v[j]);
      return Py_BuildValue("iK", NOT_HANDLED, 0ULL);
    }
  }
  const Py_ssize_t batch = v[3].shape[0];
  int st;
  uint64_t epoch = 0;
  if (v[0].shape[0] != batch + 1 || v[1].shape[0] != batch + 1 || batch > INT32_MAX ||
      (batch > 0 && v[2].shape[0] < ((const int32_t *)v[1].buf)[batch])) {
    st = NOT_HANDLED;   /* the general path reports the shape error */
  } else {
    st = g_plan_tree((void *)(uintptr_t)ctx, (const int32_t *)v[0].buf, (const int32_t *)v[1].buf,
                     v[2].shape[0] ? (const int32_t *)v[2].buf : NULL, (const int32_t *)v[3].buf,
                     (int32_t)batch, causal, window, (void *)(uintptr_t)stream, &epoch);
  }
  for (int k = 0; k < 4; ++k) PyBuffer_Release(&v[k]);
  return Py_BuildValue("iK", st, (unsigned long long)epoch);
}

static PyObject *run_tree(PyObject *self, PyObject *args) {
  unsigned long long ctx, q, kv, out, lse, mask, depths, slopes, epoch, stream;
  int rows, words;
  float scale, cap, ks, vs;
  (void)self;
  if (!PyArg_ParseTuple(args, "KKiKKKKiKKffffKK", &ctx, &q, &rows, &kv, &out, &lse, &mask, &words,
                        &depths, &slopes, &scale, &cap, &ks, &vs, &epoch, &stream))
    return NULL;
  if (g_run_tree == NULL) return PyLong_FromLong(NOT_HANDLED);
  return PyLong_FromLong(g_run_tree(ADDR(ctx), ADDR(q), rows, ADDR(kv), ADDR(out),
                                    (float *)ADDR(lse), (const uint32_t *)ADDR(mask), words,
                                    (const int32_t *)ADDR(depths), (const float *)ADDR(slopes),
                                    scale, cap, ks, vs, (uint64_t)epoch, ADDR(stream)));
}

static PyObject *rotate_append(PyObject *self, PyObject *args) {
  unsigned long long q, qo, k, v, qn, kn, turns, axes, rp, bi, pos, ip, ix, la, kv, err, stream;
  long long qt, qh, ot, oh, kt, kh, vt, vh;
  int f32, rotary, pairs, n_axes, n, nnz, batch, pages, page, hq, hkv, dim;
  float eps, rs, ks, vs;
  unsigned int flags;
  (void)self;
  if (!PyArg_ParseTuple(args, "KLLKLLKLLKLLKKifKKiifKiKKiKKiKiKiiiiiffIKK", &q, &qt, &qh, &qo, &ot,
                        &oh, &k, &kt, &kh, &v, &vt, &vh, &qn, &kn, &f32, &eps, &turns, &axes,
                        &rotary, &pairs, &rs, &rp, &n_axes, &bi, &pos, &n, &ip, &ix, &nnz, &la,
                        &batch, &kv, &pages, &page, &hq, &hkv, &dim, &ks, &vs, &flags, &err,
                        &stream))
    return NULL;
  if (g_rotate == NULL) return PyLong_FromLong(NOT_HANDLED);
  return PyLong_FromLong(g_rotate(
      ADDR(q), qt, qh, ADDR(qo), ot, oh, ADDR(k), kt, kh, ADDR(v), vt, vh, ADDR(qn), ADDR(kn), f32,
      eps, (const uint64_t *)ADDR(turns), (const int32_t *)ADDR(axes), rotary, pairs, rs,
      (const int32_t *)ADDR(rp), n_axes, (const int32_t *)ADDR(bi), (const int32_t *)ADDR(pos), n,
      (const int32_t *)ADDR(ip), (const int32_t *)ADDR(ix), nnz, (const int32_t *)ADDR(la), batch,
      ADDR(kv), pages, page, hq, hkv, dim, ks, vs, (uint32_t)flags, (int32_t *)ADDR(err),
      ADDR(stream)));
}

static PyObject *accept_kv(PyObject *self, PyObject *args) {
  PyObject *kv;
  unsigned long long acc, dr, ip, ix, la, err, stream;
  int width, nnz, batch, pages, page, hkv, dim;
  unsigned int flags;
  void *kvs[MAX_LAYERS];
  (void)self;
  if (!PyArg_ParseTuple(args, "OKiKKKiKiiiiiIKK", &kv, &acc, &width, &dr, &ip, &ix, &nnz, &la,
                        &batch, &pages, &page, &hkv, &dim, &flags, &err, &stream))
    return NULL;
  const Py_ssize_t layers = PyList_Check(kv) ? PyList_GET_SIZE(kv) : 0;
  if (g_accept == NULL || layers < 1 || layers > MAX_LAYERS || !addresses(kv, layers, kvs))
    return PyLong_FromLong(NOT_HANDLED);
  return PyLong_FromLong(g_accept((int32_t)layers, kvs, (const int32_t *)ADDR(acc), width,
                                  (const int32_t *)ADDR(dr), (const int32_t *)ADDR(ip),
                                  (const int32_t *)ADDR(ix), nnz, (const int32_t *)ADDR(la), batch,
                                  pages, page, hkv, dim, (uint32_t)flags, (int32_t *)ADDR(err),
                                  ADDR(stream)));
}

static PyMethodDef methods[] = {
    {"init_step", init_step, METH_VARARGS,
     "init_step(plan_tree_address, run_tree_address, rotate_append_address, accept_address)"},
    {"plan_tree", plan_tree, METH_VARARGS,
     "plan_tree(ctx, q_indptr, indptr, indices, last, causal, window, stream) -> (status, epoch)"},
    {"run_tree", run_tree, METH_VARARGS, "pkd_run_tree_scaled -> status"},
    {"rotate_append", rotate_append, METH_VARARGS, "pkd_rotate_append_kv -> status"},
    {"accept_kv", accept_kv, METH_VARARGS, "pkd_accept_kv (a list of addresses) -> status"},
    {"init_ops", init_ops, METH_VARARGS,
     "init_ops(accumulate_weights_address, append_latent_address, evict_address, "
     "evict_workspace_bytes_address)"},
    {"evict_bytes", evict_bytes, METH_VARARGS, "pkd_evict_workspace_bytes -> bytes"},
    {"accumulate", accumulate, METH_VARARGS, "pkd_accumulate_weights -> status"},
    {"append_latent", append_latent, METH_VARARGS, "pkd_append_latent -> status"},
    {"evict", evict, METH_VARARGS, "pkd_evict_kv (lists of addresses per layer) -> status"},
    {"plan_cascade", plan_cascade, METH_VARARGS,
     "plan_cascade(ctx, group_indptr, p_indptr, p_indices, p_last, s_indptr, s_indices, "
     "s_last, stream) -> (status, epoch)"},
    {"init", init, METH_VARARGS,
     "init(plan_address, plan_shared_address[, plan_cascade_address[, run_scaled_address]])"},
    {"run", run, METH_VARARGS,
     "run(ctx, q, kv, out, lse, k_scale, v_scale, expect_epoch, stream) -> status"},
    {"plan", plan, METH_VARARGS, "plan(ctx, indptr, indices, last, stream) -> (status, epoch)"},
    {"plan_shared", plan_shared, METH_VARARGS,
     "plan_shared(ctx, group_indptr, indptr, indices, last, stream) -> (status, epoch)"},
    {NULL, NULL, 0, NULL}};

static struct PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pkd_plan", NULL, -1, methods,
                                    NULL, NULL, NULL, NULL};

PyMODINIT_FUNC PyInit__pkd_plan(void) { return PyModule_Create(&module); }
