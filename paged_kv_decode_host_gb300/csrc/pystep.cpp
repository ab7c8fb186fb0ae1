// The calls of drafts.py on tensors directly: pkd_rotate_append_kv,
// pkd_run_tree_scaled and pkd_accept_kv with their arguments checked, outputs
// allocated and addresses taken in C++ (a call's host time from 16-20 us to
// about 5: these run once per layer, and an accept names every layer's cache).
//
// Each function handles the common call -- the current stream, on the current
// device, every tensor as the call wants it -- and returns NotImplemented,
// having done nothing, for any other: the binding's own path then takes it, or
// says what is wrong.  The entry points are the C ABI's, whose addresses the
// binding hands over once (init), so this module does not link libpkd.
#include <Python.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <cstring>

#include "pkd.h"

namespace {

decltype(&pkd_rotate_append_kv) g_rotate = nullptr;
decltype(&pkd_run_tree_scaled) g_run_tree = nullptr;
decltype(&pkd_accept_kv) g_accept = nullptr;

constexpr int kLayers = 128;

PyObject* other() {
  PyErr_Clear();
  Py_RETURN_NOTIMPLEMENTED;
}

// A tensor argument; `ok` is cleared for anything else.
const at::Tensor* tensor(PyObject* o, bool& ok) {
  if (THPVariable_Check(o)) return &THPVariable_Unpack(o);
  ok = false;
  return nullptr;
}
const at::Tensor* tensor_or_none(PyObject* o, bool& ok) { return o == Py_None ? nullptr : tensor(o, ok); }

bool on(const at::Tensor& t, at::ScalarType type, int dev) {
  return t.scalar_type() == type && t.is_cuda() && t.get_device() == dev;
}
bool whole(const at::Tensor& t, at::ScalarType type, int dev) { return on(t, type, dev) && t.is_contiguous(); }

bool is_shape(const at::Tensor& t, at::IntArrayRef want) { return t.sizes() == want; }

// The device table; its batch in *batch.
bool table(const at::Tensor& indptr, const at::Tensor& indices, const at::Tensor& last, int dev, int64_t* batch) {
  *batch = last.numel();
  return whole(indptr, at::kInt, dev) && whole(indices, at::kInt, dev) && whole(last, at::kInt, dev) &&
         indptr.numel() == *batch + 1 && indices.numel() <= INT32_MAX && *batch <= INT32_MAX;
}

void* address(const at::Tensor* t) { return t == nullptr ? nullptr : t->data_ptr(); }

// The shape of a K / V cache.
struct Cache {
  bool fp8;
  int64_t pages, page, heads, dim;
};
bool cache_of(const at::Tensor& kv, bool hnd, Cache* c) {
  if (!kv.is_cuda() || kv.dim() != 5 || kv.size(1) != 2 || !kv.is_contiguous()) return false;
  c->fp8 = kv.scalar_type() == at::kFloat8_e4m3fn;
  if (!c->fp8 && kv.scalar_type() != at::kBFloat16) return false;
  c->pages = kv.size(0);
  c->page = kv.size(hnd ? 3 : 2);
  c->heads = kv.size(hnd ? 2 : 3);
  c->dim = kv.size(4);
  return c->pages <= INT32_MAX && c->page <= INT32_MAX && c->heads <= INT32_MAX && c->dim <= INT32_MAX;
}

// Contiguous heads of [n][heads][dim] on 16-byte boundaries.
bool rows(const at::Tensor& t, int dev, int64_t n, int64_t dim) {
  return on(t, at::kBFloat16, dev) && t.dim() == 3 && t.size(0) == n && t.size(2) == dim && t.stride(2) == 1 &&
         (n <= 1 || t.stride(0) % 8 == 0) && (t.size(1) <= 1 || t.stride(1) % 8 == 0) &&
         reinterpret_cast<uintptr_t>(t.data_ptr()) % 16 == 0 && t.size(1) <= INT32_MAX;
}

// rotate_append(q, k, v, rope_args, rope_axes, rope_dev, batch_indices, positions, indptr, indices,
//               last, kv, rope_positions, q_norm, k_norm, eps, k_scale, v_scale, hnd, err)
//   -> (status, q_out); rope_args: a tuple (turns, axes, rotary_dim, interleaved, scale) or None
PyObject* rotate_append(PyObject*, PyObject* const* a, Py_ssize_t count) try {
  if (g_rotate == nullptr || count != 20) return other();
  bool ok = true;
  const at::Tensor *q = tensor_or_none(a[0], ok), *k = tensor(a[1], ok), *v = tensor(a[2], ok),
                   *rows_of = tensor(a[6], ok), *places = tensor(a[7], ok), *indptr = tensor(a[8], ok),
                   *indices = tensor(a[9], ok), *last = tensor(a[10], ok), *kv = tensor(a[11], ok),
                   *at = tensor_or_none(a[12], ok), *qn = tensor_or_none(a[13], ok),
                   *kn = tensor_or_none(a[14], ok), *err = tensor_or_none(a[19], ok);
  if (!ok) return other();
  const double eps = PyFloat_AsDouble(a[15]), ks = PyFloat_AsDouble(a[16]), vs = PyFloat_AsDouble(a[17]);
  const long hnd = PyLong_AsLong(a[18]);
  Cache c;
  if (PyErr_Occurred() || !cache_of(*kv, hnd != 0, &c)) return other();
  const int dev = kv->get_device();
  if (c10::cuda::current_device() != dev) return other();
  const int64_t n = rows_of->numel();
  int64_t batch;
  if (!whole(*rows_of, at::kInt, dev) || !whole(*places, at::kInt, dev) || places->numel() != n || n > INT32_MAX ||
      !table(*indptr, *indices, *last, dev, &batch) || n == 0 || !rows(*k, dev, n, c.dim) ||
      !rows(*v, dev, n, c.dim) || k->size(1) != c.heads || v->size(1) != c.heads)
    return other();
  if (q != nullptr ? !rows(*q, dev, n, c.dim) : qn != nullptr) return other();
  if (err != nullptr && (!on(*err, at::kInt, dev) || err->numel() < 1)) return other();
  // the rotation
  const void *turns = nullptr, *axes = nullptr;
  long rotary = 0, pairs = 0;
  double scale = 1.0;
  int64_t num_axes = 1;
  const at::Tensor* where = nullptr;
  if (a[3] != Py_None) {
    if (!PyTuple_Check(a[3]) || PyTuple_GET_SIZE(a[3]) != 5) return other();
    turns = PyLong_AsVoidPtr(PyTuple_GET_ITEM(a[3], 0));
    axes = PyLong_AsVoidPtr(PyTuple_GET_ITEM(a[3], 1));
    rotary = PyLong_AsLong(PyTuple_GET_ITEM(a[3], 2));
    pairs = PyLong_AsLong(PyTuple_GET_ITEM(a[3], 3));
    scale = PyFloat_AsDouble(PyTuple_GET_ITEM(a[3], 4));
    const long most = PyLong_AsLong(a[4]), rope_dev = PyLong_AsLong(a[5]);
    if (PyErr_Occurred()) return other();
    where = at == nullptr ? places : at;
    if (where->dim() == 2) num_axes = where->size(1);
    if (rope_dev != dev || !whole(*where, at::kInt, dev) || where->numel() != n * num_axes || most > num_axes ||
        num_axes > 4 || rotary > c.dim)
      return other();
  }
  int f32 = -1;
  for (const at::Tensor* w : {qn, kn}) {
    if (w == nullptr) continue;
    const int kind = w->scalar_type() == at::kFloat ? 1 : 0;
    if ((kind == 0 && w->scalar_type() != at::kBFloat16) || (f32 >= 0 && f32 != kind) || !w->is_cuda() ||
        w->get_device() != dev || w->dim() != 1 || w->size(0) != c.dim || !w->is_contiguous())
      return other();
    f32 = kind;
  }
  at::Tensor out;
  int64_t hq = 0;
  if (q != nullptr) {
    hq = q->size(1);
    out = at::empty({n, hq, c.dim}, q->options());
  }
  const int st = g_rotate(
      address(q), q ? q->stride(0) : 0, q ? q->stride(1) : 0, q ? out.data_ptr() : nullptr, hq * c.dim, c.dim,
      k->data_ptr(), k->stride(0), k->stride(1), v->data_ptr(), v->stride(0), v->stride(1), address(qn), address(kn),
      f32 == 1, (float)eps, static_cast<const uint64_t*>(turns), static_cast<const int32_t*>(axes), (int32_t)rotary,
      (int32_t)pairs, (float)scale, static_cast<const int32_t*>(address(where)), (int32_t)num_axes,
      static_cast<const int32_t*>(rows_of->data_ptr()), static_cast<const int32_t*>(places->data_ptr()), (int32_t)n,
      static_cast<const int32_t*>(indptr->data_ptr()), static_cast<const int32_t*>(indices->data_ptr()),
      (int32_t)indices->numel(), static_cast<const int32_t*>(last->data_ptr()), (int32_t)batch, kv->data_ptr(),
      (int32_t)c.pages, (int32_t)c.page, (int32_t)hq, (int32_t)c.heads, (int32_t)c.dim, (float)ks, (float)vs,
      (hnd ? PKD_FLAG_HND : 0u) | (c.fp8 ? PKD_FLAG_KV_FP8 : 0u), static_cast<int32_t*>(address(err)),
      c10::cuda::getCurrentCUDAStream(dev).stream());
  PyObject* res = q ? THPVariable_Wrap(std::move(out)) : Py_NewRef(Py_None);
  return res == nullptr ? nullptr : Py_BuildValue("iN", st, res);
} catch (...) {   // (no memory for the output, say: the binding's path raises it)
  return other();
}

// run_tree(ctx, device, tokens, causal, kv_shape, q, kv, mask, depths, slopes, scale, score_cap, out,
//          lse, return_lse, expect_epoch, k_scale, v_scale, fp8) -> (status, out, lse or None); kv_shape: the context's
//          (pages, 2, P, Hkv, D) or (pages, 2, Hkv, P, D), then Hq
PyObject* run_tree(PyObject*, PyObject* const* a, Py_ssize_t count) try {
  if (g_run_tree == nullptr || count != 19) return other();
  bool ok = true;
  const at::Tensor *q = tensor(a[5], ok), *kv = tensor(a[6], ok), *mask = tensor_or_none(a[7], ok),
                   *depths = tensor_or_none(a[8], ok), *slopes = tensor_or_none(a[9], ok),
                   *out = tensor_or_none(a[12], ok), *lse = tensor_or_none(a[13], ok);
  if (!ok || !PyTuple_Check(a[4]) || PyTuple_GET_SIZE(a[4]) != 6) return other();
  void* ctx = PyLong_AsVoidPtr(a[0]);
  const long dev = PyLong_AsLong(a[1]), tokens = PyLong_AsLong(a[2]), causal = PyLong_AsLong(a[3]);
  const double scale = PyFloat_AsDouble(a[10]), cap = PyFloat_AsDouble(a[11]);
  const long want_lse = PyLong_AsLong(a[14]);
  const unsigned long long epoch = PyLong_AsUnsignedLongLong(a[15]);
  const double ks = PyFloat_AsDouble(a[16]), vs = PyFloat_AsDouble(a[17]);
  const at::ScalarType kv_type = PyLong_AsLong(a[18]) ? at::kFloat8_e4m3fn : at::kBFloat16;
  int64_t shape[6];
  for (int i = 0; i < 6; ++i) shape[i] = PyLong_AsLongLong(PyTuple_GET_ITEM(a[4], i));
  if (PyErr_Occurred() || c10::cuda::current_device() != dev) return other();
  const int64_t hq = shape[5], dim = shape[4];
  if (q->dim() != 3) return other();
  const int64_t n = q->size(0), words = mask != nullptr && mask->dim() == 2 ? mask->size(1) : 0;
  const int64_t q_shape[3] = {n, hq, dim};
  const at::IntArrayRef heads(q_shape, 2);
  if (n < tokens || n > INT32_MAX || words > INT32_MAX || !whole(*q, at::kBFloat16, dev) ||
      !is_shape(*q, q_shape) || !whole(*kv, kv_type, dev) || !is_shape(*kv, at::IntArrayRef(shape, 5)) ||
      (mask && (!whole(*mask, at::kInt, dev) || mask->dim() != 2 || mask->size(0) != n)) ||
      (depths && (!whole(*depths, at::kInt, dev) || !is_shape(*depths, {n}))) ||
      (slopes && (!whole(*slopes, at::kFloat, dev) || !is_shape(*slopes, {hq}))) ||
      (out && (!whole(*out, at::kBFloat16, dev) || !is_shape(*out, q_shape))) ||
      (lse && (!whole(*lse, at::kFloat, dev) || !is_shape(*lse, heads))) ||
      (causal ? mask || depths : !mask && tokens > 0))
    return other();
  at::Tensor o = out ? *out : at::empty(q_shape, q->options());
  at::Tensor l;
  if (lse)
    l = *lse;
  else if (want_lse)
    l = at::empty(heads, q->options().dtype(at::kFloat));
  const int st = g_run_tree(static_cast<pkd_ctx*>(ctx), q->data_ptr(), (int32_t)n, kv->data_ptr(), o.data_ptr(),
                            l.defined() ? static_cast<float*>(l.data_ptr()) : nullptr,
                            static_cast<const uint32_t*>(address(mask)), (int32_t)words,
                            static_cast<const int32_t*>(address(depths)),
                            static_cast<const float*>(address(slopes)), (float)scale, (float)cap, (float)ks, (float)vs,
                            epoch,
                            c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream());
  PyObject* po = out ? Py_NewRef(a[12]) : THPVariable_Wrap(std::move(o));
  PyObject* pl = lse ? Py_NewRef(a[13]) : l.defined() ? THPVariable_Wrap(std::move(l)) : Py_NewRef(Py_None);
  if (po == nullptr || pl == nullptr) {
    Py_XDECREF(po);
    Py_XDECREF(pl);
    return nullptr;
  }
  return Py_BuildValue("iNN", st, po, pl);
} catch (...) {
  return other();
}

// accept_kv(kv_caches, accepted, drafted, indptr, indices, last, hnd, err) -> status
PyObject* accept_kv(PyObject*, PyObject* const* a, Py_ssize_t count) try {
  if (g_accept == nullptr || count != 8 || !(PyList_Check(a[0]) || PyTuple_Check(a[0]))) return other();
  const Py_ssize_t layers = PySequence_Fast_GET_SIZE(a[0]);
  if (layers < 1 || layers > kLayers) return other();
  bool ok = true;
  const at::Tensor *accepted = tensor(a[1], ok), *drafted = tensor(a[2], ok), *indptr = tensor(a[3], ok),
                   *indices = tensor(a[4], ok), *last = tensor(a[5], ok), *err = tensor_or_none(a[7], ok);
  const long hnd = PyLong_AsLong(a[6]);
  if (!ok || PyErr_Occurred()) return other();
  void* kv[kLayers];
  Cache c;
  int dev = -1;
  PyObject** items = PySequence_Fast_ITEMS(a[0]);
  const at::Tensor* first = nullptr;
  for (Py_ssize_t l = 0; l < layers; ++l) {
    const at::Tensor* t = tensor(items[l], ok);
    if (!ok) return other();
    if (l == 0) {
      if (!cache_of(*t, hnd != 0, &c)) return other();
      first = t;
      dev = t->get_device();
    } else if (!whole(*t, first->scalar_type(), dev) || !is_shape(*t, first->sizes())) {
      return other();
    }
    kv[l] = t->data_ptr();
  }
  int64_t batch;
  if (c10::cuda::current_device() != dev || !table(*indptr, *indices, *last, dev, &batch) ||
      !whole(*accepted, at::kInt, dev) || accepted->dim() != 2 || accepted->size(0) != batch ||
      accepted->size(1) > INT32_MAX || !whole(*drafted, at::kInt, dev) || drafted->numel() != batch ||
      (err != nullptr && (!on(*err, at::kInt, dev) || err->numel() < 1)))
    return other();
  return PyLong_FromLong(g_accept(
      (int32_t)layers, kv, static_cast<const int32_t*>(accepted->data_ptr()), (int32_t)accepted->size(1),
      static_cast<const int32_t*>(drafted->data_ptr()), static_cast<const int32_t*>(indptr->data_ptr()),
      static_cast<const int32_t*>(indices->data_ptr()), (int32_t)indices->numel(),
      static_cast<const int32_t*>(last->data_ptr()), (int32_t)batch, (int32_t)c.pages, (int32_t)c.page,
      (int32_t)c.heads, (int32_t)c.dim, (hnd ? PKD_FLAG_HND : 0u) | (c.fp8 ? PKD_FLAG_KV_FP8 : 0u),
      static_cast<int32_t*>(address(err)), c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev).stream()));
} catch (...) {
  return other();
}

// init(abi, torch_version, rotate_append_address, run_tree_address, accept_address); ImportError
// where the module was built for other entry points or another torch
PyObject* init(PyObject*, PyObject* args) {
  int abi;
  const char* torch;
  unsigned long long r, t, c;
  if (!PyArg_ParseTuple(args, "isKKK", &abi, &torch, &r, &t, &c)) return nullptr;
  if (abi != PKD_STEP_ABI || std::strcmp(torch, PKD_TORCH) != 0) {
    PyErr_SetString(PyExc_ImportError, "_pkd_step was built for another libpkd or torch");
    return nullptr;
  }
  g_rotate = reinterpret_cast<decltype(g_rotate)>((uintptr_t)r);
  g_run_tree = reinterpret_cast<decltype(g_run_tree)>((uintptr_t)t);
  g_accept = reinterpret_cast<decltype(g_accept)>((uintptr_t)c);
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"init", init, METH_VARARGS, "init(abi, torch_version, rotate_append_address, run_tree_address, accept_address)"},
    {"rotate_append", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&rotate_append)), METH_FASTCALL,
     "pkd_rotate_append_kv on tensors -> (status, q_out), or NotImplemented"},
    {"run_tree", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&run_tree)), METH_FASTCALL,
     "pkd_run_tree_scaled on tensors -> (status, out, lse), or NotImplemented"},
    {"accept_kv", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&accept_kv)), METH_FASTCALL,
     "pkd_accept_kv on tensors -> status, or NotImplemented"},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pkd_step", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pkd_step(void) { return PyModule_Create(&module); }
