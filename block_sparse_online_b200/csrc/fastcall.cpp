// fastcall.cpp -- a short way from Python to the dense attention and cache entry points.
//
// These calls take 3 to 10 us on the GPU at the sizes of single tokens, and checking a call's
// tensors attribute by attribute in Python takes as long. The functions here check the usual
// call (every tensor given, on the current device, on the current stream or a given one of that device) and make it. They
// return the library's status, or None for anything else: the caller then takes the Python way, which
// says what is wrong or does what is left. The library's function is passed as an address, so
// that a call goes to the library that the Python side has loaded.
#include <Python.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "solattn.h"

namespace {

const at::Tensor *tensor(PyObject *x) { return THPVariable_Check(x) ? &THPVariable_Unpack(x) : nullptr; }

int dtype_of(const at::Tensor &t) {
  return t.scalar_type() == at::kBFloat16 ? SOLATTN_BF16 : t.scalar_type() == at::kHalf ? SOLATTN_FP16 : -1;
}

bool on(const at::Tensor &t, int dev) { return t.is_cuda() && t.get_device() == dev && t.layout() == at::kStrided; }

// A [B][heads][n][d] tensor, or packed rows [n][heads][d] (dims = 3).
bool view(PyObject *o, int dev, int dt, int dims, int64_t B, int64_t h, int64_t n, int64_t d, solattn_view *v) {
  const at::Tensor *t = tensor(o);
  if (!t || !on(*t, dev) || dtype_of(*t) != dt || t->dim() != dims) return false;
  const auto s = t->sizes();
  const auto st = t->strides();
  if (dims == 4 ? s[0] != B || s[1] != h || s[2] != n || s[3] != d : s[0] != n || s[1] != h || s[2] != d) return false;
  if (st[dims - 1] != 1 || t->numel() == 0) return false;
  *v = dims == 4 ? solattn_view{t->data_ptr(), st[0], st[1], st[2]} : solattn_view{t->data_ptr(), 0, st[1], st[0]};
  return true;
}

const int32_t *ints(PyObject *o, int dev, int64_t n) {
  const at::Tensor *t = tensor(o);
  if (!t || !on(*t, dev) || t->scalar_type() != at::kInt || !t->is_contiguous() || t->numel() < n) return nullptr;
  return static_cast<const int32_t *>(t->data_ptr());
}

bool bytes(PyObject *o, int dev, void **ptr, size_t *n) {
  const at::Tensor *t = tensor(o);
  if (!t || !on(*t, dev) || t->scalar_type() != at::kByte || !t->is_contiguous()) return false;
  *ptr = t->data_ptr();
  *n = static_cast<size_t>(t->numel());
  return true;
}

bool seqs(PyObject *table, PyObject *cu, PyObject *len, int dev, int64_t total, solattn_seqs *s) {
  const at::Tensor *t = tensor(table);
  if (!t || t->dim() != 2 || t->numel() == 0 || total > INT32_MAX || t->numel() > INT32_MAX) return false;
  s->B = static_cast<int>(t->size(0));
  s->width = static_cast<int>(t->size(1));
  s->total = static_cast<int>(total);
  s->table = ints(table, dev, 1);
  s->cu = ints(cu, dev, s->B + 1);
  s->len = ints(len, dev, s->B);
  return s->table && s->cu && s->len;
}

void *address(PyObject *x) { return PyLong_AsVoidPtr(x); }

PyObject *status(int rc) { return PyLong_FromLong(rc); }

// The call's stream: the current one for None, else that of a torch.cuda.Stream of the device.
bool stream_of(PyObject *s, int dev, void **out) {
  if (s == Py_None) {
    *out = c10::cuda::getCurrentCUDAStream(dev).stream();
    return true;
  }
  PyObject *d = PyObject_GetAttrString(s, "device_index"), *h = d ? PyObject_GetAttrString(s, "cuda_stream") : nullptr;
  const bool ok = h && PyLong_Check(d) && PyLong_Check(h) && PyLong_AsLong(d) == dev;
  if (ok) *out = PyLong_AsVoidPtr(h);
  Py_XDECREF(d);
  Py_XDECREF(h);
  return ok && !PyErr_Occurred();
}

// (function, q, k, v, key_len or None, out, workspace, stream or None)
PyObject *cross(PyObject *, PyObject *const *a, Py_ssize_t n) {
  if (n != 8) Py_RETURN_NONE;
  const at::Tensor *q = tensor(a[1]), *k = tensor(a[2]);
  if (!q || !k || !q->is_cuda() || q->dim() != 4 || k->dim() != 4) Py_RETURN_NONE;
  const int dev = q->get_device(), dt = dtype_of(*q);
  if (dt < 0 || c10::cuda::current_device() != dev) Py_RETURN_NONE;
  const auto s = q->sizes(), ks = k->sizes();
  for (int64_t x : {s[0], s[1], s[2], s[3], ks[1], ks[2]})
    if (x > INT32_MAX) Py_RETURN_NONE;
  solattn_view vq, vk, vv, vo;
  void *ws, *st;
  size_t wn;
  const int32_t *len = nullptr;
  if (!view(a[1], dev, dt, 4, s[0], s[1], s[2], s[3], &vq) || !view(a[2], dev, dt, 4, s[0], ks[1], ks[2], s[3], &vk) ||
      !view(a[3], dev, dt, 4, s[0], ks[1], ks[2], s[3], &vv) || !view(a[5], dev, dt, 4, s[0], s[1], s[2], s[3], &vo) ||
      !bytes(a[6], dev, &ws, &wn) || (a[4] != Py_None && !(len = ints(a[4], dev, s[0]))) || !stream_of(a[7], dev, &st))
    Py_RETURN_NONE;
  const auto fn = reinterpret_cast<decltype(&solattn_cross)>(address(a[0]));
  return status(fn(&vq, &vk, &vv, &vo, len, static_cast<int>(s[0]), static_cast<int>(s[1]), static_cast<int>(ks[1]),
                   static_cast<int>(s[2]), static_cast<int>(ks[2]), static_cast<int>(s[3]), dt, ws, wn, st));
}

// (function, cache, its device, its 16-bit dtype or -1, q, table, cu, length, max_new, causal, out, workspace, stream or None)
PyObject *paged(PyObject *, PyObject *const *a, Py_ssize_t n) {
  if (n != 13) Py_RETURN_NONE;
  const auto *c = static_cast<const solattn_cache *>(address(a[1]));
  const int dev = static_cast<int>(PyLong_AsLong(a[2])), cdt = static_cast<int>(PyLong_AsLong(a[3]));
  const at::Tensor *q = tensor(a[4]);
  if (!q || q->dim() != 3 || !PyLong_Check(a[8]) || c10::cuda::current_device() != dev) Py_RETURN_NONE;
  const int dt = dtype_of(*q);
  if (dt < 0 || (cdt >= 0 && cdt != dt)) Py_RETURN_NONE;
  const int64_t total = q->size(0), H = q->size(1);
  int over = 0;
  const long max_new = PyLong_AsLongAndOverflow(a[8], &over);
  const int causal = PyObject_IsTrue(a[9]);
  solattn_seqs s;
  solattn_view vq, vo;
  void *ws, *st;
  size_t wn;
  if (over || max_new < 0 || max_new > INT32_MAX || causal < 0 || H > INT32_MAX || !seqs(a[5], a[6], a[7], dev, total, &s) ||
      !view(a[4], dev, dt, 3, 1, H, total, c->d, &vq) || !view(a[10], dev, dt, 3, 1, H, total, c->d, &vo) ||
      !bytes(a[11], dev, &ws, &wn) || !stream_of(a[12], dev, &st)) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
  const auto fn = reinterpret_cast<decltype(&solattn_paged_forward)>(address(a[0]));
  return status(fn(&vq, &vo, c, &s, static_cast<int>(H), static_cast<int>(max_new), causal, dt, ws, wn, st));
}

// (function, write, cache, its device, its 16-bit dtype or -1, k rows, v rows, table, cu, length, workspace, stream or None)
PyObject *cache_rows(PyObject *, PyObject *const *a, Py_ssize_t n) {
  if (n != 12) Py_RETURN_NONE;
  const auto *c = static_cast<const solattn_cache *>(address(a[2]));
  const int dev = static_cast<int>(PyLong_AsLong(a[3])), cdt = static_cast<int>(PyLong_AsLong(a[4]));
  const at::Tensor *k = tensor(a[5]);
  if (!k || k->dim() != 3 || c10::cuda::current_device() != dev) Py_RETURN_NONE;
  const int dt = dtype_of(*k);
  if (dt < 0 || (cdt >= 0 && cdt != dt)) Py_RETURN_NONE;
  const int64_t total = k->size(0);
  solattn_seqs s;
  solattn_view vk, vv;
  void *ws, *st;
  size_t wn;
  if (!seqs(a[7], a[8], a[9], dev, total, &s) || !view(a[5], dev, dt, 3, 1, c->Hkv, total, c->d, &vk) ||
      !view(a[6], dev, dt, 3, 1, c->Hkv, total, c->d, &vv) || !bytes(a[10], dev, &ws, &wn) || wn < 256 || !stream_of(a[11], dev, &st))
    Py_RETURN_NONE;
  if (a[1] == Py_True) return status(reinterpret_cast<decltype(&solattn_cache_append)>(address(a[0]))(c, &vk, &vv, &s, dt, ws, st));
  return status(reinterpret_cast<decltype(&solattn_cache_read)>(address(a[0]))(c, &s, &vk, &vv, dt, ws, st));
}

// An exception of a tensor accessor must not pass through the interpreter: the Python way reports it.
template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyObject *guarded(PyObject *self, PyObject *const *a, Py_ssize_t n) {
  try {
    PyObject *r = F(self, a, n);
    if (r == Py_None) PyErr_Clear();
    return r;
  } catch (...) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
}

template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
PyMethodDef method(const char *name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&guarded<F>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {method<cross>("cross"), method<paged>("paged"), method<cache_rows>("cache_rows"), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fastcall", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fastcall() { return PyModule_Create(&module); }
