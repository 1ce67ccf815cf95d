// Native argument marshalling of the attention calls for the Python binding.
//
// The calls run once or more per layer of a decode step, and looking at each
// tensor's type, shape and strides from Python takes longer than a small
// kernel.  Each function here takes a call's arguments, checks them as the
// binding's Python code does, and calls libtg; where anything is not as it
// should be it returns None, and the Python code, which then looks again, says
// what is wrong.  It computes nothing.
#include <cstdint>
#include <new>

#include <torch/csrc/autograd/python_variable.h>
#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAStream.h>

#include "../../include/tg.h"

namespace {

typedef tg_status (*AppendFn)(const void*, int64_t, const void*, int64_t, const void*, int64_t, const int64_t*, int32_t,
                              const tg_cache*, const tg_attn*, void*, void*, tg_stream);
typedef tg_status (*StepFn)(const void*, int64_t, int32_t, const tg_cache*, const tg_attn*, void*, float*, tg_stream);
typedef tg_status (*ReadFn)(const int64_t*, int32_t, const tg_cache*, const tg_attn*, void*, int64_t, void*, int64_t, tg_stream);
typedef tg_status (*SharedFn)(const void*, int64_t, int32_t, const tg_cache*, const int64_t*, const int32_t*, int32_t, const tg_attn*,
                              void*, float*, tg_stream);
typedef tg_status (*PromptFn)(const void*, int64_t, const void*, int64_t, const void*, int64_t, const int64_t*,
                              const int64_t*, int32_t, int32_t, int32_t, int32_t, const tg_attn*, void*, float*, tg_stream);

// What a handle's tensors must look like (make()).
struct Handle {
  const tg_attn* cfg;
  int64_t H, G, D, p1, p2;  // a page is [p1, p2, D], of an i8 cache p1 bytes
  at::ScalarType type, cache;
  AppendFn append;
  ReadFn read;
  StepFn step;
  SharedFn shared;
  PromptFn prompt;
};

const char* kName = "tg_attention_handle";

void drop(PyObject* capsule) { delete static_cast<Handle*>(PyCapsule_GetPointer(capsule, kName)); }

at::ScalarType scalar(long code) {
  return code == TG_DTYPE_BF16 ? at::kBFloat16 : code == TG_DTYPE_F16 ? at::kHalf : code == TG_DTYPE_I8 ? at::kByte : at::kFloat8_e4m3fn;
}

// make(handle, H, G, D, p1, p2, dtype, cache_dtype, append, step, prompt[, read, shared]): addresses as integers
PyObject* make(PyObject*, PyObject* args) {
  unsigned long long h, fa, fs, fp, fr = 0, fh = 0;
  long long H, G, D, p1, p2;
  long dt, ct;
  if (!PyArg_ParseTuple(args, "KLLLLLllKKK|KK", &h, &H, &G, &D, &p1, &p2, &dt, &ct, &fa, &fs, &fp, &fr, &fh)) return nullptr;
  auto* x = new (std::nothrow) Handle{reinterpret_cast<const tg_attn*>(h), H, G, D, p1, p2, scalar(dt), scalar(ct),
                       reinterpret_cast<AppendFn>(fa), reinterpret_cast<ReadFn>(fr), reinterpret_cast<StepFn>(fs),
                       reinterpret_cast<SharedFn>(fh), reinterpret_cast<PromptFn>(fp)};
  if (!x) return PyErr_NoMemory();
  return PyCapsule_New(x, kName, drop);
}

inline const at::Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

// Rows of `heads` contiguous heads, evenly spaced: the row stride, or -1.
inline int64_t rows(const at::Tensor* t, int64_t dims, int64_t heads, const Handle* h) {
  if (!t || t->dim() != dims || !t->is_cuda() || t->scalar_type() != h->type) return -1;
  const auto s = t->sizes(), st = t->strides();
  const int64_t n = dims;
  if (s[n - 2] != heads || s[n - 1] != h->D || st[n - 1] != 1 || (heads > 1 && st[n - 2] != h->D)) return -1;
  const int64_t inner = s[n - 3], outer = dims == 4 ? s[0] : 1;
  if (inner == 0 || outer == 0 || (inner == 1 && outer == 1)) return heads * h->D;  // no row, or one
  const int64_t row = inner > 1 ? st[n - 3] : st[0];
  if (row == 0 || (inner > 1 && outer > 1 && st[0] != row * inner)) return -1;  // a broadcast row, or two spacings
  return row;
}

inline bool whole(const at::Tensor* t, at::ScalarType type, int64_t numel) {
  return t && t->is_cuda() && t->scalar_type() == type && t->is_contiguous() && t->numel() >= numel;
}

inline bool pages(const at::Tensor* t, const Handle* h, int64_t* stride) {
  if (!t || !t->is_cuda() || t->scalar_type() != h->cache) return false;
  if (h->cache == at::kByte) {
    if (t->dim() != 2 || t->size(1) < h->p1 || t->stride(1) != 1) return false;
    *stride = t->size(0) > 1 ? t->stride(0) : (t->size(1) + 15) / 16 * 16;
    return true;
  }
  if (t->dim() != 4) return false;
  const auto s = t->sizes(), st = t->strides();
  if (s[1] != h->p1 || s[2] != h->p2 || s[3] != h->D || st[3] != 1 || (h->p2 > 1 && st[2] != h->D) ||
      (h->p1 > 1 && st[1] != h->p2 * h->D))
    return false;
  *stride = s[0] > 1 ? st[0] : h->p1 * h->p2 * h->D;
  return true;
}

inline bool cache(PyObject* kv_lens, PyObject* table, PyObject* k, PyObject* v, const Handle* h, tg_cache* c) {
  const at::Tensor *l = tensor(kv_lens), *t = tensor(table), *kp = tensor(k), *vp = tensor(v);
  if (!pages(kp, h, &c->k_page_stride) || !pages(vp, h, &c->v_page_stride) || kp->size(0) != vp->size(0)) return false;
  if (!t || t->dim() != 2 || !t->is_cuda() || t->scalar_type() != at::kInt) return false;
  const int64_t B = t->size(0), most = t->size(1);
  if (most > 1 && t->stride(1) != 1) return false;
  if (!whole(l, at::kInt, B)) return false;
  c->k_pages = kp->data_ptr();
  c->v_pages = vp->data_ptr();
  c->num_pages = static_cast<int32_t>(kp->size(0));
  c->page_table = static_cast<const int32_t*>(t->data_ptr());
  c->table_stride = B > 1 ? t->stride(0) : most;
  c->max_pages = static_cast<int32_t>(most);
  c->kv_lens = static_cast<const int32_t*>(l->data_ptr());
  c->batch = static_cast<int32_t>(B);
  return true;
}

// The given stream's handle (an integer), or the current one of the tensor's device.
inline bool stream_of(PyObject* o, const at::Tensor* t, tg_stream* s) {
  if (o == Py_None) {
    *s = reinterpret_cast<tg_stream>(c10::cuda::getCurrentCUDAStream(t->get_device()).stream());
    return true;
  }
  const unsigned long long v = PyLong_AsUnsignedLongLong(o);
  if (PyErr_Occurred()) { PyErr_Clear(); return false; }
  *s = reinterpret_cast<tg_stream>(v);
  return true;
}

inline const Handle* handle(PyObject* o) {
  auto* h = static_cast<const Handle*>(PyCapsule_GetPointer(o, kName));
  if (!h) PyErr_Clear();
  return h;
}

constexpr int64_t kInt32 = 0x7fffffff;

// append(q, k, v, q_offsets, kv_lens, page_table, k_pages, v_pages, handle, q_out, k_out, stream)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) try {
  const Handle* h = n == 12 ? handle(a[8]) : nullptr;
  if (!h) Py_RETURN_NONE;
  const at::Tensor *k = tensor(a[1]), *v = tensor(a[2]), *off = tensor(a[3]);
  const bool has_q = a[0] != Py_None;
  const int64_t ks = rows(k, 3, h->G, h), vs = rows(v, 3, h->G, h);
  if (ks < 0 || vs < 0 || has_q != (a[9] != Py_None)) Py_RETURN_NONE;
  const int64_t T = k->size(0);
  if (v->size(0) != T || T > kInt32) Py_RETURN_NONE;
  const at::Tensor *q = nullptr, *qo = nullptr, *kout = nullptr;
  int64_t qs = 0;
  if (has_q) {
    q = tensor(a[0]);
    qo = tensor(a[9]);
    qs = rows(q, 3, h->H, h);
    if (qs < 0 || q->size(0) != T || !whole(qo, h->type, T * h->H * h->D)) Py_RETURN_NONE;
  }
  if (a[10] != Py_None) {
    kout = tensor(a[10]);
    if (!whole(kout, h->type, T * h->G * h->D)) Py_RETURN_NONE;
  }
  tg_cache c;
  tg_stream s;
  if (!cache(a[4], a[5], a[6], a[7], h, &c) || !whole(off, at::kLong, c.batch + 1ll) || !stream_of(a[11], k, &s)) Py_RETURN_NONE;
  return PyLong_FromLong(h->append(q ? q->data_ptr() : nullptr, qs, k->data_ptr(), ks, v->data_ptr(), vs,
                                   static_cast<const int64_t*>(off->data_ptr()), static_cast<int32_t>(T), &c, h->cfg,
                                   qo ? qo->data_ptr() : nullptr, kout ? kout->data_ptr() : nullptr, s));
} catch (...) {  // a tensor without storage
  Py_RETURN_NONE;
}

// step(q, kv_lens, page_table, k_pages, v_pages, handle, out, out_lse, stream)
PyObject* step(PyObject*, PyObject* const* a, Py_ssize_t n) try {
  const Handle* h = n == 9 ? handle(a[5]) : nullptr;
  if (!h) Py_RETURN_NONE;
  const at::Tensor *q = tensor(a[0]), *out = tensor(a[6]), *lse = nullptr;
  const int64_t qs = rows(q, 4, h->H, h);
  tg_cache c;
  tg_stream s;
  if (qs < 0 || !cache(a[1], a[2], a[3], a[4], h, &c) || q->size(0) != c.batch || q->size(1) > kInt32) Py_RETURN_NONE;
  const int64_t all = q->size(0) * q->size(1) * h->H;
  if (!whole(out, h->type, all * h->D)) Py_RETURN_NONE;
  if (a[7] != Py_None) {
    lse = tensor(a[7]);
    if (!whole(lse, at::kFloat, all)) Py_RETURN_NONE;
  }
  if (!stream_of(a[8], q, &s)) Py_RETURN_NONE;
  return PyLong_FromLong(h->step(q->data_ptr(), qs, static_cast<int32_t>(q->size(1)), &c, h->cfg, out->data_ptr(),
                                 lse ? static_cast<float*>(lse->data_ptr()) : nullptr, s));
} catch (...) {  // a tensor without storage
  Py_RETURN_NONE;
}

// read(offsets, kv_lens, page_table, k_pages, v_pages, handle, k, v, stream)
PyObject* read(PyObject*, PyObject* const* a, Py_ssize_t n) try {
  const Handle* h = n == 9 ? handle(a[5]) : nullptr;
  if (!h || !h->read) Py_RETURN_NONE;
  const at::Tensor* t[2] = {nullptr, nullptr};
  int64_t stride[2] = {0, 0}, T = -1;
  for (int w = 0; w < 2; ++w) {
    if (a[6 + w] == Py_None) continue;
    t[w] = tensor(a[6 + w]);
    stride[w] = rows(t[w], 3, h->G, h);
    if (stride[w] < 0 || (T >= 0 && t[w]->size(0) != T)) Py_RETURN_NONE;
    T = t[w]->size(0);
  }
  const at::Tensor* off = tensor(a[0]);
  tg_cache c;
  tg_stream s;
  if (T < 0 || T > kInt32 || !cache(a[1], a[2], a[3], a[4], h, &c) || !whole(off, at::kLong, c.batch + 1ll) ||
      !stream_of(a[8], off, &s))
    Py_RETURN_NONE;
  return PyLong_FromLong(h->read(static_cast<const int64_t*>(off->data_ptr()), static_cast<int32_t>(T), &c, h->cfg,
                                 t[0] ? t[0]->data_ptr() : nullptr, stride[0], t[1] ? t[1]->data_ptr() : nullptr, stride[1], s));
} catch (...) {  // a tensor without storage
  Py_RETURN_NONE;
}

// shared(q, kv_lens, page_table, k_pages, v_pages, group_offsets, prefix_lens, handle, out, out_lse, stream)
PyObject* shared(PyObject*, PyObject* const* a, Py_ssize_t n) try {
  const Handle* h = n == 11 ? handle(a[7]) : nullptr;
  if (!h || !h->shared) Py_RETURN_NONE;
  const at::Tensor *q = tensor(a[0]), *go = tensor(a[5]), *pl = tensor(a[6]), *out = tensor(a[8]), *lse = nullptr;
  const int64_t qs = rows(q, 4, h->H, h);
  tg_cache c;
  tg_stream s;
  if (qs < 0 || !cache(a[1], a[2], a[3], a[4], h, &c) || q->size(0) != c.batch || q->size(1) > kInt32) Py_RETURN_NONE;
  const int64_t all = q->size(0) * q->size(1) * h->H, groups = pl ? pl->numel() : 0;
  if (groups > kInt32 || !whole(pl, at::kInt, groups) || !whole(go, at::kLong, groups + 1) || !whole(out, h->type, all * h->D))
    Py_RETURN_NONE;
  if (a[9] != Py_None) {
    lse = tensor(a[9]);
    if (!whole(lse, at::kFloat, all)) Py_RETURN_NONE;
  }
  if (!stream_of(a[10], q, &s)) Py_RETURN_NONE;
  return PyLong_FromLong(h->shared(q->data_ptr(), qs, static_cast<int32_t>(q->size(1)), &c,
                                   static_cast<const int64_t*>(go->data_ptr()), static_cast<const int32_t*>(pl->data_ptr()),
                                   static_cast<int32_t>(groups), h->cfg, out->data_ptr(),
                                   lse ? static_cast<float*>(lse->data_ptr()) : nullptr, s));
} catch (...) {  // a tensor without storage
  Py_RETURN_NONE;
}

// prompt(q, k, v, q_offsets, kv_offsets, handle, out, out_lse, causal, stream)
PyObject* prompt(PyObject*, PyObject* const* a, Py_ssize_t n) try {
  const Handle* h = n == 10 ? handle(a[5]) : nullptr;
  if (!h) Py_RETURN_NONE;
  const at::Tensor *q = tensor(a[0]), *k = tensor(a[1]), *v = tensor(a[2]), *qo = tensor(a[3]), *ko = nullptr, *out = tensor(a[6]),
                   *lse = nullptr;
  const int64_t qs = rows(q, 3, h->H, h), ks = rows(k, 3, h->G, h), vs = rows(v, 3, h->G, h);
  if (qs < 0 || ks < 0 || vs < 0 || !qo) Py_RETURN_NONE;
  const int64_t Tq = q->size(0), Tk = k->size(0), B = qo->numel() - 1;
  if (v->size(0) != Tk || B < 0 || Tq > kInt32 || Tk > kInt32 || !whole(qo, at::kLong, B + 1)) Py_RETURN_NONE;
  if (a[4] != Py_None) {
    ko = tensor(a[4]);
    if (!whole(ko, at::kLong, B + 1)) Py_RETURN_NONE;
  }
  if (!whole(out, h->type, Tq * h->H * h->D)) Py_RETURN_NONE;
  if (a[7] != Py_None) {
    lse = tensor(a[7]);
    if (!whole(lse, at::kFloat, Tq * h->H)) Py_RETURN_NONE;
  }
  tg_stream s;
  const int causal = PyObject_IsTrue(a[8]);
  if (causal < 0 || !stream_of(a[9], q, &s)) { PyErr_Clear(); Py_RETURN_NONE; }
  return PyLong_FromLong(h->prompt(q->data_ptr(), qs, k->data_ptr(), ks, v->data_ptr(), vs,
                                   static_cast<const int64_t*>(qo->data_ptr()),
                                   ko ? static_cast<const int64_t*>(ko->data_ptr()) : nullptr, static_cast<int32_t>(B),
                                   static_cast<int32_t>(Tq), static_cast<int32_t>(Tk), causal, h->cfg, out->data_ptr(),
                                   lse ? static_cast<float*>(lse->data_ptr()) : nullptr, s));
} catch (...) {  // a tensor without storage
  Py_RETURN_NONE;
}

PyMethodDef kMethods[] = {
    {"make", make, METH_VARARGS, "A handle for the calls below."},
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(append)), METH_FASTCALL, "tg_cache_append, or None."},
    {"step", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(step)), METH_FASTCALL, "tg_attend_step, or None."},
    {"read", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(read)), METH_FASTCALL, "tg_cache_read, or None."},
    {"shared", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(shared)), METH_FASTCALL, "tg_attend_shared, or None."},
    {"prompt", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(prompt)), METH_FASTCALL, "tg_attend_prompt, or None."},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "tg_binding", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_tg_binding() { return PyModule_Create(&kModule); }
