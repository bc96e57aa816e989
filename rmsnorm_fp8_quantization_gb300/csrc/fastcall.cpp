// Host-side shortcut of the rotary and paged wrappers (ops.py).
//
// A step of a serving loop launches kernels of 2 to 10 us; the wrappers' checks,
// allocations and argument packing in Python cost 16 to 27 us of host time a
// call.  These functions do the same for the USUAL call -- plain CUDA tensors of
// the expected types, shapes and layout, no outputs given -- and return None for
// any other, which then takes the wrapper's own way with its checks and errors.
// The arguments go to the C entry points of include/gbnorm.h, whose addresses the
// wrappers hand over; nothing is computed here.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <cfloat>
#include <cmath>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "gbnorm.h"

namespace {

using RopeFn = gbn_status (*)(const gbn_rope_args*, cudaStream_t);
using AppendFn = gbn_status (*)(const gbn_paged_append_args*, cudaStream_t);
using AttendFn = gbn_status (*)(const gbn_paged_attention_args*, cudaStream_t);
using BytesFn = gbn_status (*)(int64_t, int64_t, int64_t, int64_t, int64_t, int64_t, int64_t,
                               int64_t, int64_t, int64_t, int, gbn_dtype, gbn_dtype, size_t*);
RopeFn g_rope[2];
AppendFn g_append;
AttendFn g_attend;
BytesFn g_bytes;

// A plain tensor (no subclass), or null.
const at::Tensor* plain(PyObject* o) {
  return THPVariable_CheckExact(o) ? &THPVariable_Unpack(o) : nullptr;
}
int gbn_type(at::ScalarType t) {
  switch (t) {
    case at::kFloat: return GBN_F32;
    case at::kBFloat16: return GBN_BF16;
    case at::kHalf: return GBN_F16;
    case at::kByte:
    case at::kFloat8_e4m3fn: return GBN_E4M3;
    default: return -1;
  }
}
bool inner_ok(const at::Tensor& t) { return t.stride(-1) == 1; }
// An output like t, the elements of a head side by side.  (Where t's elements share
// memory, empty_like orders the dimensions by their strides, and the last may not be
// the innermost.)
at::Tensor output_like(const at::Tensor& t) {
  at::Tensor o = at::empty_like(t);
  return inner_ok(o) ? o : at::empty(t.sizes(), t.options());
}

// Keeps the interpreter's rules: a C++ exception becomes "not the usual call".
template <typename F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (...) {
    PyErr_Clear();
    Py_RETURN_NONE;
  }
}

// The status of a refused call, for the wrapper to raise.
PyObject* status(gbn_status st) { return PyLong_FromLong(static_cast<long>(st)); }

PyObject* setup(PyObject*, PyObject* args) {
  unsigned long long a, b, c, d, e;
  if (!PyArg_ParseTuple(args, "KKKKK", &a, &b, &c, &d, &e)) return nullptr;
  g_rope[0] = reinterpret_cast<RopeFn>(a);
  g_rope[1] = reinterpret_cast<RopeFn>(b);
  g_append = reinterpret_cast<AppendFn>(c);
  g_attend = reinterpret_cast<AttendFn>(d);
  g_bytes = reinterpret_cast<BytesFn>(e);
  Py_RETURN_NONE;
}

// A number that fp32 has room for (the wrapper's own way says so where it has not).
bool number(PyObject* o, double* v) {
  if (PyFloat_CheckExact(o)) *v = PyFloat_AS_DOUBLE(o);
  else if (PyLong_CheckExact(o)) *v = PyLong_AsDouble(o);
  else return false;
  if (*v == -1.0 && PyErr_Occurred()) {
    PyErr_Clear();
    return false;
  }
  return !(std::fabs(*v) > FLT_MAX) || std::isinf(*v);
}
bool whole(PyObject* o, int64_t* v) {
  if (!PyLong_CheckExact(o)) return false;
  int over = 0;
  *v = PyLong_AsLongLongAndOverflow(o, &over);
  return over == 0;
}

// rope(backward, q, k, inv_freq, positions, layout, mscale)
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    int64_t backward, layout;
    double mscale;
    const at::Tensor *q, *k, *f, *pos;
    if (n != 7 || !whole(a[0], &backward) || !(q = plain(a[1])) || !(k = plain(a[2])) ||
        !(f = plain(a[3])) || !(pos = plain(a[4])) || !whole(a[5], &layout) || !number(a[6], &mscale))
      Py_RETURN_NONE;
    const int type = gbn_type(q->scalar_type());
    const int dev = q->is_cuda() ? q->get_device() : -1;
    if (dev < 0 || q->dim() != 4 || k->dim() != 4 || q->scalar_type() != k->scalar_type() ||
        type < 0 || type == GBN_E4M3 || !inner_ok(*q) || !inner_ok(*k) || q->size(0) != k->size(0) ||
        q->size(1) != k->size(1) || q->size(3) != k->size(3) || f->scalar_type() != at::kDouble ||
        f->dim() != 1 || !f->is_contiguous() || pos->dim() != 2 || !pos->is_contiguous() ||
        (pos->scalar_type() != at::kLong && pos->scalar_type() != at::kInt) ||
        pos->size(0) != q->size(0) || pos->size(1) != q->size(1) || !k->is_cuda() ||
        !f->is_cuda() || !pos->is_cuda() || k->get_device() != dev || f->get_device() != dev ||
        pos->get_device() != dev || c10::cuda::current_device() != dev)
      Py_RETURN_NONE;
    at::Tensor qo = output_like(*q), ko = output_like(*k);
    gbn_rope_args g;
    g.q = q->data_ptr();
    g.k = k->data_ptr();
    g.positions = pos->data_ptr();
    g.inv_freq = static_cast<const double*>(f->data_ptr());
    g.q_out = qo.data_ptr();
    g.k_out = ko.data_ptr();
    g.batches = q->size(0);
    g.seq = q->size(1);
    g.q_heads = q->size(2);
    g.k_heads = k->size(2);
    g.head_dim = q->size(3);
    g.rotary_dim = 2 * f->size(0);
    for (int i = 0; i < 3; ++i) {
      g.q_strides[i] = q->stride(i);
      g.k_strides[i] = k->stride(i);
      g.q_out_strides[i] = qo.stride(i);
      g.k_out_strides[i] = ko.stride(i);
    }
    g.position_stride = pos->size(0) > 1 ? pos->stride(0) : 0;
    g.position_bytes = static_cast<int32_t>(pos->element_size());
    g.dtype = type;
    g.layout = static_cast<int32_t>(layout);
    g.mscale = static_cast<float>(mscale);
    const gbn_status st = g_rope[backward != 0](&g, c10::cuda::getCurrentCUDAStream(dev).stream());
    if (st != GBN_OK) return status(st);
    PyObject* r = PyTuple_New(2);
    if (!r) return nullptr;
    PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(std::move(qo)));
    PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(std::move(ko)));
    return r;
  });
}

struct Paged {
  const at::Tensor *k_cache, *v_cache, *cu, *kv, *table;
  int type, cache_type;
};
// What both paged calls share, next to x [tokens, heads, head_dim].
bool paged_ok(const at::Tensor& x, PyObject* const* a, int dev, Paged* p) {
  if (!(p->k_cache = plain(a[0])) || !(p->v_cache = plain(a[1])) || !(p->cu = plain(a[2])) ||
      !(p->kv = plain(a[3])) || !(p->table = plain(a[4])))
    return false;
  p->type = gbn_type(x.scalar_type());
  p->cache_type = gbn_type(p->k_cache->scalar_type());
  if ((p->type != GBN_BF16 && p->type != GBN_F16) ||
      (p->cache_type != p->type && p->cache_type != GBN_E4M3) ||
      gbn_type(p->v_cache->scalar_type()) != p->cache_type || x.dim() != 3 || !inner_ok(x) ||
      p->k_cache->dim() != 4 || p->v_cache->dim() != 4 || !inner_ok(*p->k_cache) ||
      !inner_ok(*p->v_cache) || p->k_cache->sizes() != p->v_cache->sizes() ||
      p->k_cache->size(3) != x.size(2))
    return false;
  for (const at::Tensor* t : {p->cu, p->kv, p->table})
    if (t->scalar_type() != at::kInt || !t->is_contiguous()) return false;
  if (p->cu->dim() != 1 || p->kv->dim() != 1 || p->table->dim() != 2 ||
      p->cu->size(0) != p->kv->size(0) + 1 || p->table->size(0) != p->kv->size(0))
    return false;
  for (const at::Tensor* t : {p->k_cache, p->v_cache, p->cu, p->kv, p->table})
    if (!t->is_cuda() || t->get_device() != dev) return false;
  return true;
}
// A given fp32 scalar on the device, or None where none is needed.
bool scalar_ok(PyObject* o, bool need, int dev, const float** v) {
  *v = nullptr;
  if (o == Py_None) return !need;
  const at::Tensor* t = plain(o);
  if (!t || t->scalar_type() != at::kFloat || t->numel() != 1 || !t->is_cuda() ||
      t->get_device() != dev)
    return false;
  *v = static_cast<const float*>(t->data_ptr());
  return true;
}

// append(k, v, k_cache, v_cache, cu, kv_lens, table, q, inv_freq, layout, mscale, k_scale, v_scale)
PyObject* append(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const at::Tensor *k, *v, *q, *f;
    int64_t layout;
    double mscale;
    Paged p;
    if (n != 13 || !(k = plain(a[0])) || !(v = plain(a[1])) || !(q = plain(a[7])) ||
        !(f = plain(a[8])) || !whole(a[9], &layout) || !number(a[10], &mscale) || !k->is_cuda())
      Py_RETURN_NONE;
    const int dev = k->get_device();
    if (c10::cuda::current_device() != dev || !paged_ok(*k, a + 2, dev, &p)) Py_RETURN_NONE;
    const bool fp8 = p.cache_type == GBN_E4M3;
    gbn_paged_append_args g;
    if (v->scalar_type() != k->scalar_type() || v->sizes() != k->sizes() || !inner_ok(*v) ||
        k->size(1) != p.k_cache->size(2) || q->scalar_type() != k->scalar_type() || q->dim() != 3 ||
        q->size(0) != k->size(0) || q->size(2) != k->size(2) || !inner_ok(*q) || !v->is_cuda() ||
        v->get_device() != dev || !q->is_cuda() || q->get_device() != dev ||
        f->scalar_type() != at::kDouble || f->dim() != 1 || !f->is_contiguous() || !f->is_cuda() ||
        f->get_device() != dev || !scalar_ok(a[11], fp8, dev, &g.k_scale) ||
        !scalar_ok(a[12], fp8, dev, &g.v_scale))
      Py_RETURN_NONE;
    at::Tensor qo = output_like(*q);
    g.q = q->data_ptr();
    g.k = k->data_ptr();
    g.v = v->data_ptr();
    g.q_out = qo.data_ptr();
    g.k_cache = p.k_cache->data_ptr();
    g.v_cache = p.v_cache->data_ptr();
    g.inv_freq = static_cast<const double*>(f->data_ptr());
    g.cu_seqlens = static_cast<const int32_t*>(p.cu->data_ptr());
    g.kv_lens = static_cast<const int32_t*>(p.kv->data_ptr());
    g.block_table = static_cast<const int32_t*>(p.table->data_ptr());
    g.tokens = k->size(0);
    g.batches = p.kv->size(0);
    g.q_heads = q->size(1);
    g.kv_heads = k->size(1);
    g.head_dim = k->size(2);
    g.rotary_dim = 2 * f->size(0);
    g.num_pages = p.k_cache->size(0);
    g.page_size = p.k_cache->size(1);
    g.table_pages = p.table->size(1);
    g.table_stride = p.table->stride(0);
    for (int i = 0; i < 2; ++i) {
      g.q_strides[i] = q->stride(i);
      g.k_strides[i] = k->stride(i);
      g.v_strides[i] = v->stride(i);
      g.q_out_strides[i] = qo.stride(i);
    }
    for (int i = 0; i < 3; ++i) {
      g.k_cache_strides[i] = p.k_cache->stride(i);
      g.v_cache_strides[i] = p.v_cache->stride(i);
    }
    g.dtype = p.type;
    g.cache_dtype = p.cache_type;
    g.layout = static_cast<int32_t>(layout);
    g.mscale = static_cast<float>(mscale);
    const gbn_status st = g_append(&g, c10::cuda::getCurrentCUDAStream(dev).stream());
    if (st != GBN_OK) return status(st);
    return THPVariable_Wrap(std::move(qo));
  });
}

// attention(q, k_cache, v_cache, cu, kv_lens, table, max_q, max_kv | None, scale | None, causal,
//           window, k_scale_inv, v_scale_inv, return_lse)
PyObject* attention(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded([&]() -> PyObject* {
    const at::Tensor* q;
    Paged p;
    gbn_paged_attention_args g;
    double scale = 0.0;
    if (n != 14 || !(q = plain(a[0])) || !q->is_cuda() || !whole(a[6], &g.max_q) ||
        !whole(a[10], &g.window) || (a[9] != Py_True && a[9] != Py_False) ||
        (a[13] != Py_True && a[13] != Py_False))
      Py_RETURN_NONE;
    const int dev = q->get_device();
    if (c10::cuda::current_device() != dev || !paged_ok(*q, a + 1, dev, &p)) Py_RETURN_NONE;
    const bool fp8 = p.cache_type == GBN_E4M3;
    if (!scalar_ok(a[11], fp8, dev, &g.k_scale_inv) || !scalar_ok(a[12], fp8, dev, &g.v_scale_inv))
      Py_RETURN_NONE;
    g.tokens = q->size(0);
    g.batches = p.kv->size(0);
    g.q_heads = q->size(1);
    g.kv_heads = p.k_cache->size(2);
    g.head_dim = q->size(2);
    g.num_pages = p.k_cache->size(0);
    g.page_size = p.k_cache->size(1);
    g.table_pages = p.table->size(1);
    g.table_stride = p.table->stride(0);
    if (a[7] == Py_None) {
      const int64_t room = g.table_pages * g.page_size;
      g.max_kv = room < (1 << 30) ? room : (1 << 30);
    } else if (!whole(a[7], &g.max_kv)) {
      Py_RETURN_NONE;
    }
    if (a[8] == Py_None) scale = 1.0 / std::sqrt(static_cast<double>(g.head_dim));
    else if (!number(a[8], &scale)) Py_RETURN_NONE;
    g.dtype = p.type;
    g.cache_dtype = p.cache_type;
    g.causal = a[9] == Py_True;
    g.scale = static_cast<float>(scale);
    size_t bytes = 0;
    gbn_status st = g_bytes(g.tokens, g.batches, g.q_heads, g.kv_heads, g.head_dim, g.page_size,
                            g.table_pages, g.max_q, g.max_kv, g.window, g.causal,
                            static_cast<gbn_dtype>(g.dtype), static_cast<gbn_dtype>(g.cache_dtype),
                            &bytes);
    if (st != GBN_OK) return status(st);
    at::Tensor out = output_like(*q), lse, work;
    if (a[13] == Py_True) lse = at::empty({g.tokens, g.q_heads}, q->options().dtype(at::kFloat));
    if (bytes) work = at::empty({static_cast<int64_t>(bytes)}, q->options().dtype(at::kByte));
    g.q = q->data_ptr();
    g.k_cache = p.k_cache->data_ptr();
    g.v_cache = p.v_cache->data_ptr();
    g.cu_seqlens = static_cast<const int32_t*>(p.cu->data_ptr());
    g.kv_lens = static_cast<const int32_t*>(p.kv->data_ptr());
    g.block_table = static_cast<const int32_t*>(p.table->data_ptr());
    g.out = out.data_ptr();
    g.lse = lse.defined() ? static_cast<float*>(lse.data_ptr()) : nullptr;
    g.workspace = bytes ? work.data_ptr() : nullptr;
    g.workspace_bytes = bytes;
    for (int i = 0; i < 2; ++i) {
      g.q_strides[i] = q->stride(i);
      g.out_strides[i] = out.stride(i);
    }
    for (int i = 0; i < 3; ++i) {
      g.k_cache_strides[i] = p.k_cache->stride(i);
      g.v_cache_strides[i] = p.v_cache->stride(i);
    }
    st = g_attend(&g, c10::cuda::getCurrentCUDAStream(dev).stream());
    if (st != GBN_OK) return status(st);
    if (!lse.defined()) return THPVariable_Wrap(std::move(out));
    PyObject* r = PyTuple_New(2);
    if (!r) return nullptr;
    PyTuple_SET_ITEM(r, 0, THPVariable_Wrap(std::move(out)));
    PyTuple_SET_ITEM(r, 1, THPVariable_Wrap(std::move(lse)));
    return r;
  });
}

PyMethodDef kMethods[] = {
    {"setup", setup, METH_VARARGS, "Addresses of the C entry points."},
    {"rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(rope)), METH_FASTCALL, ""},
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(append)), METH_FASTCALL, ""},
    {"attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(attention)),
     METH_FASTCALL, ""},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_fastcall", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fastcall() {
  PyObject* m = PyModule_Create(&kModule);
  // The torch whose headers this was compiled with: the wrappers use it with no other.
  if (m && PyModule_AddStringConstant(m, "built_for", GBN_BUILT_FOR) < 0) Py_CLEAR(m);
  return m;
}
