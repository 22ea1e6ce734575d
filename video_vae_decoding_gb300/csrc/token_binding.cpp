// The short way from Python to the token operators: marshals the tensors of an
// ordinary call in C++.  A step of a streaming model makes such calls by the
// hundred, each for a few microseconds of the GPU's time, and reading a dozen
// attributes per tensor in Python takes longer than that.
//
// Every function returns None for a call that it does not take (another device
// than the current one, a stream of its own, a type or shape it does not expect,
// a gradient required, an error of the library): tokens.py then does the same in
// Python, with its checks and messages.  So nothing here raises.
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAStream.h>

#include <math.h>
#include <stdint.h>

#include "wan_vae.h"

namespace {

decltype(&wan_rotary) f_rotary;
decltype(&wan_kv_append) f_append;
decltype(&wan_kv_attention) f_attention;
decltype(&wan_kv_attention_workspace) f_workspace;

// A plain tensor (no subclass) that needs no gradient and carries no tangent; null for anything else.
const at::Tensor* tensor(PyObject* o) {
  if (!THPVariable_CheckExact(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (t.layout() != at::kStrided || (t.requires_grad() && at::GradMode::is_enabled()) || t._fw_grad(0).defined())
    return nullptr;
  return &t;
}

int code(const at::Tensor& t) {
  const auto d = t.scalar_type();
  return d == at::kFloat ? WAN_F32 : d == at::kBFloat16 ? WAN_BF16 : d == at::kHalf ? WAN_F16 : -1;
}
bool ints(const at::Tensor& t, at::Device dev, int dims) {
  return t.scalar_type() == at::kInt && t.device() == dev && t.dim() == dims;
}
bool positions_ok(const at::Tensor& t, at::Device dev) {
  return (t.scalar_type() == at::kInt || t.scalar_type() == at::kLong) && t.device() == dev && t.is_contiguous();
}
bool rows(const at::Tensor& t) { return t.size(-1) <= 1 || t.stride(-1) == 1; }
bool fits(int64_t n) { return n >= 0 && n <= 0x7fffffff; }

// Whether dev is the current GPU, and its current stream.
bool stream_of(at::Device dev, wan_cuda_stream* s) {
  if (!dev.is_cuda() || c10::cuda::current_device() != dev.index()) return false;
  *s = c10::cuda::getCurrentCUDAStream(dev.index()).stream();
  return true;
}

// The result of a call: out, or new memory like t where out is None.
bool result(PyObject* out, const at::Tensor& t, at::Tensor* r) {
  if (out == Py_None) {
    *r = at::empty(t.sizes(), t.options().requires_grad(false));
    return true;
  }
  const at::Tensor* o = tensor(out);
  if (!o || o->scalar_type() != t.scalar_type() || o->device() != t.device() || o->sizes() != t.sizes() || !rows(*o))
    return false;
  *r = *o;
  return true;
}
// Counts the version of a tensor that a call wrote to, for autograd's check of what it saved.
void written(const at::Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}
PyObject* give(PyObject* out, at::Tensor&& r) {
  if (out == Py_None) return THPVariable_Wrap(std::move(r));
  written(r);
  Py_INCREF(out);
  return out;
}

PyObject* decline() {
  PyErr_Clear();
  Py_RETURN_NONE;
}
// An exception (memory that cannot be had, for one) is met again, and told, on the way in Python.
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n) {
  try {
    if (n == N && f_rotary) {
      PyObject* r = F(a);
      if (r) return r;
    }
  } catch (...) {
  }
  return decline();
}

// rotary(x, positions, rotation's address, axes, out or None, inverse)
PyObject* rotary(PyObject* const* a) {
  const at::Tensor *x = tensor(a[0]), *p = tensor(a[1]);
  if (!x || !p) return nullptr;
  const int dt = code(*x);
  if (dt < 0 || (x->dim() != 3 && x->dim() != 4) || !rows(*x) || !positions_ok(*p, x->device())) return nullptr;
  const int k = (int)x->dim() - 3;
  const int64_t B = k ? x->size(0) : 1, T = x->size(k), H = x->size(k + 1), D = x->size(k + 2);
  const long axes = PyLong_AsLong(a[3]), inverse = PyLong_AsLong(a[5]);
  const bool shared = p->dim() == 2 && p->size(0) == T && p->size(1) == axes;
  if (!shared && !(p->dim() == 3 && p->size(0) == B && p->size(1) == T && p->size(2) == axes)) return nullptr;
  const wan_rotation* rot = (const wan_rotation*)PyLong_AsVoidPtr(a[2]);
  wan_cuda_stream s;
  at::Tensor out;
  if (PyErr_Occurred() || !fits(B) || !fits(T) || !fits(H) || !fits(D) || !stream_of(x->device(), &s) ||
      !result(a[4], *x, &out))
    return nullptr;
  const int64_t xs[3] = {k ? x->stride(0) : 0, x->stride(k), x->stride(k + 1)};
  const int64_t os[3] = {k ? out.stride(0) : 0, out.stride(k), out.stride(k + 1)};
  if (f_rotary(x->data_ptr(), xs, out.data_ptr(), os, dt, (int32_t)B, (int32_t)T, (int32_t)H, (int32_t)D, p->data_ptr(),
               p->scalar_type() == at::kLong, shared ? 0 : T * axes, rot, (int32_t)inverse, s) != WAN_OK)
    return nullptr;
  return give(a[4], std::move(out));
}

bool cache_of(const at::Tensor& k, const at::Tensor& v, wan_kv_cache* c) {
  const int dt = code(k);
  if ((dt != WAN_BF16 && dt != WAN_F16) || v.scalar_type() != k.scalar_type() || v.device() != k.device() || k.dim() != 4 ||
      v.sizes() != k.sizes() || !rows(k) || !rows(v) || !fits(k.size(1)) || !fits(k.size(2)) || !fits(k.size(3)))
    return false;
  *c = wan_kv_cache{k.data_ptr(), v.data_ptr(), dt,          (int32_t)k.size(1), (int32_t)k.size(2), (int32_t)k.size(3),
                    k.size(0),    k.stride(0),  k.stride(1), k.stride(2),        v.stride(0),        v.stride(1),
                    v.stride(2)};
  return true;
}

// The tables of a call; cu and status may be None.
bool batch_of(at::Device dev, PyObject* pages, PyObject* lengths, PyObject* cu, PyObject* status, int64_t tokens,
              wan_kv_batch* b) {
  const at::Tensor *p = tensor(pages), *l = tensor(lengths);
  if (!p || !l || !ints(*p, dev, 2) || !ints(*l, dev, 1)) return false;
  const int64_t B = l->size(0);
  if (p->size(0) != B || (p->size(1) > 1 && p->stride(1) != 1) || !l->is_contiguous() || !fits(tokens) || !fits(B) ||
      !fits(p->size(1)))
    return false;
  const int32_t* c = nullptr;
  int32_t* s = nullptr;
  if (cu != Py_None) {
    const at::Tensor* t = tensor(cu);
    if (!t || !ints(*t, dev, 1) || t->size(0) != B + 1 || !t->is_contiguous()) return false;
    c = (const int32_t*)t->data_ptr();
  }
  if (status != Py_None) {
    const at::Tensor* t = tensor(status);
    if (!t || !ints(*t, dev, 1) || t->size(0) != 1) return false;
    s = (int32_t*)t->data_ptr();
  }
  *b = wan_kv_batch{(const int32_t*)p->data_ptr(), p->stride(0), (int32_t)p->size(1), (int32_t)B,
                    (const int32_t*)l->data_ptr(), c,            (int32_t)tokens,     s};
  return true;
}

// append(k, v, k_cache, v_cache, pages, lengths, cu, positions, rotation's address (0: none), axes, q, q_out, status): the
// turned q, True without q
PyObject* append(PyObject* const* a) {
  const at::Tensor *k = tensor(a[0]), *v = tensor(a[1]), *kc = tensor(a[2]), *vc = tensor(a[3]);
  wan_kv_cache c;
  wan_kv_batch b;
  if (!k || !v || !kc || !vc || !cache_of(*kc, *vc, &c)) return nullptr;
  const at::Device dev = kc->device();
  const auto type = kc->scalar_type();
  if (k->scalar_type() != type || v->scalar_type() != type || k->device() != dev || v->device() != dev || k->dim() != 3 ||
      v->sizes() != k->sizes() || k->size(1) != c.heads || k->size(2) != c.head_dim || !rows(*k) || !rows(*v))
    return nullptr;
  const int64_t T = k->size(0);
  if (T == 0 || !batch_of(dev, a[4], a[5], a[6], a[12], T, &b)) return nullptr;
  const wan_rotation* rot = (const wan_rotation*)PyLong_AsVoidPtr(a[8]);
  const long axes = PyLong_AsLong(a[9]);
  if (PyErr_Occurred()) return nullptr;
  const at::Tensor* p = nullptr;
  if (rot) {
    p = tensor(a[7]);
    if (!p || !positions_ok(*p, dev) || p->dim() != 2 || p->size(0) != T || p->size(1) != axes) return nullptr;
  } else if (a[7] != Py_None) {
    return nullptr;
  }
  wan_cuda_stream s;
  if (!stream_of(dev, &s)) return nullptr;
  const at::Tensor* q = nullptr;
  at::Tensor out;
  if (a[10] != Py_None) {
    q = tensor(a[10]);
    if (!q || q->scalar_type() != type || q->device() != dev || q->dim() != 3 || q->size(0) != T || q->size(1) < 1 ||
        !fits(q->size(1)) || q->size(2) != c.head_dim || !rows(*q) || !result(a[11], *q, &out))
      return nullptr;
  } else if (a[11] != Py_None) {
    return nullptr;
  }
  if (f_append(&c, &b, k->data_ptr(), k->stride(0), k->stride(1), v->data_ptr(), v->stride(0), v->stride(1),
               q ? q->data_ptr() : nullptr, q ? (int32_t)q->size(1) : 0, q ? q->stride(0) : 0, q ? q->stride(1) : 0,
               q ? out.data_ptr() : nullptr, q ? out.stride(0) : 0, q ? out.stride(1) : 0, rot, p ? p->data_ptr() : nullptr,
               p && p->scalar_type() == at::kLong, s) != WAN_OK)
    return nullptr;
  written(*kc);
  written(*vc);
  if (!q) Py_RETURN_TRUE;
  return give(a[11], std::move(out));
}

// attention(q, k_cache, v_cache, pages, lengths, cu, ranges, scale or None, out, return_lse, status): out, or (out, lse)
PyObject* attention(PyObject* const* a) {
  const at::Tensor *q = tensor(a[0]), *kc = tensor(a[1]), *vc = tensor(a[2]);
  wan_kv_cache c;
  wan_kv_batch b;
  if (!q || !kc || !vc || !cache_of(*kc, *vc, &c)) return nullptr;
  const at::Device dev = kc->device();
  if (q->scalar_type() != kc->scalar_type() || q->device() != dev || q->dim() != 3 || q->size(2) != c.head_dim ||
      !fits(q->size(1)) || !rows(*q))
    return nullptr;
  const int64_t T = q->size(0), H = q->size(1);
  if (T == 0 || !batch_of(dev, a[3], a[4], a[5], a[10], T, &b)) return nullptr;
  const int32_t* ranges = nullptr;
  if (a[6] != Py_None) {
    const at::Tensor* r = tensor(a[6]);
    if (!r || !ints(*r, dev, 2) || r->size(0) != T || r->size(1) != 2 || !r->is_contiguous()) return nullptr;
    ranges = (const int32_t*)r->data_ptr();
  }
  const double scale = a[7] == Py_None ? 1.0 / sqrt((double)c.head_dim) : PyFloat_AsDouble(a[7]);
  const int with_lse = PyObject_IsTrue(a[9]);
  wan_cuda_stream s;
  if (PyErr_Occurred() || !stream_of(dev, &s)) return nullptr;
  const int64_t bytes = f_workspace(&c, &b, (int32_t)H);
  at::Tensor out, lse;
  if (bytes < 0 || !result(a[8], *q, &out)) return nullptr;
  // freed at the end of this call, so the caching allocator gives it to later work of this stream only
  const at::Tensor ws = at::empty({bytes}, at::TensorOptions().dtype(at::kByte).device(dev));
  if (with_lse) lse = at::empty({T, H}, at::TensorOptions().dtype(at::kFloat).device(dev));
  if (f_attention(&c, &b, q->data_ptr(), (int32_t)H, q->stride(0), q->stride(1), ranges, (float)scale, out.data_ptr(),
                  out.stride(0), out.stride(1), with_lse ? (float*)lse.data_ptr() : nullptr, ws.data_ptr(), bytes,
                  s) != WAN_OK)
    return nullptr;
  PyObject* r = give(a[8], std::move(out));
  if (!with_lse || !r) return r;
  PyObject* l = THPVariable_Wrap(std::move(lse));
  PyObject* both = l ? PyTuple_Pack(2, r, l) : nullptr;
  Py_DECREF(r);
  Py_XDECREF(l);
  return both;
}

// init(addresses of the library's four functions)
PyObject* init(PyObject*, PyObject* args) {
  unsigned long long f[4];
  if (!PyArg_ParseTuple(args, "KKKK", &f[0], &f[1], &f[2], &f[3])) return nullptr;
  f_append = (decltype(f_append))(uintptr_t)f[1];
  f_attention = (decltype(f_attention))(uintptr_t)f[2];
  f_workspace = (decltype(f_workspace))(uintptr_t)f[3];
  f_rotary = (decltype(f_rotary))(uintptr_t)f[0];
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"init", init, METH_VARARGS, nullptr},
    {"rotary", (PyCFunction)(void (*)(void))entry<rotary, 6>, METH_FASTCALL, nullptr},
    {"append", (PyCFunction)(void (*)(void))entry<append, 13>, METH_FASTCALL, nullptr},
    {"attention", (PyCFunction)(void (*)(void))entry<attention, 11>, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tokens", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tokens() { return PyModule_Create(&module); }
