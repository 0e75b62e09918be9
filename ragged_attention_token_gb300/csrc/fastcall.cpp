// Argument marshalling of the block operators in C++: the checks that rra.py
// makes of its tensors, then the call into librra, for calls whose arguments are
// all as they should be.  Any other call returns -1 with nothing done, and
// rra.py's own checks say what is wrong (or marshal it themselves).
//
// The smallest of these operators take 3 to 8 us on the GPU; read attribute
// by attribute from Python, their ten tensors cost the host as long again.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>

#include "../../include/rra.h"

namespace {

decltype(&rra_linear_epilogue) f_linear = nullptr;
decltype(&rra_qk_norm_rope) f_rope = nullptr;
decltype(&rra_attend_prompt) f_prompt = nullptr;
decltype(&rra_attend_cache) f_cache = nullptr;

// One call's arguments, taken in order; `ok` turns false at the first that is not plain.
struct Args {
  PyObject* const* v;
  Py_ssize_t n, i = 0;
  bool ok = true;
  int dev = -1;

  PyObject* next() {
    if (i >= n) {
      ok = false;
      return Py_None;
    }
    return v[i++];
  }
  // A strided CUDA tensor on the current device; null for None.
  const at::Tensor* tensor(bool optional = false) {
    PyObject* o = next();
    if (!ok || (o == Py_None && optional)) return nullptr;
    if (!THPVariable_Check(o)) {
      ok = false;
      return nullptr;
    }
    const at::Tensor& t = THPVariable_Unpack(o);
    if (!t.defined() || t.layout() != at::kStrided || !t.is_cuda()) {
      ok = false;
      return nullptr;
    }
    if (dev < 0) dev = c10::cuda::current_device();
    if (t.get_device() != dev) {
      ok = false;
      return nullptr;
    }
    return &t;
  }
  long long integer() {
    PyObject* o = next();
    if (!ok || !PyLong_Check(o)) {
      ok = false;
      return 0;
    }
    const long long x = PyLong_AsLongLong(o);
    if ((x == -1 && PyErr_Occurred()) || x < INT_MIN || x > INT_MAX) {
      PyErr_Clear();
      ok = false;
    }
    return x;
  }
  float real() {
    PyObject* o = next();
    if (!ok || !PyFloat_Check(o)) {
      ok = false;
      return 0.f;
    }
    return static_cast<float>(PyFloat_AS_DOUBLE(o));
  }
  // The stream handle given, or the current stream's.
  void* stream() {
    PyObject* o = next();
    if (!ok) return nullptr;
    if (o == Py_None) return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
    void* p = PyLong_Check(o) ? PyLong_AsVoidPtr(o) : nullptr;
    if (!PyLong_Check(o) || PyErr_Occurred()) {
      PyErr_Clear();
      ok = false;
    }
    return p;
  }

  bool take(bool c) { return ok = ok && c; }
};

bool code(const at::Tensor& t, rra_dtype& dt) {
  switch (t.scalar_type()) {
    case at::kHalf: dt = RRA_F16; return true;
    case at::kBFloat16: dt = RRA_BF16; return true;
    case at::kFloat: dt = RRA_F32; return true;
    default: return false;
  }
}

// Contiguous, of this type and these sizes (-1: any).
template <typename T = void>
const T* dense(Args& a, const at::Tensor* t, at::ScalarType st, std::initializer_list<int64_t> sizes) {
  if (t == nullptr) return nullptr;
  a.take(t->scalar_type() == st && t->is_contiguous() && t->dim() == static_cast<int64_t>(sizes.size()));
  int64_t k = 0;
  for (int64_t s : sizes) {
    if (!a.ok) return nullptr;
    a.take(s < 0 || t->size(k) == s);
    ++k;
  }
  return a.ok ? static_cast<const T*>(t->data_ptr()) : nullptr;
}

struct Rows {
  void* p = nullptr;
  long long stride = 0;
};
// [rows, H, d] whose rows are contiguous and may lie apart.
Rows spread(Args& a, const at::Tensor* t, at::ScalarType st, int64_t rows, int64_t H, int64_t d) {
  Rows r;
  if (t == nullptr || !a.take(t->scalar_type() == st && t->dim() == 3 && t->size(0) == rows && t->size(1) == H && t->size(2) == d &&
                              (d <= 1 || t->stride(2) == 1) && (H <= 1 || t->stride(1) == d)))
    return r;
  r.p = t->data_ptr();
  r.stride = rows > 1 ? t->stride(0) : H * d;
  return r;
}

const int32_t* offsets(Args& a, const at::Tensor* t, long long B) {
  if (t == nullptr || !a.take(t->scalar_type() == at::kInt && t->is_contiguous() && t->numel() >= B + 1)) return nullptr;
  return static_cast<const int32_t*>(t->data_ptr());
}

PyObject* result(long status) { return PyLong_FromLong(status); }

bool fits(int64_t x) { return x >= 0 && x <= INT_MAX; }

// linear(a, w, cu_seqlens, B, c, bias, act, residual, stream)
PyObject* linear(PyObject*, PyObject* const* v, Py_ssize_t n) {
  try {
    Args a{v, n};
    const at::Tensor *x = a.tensor(), *w = a.tensor(), *cu = a.tensor();
    const long long B = a.integer();
    const at::Tensor *c = a.tensor(), *bias = a.tensor(true);
    const long long act = a.integer();
    const at::Tensor* res = a.tensor(true);
    void* s = a.stream();
    rra_dtype in, out;
    if (!a.ok || x->dim() != 2 || w->dim() != 2 || !code(*x, in) || !code(*c, out)) return result(-1);
    const int64_t cap = x->size(0), K = x->size(1), N = w->size(0);
    const void* px = dense(a, x, x->scalar_type(), {-1, -1});
    const void* pw = dense(a, w, x->scalar_type(), {-1, K});
    const float* pb = dense<float>(a, bias, at::kFloat, {N});
    const void* pr = dense(a, res, c->scalar_type(), {cap, N});
    void* pc = const_cast<void*>(dense(a, c, c->scalar_type(), {cap, N}));
    const int32_t* pcu = offsets(a, cu, B);
    if (!a.ok || !fits(cap) || !fits(K) || !fits(N)) return result(-1);
    rra_status st;
    Py_BEGIN_ALLOW_THREADS
    st = f_linear(px, pw, pb, pr, pcu, static_cast<int>(B), static_cast<int>(cap), static_cast<int>(K), static_cast<int>(N),
                  in, static_cast<rra_activation>(act), pc, out, s);
    Py_END_ALLOW_THREADS
    return result(st);
  } catch (...) {
    return result(-1);
  }
}

// rope(q, k, positions, cu_seqlens, B, q_out, k_out, inv_freq, q_weight, k_weight, eps, interleaved, rope_scale, v,
//      v_out, kv_rows, stream)
PyObject* rope(PyObject*, PyObject* const* v, Py_ssize_t n) {
  try {
    Args a{v, n};
    const at::Tensor *q = a.tensor(), *k = a.tensor(), *pos = a.tensor(true), *cu = a.tensor();
    const long long B = a.integer();
    const at::Tensor *qo = a.tensor(), *ko = a.tensor(), *f = a.tensor(true), *qw = a.tensor(true), *kw = a.tensor(true);
    const float eps = a.real();
    const long long il = a.integer();
    const float scale = a.real();
    const at::Tensor *vi = a.tensor(true), *vo = a.tensor(true), *slots = a.tensor(true);
    void* s = a.stream();
    rra_dtype dt;
    if (!a.ok || q->dim() != 3 || k->dim() != 3 || ko->dim() != 3 || !code(*q, dt) || (vi == nullptr) != (vo == nullptr) ||
        (pos == nullptr) != (f == nullptr))
      return result(-1);
    const at::ScalarType t = q->scalar_type();
    const int64_t cap = q->size(0), Hq = q->size(1), d = q->size(2), Hkv = k->size(1);
    const int64_t rows = slots != nullptr ? ko->size(0) : cap;
    const Rows rq = spread(a, q, t, cap, Hq, d), rk = spread(a, k, t, cap, Hkv, d);
    const Rows rqo = spread(a, qo, t, cap, Hq, d), rko = spread(a, ko, t, rows, Hkv, d);
    Rows rv, rvo;
    if (vi != nullptr) {
      rv = spread(a, vi, t, cap, Hkv, d);
      rvo = spread(a, vo, t, rows, Hkv, d);
    }
    const int32_t* ppos = dense<int32_t>(a, pos, at::kInt, {cap});
    const float* pf = dense<float>(a, f, at::kFloat, {-1});
    const float* pqw = dense<float>(a, qw, at::kFloat, {d});
    const float* pkw = dense<float>(a, kw, at::kFloat, {d});
    const int32_t* pslots = dense<int32_t>(a, slots, at::kInt, {cap});
    const int32_t* pcu = offsets(a, cu, B);
    const int64_t rot = f != nullptr ? 2 * f->numel() : 0;
    if (!a.ok || !fits(cap) || !fits(Hq) || !fits(Hkv) || !fits(d) || !fits(rot)) return result(-1);
    rra_status st;
    Py_BEGIN_ALLOW_THREADS
    st = f_rope(rq.p, rq.stride, rk.p, rk.stride, rv.p, rv.stride, ppos, pcu, static_cast<int>(B), static_cast<int>(cap),
                static_cast<int>(Hq), static_cast<int>(Hkv), static_cast<int>(d), dt, pqw, pkw, eps, pf,
                static_cast<int>(rot), static_cast<int>(il), scale, rqo.p, rqo.stride, rko.p, rko.stride, rvo.p, rvo.stride,
                pslots, rows, s);
    Py_END_ALLOW_THREADS
    return result(st);
  } catch (...) {
    return result(-1);
  }
}

// prompt(q, k, v, cu_seqlens, B, max_seqlen, o, scale, causal, stream)
PyObject* prompt(PyObject*, PyObject* const* v, Py_ssize_t n) {
  try {
    Args a{v, n};
    const at::Tensor *q = a.tensor(), *k = a.tensor(), *vi = a.tensor(), *cu = a.tensor();
    const long long B = a.integer(), most = a.integer();
    const at::Tensor* o = a.tensor();
    const float scale = a.real();
    const long long causal = a.integer();
    void* s = a.stream();
    rra_dtype dt;
    if (!a.ok || q->dim() != 3 || k->dim() != 3 || !code(*q, dt)) return result(-1);
    const at::ScalarType t = q->scalar_type();
    const int64_t cap = q->size(0), Hq = q->size(1), d = q->size(2), Hkv = k->size(1);
    const Rows rq = spread(a, q, t, cap, Hq, d), rk = spread(a, k, t, cap, Hkv, d), rv = spread(a, vi, t, cap, Hkv, d);
    void* po = const_cast<void*>(dense(a, o, t, {cap, Hq, d}));
    const int32_t* pcu = offsets(a, cu, B);
    if (!a.ok || !fits(cap) || !fits(Hq) || !fits(Hkv) || !fits(d)) return result(-1);
    rra_status st;
    Py_BEGIN_ALLOW_THREADS
    st = f_prompt(rq.p, rq.stride, rk.p, rk.stride, rv.p, rv.stride, pcu, static_cast<int>(B), static_cast<int>(cap),
                  static_cast<int>(most), static_cast<int>(Hq), static_cast<int>(Hkv), static_cast<int>(d), scale,
                  static_cast<int>(causal), dt, po, s);
    Py_END_ALLOW_THREADS
    return result(st);
  } catch (...) {
    return result(-1);
  }
}

// cache(q, k_cache, v_cache, kv_len, o, scale, stream)
PyObject* cache(PyObject*, PyObject* const* v, Py_ssize_t n) {
  try {
    Args a{v, n};
    const at::Tensor *q = a.tensor(), *k = a.tensor(), *vc = a.tensor(), *len = a.tensor(), *o = a.tensor();
    const float scale = a.real();
    void* s = a.stream();
    rra_dtype dt;
    if (!a.ok || q->dim() != 3 || k->dim() != 4 || !code(*q, dt)) return result(-1);
    const at::ScalarType t = q->scalar_type();
    const int64_t B = k->size(0), cap = k->size(1), Hkv = k->size(2), d = k->size(3), rows = q->size(0), Hq = q->size(1);
    if (B < 1 || rows % B != 0) return result(-1);
    const Rows rq = spread(a, q, t, rows, Hq, d);
    const void *pk = dense(a, k, t, {B, cap, Hkv, d}), *pv = dense(a, vc, t, {B, cap, Hkv, d});
    const int32_t* pl = dense<int32_t>(a, len, at::kInt, {B});
    void* po = const_cast<void*>(dense(a, o, t, {rows, Hq, d}));
    if (!a.ok || !fits(B) || !fits(rows) || !fits(cap) || !fits(Hq) || !fits(Hkv) || !fits(d)) return result(-1);
    rra_status st;
    Py_BEGIN_ALLOW_THREADS
    st = f_cache(rq.p, rq.stride, pk, pv, pl, static_cast<int>(B), static_cast<int>(rows / B), static_cast<int>(cap),
                 static_cast<int>(Hq), static_cast<int>(Hkv), static_cast<int>(d), scale, dt, po, s);
    Py_END_ALLOW_THREADS
    return result(st);
  } catch (...) {
    return result(-1);
  }
}

// bind(linear, rope, prompt, cache): the addresses of librra's functions.
PyObject* bind(PyObject*, PyObject* const* v, Py_ssize_t n) {
  if (n != 4) {
    PyErr_SetString(PyExc_TypeError, "bind takes four addresses");
    return nullptr;
  }
  void* p[4];
  for (int i = 0; i < 4; ++i) {
    p[i] = PyLong_AsVoidPtr(v[i]);
    if (p[i] == nullptr) {
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "null address");
      return nullptr;
    }
  }
  f_linear = reinterpret_cast<decltype(f_linear)>(p[0]);
  f_rope = reinterpret_cast<decltype(f_rope)>(p[1]);
  f_prompt = reinterpret_cast<decltype(f_prompt)>(p[2]);
  f_cache = reinterpret_cast<decltype(f_cache)>(p[3]);
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"bind", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(bind)), METH_FASTCALL, nullptr},
    {"linear", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(linear)), METH_FASTCALL, nullptr},
    {"rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(rope)), METH_FASTCALL, nullptr},
    {"prompt", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(prompt)), METH_FASTCALL, nullptr},
    {"cache", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(cache)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_rra_fast", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__rra_fast() { return PyModule_Create(&module); }
