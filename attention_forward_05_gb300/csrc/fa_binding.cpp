// fa_binding.cpp -- Python binding of the position and paged-cache entry points (include/fa.h): fa_rope,
// fa_paged_append, fa_decode_paged_prefix.
//
// These are called once a token or once a layer, often on a few kilobytes, where the host path is the larger
// part of a call: checks, allocations and argument conversion take about 2 us here, against 12 to 20 us by way
// of ctypes.  Like the rest of the binding it only checks tensors, allocates outputs and workspaces with
// PyTorch's allocator on the current stream, and calls the C ABI.  A call returns its tensors, or the
// fa_status code of a call that the library refused.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <cstdio>
#include <optional>

#include "fa.h"

namespace {

using at::Tensor;

// A Python exception to raise; type nullptr: one that is set already.
struct Refusal {
  PyObject* type;
  char text[160];
};

template <typename... A>
Refusal refusal(PyObject* type, const char* format, A... a) {
  Refusal r{type, {}};
  snprintf(r.text, sizeof(r.text), format, a...);
  return r;
}
template <typename... A>
Refusal ValueError(const char* format, A... a) {
  return refusal(PyExc_ValueError, format, a...);
}
template <typename... A>
Refusal TypeError(const char* format, A... a) {
  return refusal(PyExc_TypeError, format, a...);
}
Refusal raised() { return Refusal{nullptr, {}}; }

// Runs `f`; what it throws becomes a Python exception.
template <typename F>
PyObject* guarded(F&& f) {
  HANDLE_TH_ERRORS
  try {
    return f();
  } catch (const Refusal& r) {
    if (r.type) PyErr_SetString(r.type, r.text);
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// An argument that may be None.
struct Arg {
  const char* name;
  const Tensor* t;  // nullptr: None
  const Tensor& operator*() const { return *t; }
  const Tensor* operator->() const { return t; }
  explicit operator bool() const { return t != nullptr; }
  // Throws for a tensor without memory (a fake one): taken before the GIL is let go.
  void* ptr() const {
    void* const p = t ? t->data_ptr() : nullptr;
    if (p == nullptr && t && t->numel() > 0) throw refusal(PyExc_ValueError, "%s has no memory", name);
    return p;
  }
};

Arg arg(PyObject* o, const char* name, bool optional = false) {
  if (optional && o == Py_None) return {name, nullptr};
  if (!THPVariable_Check(o)) throw TypeError("%s must be a tensor", name);
  return {name, &THPVariable_Unpack(o)};
}

// All tensors on the current device; returns its index.
template <typename... A>
int same_device(const A&... args) {
  const int cur = c10::cuda::current_device();
  for (const Arg* a : {&args...}) {
    if (!*a) continue;
    if (!(*a)->is_cuda()) throw ValueError("%s must be a CUDA tensor", a->name);
    if ((*a)->get_device() != cur)
      throw ValueError("%s is on cuda:%d, not on the current device cuda:%d", a->name,
                       static_cast<int>((*a)->get_device()), cur);
  }
  return cur;
}

// CUDA tensors come before the current device is asked for: without a GPU that would raise another error.
template <typename... A>
void need_cuda(const A&... args) {
  for (const Arg* a : {&args...})
    if (*a && !(*a)->is_cuda()) throw ValueError("%s must be a CUDA tensor", a->name);
}

void need_type(const Arg& a, at::ScalarType type, const char* what) {
  if (a && a->scalar_type() != type) throw ValueError("%s must be %s", a.name, what);
}

void need_contiguous(const Arg& a) {
  if (a && !a->is_contiguous()) throw ValueError("%s must be contiguous", a.name);
}

// The strides of all dimensions but the last, which must be contiguous; 0 for those of one entry, whose stride says
// nothing.
void strides_of(const Arg& a, long long* out) {
  const int n = static_cast<int>(a->dim()) - 1;
  if (a->stride(n) != 1) throw ValueError("%s's last dimension must be contiguous", a.name);
  for (int i = 0; i < n; ++i) out[i] = a->size(i) == 1 ? 0 : a->stride(i);
}

int as_int(int64_t v, const char* name) {
  if (v < 0 || v > 0x7FFFFFFF) throw ValueError("%s is out of range", name);
  return static_cast<int>(v);
}

fa_stream_t stream_of(int dev) {
  return reinterpret_cast<fa_stream_t>(c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream());
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw raised();
  return v != 0;
}

// A new tensor beside `t`, from PyTorch's allocator on the current stream.
Tensor empty_like_shape(at::IntArrayRef sizes, const Tensor& t, at::ScalarType type) {
  return Tensor(at::detail::empty_cuda(sizes, type, t.device(), std::nullopt));
}

// Frequencies and axes of a rotation.
void check_rotation(const Arg& positions, const Arg& freqs, const Arg& axes) {
  need_type(positions, at::kInt, "int32");
  need_contiguous(positions);
  if (freqs->scalar_type() != at::kDouble || freqs->dim() != 1 || !freqs->is_contiguous())
    throw ValueError("freqs must be a contiguous float64 vector (radians per position)");
  if (axes && (axes->scalar_type() != at::kInt || axes->sizes() != freqs->sizes() || !axes->is_contiguous()))
    throw ValueError("axes must be contiguous int32, one entry a frequency");
}

// (a, b); takes both references.  A nullptr is an object that could not be made, with its exception set.
PyObject* pair(PyObject* a, PyObject* b) {
  PyObject* out = a && b ? PyTuple_Pack(2, a, b) : nullptr;
  Py_XDECREF(a);
  Py_XDECREF(b);
  return out;
}

void need_args(Py_ssize_t n, Py_ssize_t want) {
  if (n != want) throw TypeError("%d arguments expected", static_cast<int>(want));
}

// rope(q, k, positions, freqs, axes, interleaved, q_out, k_out, inverse) -> (q_out, k_out)
PyObject* rope(PyObject*, PyObject* const* in, Py_ssize_t n_in) {
  return guarded([&]() -> PyObject* {
    need_args(n_in, 9);
    const Arg q = arg(in[0], "q"), k = arg(in[1], "k", true), pos = arg(in[2], "positions"), freqs = arg(in[3], "freqs"),
              axes = arg(in[4], "axes", true);
    Arg qo = arg(in[6], "q_out", true), ko = arg(in[7], "k_out", true);
    need_cuda(q, k, pos, freqs, axes, qo, ko);
    const int dev = same_device(q, k, pos, freqs, axes, qo, ko);
    check_rotation(pos, freqs, axes);
    if (q->dim() != 4 || (k && (k->dim() != 4 || k->size(0) != q->size(0) || k->size(2) != q->size(2) ||
                                k->size(3) != q->size(3))))
      throw ValueError("q [B,H,N,d], k [B,Hkv,N,d] expected");
    const at::ScalarType type = q->scalar_type();
    if (type != at::kBFloat16 && type != at::kFloat) throw TypeError("unsupported dtype: bf16 or fp32");
    if (k && k->scalar_type() != type) throw TypeError("q and k must share a dtype");
    if (!k && ko) throw ValueError("k_out without k");
    const int64_t B = q->size(0), N = q->size(2);
    int64_t n_axes = 1;
    bool shared = false, fits;
    if (pos->dim() == 1) {  // [N]: one axis, the same for every batch entry
      shared = true;
      fits = pos->size(0) == N;
    } else if (pos->dim() == 2) {  // [B, N]: one axis
      fits = pos->size(0) == B && pos->size(1) == N;
    } else {  // [axes, B, N] or, the same for every batch entry, [axes, 1, N]
      fits = pos->dim() == 3 && (pos->size(1) == B || pos->size(1) == 1) && pos->size(2) == N;
      n_axes = pos->dim() == 3 ? pos->size(0) : 1;
      shared = fits && pos->size(1) == 1 && B > 1;
    }
    if (!fits) throw ValueError("positions [N], [B,N], [axes,B,N] or [axes,1,N] expected");
    Tensor q_new, k_new;
    if (!qo) {
      q_new = empty_like_shape(q->sizes(), *q, type);
      qo.t = &q_new;
    }
    if (k && !ko) {
      k_new = empty_like_shape(k->sizes(), *k, type);
      ko.t = &k_new;
    }
    long long strides[12] = {};
    const Arg* each[4] = {&q, &k, &qo, &ko};
    for (int i = 0; i < 4; ++i) {
      if (!*each[i]) continue;
      if ((*each[i])->sizes() != (*each[i & 1])->sizes() || (*each[i])->scalar_type() != type)
        throw ValueError("%s must match its input", each[i]->name);
      strides_of(*each[i], strides + 3 * i);
    }
    const int H = as_int(q->size(1), "H"), Hkv = k ? as_int(k->size(1), "Hkv") : 0;
    const int Bi = as_int(B, "B"), Ni = as_int(N, "N"), d = as_int(q->size(3), "d"), ax = as_int(n_axes, "axes");
    const int rot = as_int(2 * freqs->size(0), "freqs");
    const bool inter = truth(in[5]), inverse = truth(in[8]);
    void *const qp = q.ptr(), *const kp = k.ptr(), *const qop = qo.ptr(), *const kop = ko.ptr();
    const int *const posp = static_cast<const int*>(pos.ptr()), *const axp = static_cast<const int*>(axes.ptr());
    const double* const fp = static_cast<const double*>(freqs.ptr());
    const fa_stream_t stream = stream_of(dev);
    int st = FA_OK;
    if (B > 0 && N > 0) {  // an empty tensor has no address; there is nothing to rotate
      Py_BEGIN_ALLOW_THREADS;
      st = fa_rope(qp, kp, qop, kop, strides, Bi, H, Hkv, Ni, d, type == at::kFloat ? FA_FP32 : FA_BF16, posp, shared, fp,
                   axp, ax, rot, inter, inverse, stream);
      Py_END_ALLOW_THREADS;
    }
    if (st != FA_OK) return PyLong_FromLong(st);
    PyObject* a = q_new.defined() ? THPVariable_Wrap(std::move(q_new)) : Py_NewRef(in[6]);
    PyObject* b = k_new.defined() ? THPVariable_Wrap(std::move(k_new)) : Py_NewRef(in[7]);
    return pair(a, b);
  });
}

// Shape, dtype and strides of a pair of caches.
void check_cache(const Arg& kc, const Arg& vc, long long (&strides)[3]) {
  if (kc->dim() != 4 || kc->sizes() != vc->sizes())
    throw ValueError("k_cache/v_cache [num_pages,Hkv,page_size,d] expected");
  if (kc->scalar_type() != at::kBFloat16 || vc->scalar_type() != at::kBFloat16) throw TypeError("the cache is bf16");
  long long sv[3];
  strides_of(kc, strides);
  strides_of(vc, sv);
  if (strides[0] != sv[0] || strides[1] != sv[1] || strides[2] != sv[2])
    throw ValueError("k_cache and v_cache must have the same strides");
}

// append(k, v, k_cache, v_cache, slots, q, positions, freqs, axes, interleaved, q_out) -> q_out or None
PyObject* append(PyObject*, PyObject* const* in, Py_ssize_t n_in) {
  return guarded([&]() -> PyObject* {
    need_args(n_in, 11);
    const Arg k = arg(in[0], "k"), v = arg(in[1], "v"), kc = arg(in[2], "k_cache"), vc = arg(in[3], "v_cache"),
              slots = arg(in[4], "slots"), q = arg(in[5], "q", true), pos = arg(in[6], "positions", true),
              freqs = arg(in[7], "freqs", true), axes = arg(in[8], "axes", true);
    Arg qo = arg(in[10], "q_out", true);
    need_cuda(k, v, kc, vc, slots, q, pos, freqs, axes, qo);
    const int dev = same_device(k, v, kc, vc, slots, q, pos, freqs, axes, qo);
    long long cs[3];
    check_cache(kc, vc, cs);
    const int64_t Hkv = kc->size(1), d = kc->size(3);
    if (k->dim() != 3 || k->sizes() != v->sizes() || k->size(1) != Hkv || k->size(2) != d)
      throw ValueError("k/v [T,Hkv,d] of the cache's Hkv and d expected");
    const int64_t T = k->size(0);
    if (k->scalar_type() != at::kBFloat16 || v->scalar_type() != at::kBFloat16 ||
        (q && q->scalar_type() != at::kBFloat16))
      throw TypeError("k, v and q are bf16");
    if (slots->scalar_type() != at::kLong || slots->dim() != 1 || slots->size(0) != T || !slots->is_contiguous())
      throw ValueError("slots must be contiguous int64 [T]");
    if (static_cast<bool>(pos) != static_cast<bool>(freqs)) throw ValueError("positions and freqs go together");
    int64_t n_axes = 1, rot = 0;
    if (pos) {
      check_rotation(pos, freqs, axes);
      if (pos->dim() == 2) n_axes = pos->size(0);
      if (pos->dim() < 1 || pos->dim() > 2 || pos->size(pos->dim() - 1) != T)
        throw ValueError("positions [T] or [axes,T] expected");
      rot = 2 * freqs->size(0);
    }
    if (q && (q->dim() != 3 || q->size(0) != T || q->size(2) != d)) throw ValueError("q [T,H,d] expected");
    if (!q && qo) throw ValueError("q_out without q");
    if (qo && (qo->sizes() != q->sizes() || qo->scalar_type() != at::kBFloat16 || !qo->is_contiguous()))
      throw ValueError("q_out must be contiguous and match q");
    Tensor q_new;
    if (q && !qo) {
      q_new = empty_like_shape(q->sizes(), *q, at::kBFloat16);
      qo.t = &q_new;
    }
    long long s[6] = {};
    strides_of(k, s);
    strides_of(v, s + 2);
    if (q) strides_of(q, s + 4);
    const int Ti = as_int(T, "T"), H = q ? as_int(q->size(1), "H") : 0, pages = as_int(kc->size(0), "num_pages"),
              ps = as_int(kc->size(2), "page_size"), di = as_int(d, "d"), hk = as_int(Hkv, "Hkv"),
              ax = as_int(n_axes, "axes"), r = as_int(rot, "freqs");
    const bool inter = truth(in[9]);
    int st = FA_OK;
    if (T > 0) {  // an empty tensor has no address; there is nothing to append
      void *const kp = k.ptr(), *const vp = v.ptr(), *const qp = q.ptr(), *const qop = qo.ptr();
      void *const kcp = kc.ptr(), *const vcp = vc.ptr();
      const long long* const sp = static_cast<const long long*>(slots.ptr());
      const int *const posp = static_cast<const int*>(pos.ptr()), *const axp = static_cast<const int*>(axes.ptr());
      const double* const fp = static_cast<const double*>(freqs.ptr());
      const fa_stream_t stream = stream_of(dev);
      Py_BEGIN_ALLOW_THREADS;
      st = fa_paged_append(kp, vp, qp, qop, kcp, vcp, s, cs, sp, Ti, H, hk, di, pages, ps, posp, fp, axp, ax, r, inter,
                           stream);
      Py_END_ALLOW_THREADS;
    }
    if (st != FA_OK) return PyLong_FromLong(st);
    return q_new.defined() ? THPVariable_Wrap(std::move(q_new)) : Py_NewRef(in[10]);
  });
}

// decode(q, k_cache, v_cache, prefix_pages, prefix_len, page_table, seq_lens, scale, workspace, with_lse, o) -> (o, lse)
PyObject* decode(PyObject*, PyObject* const* in, Py_ssize_t n_in) {
  return guarded([&]() -> PyObject* {
    need_args(n_in, 11);
    const Arg q = arg(in[0], "q"), kc = arg(in[1], "k_cache"), vc = arg(in[2], "v_cache"),
              pre = arg(in[3], "prefix_pages", true), table = arg(in[5], "page_table"), lens = arg(in[6], "seq_lens");
    const Arg ws = arg(in[8], "workspace", true);
    Arg o = arg(in[10], "o", true);
    need_cuda(q, kc, vc, pre, table, lens, ws, o);
    const int dev = same_device(q, kc, vc, pre, table, lens, ws, o);
    long long cs[3];
    check_cache(kc, vc, cs);
    const int64_t Hkv = kc->size(1), ps = kc->size(2), d = kc->size(3), qd = q->dim();
    if ((qd != 3 && qd != 4) || q->size(qd - 1) != d || (qd == 4 && q->size(2) != 1) || !q->is_contiguous())
      throw ValueError("contiguous q [B,H,d] or [B,H,1,d] expected");
    if (q->scalar_type() != at::kBFloat16) throw TypeError("decode takes bf16 q, k, v");
    const int64_t B = q->size(0), H = q->size(1);
    if (Hkv < 1 || H % Hkv != 0) throw ValueError("query heads must be a multiple of key/value heads");
    if (table->scalar_type() != at::kInt || table->dim() != 2 || table->size(0) != B || table->size(1) < 1)
      throw ValueError("page_table must be int32 [B, max_pages] with a column");
    const int64_t max_pages = table->size(1);
    if (table->stride(1) != 1 && max_pages > 1) throw ValueError("page_table's rows must be contiguous");
    if (lens->scalar_type() != at::kInt || lens->dim() != 1 || lens->size(0) != B || !lens->is_contiguous())
      throw ValueError("seq_lens must be contiguous int32 [B]");
    const long long plen = PyLong_AsLongLong(in[4]);
    if (plen == -1 && PyErr_Occurred()) throw raised();
    if (plen != 0 && (!pre || pre->scalar_type() != at::kInt || pre->dim() != 1 || !pre->is_contiguous() || plen < 0 ||
                      plen > pre->size(0) * ps || plen > 0x7FFFFFFF))
      throw ValueError("prefix_pages must be contiguous int32 and hold the prefix");
    double scale = 1.0 / std::sqrt(static_cast<double>(d));
    if (in[7] != Py_None) {
      scale = PyFloat_AsDouble(in[7]);
      if (scale == -1.0 && PyErr_Occurred()) throw raised();
    }
    if (o && (o->scalar_type() != at::kBFloat16 || o->numel() != B * H * d || !o->is_contiguous()))
      throw ValueError("o must be contiguous bf16 [B,H,d]");
    need_contiguous(ws);
    const int Bi = as_int(B, "B"), Hi = as_int(H, "H"), hk = as_int(Hkv, "Hkv"), di = as_int(d, "d"),
              psi = as_int(ps, "page_size"), pages = as_int(kc->size(0), "num_pages"), mp = as_int(max_pages, "max_pages");
    Tensor o_new, lse;
    if (!o) {
      o_new = empty_like_shape({B, H, d}, *q, at::kBFloat16);
      o.t = &o_new;
    }
    if (truth(in[9])) lse = empty_like_shape({B, H}, *q, at::kFloat);
    // The workspace goes back to the allocator when this returns: later work that gets it is behind this call's on the
    // current stream.
    c10::DataPtr own_ws;
    void* ws_ptr = ws.ptr();
    size_t ws_bytes = ws ? ws->nbytes() : 0;
    if (!ws && B > 0) {
      ws_bytes = fa_decode_paged_call_bytes(Bi, Hi, hk, di, psi, mp, static_cast<int>(plen));
      if (ws_bytes > 0) {  // 0: none needed, or arguments that the call below refuses
        own_ws = c10::cuda::CUDACachingAllocator::get()->allocate(ws_bytes);
        ws_ptr = own_ws.get();
      }
    }
    const long long row = B == 1 ? mp : table->stride(0);
    void *const qp = q.ptr(), *const kcp = kc.ptr(), *const vcp = vc.ptr(), *const op = o.ptr();
    const int* const prep = plen ? static_cast<const int*>(pre.ptr()) : nullptr;
    const int *const tp = static_cast<const int*>(table.ptr()), *const lp = static_cast<const int*>(lens.ptr());
    float* const lsep = lse.defined() ? static_cast<float*>(lse.data_ptr()) : nullptr;
    const fa_stream_t stream = stream_of(dev);
    int st = FA_OK;
    if (B > 0) {  // a step without sequences: empty results
      Py_BEGIN_ALLOW_THREADS;
      st = fa_decode_paged_prefix(qp, kcp, vcp, op, prep, static_cast<int>(plen), tp, row, lp, Bi, Hi, hk, di, pages, psi,
                                  mp, cs, static_cast<float>(scale), ws_ptr, ws_bytes, lsep, stream);
      Py_END_ALLOW_THREADS;
    }
    if (st != FA_OK) return PyLong_FromLong(st);
    PyObject* a = o_new.defined() ? THPVariable_Wrap(std::move(o_new)) : Py_NewRef(in[10]);
    PyObject* b = lse.defined() ? THPVariable_Wrap(std::move(lse)) : Py_NewRef(Py_None);
    return pair(a, b);
  });
}

PyMethodDef kMethods[] = {
    {"rope", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(rope)), METH_FASTCALL, nullptr},
    {"append", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(append)), METH_FASTCALL, nullptr},
    {"decode", reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(decode)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_fa_binding", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fa_binding() { return PyModule_Create(&kModule); }
