// binding.cpp - the Python binding's checks and marshalling for the calls around a paged cache
// and a training step's norms, in C++: a call on one new token spends less time on the GPU
// (2 to 4 us) than ctypes and Python take to look at its tensors (25 us; 7 us this way).
//
// It checks tensors as the Python wrappers document, allocates results and workspace where none
// are given, and calls an entry point of the C library by its address on the current torch stream.
// Each function returns its results, or the library's nonzero status as an int.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <array>
#include <cmath>
#include <cstdint>
#include <string>

#include "attn_fwd.h"

namespace {

struct Refused {
  PyObject* type;
  std::string what;
};
[[noreturn]] void type_error(const std::string& what) { throw Refused{PyExc_TypeError, what}; }
[[noreturn]] void value_error(const std::string& what) { throw Refused{PyExc_ValueError, what}; }

const at::Tensor* tensor(PyObject* o) { return THPVariable_Check(o) ? &THPVariable_Unpack(o) : nullptr; }

std::string shape_str(at::IntArrayRef s) {
  std::string r = "(";
  for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
  return r + (s.size() == 1 ? ",)" : ")");
}

const at::Tensor& bf16(const char* name, PyObject* o, int device = -1) {
  const at::Tensor* t = tensor(o);
  if (!t || t->scalar_type() != at::kBFloat16 || !t->is_cuda()) type_error(std::string(name) + " must be a bf16 CUDA tensor");
  if (device >= 0 && t->get_device() != device) value_error(std::string(name) + " must be on the device of the others");
  return *t;
}

// A contiguous tensor of a type and shape on a device.
const at::Tensor& plain(const char* name, PyObject* o, at::ScalarType type, const char* type_name, at::IntArrayRef shape,
                        int device) {
  const at::Tensor* t = tensor(o);
  if (!t || t->scalar_type() != type || t->sizes() != shape || !t->is_contiguous() || !t->is_cuda() ||
      t->get_device() != device)
    value_error(std::string(name) + " must be a contiguous " + type_name + " tensor of shape " + shape_str(shape) +
                " on the device of the others");
  return *t;
}

// (tokens, heads, d), or 4-D in the layout: sizes and element strides.
struct Rows {
  int64_t B, S, H, D;
  std::array<int64_t, 3> at;
};
Rows rows_of(const char* name, const at::Tensor& t, int layout) {
  Rows r;
  const auto n = t.sizes(), s = t.strides();
  if (n.size() == 4) {
    const int token = layout == ATTN_LAYOUT_BSHD ? 1 : 2, head = 3 - token;
    r = {n[0], n[token], n[head], n[3], {s[0], s[token], s[head]}};
  } else if (n.size() == 3) {
    r = {1, n[0], n[1], n[2], {0, s[0], s[1]}};
  } else {
    value_error(std::string(name) + " must be (tokens, heads, d) or 4-D");
  }
  if (s.back() != 1 && n.back() != 1) value_error(std::string(name) + "'s last dimension must be contiguous");
  return r;
}

// A result as given, or a new one: the tensor, and the object to return.
struct Result {
  at::Tensor t;
  PyObject* given;
  PyObject* object() const { return given ? Py_NewRef(given) : THPVariable_Wrap(t); }
};
at::Tensor fresh(at::IntArrayRef shape, at::ScalarType type, const at::Tensor& like) {
  return at::empty(shape, at::TensorOptions().dtype(type).device(like.device()));
}
Result rows_out(const char* name, PyObject* o, const at::Tensor& like, int device) {
  if (o == Py_None) return {fresh(like.sizes(), at::kBFloat16, like), nullptr};
  const at::Tensor& t = bf16(name, o, device);
  if (t.sizes() != like.sizes()) value_error(std::string(name) + " must be a bf16 CUDA tensor of shape " + shape_str(like.sizes()));
  return {t, o};
}
Result plain_out(const char* name, PyObject* o, at::ScalarType type, const char* type_name, at::IntArrayRef shape,
                 const at::Tensor& like) {
  if (o == Py_None) return {fresh(shape, type, like), nullptr};
  return {plain(name, o, type, type_name, shape, like.get_device()), o};
}

// A workspace as given, or a new one of `need` bytes.
struct Workspace {
  at::Tensor t;
  void* p;
  int64_t n;
};
Workspace workspace_of(PyObject* o, int64_t need, const at::Tensor& like) {
  Workspace w;
  if (o == Py_None) {
    w.t = fresh({need}, at::kByte, like);
  } else {
    const at::Tensor* t = tensor(o);
    if (!t || !t->is_cuda() || t->get_device() != like.get_device() || !t->is_contiguous())
      value_error("workspace must be a contiguous CUDA tensor on the device of the others");
    w.t = *t;
  }
  w.p = w.t.data_ptr();
  w.n = static_cast<int64_t>(w.t.nbytes());
  return w;
}

// What the norm-and-rotation calls share.
struct Rope {
  const at::Tensor *q, *k, *wq, *wk, *cos, *sin, *positions;
  Rows rq, rk;
  int device;
  int64_t max_pos, rot;
  at::DimVector per_token;  // shape of what is one a token
};
Rope rope_of(PyObject* const* a, int layout) {  // q, k, q_weight, k_weight, cos, sin, positions
  Rope r;
  r.q = &bf16("q", a[0]);
  r.device = r.q->get_device();
  r.k = &bf16("k", a[1], r.device);
  r.rq = rows_of("q", *r.q, layout);
  r.rk = rows_of("k", *r.k, layout);
  if (r.rk.B != r.rq.B || r.rk.S != r.rq.S || r.rk.D != r.rq.D || r.q->dim() != r.k->dim()) value_error("shape mismatch");
  const at::Tensor** w[2] = {&r.wq, &r.wk};
  for (int i = 0; i < 2; ++i)
    *w[i] = &plain(i ? "k_weight" : "q_weight", a[2 + i], at::kBFloat16, "bf16", {r.rq.D}, r.device);
  r.cos = tensor(a[4]);
  if (!r.cos || r.cos->dim() != 2) value_error("cos must be a contiguous fp32 tensor of shape (max_pos, rotary_dim / 2)");
  r.cos = &plain("cos", a[4], at::kFloat, "fp32", r.cos->sizes(), r.device);
  r.sin = &plain("sin", a[5], at::kFloat, "fp32", r.cos->sizes(), r.device);
  r.max_pos = r.cos->size(0);
  r.rot = 2 * r.cos->size(1);
  if (r.q->dim() == 3)
    r.per_token = {r.rq.S};
  else
    r.per_token = {r.rq.B, r.rq.S};
  r.positions = &plain("positions", a[6], at::kInt, "int32", r.per_token, r.device);
  return r;
}

// A cache's pages: 4-D tensors whose pages are dense and may lie apart.
struct Pages {
  const at::Tensor *k, *v;
  int64_t n, page, Hkv, D, stride;
};
Pages pages_of(PyObject* ko, PyObject* vo, int layout, int device = -1) {
  Pages p;
  p.k = &bf16("k_pages", ko, device);
  p.v = &bf16("v_pages", vo, p.k->get_device());
  const auto n = p.k->sizes(), s = p.k->strides();
  const auto vs = p.v->strides();
  if (n.size() != 4 || p.v->sizes() != n) value_error("k_pages and v_pages must be 4-D tensors of one shape and strides");
  // A dimension of one entry has no stride: what stands there is not looked at.
  const int64_t dense[4] = {0, n[2] * n[3], n[3], 1};
  for (int i = 0; i < 4; ++i) {
    if (n[i] <= 1) continue;
    if (vs[i] != s[i]) value_error("k_pages and v_pages must be 4-D tensors of one shape and strides");
    if (i > 0 && s[i] != dense[i]) value_error("a page of k_pages and v_pages must be contiguous");
  }
  const bool bshd = layout == ATTN_LAYOUT_BSHD;
  p.n = n[0];
  p.page = bshd ? n[1] : n[2];
  p.Hkv = bshd ? n[2] : n[1];
  p.D = n[3];
  p.stride = n[0] > 1 ? s[0] : n[1] * n[2] * n[3];
  return p;
}

// (B, max_pages) and the lengths that go with it.
struct Table {
  const at::Tensor *pages, *lens;
  int64_t B, max_pages;
};
const at::Tensor& int32_of(const char* name, PyObject* o, int dim, int device) {
  const at::Tensor* t = tensor(o);
  if (!t || t->scalar_type() != at::kInt || !t->is_cuda() || t->dim() != dim || !t->is_contiguous())
    type_error(std::string(name) + " must be a contiguous " + std::to_string(dim) + "-D int32 CUDA tensor");
  if (t->get_device() != device) value_error(std::string(name) + " must be on the pages' device");
  return *t;
}
Table table_of(PyObject* pages, PyObject* lens, int device) {
  Table t;
  t.pages = &int32_of("page_table", pages, 2, device);
  t.lens = &int32_of("seqlens", lens, 1, device);
  t.B = t.pages->size(0);
  t.max_pages = t.pages->size(1);
  if (t.lens->size(0) != t.B) value_error("seqlens must have an entry for each row of page_table");
  return t;
}

template <typename Fn>
Fn* address(PyObject* o) {
  void* p = PyLong_AsVoidPtr(o);
  if (!p) value_error("no entry point");
  return reinterpret_cast<Fn*>(p);
}
int int_of(PyObject* o) {
  const long x = PyLong_AsLong(o);
  if (x == -1 && PyErr_Occurred()) throw python_error();
  return static_cast<int>(x);
}
int64_t int64_of(PyObject* o) {
  const long long x = PyLong_AsLongLong(o);
  if (x == -1 && PyErr_Occurred()) throw python_error();
  return x;
}
float float_of(PyObject* o) {
  const double x = PyFloat_AsDouble(o);
  if (x == -1.0 && PyErr_Occurred()) throw python_error();
  return static_cast<float>(x);
}
void* ptr(const at::Tensor& t) { return t.data_ptr(); }
void* stream_of(int device) { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device)).stream(); }

// The call itself, without the interpreter's lock.
template <typename F>
int unlocked(F&& f) {
  PyThreadState* s = PyEval_SaveThread();
  const int st = f();
  PyEval_RestoreThread(s);
  return st;
}

PyObject* answer(int st, std::initializer_list<const Result*> results) {
  if (st != ATTN_OK) return PyLong_FromLong(st);
  PyObject* t = PyTuple_New(static_cast<Py_ssize_t>(results.size()));
  if (!t) return nullptr;
  Py_ssize_t i = 0;
  for (const Result* r : results) {
    PyObject* o = r->object();
    if (!o) {
      Py_DECREF(t);
      return nullptr;
    }
    PyTuple_SET_ITEM(t, i++, o);
  }
  return t;
}

// norm_rope(entry, q, k, q_weight, k_weight, cos, sin, positions, q_out, k_out, eps, layout, rounding, flags)
PyObject* norm_rope(PyObject* const* a) {
  auto* fn = address<decltype(attn_qk_norm_rope)>(a[0]);
  const int layout = int_of(a[11]), mode = int_of(a[12]), flags = int_of(a[13]);
  const float eps = float_of(a[10]);
  const Rope r = rope_of(a + 1, layout);
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(r.device));
  const Result qo = rows_out("q_out", a[8], *r.q, r.device), ko = rows_out("k_out", a[9], *r.k, r.device);
  const Rows rqo = rows_of("q_out", qo.t, layout), rko = rows_of("k_out", ko.t, layout);
  void* stream = stream_of(r.device);
  const int st = unlocked([&] {
    return fn(ptr(*r.q), ptr(*r.k), ptr(*r.wq), ptr(*r.wk), static_cast<const float*>(ptr(*r.cos)),
              static_cast<const float*>(ptr(*r.sin)), static_cast<const int32_t*>(ptr(*r.positions)), ptr(qo.t),
              ptr(ko.t), r.rq.at.data(), r.rk.at.data(), rqo.at.data(), rko.at.data(), r.rq.B, r.rq.S, r.rq.H, r.rk.H,
              r.rq.D, r.max_pos, r.rot, eps, mode, flags, stream);
  });
  return answer(st, {&qo, &ko});
}

// norm_rope_paged(entry, q, k, q_weight, k_weight, cos, sin, positions, v, slots, k_pages, v_pages, q_out, eps, layout,
//                 rounding, flags)
PyObject* norm_rope_paged(PyObject* const* a) {
  auto* fn = address<decltype(attn_qk_norm_rope_paged)>(a[0]);
  const int layout = int_of(a[14]), mode = int_of(a[15]), flags = int_of(a[16]);
  const float eps = float_of(a[13]);
  const Rope r = rope_of(a + 1, layout);
  const at::Tensor& v = bf16("v", a[8], r.device);
  const Rows rv = rows_of("v", v, layout);
  const Pages p = pages_of(a[10], a[11], layout, r.device);
  if (v.sizes() != r.k->sizes() || p.Hkv != r.rk.H || p.D != r.rk.D) value_error("shape mismatch");
  const at::Tensor& slots = plain("slots", a[9], at::kInt, "int32", r.per_token, r.device);
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(r.device));
  const Result qo = rows_out("q_out", a[12], *r.q, r.device);
  const Rows rqo = rows_of("q_out", qo.t, layout);
  void* stream = stream_of(r.device);
  const int st = unlocked([&] {
    return fn(ptr(*r.q), ptr(*r.k), ptr(v), ptr(*r.wq), ptr(*r.wk), static_cast<const float*>(ptr(*r.cos)),
              static_cast<const float*>(ptr(*r.sin)), static_cast<const int32_t*>(ptr(*r.positions)),
              static_cast<const int32_t*>(ptr(slots)), ptr(qo.t), ptr(*p.k), ptr(*p.v), r.rq.at.data(), r.rk.at.data(),
              rv.at.data(), rqo.at.data(), layout, r.rq.B, r.rq.S, r.rq.H, r.rk.H, p.n, p.page, p.stride, r.rq.D,
              r.max_pos, r.rot, eps, mode, flags, stream);
  });
  return answer(st, {&qo});
}

// norm_rope_bwd(entry, workspace_bytes, q, k, q_weight, k_weight, cos, sin, positions, dq_out, dk_out, dq, dk,
//               dq_weight, dk_weight, workspace, eps, layout, rounding, flags)
PyObject* norm_rope_bwd(PyObject* const* a) {
  auto* fn = address<decltype(attn_qk_norm_rope_bwd)>(a[0]);
  auto* bytes = address<decltype(attn_qk_norm_rope_bwd_workspace_bytes)>(a[1]);
  const int layout = int_of(a[17]), mode = int_of(a[18]), flags = int_of(a[19]);
  const float eps = float_of(a[16]);
  const Rope r = rope_of(a + 2, layout);
  const at::Tensor &gq = bf16("dq_out", a[9], r.device), &gk = bf16("dk_out", a[10], r.device);
  if (gq.sizes() != r.q->sizes() || gk.sizes() != r.k->sizes()) value_error("shape mismatch");
  const Rows rgq = rows_of("dq_out", gq, layout), rgk = rows_of("dk_out", gk, layout);
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(r.device));
  const Result dq = rows_out("dq", a[11], *r.q, r.device), dk = rows_out("dk", a[12], *r.k, r.device);
  const Rows rdq = rows_of("dq", dq.t, layout), rdk = rows_of("dk", dk.t, layout);
  const Result wq = plain_out("dq_weight", a[13], at::kFloat, "fp32", {r.rq.D}, *r.q);
  const Result wk = plain_out("dk_weight", a[14], at::kFloat, "fp32", {r.rq.D}, *r.q);
  const int64_t need = bytes(r.rq.B, r.rq.S, r.rq.H, r.rk.H, r.rq.D);
  if (need < 0) return PyLong_FromLongLong(need);
  const Workspace ws = workspace_of(a[15], need, *r.q);
  void* stream = stream_of(r.device);
  const int st = unlocked([&] {
    return fn(ptr(gq), ptr(gk), ptr(*r.q), ptr(*r.k), ptr(*r.wq), ptr(*r.wk), static_cast<const float*>(ptr(*r.cos)),
              static_cast<const float*>(ptr(*r.sin)), static_cast<const int32_t*>(ptr(*r.positions)), ptr(dq.t),
              ptr(dk.t), static_cast<float*>(ptr(wq.t)), static_cast<float*>(ptr(wk.t)), rgq.at.data(), rgk.at.data(),
              r.rq.at.data(), r.rk.at.data(), rdq.at.data(), rdk.at.data(), r.rq.B, r.rq.S, r.rq.H, r.rk.H, r.rq.D,
              r.max_pos, r.rot, eps, mode, flags, ws.p, ws.n, stream);
  });
  return answer(st, {&dq, &dk, &wq, &wk});
}

// fwd_paged(entry, workspace_bytes, q, k_pages, v_pages, page_table, seqlens, out, lse, mass, workspace, scale, layout,
//           rounding, flags)
PyObject* fwd_paged(PyObject* const* a) {
  auto* fn = address<decltype(attn_fwd_paged)>(a[0]);
  auto* bytes = address<decltype(attn_fwd_paged_workspace_bytes)>(a[1]);
  const int layout = int_of(a[12]), mode = int_of(a[13]), flags = int_of(a[14]);
  const at::Tensor& q = bf16("q", a[2]);
  if (q.dim() != 4 || !q.is_contiguous()) value_error("q must be a contiguous 4-D tensor");
  const int device = q.get_device();
  const Rows r = rows_of("q", q, layout);
  const Pages p = pages_of(a[3], a[4], layout, device);
  const Table t = table_of(a[5], a[6], device);
  if (t.B != r.B || p.D != r.D || p.Hkv < 1 || r.H % p.Hkv) value_error("shape mismatch");
  float* mass = nullptr;
  if (a[9] != Py_None)
    mass = static_cast<float*>(ptr(plain("mass", a[9], at::kFloat, "fp32", {r.B, p.Hkv, t.max_pages * p.page}, device)));
  const float scale = a[11] == Py_None ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(r.D))) : float_of(a[11]);
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(device));
  const Result out = plain_out("out", a[7], at::kBFloat16, "bf16", q.sizes(), q);
  const Result lse = plain_out("lse", a[8], at::kFloat, "fp32", {r.B, r.H, r.S}, q);
  const int64_t need = bytes(r.B, r.H, p.Hkv, r.S, p.page, t.max_pages, r.D, mass != nullptr);
  if (need < 0) return PyLong_FromLongLong(need);
  const Workspace ws = workspace_of(a[10], need, q);
  void* stream = stream_of(device);
  const int st = unlocked([&] {
    return fn(ptr(q), ptr(*p.k), ptr(*p.v), static_cast<const int32_t*>(ptr(*t.pages)),
              static_cast<const int32_t*>(ptr(*t.lens)), ptr(out.t), static_cast<float*>(ptr(lse.t)), mass, layout, r.B,
              r.H, p.Hkv, r.S, p.n, p.page, p.stride, t.max_pages, r.D, scale, mode, flags, ws.p, ws.n, stream);
  });
  return answer(st, {&out, &lse});
}

// cache_evict(entry, workspace_bytes, k_pages, v_pages, page_table, seqlens, mass, mass_out, seqlens_out, workspace,
//             budget, recent, layout)
PyObject* cache_evict(PyObject* const* a) {
  auto* fn = address<decltype(attn_cache_evict)>(a[0]);
  auto* bytes = address<decltype(attn_cache_evict_workspace_bytes)>(a[1]);
  const int layout = int_of(a[12]);
  const int64_t budget = int64_of(a[10]), recent = int64_of(a[11]);
  const Pages p = pages_of(a[2], a[3], layout);
  const int device = p.k->get_device();
  const Table t = table_of(a[4], a[5], device);
  const std::array<int64_t, 3> shape = {t.B, p.Hkv, t.max_pages * p.page};
  const at::Tensor& mass = plain("mass", a[6], at::kFloat, "fp32", shape, device);
  const c10::cuda::CUDAGuard guard(static_cast<c10::DeviceIndex>(device));
  const Result mass_out = plain_out("mass_out", a[7], at::kFloat, "fp32", shape, mass);
  const Result lens_out = plain_out("seqlens_out", a[8], at::kInt, "int32", {t.B}, mass);
  const int64_t need = bytes(t.B, p.Hkv, p.n, p.page, t.max_pages, budget);
  if (need < 0) return PyLong_FromLongLong(need);
  const Workspace ws = workspace_of(a[9], need, mass);
  void* stream = stream_of(device);
  const int st = unlocked([&] {
    return fn(ptr(*p.k), ptr(*p.v), static_cast<const int32_t*>(ptr(*t.pages)), static_cast<const int32_t*>(ptr(*t.lens)),
              static_cast<const float*>(ptr(mass)), static_cast<float*>(ptr(mass_out.t)),
              static_cast<int32_t*>(ptr(lens_out.t)), layout, t.B, p.Hkv, p.n, p.page, p.stride, t.max_pages, p.D,
              budget, recent, ws.p, ws.n, stream);
  });
  return answer(st, {&lens_out, &mass_out});
}

template <PyObject* (*kFn)(PyObject* const*), int kArgs>
PyObject* entry(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != kArgs) {
    PyErr_Format(PyExc_TypeError, "%d arguments wanted, %zd given", kArgs, n);
    return nullptr;
  }
  try {
    return kFn(a);
  } catch (const Refused& r) {
    PyErr_SetString(r.type, r.what.c_str());
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

template <PyObject* (*kFn)(PyObject* const*), int kArgs>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&entry<kFn, kArgs>)), METH_FASTCALL, nullptr};
}
PyMethodDef g_methods[] = {method<norm_rope, 14>("norm_rope"),
                           method<norm_rope_paged, 17>("norm_rope_paged"),
                           method<norm_rope_bwd, 20>("norm_rope_bwd"),
                           method<fwd_paged, 15>("fwd_paged"),
                           method<cache_evict, 13>("cache_evict"),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "attn_binding", nullptr, -1, g_methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" PyMODINIT_FUNC PyInit_attn_binding(void) { return PyModule_Create(&g_module); }
