// marshal.cpp - argument checks and tables of the calls whose host side would
// otherwise outlast their kernels: a step over 50 vectors takes 5 us on the
// device and took 60 to check from Python, one row's norms 3 us and 14.
//
// A Python extension module (host code only).  It reads tensors through
// torch's C++ interface, raises the same exceptions as the Python checks
// beside it, and calls the library through the addresses that the Python
// side passes.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/empty_like.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <string>
#include <vector>

#include "../../include/nsortho.h"

namespace {

constexpr int64_t kStateBlock = 256;  // elements of an 8-bit moment that share a scale

PyObject* fail(PyObject* type, const std::string& what) {
  PyErr_SetString(type, what.c_str());
  return nullptr;
}

// The ns_dtype of a tensor; -1 for another type.
int dtype_of(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return NS_BF16;
    case at::kHalf: return NS_FP16;
    case at::kFloat: return NS_FP32;
    default: return -1;
  }
}

bool tensor_of(PyObject* o, at::Tensor& t, const char* name) {
  if (!THPVariable_Check(o)) {
    fail(PyExc_TypeError, std::string(name) + " must be a tensor");
    return false;
  }
  t = THPVariable_Unpack(o);
  return true;
}

// A Python sequence, held.
struct Sequence {
  PyObject* fast = nullptr;
  explicit Sequence(PyObject* o) : fast(PySequence_Fast(o, "expects a sequence")) {}
  ~Sequence() { Py_XDECREF(fast); }
  Sequence(const Sequence&) = delete;
  Sequence& operator=(const Sequence&) = delete;
  Py_ssize_t size() const { return PySequence_Fast_GET_SIZE(fast); }
  PyObject* at(Py_ssize_t i) const { return PySequence_Fast_GET_ITEM(fast, i); }
};

// A number, or one per tensor.
struct Numbers {
  bool single = false;
  double value = 0.0;
  std::vector<double> values;
  bool read(PyObject* o, Py_ssize_t count, const char* name) {
    if (PyFloat_Check(o) || PyLong_Check(o)) {
      single = true;
      value = PyFloat_AsDouble(o);
      return !PyErr_Occurred();
    }
    Sequence s(o);
    if (!s.fast) return false;
    if (s.size() != count) {
      fail(PyExc_ValueError, std::string(name) + " must be one number or one per tensor");
      return false;
    }
    values.resize(count);
    for (Py_ssize_t i = 0; i < count; ++i) {
      values[i] = PyFloat_AsDouble(s.at(i));
      if (values[i] == -1.0 && PyErr_Occurred()) return false;
    }
    return true;
  }
  float at(Py_ssize_t i) const { return (float)(single ? value : values[i]); }
};

// adamw_table(params, grads, m, v, scales, copies, lr, weight_decay): the
// ns_adamw_tensor array of a step as bytes.  Lists of one length; scales and
// copies may be None; all tensors on the first parameter's device.
PyObject* adamw_table(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  if (nargs != 8) return fail(PyExc_TypeError, "adamw_table takes 8 arguments");
  Sequence params(args[0]), grads(args[1]), ms(args[2]), vs(args[3]);
  if (!params.fast || !grads.fast || !ms.fast || !vs.fast) return nullptr;
  const Py_ssize_t count = params.size();
  Sequence scales(args[4] == Py_None ? args[0] : args[4]), copies(args[5] == Py_None ? args[0] : args[5]);
  if (!scales.fast || !copies.fast) return nullptr;
  if (grads.size() != count || ms.size() != count || vs.size() != count)
    return fail(PyExc_ValueError, "params, grads, m and v must have one entry per tensor");
  if (scales.size() != count) return fail(PyExc_ValueError, "scales must have one entry (or None) per tensor");
  if (copies.size() != count) return fail(PyExc_ValueError, "copies must have one entry (or None) per tensor");
  Numbers lr, decay;
  if (!lr.read(args[6], count, "lr") || !decay.read(args[7], count, "weight_decay")) return nullptr;
  PyObject* out = PyBytes_FromStringAndSize(nullptr, (Py_ssize_t)sizeof(ns_adamw_tensor) * count);
  if (!out) return nullptr;
  struct Drop {
    PyObject* o;
    ~Drop() { Py_XDECREF(o); }
  } drop{out};
  ns_adamw_tensor* table = reinterpret_cast<ns_adamw_tensor*>(PyBytes_AS_STRING(out));
  std::vector<const void*> written;
  written.reserve(5 * count);
  at::Tensor p, g, m, v, s, c;
  at::Device device(at::kCPU);
  for (Py_ssize_t i = 0; i < count; ++i) {
    if (!tensor_of(params.at(i), p, "params") || !tensor_of(grads.at(i), g, "grads") || !tensor_of(ms.at(i), m, "m") ||
        !tensor_of(vs.at(i), v, "v"))
      return nullptr;
    if (i == 0) device = p.device();
    const at::Tensor* all[] = {&p, &g, &m, &v};
    for (const at::Tensor* t : all) {
      if (!t->is_cuda() || t->device() != device) return fail(PyExc_ValueError, "every tensor must be on one device");
      if (!t->is_contiguous()) return fail(PyExc_ValueError, "every tensor must be contiguous");
    }
    const int pt = dtype_of(p), gt = dtype_of(g);
    if (pt < 0 || gt < 0) return fail(PyExc_TypeError, "params and grads must be bf16, fp16 or fp32");
    const bool coded = m.scalar_type() == at::kFloat8_e4m3fn;
    if ((!coded && m.scalar_type() != at::kFloat) || v.scalar_type() != m.scalar_type())
      return fail(PyExc_TypeError, "m and v must both be float32 or both float8_e4m3fn");
    const int64_t n = p.numel();
    if (g.sizes() != p.sizes()) return fail(PyExc_ValueError, "grads must have their parameters' shapes");
    if (m.numel() != n || v.numel() != n)
      return fail(PyExc_ValueError, "m and v must have as many elements as their parameters");
    ns_adamw_tensor& e = table[i];
    e.scales = nullptr;
    e.copy = nullptr;
    e.copy_dtype = NS_BF16;
    PyObject* so = args[4] == Py_None ? Py_None : scales.at(i);
    if ((so != Py_None) != coded)
      return fail(PyExc_ValueError, "scales go with float8_e4m3fn moments, one tensor each");
    if (coded) {
      if (!tensor_of(so, s, "scales")) return nullptr;
      if (s.scalar_type() != at::kFloat || s.numel() != 2 * ((n + kStateBlock - 1) / kStateBlock) ||
          s.device() != device || !s.is_contiguous())
        return fail(PyExc_ValueError, "scales must be contiguous float32 tensors [2, ceil(numel / 256)] on the device");
      e.scales = static_cast<float*>(s.data_ptr());
    }
    PyObject* co = args[5] == Py_None ? Py_None : copies.at(i);
    if (co != Py_None) {
      if (!tensor_of(co, c, "copies")) return nullptr;
      const int ct = dtype_of(c);
      if (ct < 0 || c.sizes() != p.sizes() || c.device() != device || !c.is_contiguous())
        return fail(PyExc_ValueError, "copies must be contiguous bf16, fp16 or fp32 tensors of their parameter's shape");
      e.copy = c.data_ptr();
      e.copy_dtype = (ns_dtype)ct;
    }
    e.param = p.data_ptr();
    e.grad = g.data_ptr();
    e.exp_avg = m.data_ptr();
    e.exp_avg_sq = v.data_ptr();
    e.numel = n;
    e.lr = lr.at(i);
    e.weight_decay = decay.at(i);
    e.param_dtype = (ns_dtype)pt;
    e.grad_dtype = (ns_dtype)gt;
    e.reserved = 0;
    if (n > 0) {
      written.insert(written.end(), {e.param, e.exp_avg, e.exp_avg_sq});
      if (e.scales) written.push_back(e.scales);
      if (e.copy) written.push_back(e.copy);
    }
  }
  std::sort(written.begin(), written.end());
  if (std::adjacent_find(written.begin(), written.end()) != written.end())
    return fail(PyExc_ValueError, "a tensor is given twice");
  drop.o = nullptr;
  return out;
  END_HANDLE_TH_ERRORS
}

// ---------------------------------------------------------------------------
// Residual norms.
// ---------------------------------------------------------------------------

// A tensor seen as a matrix of its last axis: 2-D with contiguous rows, or
// contiguous of any rank.
struct Rows {
  int64_t rows = 0, cols = 0, ld = 0;
  bool read(const at::Tensor& t, const char* name) {
    const auto sizes = t.sizes();
    auto bad = [&](const char* what) {
      fail(PyExc_ValueError, std::string(name) + what);
      return false;
    };
    if (sizes.empty()) return bad(" must have at least one axis");
    cols = sizes.back();
    if (cols < 1) return bad("'s last axis must not be empty");
    rows = t.numel() / cols;
    ld = cols;
    if (t.is_contiguous()) return true;
    if (sizes.size() != 2) return bad(" must be contiguous (or 2-D)");
    if (t.stride(1) != 1 && cols > 1) return bad("'s rows must be contiguous (stride(-1) == 1)");
    if (rows > 1 && t.stride(0) < cols) return bad("'s rows must not overlap");
    if (rows > 1) ld = t.stride(0);
    return true;
  }
};

// A tensor of x's shape, type and device; its row stride.
bool like(const at::Tensor& t, const at::Tensor& x, const char* name, int64_t& ld) {
  if (t.sizes() != x.sizes() || t.scalar_type() != x.scalar_type() || t.device() != x.device()) {
    fail(PyExc_ValueError, std::string(name) + " must have the shape, dtype and device of the other tensors");
    return false;
  }
  Rows r;
  if (!r.read(t, name)) return false;
  ld = r.ld;
  return true;
}

using ResidualNorm = ns_status (*)(const void*, int64_t, const void*, int64_t, int64_t, int64_t, ns_dtype, const void*,
                                   int64_t, const void*, const void*, ns_dtype, float, int32_t, float, void*, int64_t,
                                   void*, int64_t, float*, float*, int32_t*, ns_stream_t);

// residual_norm(address, residual, branch, gate, scale, branch_weight, weight,
// norm_branch, norm_out, eps, stats, out, out_norm, status pointer, stream):
// (stream, normed, branch_rstd, rstd), or the call's status where it is not
// NS_OK.  The caller has made the tensors' device the current one.
PyObject* residual_norm(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  if (nargs != 15) return fail(PyExc_TypeError, "residual_norm takes 15 arguments");
  const ResidualNorm fn = reinterpret_cast<ResidualNorm>(PyLong_AsVoidPtr(args[0]));
  at::Tensor x, z, gate, wb, w, s, y, rb, rs;
  if (!tensor_of(args[1], x, "residual")) return nullptr;
  Rows r;
  if (!r.read(x, "residual")) return nullptr;
  const int dt = dtype_of(x);
  if (dt < 0) return fail(PyExc_TypeError, "unsupported dtype; use bf16, fp16 or fp32");
  const bool has_z = args[2] != Py_None;
  const double scale = PyFloat_AsDouble(args[4]), eps = PyFloat_AsDouble(args[9]);
  const int norm_branch = PyObject_IsTrue(args[7]), norm_out = PyObject_IsTrue(args[8]), stats = PyObject_IsTrue(args[10]);
  if (PyErr_Occurred()) return nullptr;
  if (!has_z) {
    if (args[3] != Py_None || args[5] != Py_None || args[11] != Py_None || scale != 1.0)
      return fail(PyExc_ValueError, "gate, branch_weight, out and scale go with a branch");
    if (!norm_out) return fail(PyExc_ValueError, "nothing to compute");
  }
  int64_t ldz = 0, lds = 0, ldy = 0, groups = 0;
  if (has_z && (!tensor_of(args[2], z, "branch") || !like(z, x, "branch", ldz))) return nullptr;
  // The gate and the weights have one type, x's or float32.
  int pt = -1;
  auto param = [&](PyObject* o, at::Tensor& t, const char* name) {
    if (!tensor_of(o, t, name)) return false;
    const int type = dtype_of(t);
    if (type != dt && type != NS_FP32) {
      fail(PyExc_TypeError, std::string(name) + " must have the data's dtype or float32");
      return false;
    }
    if (pt >= 0 && type != pt) {
      fail(PyExc_TypeError, "gate, branch_weight and weight must have the same dtype");
      return false;
    }
    pt = type;
    if (t.device() != x.device() || !t.is_contiguous() || t.dim() < 1) {
      fail(PyExc_ValueError, std::string(name) + " must be contiguous and on the data's device");
      return false;
    }
    return true;
  };
  if (args[3] != Py_None) {
    if (!param(args[3], gate, "gate")) return nullptr;
    if (gate.size(-1) != r.cols) return fail(PyExc_ValueError, "gate's last axis must be as long as the data's");
    groups = gate.numel() / r.cols;
    if (groups < 1 || (r.rows && (groups > r.rows || r.rows % groups)))
      return fail(PyExc_ValueError, "gate must have rows that divide the data's");
  }
  for (auto [o, t, name] : {std::tuple<PyObject*, at::Tensor*, const char*>{args[5], &wb, "branch_weight"},
                            {args[6], &w, "weight"}}) {
    if (o == Py_None) continue;
    if (!param(o, *t, name)) return nullptr;
    if (t->numel() != r.cols) return fail(PyExc_ValueError, std::string(name) + " must have one element per column");
  }
  auto output = [&](PyObject* o, at::Tensor& t, const char* name, int64_t& ld) {
    if (o != Py_None) return tensor_of(o, t, name) && like(t, x, name, ld);
    t = x.is_contiguous() ? at::empty_like(x) : at::empty(x.sizes(), x.options());
    ld = r.cols;
    return true;
  };
  if (has_z && !output(args[11], s, "out", lds)) return nullptr;
  if (norm_out && !output(args[12], y, "out_norm", ldy)) return nullptr;
  const auto lead = x.sizes().slice(0, x.dim() - 1);
  if (stats && has_z && norm_branch) rb = at::empty(lead, x.options().dtype(at::kFloat));
  if (stats && norm_out) rs = at::empty(lead, x.options().dtype(at::kFloat));
  auto ptr = [](const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; };
  const ns_status st = fn(x.data_ptr(), r.ld, ptr(z), ldz, r.rows, r.cols, (ns_dtype)dt, ptr(gate), groups, ptr(wb), ptr(w),
                          (ns_dtype)(pt < 0 ? dt : pt), (float)scale, norm_branch, (float)eps, ptr(s), lds, ptr(y), ldy,
                          static_cast<float*>(ptr(rb)), static_cast<float*>(ptr(rs)),
                          static_cast<int32_t*>(args[13] == Py_None ? nullptr : PyLong_AsVoidPtr(args[13])),
                          PyLong_AsVoidPtr(args[14]));
  if (PyErr_Occurred()) return nullptr;
  if (st != NS_OK) return PyLong_FromLong(st);
  PyObject* out = PyTuple_New(4);
  if (!out) return nullptr;
  auto give = [&](int i, PyObject* given, const at::Tensor& t) {
    PyObject* o = given != Py_None ? given : t.defined() ? THPVariable_Wrap(t) : Py_None;
    if (o == given || o == Py_None) Py_INCREF(o);
    PyTuple_SET_ITEM(out, i, o);
  };
  give(0, has_z ? args[11] : args[1], s);
  give(1, norm_out ? args[12] : Py_None, y);
  give(2, Py_None, rb);
  give(3, Py_None, rs);
  return out;
  END_HANDLE_TH_ERRORS
}

PyMethodDef kMethods[] = {
    {"adamw_table", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(adamw_table)), METH_FASTCALL, nullptr},
    {"residual_norm", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(residual_norm)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_marshal", "Checks and tables of small calls.", -1, kMethods,
                       nullptr,               nullptr,    nullptr,                             nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&kModule); }
