// marshal.cpp - argument checks and tables of the calls whose host side would
// otherwise outlast their kernels.  Checked from Python, a step over 50
// vectors took 60 us of host time, one row's norms 14 and their gradients
// 22, a feed-forward block 18 and its gradients 28; the kernels of small
// calls take 3 to 20.
//
// A Python extension module (host code only).  It reads tensors through
// torch's C++ interface, raises the same exceptions as the Python checks
// beside it, and calls the library through the addresses that the Python
// side passes.  Other threads have the interpreter while it allocates or the
// library runs: either may wait for the device.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
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

// What f() gives, the interpreter left to other threads meanwhile: f touches no
// Python object.
template <class F>
auto unlocked(F&& f) {
  struct Released {
    PyThreadState* state = PyEval_SaveThread();
    ~Released() { PyEval_RestoreThread(state); }
  } released;
  return f();
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

// The same without a reference of its own, for lists of many tensors whose
// sequence holds them.
const at::Tensor* borrowed(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) {
    fail(PyExc_TypeError, std::string(name) + " must be a tensor");
    return nullptr;
  }
  return &THPVariable_Unpack(o);
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
  at::Device device(at::kCPU);
  for (Py_ssize_t i = 0; i < count; ++i) {
    const at::Tensor *pp = borrowed(params.at(i), "params"), *gp = pp ? borrowed(grads.at(i), "grads") : nullptr,
                     *mp = gp ? borrowed(ms.at(i), "m") : nullptr, *vp = mp ? borrowed(vs.at(i), "v") : nullptr;
    if (!vp) return nullptr;
    const at::Tensor &p = *pp, &g = *gp, &m = *mp, &v = *vp;
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
      const at::Tensor* s = borrowed(so, "scales");
      if (!s) return nullptr;
      if (s->scalar_type() != at::kFloat || s->numel() != 2 * ((n + kStateBlock - 1) / kStateBlock) ||
          s->device() != device || !s->is_contiguous())
        return fail(PyExc_ValueError, "scales must be contiguous float32 tensors [2, ceil(numel / 256)] on the device");
      e.scales = static_cast<float*>(s->data_ptr());
    }
    PyObject* co = args[5] == Py_None ? Py_None : copies.at(i);
    if (co != Py_None) {
      const at::Tensor* c = borrowed(co, "copies");
      if (!c) return nullptr;
      const int ct = dtype_of(*c);
      if (ct < 0 || c->sizes() != p.sizes() || c->device() != device || !c->is_contiguous())
        return fail(PyExc_ValueError, "copies must be contiguous bf16, fp16 or fp32 tensors of their parameter's shape");
      e.copy = c->data_ptr();
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
// Tensors as matrices.
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

// A tensor of the given shape, type and x's device; its row stride.
bool shaped(const at::Tensor& t, at::IntArrayRef sizes, at::ScalarType type, const at::Tensor& x, const char* name,
            int64_t& ld) {
  if (t.sizes() != sizes || t.scalar_type() != type || t.device() != x.device()) {
    fail(PyExc_ValueError, std::string(name) + " must have the shape, dtype and device that go with the other tensors");
    return false;
  }
  Rows r;
  if (!r.read(t, name)) return false;
  ld = r.ld;
  return true;
}

// A tensor of x's shape, type and device; its row stride.
bool like(const at::Tensor& t, const at::Tensor& x, const char* name, int64_t& ld) {
  return shaped(t, x.sizes(), x.scalar_type(), x, name, ld);
}

// The tensor to write if it is given (else it is made later), and its row stride.
bool output(PyObject* o, at::Tensor& t, at::IntArrayRef sizes, const at::Tensor& x, const char* name, int64_t& ld) {
  if (o != Py_None) return tensor_of(o, t, name) && shaped(t, sizes, x.scalar_type(), x, name, ld);
  ld = sizes.back();
  return true;
}
void make(at::Tensor& t, at::IntArrayRef sizes, const at::Tensor& x) {
  if (!t.defined()) t = at::empty(sizes, x.options());
}

// A parameter of x's type or float32, of one type with those before it
// (code, -1 before the first).
bool param_of(PyObject* o, at::Tensor& t, const at::Tensor& x, int& code, const char* name) {
  if (!tensor_of(o, t, name)) return false;
  const int type = dtype_of(t);
  if (t.scalar_type() != x.scalar_type() && type != NS_FP32) {
    fail(PyExc_TypeError, std::string(name) + " must have the data's dtype or float32");
    return false;
  }
  if (code >= 0 && type != code) {
    fail(PyExc_TypeError, "gate, branch_weight and weight must have the same dtype");
    return false;
  }
  code = type;
  if (t.device() != x.device() || !t.is_contiguous() || t.dim() < 1) {
    fail(PyExc_ValueError, std::string(name) + " must be contiguous and on the data's device");
    return false;
  }
  return true;
}

// The gate of a residual norm: its rows divide the data's.
bool gate_of(PyObject* o, at::Tensor& t, const at::Tensor& x, const Rows& r, int& code, int64_t& groups) {
  if (!param_of(o, t, x, code, "gate")) return false;
  if (t.size(-1) != r.cols) {
    fail(PyExc_ValueError, "gate's last axis must be as long as the data's");
    return false;
  }
  groups = t.numel() / r.cols;
  if (groups < 1 || (r.rows && (groups > r.rows || r.rows % groups))) {
    fail(PyExc_ValueError, "gate must have rows that divide the data's");
    return false;
  }
  return true;
}

// One weight per column.
bool weight_of(PyObject* o, at::Tensor& t, const at::Tensor& x, const Rows& r, int& code, const char* name) {
  if (!param_of(o, t, x, code, name)) return false;
  if (t.numel() != r.cols) {
    fail(PyExc_ValueError, std::string(name) + " must have one element per column");
    return false;
  }
  return true;
}

// A statistic of each row.
bool per_row(PyObject* o, at::Tensor& t, const at::Tensor& x, const Rows& r, const char* name) {
  if (!tensor_of(o, t, name)) return false;
  if (t.scalar_type() != at::kFloat) {
    fail(PyExc_TypeError, std::string(name) + " must be float32");
    return false;
  }
  if (t.device() != x.device() || t.numel() != r.rows || !t.is_contiguous()) {
    fail(PyExc_ValueError, std::string(name) + " must be contiguous, one element per row, on the data's device");
    return false;
  }
  return true;
}

// A workspace of the caller's, or of torch's once it is made, 256-byte aligned.
struct Workspace {
  at::Tensor held;
  void* ptr = nullptr;
  size_t bytes = 0;
  bool check(PyObject* o, const at::Tensor& x) {
    if (o == Py_None) return true;
    if (!tensor_of(o, held, "workspace")) return false;
    if (held.device() != x.device() || !held.is_contiguous()) {
      fail(PyExc_ValueError, "workspace must be contiguous and on the data's device");
      return false;
    }
    return true;
  }
  void take(size_t need, const at::Tensor& x) {
    if (!held.defined()) held = at::empty({(int64_t)need + 256}, x.options().dtype(at::kByte));
    const uintptr_t at = reinterpret_cast<uintptr_t>(held.data_ptr());
    const size_t pad = (size_t)(-at & 255), all = (size_t)held.numel() * held.element_size();
    ptr = reinterpret_cast<void*>(at + pad);
    bytes = all > pad ? all - pad : 0;
  }
};

void* data(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }

template <class T>
T address(PyObject* o) {
  return reinterpret_cast<T>(o == Py_None ? nullptr : PyLong_AsVoidPtr(o));
}

// A tuple entry: the caller's tensor, one made here, or None.
void give(PyObject* out, int i, PyObject* given, const at::Tensor& t) {
  PyObject* o = given != Py_None ? given : t.defined() ? THPVariable_Wrap(t) : Py_None;
  if (o == given || o == Py_None) Py_INCREF(o);
  PyTuple_SET_ITEM(out, i, o);
}

// ---------------------------------------------------------------------------
// Residual norms.
// ---------------------------------------------------------------------------

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
  const auto fn = address<ResidualNorm>(args[0]);
  const auto status = address<int32_t*>(args[13]);
  const auto stream = address<void*>(args[14]);
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
  int pt = -1;
  if (args[3] != Py_None && !gate_of(args[3], gate, x, r, pt, groups)) return nullptr;
  if (args[5] != Py_None && !weight_of(args[5], wb, x, r, pt, "branch_weight")) return nullptr;
  if (args[6] != Py_None && !weight_of(args[6], w, x, r, pt, "weight")) return nullptr;
  if (has_z && !output(args[11], s, x.sizes(), x, "out", lds)) return nullptr;
  if (norm_out && !output(args[12], y, x.sizes(), x, "out_norm", ldy)) return nullptr;
  const ns_status st = unlocked([&] {
    const auto lead = x.sizes().slice(0, x.dim() - 1);
    if (has_z) make(s, x.sizes(), x);
    if (norm_out) make(y, x.sizes(), x);
    if (stats && has_z && norm_branch) rb = at::empty(lead, x.options().dtype(at::kFloat));
    if (stats && norm_out) rs = at::empty(lead, x.options().dtype(at::kFloat));
    return fn(x.data_ptr(), r.ld, data(z), ldz, r.rows, r.cols, (ns_dtype)dt, data(gate), groups, data(wb), data(w),
              (ns_dtype)(pt < 0 ? dt : pt), (float)scale, norm_branch, (float)eps, data(s), lds, data(y), ldy,
              static_cast<float*>(data(rb)), static_cast<float*>(data(rs)), status, stream);
  });
  if (st != NS_OK) return PyLong_FromLong(st);
  PyObject* out = PyTuple_New(4);
  if (!out) return nullptr;
  give(out, 0, has_z ? args[11] : args[1], s);
  give(out, 1, norm_out ? args[12] : Py_None, y);
  give(out, 2, Py_None, rb);
  give(out, 3, Py_None, rs);
  return out;
  END_HANDLE_TH_ERRORS
}

using WorkspaceSize2 = size_t (*)(int64_t, int64_t);
using ResidualNormBackward = ns_status (*)(const void*, int64_t, const void*, int64_t, const void*, int64_t, const void*,
                                           int64_t, int64_t, int64_t, ns_dtype, const float*, const float*, const void*,
                                           int64_t, const void*, const void*, ns_dtype, float, void*, int64_t, void*,
                                           int64_t, void*, void*, void*, int32_t*, void*, size_t, ns_stream_t);

// residual_norm_backward(address, workspace query's address, dstream, dnormed,
// stream, branch, branch_rstd, rstd, gate, scale, branch_weight, weight,
// params, out, out_branch, workspace, status pointer, stream handle):
// (dresidual, dbranch, dgate, dbranch_weight, dweight), or the status.
PyObject* residual_norm_backward(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  if (nargs != 18) return fail(PyExc_TypeError, "residual_norm_backward takes 18 arguments");
  const auto fn = address<ResidualNormBackward>(args[0]);
  const auto query = address<WorkspaceSize2>(args[1]);
  const auto status = address<int32_t*>(args[16]);
  const auto handle = address<void*>(args[17]);
  at::Tensor ds, dy, s, z, rb, rs, gate, wb, w, dx, dz, dgate, dwb, dw;
  if (!tensor_of(args[4], s, "stream")) return nullptr;
  Rows r;
  if (!r.read(s, "stream")) return nullptr;
  const int dt = dtype_of(s);
  if (dt < 0) return fail(PyExc_TypeError, "unsupported dtype; use bf16, fp16 or fp32");
  const double scale = PyFloat_AsDouble(args[9]);
  const int params = PyObject_IsTrue(args[12]);
  if (PyErr_Occurred()) return nullptr;
  const bool has_s = args[2] != Py_None, has_y = args[3] != Py_None, has_z = args[5] != Py_None;
  if (!has_s && !has_y) return fail(PyExc_ValueError, "dstream or dnormed must be given");
  int64_t ldds = 0, lddy = 0, ldz = 0, lddx = 0, lddz = 0, groups = 0;
  if (has_s && (!tensor_of(args[2], ds, "dstream") || !like(ds, s, "dstream", ldds))) return nullptr;
  if (has_y) {
    if (!tensor_of(args[3], dy, "dnormed") || !like(dy, s, "dnormed", lddy)) return nullptr;
    if (args[7] == Py_None) return fail(PyExc_ValueError, "dnormed needs rstd");
    if (!per_row(args[7], rs, s, r, "rstd")) return nullptr;
  } else if (args[11] != Py_None) {
    return fail(PyExc_ValueError, "weight goes with dnormed");
  }
  if (!has_z) {
    if (args[8] != Py_None || args[10] != Py_None || args[6] != Py_None || scale != 1.0)
      return fail(PyExc_ValueError, "gate, branch_weight, branch_rstd and scale go with a branch");
    if (args[14] != Py_None) return fail(PyExc_ValueError, "out_branch goes with a branch");
  }
  if (has_z && (!tensor_of(args[5], z, "branch") || !like(z, s, "branch", ldz))) return nullptr;
  if (args[6] != Py_None && !per_row(args[6], rb, s, r, "branch_rstd")) return nullptr;
  int pt = -1;
  if (args[8] != Py_None && !gate_of(args[8], gate, s, r, pt, groups)) return nullptr;
  if (args[10] != Py_None && !weight_of(args[10], wb, s, r, pt, "branch_weight")) return nullptr;
  if (args[11] != Py_None && !weight_of(args[11], w, s, r, pt, "weight")) return nullptr;
  if (!output(args[13], dx, s.sizes(), s, "out", lddx)) return nullptr;
  if (has_z && !output(args[14], dz, s.sizes(), s, "out_branch", lddz)) return nullptr;
  const size_t need = query(r.rows, r.cols);
  if (need == 0) return PyLong_FromLong(NS_ERR_INVALID_ARG);
  Workspace ws;
  if (!ws.check(args[15], s)) return nullptr;
  const ns_status st = unlocked([&] {
    make(dx, s.sizes(), s);
    if (has_z) make(dz, s.sizes(), s);
    if (params && gate.defined()) make(dgate, gate.sizes(), gate);
    if (params && wb.defined()) make(dwb, wb.sizes(), wb);
    if (params && w.defined()) make(dw, w.sizes(), w);
    ws.take(need, s);
    return fn(data(ds), ldds, data(dy), lddy, s.data_ptr(), r.ld, data(z), ldz, r.rows, r.cols, (ns_dtype)dt,
              static_cast<float*>(data(rb)), static_cast<float*>(data(rs)), data(gate), groups, data(wb), data(w),
              (ns_dtype)(pt < 0 ? dt : pt), (float)scale, dx.data_ptr(), lddx, data(dz), lddz, data(dgate), data(dwb),
              data(dw), status, ws.ptr, ws.bytes, handle);
  });
  if (st != NS_OK) return PyLong_FromLong(st);
  PyObject* out = PyTuple_New(5);
  if (!out) return nullptr;
  give(out, 0, args[13], dx);
  give(out, 1, has_z ? args[14] : Py_None, dz);
  give(out, 2, Py_None, dgate);
  give(out, 3, Py_None, dwb);
  give(out, 4, Py_None, dw);
  return out;
  END_HANDLE_TH_ERRORS
}

// ---------------------------------------------------------------------------
// The gated feed-forward block.
// ---------------------------------------------------------------------------

using MlpWorkspaceSize = size_t (*)(int64_t, int64_t, int64_t, ns_dtype, int32_t, int32_t);
using GatedMlp = ns_status (*)(const void*, int64_t, const void*, int64_t, const void*, int64_t, const void*, int64_t,
                               int64_t, int64_t, int64_t, ns_dtype, ns_activation, void*, int64_t, void*, void*, int64_t,
                               ns_dtype, int32_t*, void*, size_t, ns_stream_t);
using GatedMlpBackward = ns_status (*)(const void*, int64_t, const void*, int64_t, const void*, int64_t, const void*,
                                       int64_t, const void*, int64_t, const void*, const void*, int64_t, ns_dtype, int64_t,
                                       int64_t, int64_t, ns_dtype, ns_activation, void*, int64_t, void*, int64_t, void*,
                                       int64_t, void*, int64_t, int32_t*, void*, size_t, ns_stream_t);

// x and the matrices of a block.
struct Block {
  at::Tensor x, wg, wu, wd;
  Rows r;
  int dt = -1;
  int64_t inner = 0, ldg = 0, ldu = 0, ldd = 0;
  bool read(PyObject* const* args) {
    if (!tensor_of(args[0], x, "x") || !tensor_of(args[1], wg, "w_gate") || !tensor_of(args[2], wu, "w_up") ||
        !tensor_of(args[3], wd, "w_down") || !r.read(x, "x"))
      return false;
    dt = dtype_of(x);
    if (dt < 0) {
      fail(PyExc_TypeError, "unsupported dtype; use bf16, fp16 or fp32");
      return false;
    }
    if (wg.dim() != 2 || wu.dim() != 2 || wd.dim() != 2) {
      fail(PyExc_ValueError, "w_gate, w_up and w_down must be 2-D");
      return false;
    }
    inner = wg.size(0);
    if (inner < 1 || wg.size(1) != r.cols || wu.sizes() != wg.sizes() || wd.size(0) != r.cols || wd.size(1) != inner) {
      fail(PyExc_ValueError, "w_gate and w_up must be [inner, cols] and w_down [cols, inner]");
      return false;
    }
    return shaped(wg, wg.sizes(), x.scalar_type(), x, "w_gate", ldg) &&
           shaped(wu, wu.sizes(), x.scalar_type(), x, "w_up", ldu) &&
           shaped(wd, wd.sizes(), x.scalar_type(), x, "w_down", ldd);
  }
  // [..., inner]
  at::DimVector hidden() const {
    at::DimVector sizes(x.sizes().begin(), x.sizes().end());
    sizes.back() = inner;
    return sizes;
  }
};

// Whether an operand starts on 16 bytes and steps by whole 128.
bool aligned(const at::Tensor& t, int64_t ld) {
  return reinterpret_cast<uintptr_t>(t.data_ptr()) % 16 == 0 && ld * (int64_t)t.element_size() % 128 == 0;
}

// gated_mlp(address, workspace query's address, x, w_gate, w_up, w_down,
// activation, save (None, False for x's type, True for float32), out,
// workspace, status pointer, stream): (y, gate, up), or the status.
PyObject* gated_mlp(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  if (nargs != 12) return fail(PyExc_TypeError, "gated_mlp takes 12 arguments");
  const auto fn = address<GatedMlp>(args[0]);
  const auto query = address<MlpWorkspaceSize>(args[1]);
  const auto status = address<int32_t*>(args[10]);
  const auto stream = address<void*>(args[11]);
  Block b;
  if (!b.read(args + 2)) return nullptr;
  const auto act = (ns_activation)PyLong_AsLong(args[6]);
  if (PyErr_Occurred()) return nullptr;
  at::Tensor y, gate, up;
  int64_t ldy = 0;
  if (!output(args[8], y, b.x.sizes(), b.x, "out", ldy)) return nullptr;
  int st_code = NS_FP32;
  const bool saved = args[7] != Py_None;
  const auto save_type = args[7] == Py_True ? at::kFloat : b.x.scalar_type();
  if (saved) st_code = save_type == at::kFloat ? (int)NS_FP32 : b.dt;
  const int64_t ktile = 128 / (int64_t)b.x.element_size();
  const bool even = (b.r.cols % ktile || (b.ldg == b.ldu && aligned(b.x, b.r.ld) && aligned(b.wg, b.ldg) &&
                                          aligned(b.wu, b.ldu))) &&
                    (b.inner % ktile || aligned(b.wd, b.ldd));
  const size_t need = query(b.r.rows, b.r.cols, b.inner, (ns_dtype)b.dt, even, 0);
  if (need == 0) return PyLong_FromLong(NS_ERR_INVALID_ARG);
  Workspace ws;
  if (!ws.check(args[9], b.x)) return nullptr;
  const ns_status st = unlocked([&] {
    make(y, b.x.sizes(), b.x);
    if (saved) {
      const auto sizes = b.hidden();
      gate = at::empty(sizes, b.x.options().dtype(save_type));
      up = at::empty(sizes, b.x.options().dtype(save_type));
    }
    ws.take(need, b.x);
    return fn(b.x.data_ptr(), b.r.ld, b.wg.data_ptr(), b.ldg, b.wu.data_ptr(), b.ldu, b.wd.data_ptr(), b.ldd, b.r.rows,
              b.r.cols, b.inner, (ns_dtype)b.dt, act, y.data_ptr(), ldy, data(gate), data(up), b.inner, (ns_dtype)st_code,
              status, ws.ptr, ws.bytes, stream);
  });
  if (st != NS_OK) return PyLong_FromLong(st);
  PyObject* out = PyTuple_New(3);
  if (!out) return nullptr;
  give(out, 0, args[8], y);
  give(out, 1, Py_None, gate);
  give(out, 2, Py_None, up);
  return out;
  END_HANDLE_TH_ERRORS
}

// gated_mlp_backward(address, workspace query's address, x, w_gate, w_up,
// w_down, dy, gate, up, activation, need_dx, need_dw, out_dx, out_dw_gate,
// out_dw_up, out_dw_down, workspace, status pointer, stream):
// (dx, dw_gate, dw_up, dw_down), or the status.
PyObject* gated_mlp_backward(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
  HANDLE_TH_ERRORS
  if (nargs != 19) return fail(PyExc_TypeError, "gated_mlp_backward takes 19 arguments");
  const auto fn = address<GatedMlpBackward>(args[0]);
  const auto query = address<MlpWorkspaceSize>(args[1]);
  const auto status = address<int32_t*>(args[17]);
  const auto stream = address<void*>(args[18]);
  Block b;
  if (!b.read(args + 2)) return nullptr;
  at::Tensor dy, gate, up, dx, dwg, dwu, dwd;
  int64_t lddy = 0, lds = 0, ldu = 0, lddx = 0, lddg = 0, lddu = 0, lddd = 0;
  if (!tensor_of(args[6], dy, "dy") || !like(dy, b.x, "dy", lddy) || !tensor_of(args[7], gate, "gate") ||
      !tensor_of(args[8], up, "up"))
    return nullptr;
  const auto act = (ns_activation)PyLong_AsLong(args[9]);
  const int need_dx = PyObject_IsTrue(args[10]), need_dw = PyObject_IsTrue(args[11]);
  if (PyErr_Occurred()) return nullptr;
  const auto type = gate.scalar_type();
  if (type != at::kFloat && type != b.x.scalar_type())
    return fail(PyExc_TypeError, "gate and up must be float32 or have x's dtype");
  const auto sizes = b.hidden();
  if (!shaped(gate, sizes, type, b.x, "gate", lds) || !shaped(up, sizes, type, b.x, "up", ldu)) return nullptr;
  if (lds != ldu) return fail(PyExc_ValueError, "gate and up must have the same row stride");
  if (need_dx && !output(args[12], dx, b.x.sizes(), b.x, "out_dx", lddx)) return nullptr;
  if (need_dw && (!output(args[13], dwg, b.wg.sizes(), b.x, "out_dw_gate", lddg) ||
                  !output(args[14], dwu, b.wu.sizes(), b.x, "out_dw_up", lddu) ||
                  !output(args[15], dwd, b.wd.sizes(), b.x, "out_dw_down", lddd)))
    return nullptr;
  const size_t need = query(b.r.rows, b.r.cols, b.inner, (ns_dtype)b.dt, aligned(dy, lddy), 1);
  if (need == 0) return PyLong_FromLong(NS_ERR_INVALID_ARG);
  Workspace ws;
  if (!ws.check(args[16], b.x)) return nullptr;
  const ns_status st = unlocked([&] {
    if (need_dx) make(dx, b.x.sizes(), b.x);
    if (need_dw) {
      make(dwg, b.wg.sizes(), b.x);
      make(dwu, b.wu.sizes(), b.x);
      make(dwd, b.wd.sizes(), b.x);
    }
    ws.take(need, b.x);
    return fn(dy.data_ptr(), lddy, b.x.data_ptr(), b.r.ld, b.wg.data_ptr(), b.ldg, b.wu.data_ptr(), b.ldu,
              b.wd.data_ptr(), b.ldd, gate.data_ptr(), up.data_ptr(), lds, (ns_dtype)dtype_of(gate), b.r.rows, b.r.cols,
              b.inner, (ns_dtype)b.dt, act, data(dx), lddx, data(dwg), lddg, data(dwu), lddu, data(dwd), lddd, status,
              ws.ptr, ws.bytes, stream);
  });
  if (st != NS_OK) return PyLong_FromLong(st);
  PyObject* out = PyTuple_New(4);
  if (!out) return nullptr;
  give(out, 0, need_dx ? args[12] : Py_None, dx);
  give(out, 1, need_dw ? args[13] : Py_None, dwg);
  give(out, 2, need_dw ? args[14] : Py_None, dwu);
  give(out, 3, need_dw ? args[15] : Py_None, dwd);
  return out;
  END_HANDLE_TH_ERRORS
}

#define NS_METHOD(name) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}

PyMethodDef kMethods[] = {NS_METHOD(adamw_table),
                          NS_METHOD(residual_norm),
                          NS_METHOD(residual_norm_backward),
                          NS_METHOD(gated_mlp),
                          NS_METHOD(gated_mlp_backward),
                          {nullptr, nullptr, 0, nullptr}};

PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_marshal", "Checks and tables of small calls.", -1, kMethods,
                       nullptr,               nullptr,    nullptr,                             nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__marshal() { return PyModule_Create(&kModule); }
