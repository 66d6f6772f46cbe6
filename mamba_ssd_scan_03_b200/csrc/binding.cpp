// binding.cpp -- the Python binding of the served forms and the norm (include/ssd.h) as a CPython
// extension: checks tensors, allocates outputs and workspace with PyTorch, and passes raw
// pointers plus the current CUDA stream.  A token's call is mostly host time: the same checks
// through ctypes took 13 to 17 us a call, here 6 to 7.  No kernel and no computation is here; the C
// entries are looked up in the library that the package has loaded.
#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <dlfcn.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "../../include/ssd.h"

namespace {

struct Refused {  // a Python exception to raise
  PyObject* type;
  std::string what;
};
[[noreturn]] void refuse(PyObject* type, const std::string& what) { throw Refused{type, what}; }

#define SSD_ENTRIES(X)                                                                         \
  X(ssd_conv_silu_varlen) X(ssd_conv_silu_step) X(ssd_selective_varlen_workspace_size)         \
  X(ssd_selective_scan_varlen) X(ssd_selective_step) X(ssd_group_norm_gate)                    \
  X(ssd_group_norm_gate_bwd_workspace_size) X(ssd_group_norm_gate_bwd)
#define X(name) decltype(&::name) p_##name = nullptr;
SSD_ENTRIES(X)
#undef X

std::string shape_text(at::IntArrayRef s) {
  std::string t = "(";
  for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
  return t + (s.size() == 1 ? ",)" : ")");
}

bool given(PyObject* o) { return o != Py_None; }
const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o))
    refuse(PyExc_TypeError, std::string(name) + " must be a torch.Tensor");
  return THPVariable_Unpack(o);
}
// The tensor whose device and shape the others follow.
const at::Tensor& first(PyObject* o, const char* name, int64_t ndim) {
  const at::Tensor& t = tensor(o, name);
  if (!t.is_cuda()) refuse(PyExc_ValueError, std::string(name) + " must be a CUDA tensor");
  if (t.dim() != ndim)
    refuse(PyExc_ValueError, std::string(name) + " must have " + std::to_string(ndim) +
                                 " dimensions, got " + shape_text(t.sizes()));
  return t;
}
ssd_dtype code(const at::Tensor& t, const char* name) {
  if (t.scalar_type() == at::kBFloat16) return SSD_BF16;
  if (t.scalar_type() == at::kFloat) return SSD_F32;
  refuse(PyExc_TypeError, std::string(name) + " must be bfloat16 or float32, got " +
                              at::toString(t.scalar_type()));
}
void same_place(const at::Tensor& t, const char* name, at::IntArrayRef shape, int dev) {
  if (!t.is_cuda() || t.get_device() != dev)
    refuse(PyExc_ValueError, std::string(name) + " is on " + t.device().str() +
                                 ", expected cuda:" + std::to_string(dev));
  if (t.sizes() != shape)
    refuse(PyExc_ValueError, std::string(name) + " has shape " + shape_text(t.sizes()) +
                                 ", expected " + shape_text(shape));
}
void has_type(const at::Tensor& t, const char* name, at::ScalarType type) {
  if (t.scalar_type() != type)
    refuse(PyExc_TypeError, std::string(name) + " must be " + at::toString(type) + ", got " +
                                at::toString(t.scalar_type()));
}
// A contiguous tensor's address; NULL for None.
template <typename P = void>
P* whole(PyObject* o, const char* name, at::ScalarType type, at::IntArrayRef shape, int dev) {
  if (!given(o)) return nullptr;
  const at::Tensor& t = tensor(o, name);
  same_place(t, name, shape, dev);
  has_type(t, name, type);
  if (!t.is_contiguous())
    refuse(PyExc_ValueError, std::string(name) + " must be contiguous");
  return static_cast<P*>(t.data_ptr());
}
const float* weights(PyObject* o, const char* name, at::IntArrayRef shape, int dev) {
  if (!given(o)) refuse(PyExc_TypeError, std::string(name) + " must be a torch.Tensor");
  return whole<float>(o, name, at::kFloat, shape, dev);
}
// The row stride, in elements, of a tensor of packed rows (any row stride, the values of a row
// contiguous).
int64_t row_stride(const at::Tensor& t, const char* name, at::IntArrayRef shape, int dev) {
  same_place(t, name, shape, dev);
  int64_t width = 1;
  for (size_t k = shape.size() - 1; k > 0; --k) {
    if (shape[k] > 1 && t.stride(k) != width && t.numel() > 0)
      refuse(PyExc_ValueError,
             std::string("the values of a row of ") + name + " must be contiguous");
    width *= shape[k];
  }
  if (shape[0] <= 1 || width == 0) return width;
  if (t.stride(0) < width)
    refuse(PyExc_ValueError, std::string("the rows of ") + name + " must not overlap");
  return t.stride(0);
}
// `out` where it is given (its type is then the output's), else a new tensor.
at::Tensor output(PyObject* o, const at::Tensor& like, at::IntArrayRef shape, at::ScalarType type) {
  if (given(o)) return tensor(o, "out");
  return at::empty(shape, like.options().dtype(type).requires_grad(false));
}
at::ScalarType dtype_arg(PyObject* o) {
  if (!THPDtype_Check(o)) refuse(PyExc_TypeError, "a dtype must be a torch.dtype");
  return reinterpret_cast<THPDtype*>(o)->scalar_type;
}
int64_t int_arg(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) {
    PyErr_Clear();
    refuse(PyExc_TypeError, std::string(name) + " must be an integer");
  }
  return v;
}
int int32_arg(PyObject* o, const char* name) {
  const int64_t v = int_arg(o, name);
  if (v < INT32_MIN || v > INT32_MAX)
    refuse(PyExc_ValueError, std::string(name) + " is out of range");
  return int(v);
}
int width32(int64_t v, const char* name) {
  if (v > INT32_MAX) refuse(PyExc_ValueError, std::string(name) + " is too wide");
  return int(v);
}
bool flag_arg(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) {
    PyErr_Clear();
    refuse(PyExc_TypeError, "a flag must be a truth value");
  }
  return v != 0;
}

// A packed batch's bounds [nseq + 1] int32 and flags [nseq] (bool or uint8).
struct Seqs {
  int nseq;
  const int32_t* cu;
  const uint8_t* resume;
};
Seqs seqs(PyObject* cu, PyObject* resume, int dev) {
  Seqs s{0, nullptr, nullptr};
  const at::Tensor& c = tensor(cu, "cu_seqlens");
  if (c.dim() != 1 || c.size(0) < 1)
    refuse(PyExc_ValueError, "cu_seqlens must be a tensor of nseq + 1 bounds");
  s.nseq = width32(c.size(0) - 1, "cu_seqlens");
  s.cu = whole<int32_t>(cu, "cu_seqlens", at::kInt, c.sizes(), dev);
  if (!given(resume)) return s;
  const at::Tensor& r = tensor(resume, "resume");
  if (r.scalar_type() != at::kBool && r.scalar_type() != at::kByte)
    refuse(PyExc_TypeError, "resume must be a bool or uint8 tensor");
  s.resume = whole<uint8_t>(resume, "resume", r.scalar_type(), {s.nseq}, dev);
  return s;
}
const int32_t* slot_arg(PyObject* o, int64_t n, int dev) {
  return whole<int32_t>(o, "slots", at::kInt, {n}, dev);
}

// Makes the tensors' device current for a scope.  A workspace's size follows the current device's SMs,
// so its query stands in such a scope, as the launch does.
struct OnDevice {
  c10::cuda::OptionalCUDAGuard guard;
  explicit OnDevice(int dev) : guard(c10::Device(c10::kCUDA, dev)) {}
};
// Lets other Python threads run for a scope.
struct NoGil {
  PyThreadState* const held = PyEval_SaveThread();
  NoGil() = default;
  NoGil(const NoGil&) = delete;
  ~NoGil() { PyEval_RestoreThread(held); }
};
// Calls a C entry with the device current, on its current stream.  Other Python threads run meanwhile: a
// launch waits where the driver's queue is full, perhaps for work that one of them has to start.
template <typename F>
int on_device(int dev, const F& call) {
  const OnDevice here(dev);
  const cudaStream_t stream = c10::cuda::getCurrentCUDAStream(dev).stream();
  const NoGil others;
  return int(call(stream));
}
// The output, or the status of a call that was refused.
PyObject* result(int status, const at::Tensor& out) {
  return status ? PyLong_FromLong(status) : THPVariable_Wrap(out);
}

// conv_silu_varlen(u, w, cu_seqlens, bias, conv_state, slots, resume, out) and
// conv_silu_step(conv_state, u, w, bias, slots, out)
PyObject* conv(PyObject* ou, PyObject* ow, PyObject* ocu, PyObject* obias, PyObject* ostate,
               PyObject* oslots, PyObject* oresume, PyObject* oout, bool step) {
  const at::Tensor& u = first(ou, "u", 2);
  const int dev = u.get_device();
  const int64_t rows = u.size(0), C = u.size(1);
  const ssd_dtype io = code(u, "u");
  const at::Tensor& w = tensor(ow, "w");
  if (w.dim() != 2) refuse(PyExc_ValueError, "w must be a tensor [C, K]");
  const int64_t K = w.size(1);
  const int64_t shape[2] = {rows, C};
  const int64_t us = row_stride(u, "u", shape, dev);
  const Seqs s = step ? Seqs{0, nullptr, nullptr} : seqs(ocu, oresume, dev);
  void* state = nullptr;
  int64_t nslots = 0;
  if (given(ostate)) {
    const at::Tensor& t = tensor(ostate, "conv_state");
    if (t.dim() != 3)
      refuse(PyExc_ValueError, "conv_state must be a tensor [nslots, K-1, C]");
    state = whole(ostate, "conv_state", u.scalar_type(), {t.size(0), K - 1, C}, dev);
    if (K > 1) nslots = t.size(0);
    else state = nullptr;
    // a cache without a slot is not the same as none (its address is NULL, too)
    if (K > 1 && nslots == 0 && (step ? rows : s.nseq) > 0)
      return PyLong_FromLong(SSD_ERR_INVALID_ARG);
  }
  const float* pw = weights(ow, "w", {C, K}, dev);
  const float* bias = whole<float>(obias, "bias", at::kFloat, {C}, dev);
  const int32_t* slots = slot_arg(oslots, step ? rows : s.nseq, dev);
  const at::Tensor out = output(oout, u, shape, u.scalar_type());
  const int64_t os = row_stride(out, "out", shape, dev);
  has_type(out, "out", u.scalar_type());
  const int c32 = width32(C, "u"), k32 = width32(K, "w");
  return result(on_device(dev, [&](cudaStream_t st) {
                  if (step)
                    return p_ssd_conv_silu_step(state, u.data_ptr(), us, pw, bias, slots,
                                                out.data_ptr(), os, rows, nslots, c32, k32, io,
                                                st);
                  return p_ssd_conv_silu_varlen(u.data_ptr(), us, pw, bias, s.cu, state, slots,
                                                s.resume, out.data_ptr(), os, rows, s.nseq,
                                                nslots, c32, k32, io, st);
                }),
                out);
}
PyObject* conv_silu_varlen(PyObject* const* a) {
  return conv(a[0], a[1], a[2], a[3], a[4], a[5], a[6], a[7], false);
}
PyObject* conv_silu_step(PyObject* const* a) {
  return conv(a[1], a[2], nullptr, a[3], a[0], a[4], nullptr, a[5], true);
}

// The arguments both forms of the selective scan share:
// x, dt, A, B, C, D, z, dt_bias, softplus, state, slots, out, y_dtype
struct Selective {
  ssd_selective_args args;
  at::Tensor y;
  int64_t rows;
  int dev;
  bool no_slot = false;  // a cache without a slot is not the same as none
};
void selective(PyObject* const* a, int64_t nseq, Selective* s) {
  const at::Tensor& x = first(a[0], "x", 2);
  const int dev = s->dev = x.get_device();
  const int64_t rows = s->rows = x.size(0), dim = x.size(1);
  const ssd_dtype io = code(x, "x");
  const at::Tensor &dt = tensor(a[1], "dt"), &A = tensor(a[2], "A"), &B = tensor(a[3], "B"),
                   &C = tensor(a[4], "C");
  if (A.dim() != 2) refuse(PyExc_ValueError, "A must be a tensor [dim, dstate]");
  if (B.dim() != 3) refuse(PyExc_ValueError, "B must be a tensor [rows, G, dstate]");
  if (dt.scalar_type() != at::kFloat) has_type(dt, "dt", x.scalar_type());
  has_type(B, "B", x.scalar_type());
  has_type(C, "C", x.scalar_type());
  const int64_t N = A.size(1), G = B.size(1);
  const int64_t shape[2] = {rows, dim}, bc[3] = {rows, G, N};
  ssd_selective_args& k = s->args;
  k = {};
  k.x_stride = row_stride(x, "x", shape, dev);
  k.dt_stride = row_stride(dt, "dt", shape, dev);
  k.b_stride = row_stride(B, "B", bc, dev);
  k.c_stride = row_stride(C, "C", bc, dev);
  if (given(a[6])) {
    const at::Tensor& z = tensor(a[6], "z");
    has_type(z, "z", x.scalar_type());
    k.z_stride = row_stride(z, "z", shape, dev);
    k.z = z.data_ptr();
  }
  k.A = weights(a[2], "A", {dim, N}, dev);
  k.D = whole<float>(a[5], "D", at::kFloat, {dim}, dev);
  k.dt_bias = whole<float>(a[7], "dt_bias", at::kFloat, {dim}, dev);
  k.softplus = flag_arg(a[8]);
  if (given(a[9])) {
    const at::Tensor& t = tensor(a[9], "state");
    if (t.dim() != 3) refuse(PyExc_ValueError, "state must be a tensor [nslots, dim, dstate]");
    k.nslots = t.size(0);
    k.state = whole<float>(a[9], "state", at::kFloat, {k.nslots, dim, N}, dev);
    s->no_slot = k.nslots == 0 && (nseq < 0 ? rows : nseq) > 0;
  }
  k.slots = slot_arg(a[10], nseq < 0 ? rows : nseq, dev);
  s->y = output(a[11], x, shape, given(a[11]) ? at::kFloat : dtype_arg(a[12]));
  k.y_stride = row_stride(s->y, "out", shape, dev);
  k.x = x.data_ptr();
  k.dt = dt.data_ptr();
  k.B = B.data_ptr();
  k.C = C.data_ptr();
  k.y = s->y.data_ptr();
  k.dim = width32(dim, "x");
  k.dstate = width32(N, "A");
  k.ngroups = width32(G, "B");
  k.io = io;
  k.dt_dtype = code(dt, "dt");
  k.y_dtype = code(s->y, "out");
}
// ... , cu_seqlens, resume, max_seqlen, workspace
PyObject* selective_scan_varlen(PyObject* const* a) {
  const at::Tensor& x = first(a[0], "x", 2);
  const Seqs q = seqs(a[13], a[14], x.get_device());
  Selective s;
  selective(a, q.nseq, &s);
  if (s.no_slot) return PyLong_FromLong(SSD_ERR_INVALID_ARG);
  const int64_t longest = int_arg(a[15], "max_seqlen");
  const OnDevice here(s.dev);
  size_t need = q.nseq > 0 ? p_ssd_selective_varlen_workspace_size(
                                 s.rows, q.nseq, s.args.dim, s.args.dstate, s.args.ngroups, longest)
                           : 0;
  at::Tensor ws;
  void* wp = nullptr;
  if (given(a[16])) {
    ws = tensor(a[16], "workspace");
    wp = whole(a[16], "workspace", at::kByte, ws.sizes(), s.dev);
    need = size_t(ws.numel());
  } else if (need > 0) {
    ws = at::empty({int64_t(need)}, x.options().dtype(at::kByte).requires_grad(false));
    wp = ws.data_ptr();
  }
  return result(on_device(s.dev, [&](cudaStream_t st) {
                  return p_ssd_selective_scan_varlen(&s.args, q.cu, q.resume, s.rows, q.nseq,
                                                     longest, wp, need, st);
                }),
                s.y);
}
PyObject* selective_step(PyObject* const* a) {
  Selective s;
  selective(a, -1, &s);
  if (s.no_slot) return PyLong_FromLong(SSD_ERR_INVALID_ARG);
  return result(on_device(s.dev, [&](cudaStream_t st) {
                  return p_ssd_selective_step(&s.args, s.rows, st);
                }),
                s.y);
}

// y, weight, bias, z, ngroups, eps, center, gate_first, out, out_dtype
struct Norm {
  const void *y, *z;
  const float *w, *b;
  int64_t ys, zs, rows;
  int cdim, ngroups, dev;
  float eps;
  bool center, first;
  ssd_dtype yd, zd;
};
void norm_args(PyObject* const* a, Norm* n) {
  const at::Tensor& y = first(a[0], "y", 2);
  n->dev = y.get_device();
  n->rows = y.size(0);
  n->cdim = width32(y.size(1), "y");
  const int64_t shape[2] = {n->rows, n->cdim};
  n->y = y.data_ptr();
  n->ys = row_stride(y, "y", shape, n->dev);
  n->yd = code(y, "y");
  n->w = weights(a[1], "weight", {n->cdim}, n->dev);
  n->b = whole<float>(a[2], "bias", at::kFloat, {n->cdim}, n->dev);
  n->z = nullptr;
  n->zs = 0;
  n->zd = SSD_F32;
  if (given(a[3])) {
    const at::Tensor& z = tensor(a[3], "z");
    n->zs = row_stride(z, "z", shape, n->dev);
    n->zd = code(z, "z");
    n->z = z.data_ptr();
  }
  n->ngroups = int32_arg(a[4], "ngroups");
  n->eps = float(PyFloat_AsDouble(a[5]));
  if (PyErr_Occurred()) {
    PyErr_Clear();
    refuse(PyExc_TypeError, "eps must be a number");
  }
  n->center = flag_arg(a[6]);
  n->first = flag_arg(a[7]);
}
PyObject* group_norm_gate(PyObject* const* a) {
  Norm n;
  norm_args(a, &n);
  const int64_t shape[2] = {n.rows, n.cdim};
  const at::Tensor out = output(a[8], THPVariable_Unpack(a[0]), shape,
                                given(a[8]) ? at::kFloat : dtype_arg(a[9]));
  const int64_t os = row_stride(out, "out", shape, n.dev);
  const ssd_dtype od = code(out, "out");
  return result(on_device(n.dev, [&](cudaStream_t st) {
                  return p_ssd_group_norm_gate(n.y, n.ys, n.w, n.b, n.z, n.zs, out.data_ptr(), os,
                                               n.rows, n.cdim, n.ngroups, n.eps, n.center, n.first,
                                               n.yd, n.zd, od, st);
                }),
                out);
}
// y, weight, bias, z, ngroups, eps, center, gate_first, dout, workspace -> (dy, dz, dweight, dbias)
PyObject* group_norm_gate_bwd(PyObject* const* a) {
  Norm n;
  norm_args(a, &n);
  const int64_t shape[2] = {n.rows, n.cdim};
  const at::Tensor& dout = tensor(a[8], "dout");
  const int64_t ds = row_stride(dout, "dout", shape, n.dev);
  const ssd_dtype dd = code(dout, "dout");
  const auto f32 = THPVariable_Unpack(a[0]).options().dtype(at::kFloat).requires_grad(false);
  at::Tensor dy = at::empty(shape, f32), dw = at::empty({n.cdim}, f32), dz, db, ws;
  if (given(a[3])) dz = at::empty(shape, f32.dtype(n.zd == SSD_BF16 ? at::kBFloat16 : at::kFloat));
  if (n.b) db = at::empty({n.cdim}, f32);
  const OnDevice here(n.dev);
  void* wp = nullptr;
  size_t need = p_ssd_group_norm_gate_bwd_workspace_size(n.rows, n.cdim, n.ngroups);
  if (given(a[9])) {
    ws = tensor(a[9], "workspace");
    wp = whole(a[9], "workspace", at::kByte, ws.sizes(), n.dev);
    need = size_t(ws.numel());
  } else if (need > 0) {
    ws = at::empty({int64_t(need)}, f32.dtype(at::kByte));
    wp = ws.data_ptr();
  }
  const int rc = on_device(n.dev, [&](cudaStream_t st) {
    return p_ssd_group_norm_gate_bwd(
        dout.data_ptr(), ds, n.y, n.ys, n.w, n.b, n.z, n.zs, static_cast<float*>(dy.data_ptr()),
        n.z ? dz.data_ptr() : nullptr, static_cast<float*>(dw.data_ptr()),
        n.b ? static_cast<float*>(db.data_ptr()) : nullptr, n.rows, n.cdim, n.ngroups, n.eps,
        n.center, n.first, dd, n.yd, n.zd, wp, need, st);
  });
  if (rc) return PyLong_FromLong(rc);
  auto wrap = [](const at::Tensor& t) {
    return t.defined() ? THPVariable_Wrap(t) : Py_NewRef(Py_None);
  };
  return Py_BuildValue("(NNNN)", wrap(dy), wrap(dz), wrap(dw), wrap(db));
}

// Runs F with its NARGS positional arguments; C++ exceptions become Python's.
template <PyObject* (*F)(PyObject* const*), int NARGS>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != NARGS) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Refused& r) {
    PyErr_SetString(r.type, r.what.c_str());
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

// bind(path): looks up the C entries in the library that is already loaded from `path`.
PyObject* bind_entries(PyObject*, PyObject* path) {
  const char* p = PyUnicode_AsUTF8(path);
  if (!p) return nullptr;
  void* lib = dlopen(p, RTLD_NOW | RTLD_NOLOAD);
  if (!lib) {
    PyErr_SetString(PyExc_RuntimeError, "the library is not loaded");
    return nullptr;
  }
#define X(name)                                                     \
  p_##name = reinterpret_cast<decltype(p_##name)>(dlsym(lib, #name)); \
  if (!p_##name) {                                                  \
    PyErr_SetString(PyExc_RuntimeError, "missing entry: " #name);   \
    return nullptr;                                                 \
  }
  SSD_ENTRIES(X)
#undef X
  Py_RETURN_NONE;
}

#define SSD_METHOD(name, n) \
  {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(&call<name, n>)), METH_FASTCALL, nullptr}
PyMethodDef kMethods[] = {{"bind", bind_entries, METH_O, nullptr},
                          SSD_METHOD(conv_silu_varlen, 8),
                          SSD_METHOD(conv_silu_step, 6),
                          SSD_METHOD(selective_scan_varlen, 17),
                          SSD_METHOD(selective_step, 13),
                          SSD_METHOD(group_norm_gate, 10),
                          SSD_METHOD(group_norm_gate_bwd, 10),
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods,
                       nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding(void) { return PyModule_Create(&kModule); }
