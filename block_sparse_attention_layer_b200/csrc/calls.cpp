// Python calls of the norm + rotation and 8-bit checkpoint entry points
// (norm_rope.py).  Arguments are read from the tensors and checked here, since
// the checks of seven to ten tensors in Python cost more host time (4.5 us)
// than a small call's kernel takes on the device (2.4 us for one token).
// Nothing is computed and nothing allocated: each function passes the tensors'
// addresses to the C entry, whose own checks and status codes stand behind
// these.
#include <Python.h>

#include <initializer_list>
#include <string>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <c10/util/SmallVector.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/vmoba.h"

namespace {

struct Refused {};                   // a Python error is set

[[noreturn]] void refuse(const std::string& what) {
  PyErr_SetString(PyExc_ValueError, what.c_str());
  throw Refused{};
}

// ---- the library's entry points, handed over once loaded ----

#define ENTRIES(X)                                                                      \
  X(vmoba_qk_norm_rope) X(vmoba_qk_norm_rope_act8) X(vmoba_qk_norm_rope_partition)      \
  X(vmoba_qk_norm_rope_partition_act8) X(vmoba_qk_norm_rope_bwd)                        \
  X(vmoba_qk_norm_rope_bwd_act8) X(vmoba_act8_pack) X(vmoba_act8_unpack)
#define DECLARE(f) decltype(&::f) p_##f = nullptr;
ENTRIES(DECLARE)
#undef DECLARE
PyTypeObject* act8_type = nullptr;

PyObject *s_q_weight, *s_k_weight, *s_eps, *s_table, *s_dims, *s_codes, *s_scales, *s_group,
    *s_cuda_stream, *s_device, *s_index, *s_dtype;

// An owned reference.
struct Ref {
  PyObject* p;
  explicit Ref(PyObject* o) : p(o) { if (!p) throw Refused{}; }
  ~Ref() { Py_DECREF(p); }
  Ref(const Ref&) = delete;
  Ref& operator=(const Ref&) = delete;
};

Ref attr(PyObject* o, PyObject* name) { return Ref(PyObject_GetAttr(o, name)); }

long long to_int(PyObject* o, const char* name) {
  if (!PyLong_Check(o)) refuse(std::string(name) + ": expected a whole number");
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused{};
  return v;
}

// ---- tensors ----

std::string text(at::IntArrayRef v) {
  std::string s = "(";
  for (size_t i = 0; i < v.size(); ++i)
    s += (i ? ", " : "") + std::to_string(v[i]);
  return s + (v.size() == 1 ? ",)" : ")");
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(std::string(name) + ": expected a tensor");
  return THPVariable_Unpack(o);
}

const char* type_name(at::ScalarType t) {
  return t == at::kBFloat16 ? "torch.bfloat16" : (t == at::kChar ? "torch.int8" : "torch.float32");
}

void expect_type(PyObject* o, at::ScalarType type, const char* name) {
  if (THPVariable_Unpack(o).scalar_type() == type) return;
  Ref got(PyObject_Str(attr(o, s_dtype).p));
  refuse(std::string(name) + ": expected dtype " + type_name(type) + ", got " +
         PyUnicode_AsUTF8(got.p));
}

// A call's tensors, whose devices are compared once everything else is right.
// Each is held until the call has returned: an attribute of an argument may be
// a tensor made for this one access.
struct Device {
  struct Seen { PyObject* o; const char *name, *part; };
  c10::SmallVector<Seen, 16> seen;     // 14 in a backward with separate rows and gradients
  int index = -1;
  Device() = default;
  Device(const Device&) = delete;
  Device& operator=(const Device&) = delete;
  ~Device() { for (const Seen& x : seen) Py_DECREF(x.o); }
  void take(PyObject* o, const char* name, const char* part = "") {
    Py_INCREF(o);
    seen.push_back({o, name, part});
  }
  void settle() {
    for (const Seen& x : seen) {
      const at::Tensor& t = THPVariable_Unpack(x.o);
      if (&x == seen.begin() && t.is_cuda()) index = t.get_device();
      if (t.is_cuda() && t.get_device() == index) continue;
      const std::string name = std::string(x.name) + x.part;
      if (!t.is_cuda()) refuse(name + ": expected a CUDA tensor");
      refuse(name + ": expected a tensor on cuda:" + std::to_string(index) + ", got " +
             t.device().str());
    }
  }
};

void expect_size(const at::Tensor& t, std::initializer_list<int64_t> size, const char* name) {
  const at::IntArrayRef want(size.begin(), size.size());
  if (t.sizes() != want)
    refuse(std::string(name) + ": expected shape " + text(want) + ", got " + text(t.sizes()));
}

// Address of a contiguous tensor of the call.
void* at_(PyObject* o, std::initializer_list<int64_t> size, at::ScalarType type, Device& d,
          const char* name) {
  const at::Tensor& t = tensor(o, name);
  expect_size(t, size, name);
  expect_type(o, type, name);
  if (!t.is_contiguous()) refuse(std::string(name) + ": expected a contiguous tensor");
  d.take(o, name);
  return t.data_ptr();
}

// ---- shapes ----

struct Shape {
  vmoba_shape c;
  int64_t s, h, d, blocks;
  at::ScalarType type;
};

void free_shape(PyObject* o) {
  delete static_cast<Shape*>(PyCapsule_GetPointer(o, "vmoba_shape"));
}

const Shape& shape_of(PyObject* o) {
  void* p = PyCapsule_GetPointer(o, "vmoba_shape");
  if (!p) throw Refused{};
  return *static_cast<Shape*>(p);
}

// ---- raw rows ----

// The token stride of rows whose other axes are dense.
int64_t token_stride(const at::Tensor& t, int64_t least, const char* name) {
  int64_t dense = 1;
  for (int64_t i = t.dim() - 1; i > 0; --i) {
    if (t.size(i) > 1 && t.stride(i) != dense)
      refuse(std::string(name) + ": expected dense rows, got strides " + text(t.strides()));
    dense *= t.size(i);
  }
  if (t.size(0) == 1) return least;
  if (t.stride(0) < least)
    refuse(std::string(name) + ": rows overlap, strides " + text(t.strides()));
  return t.stride(0);
}

struct Raw {
  void* at[3];
  int64_t ld;
};

// One [s][3][heads][d] tensor, or three [s][heads][d] ones.
Raw raw_rows(const Shape& sh, PyObject* o, Device& dev, const char* name) {
  Raw r;
  const int64_t row = sh.h * sh.d;
  if (PyTuple_Check(o) || PyList_Check(o)) {
    if (PySequence_Fast_GET_SIZE(o) != 3)
      refuse(std::string(name) + ": expected one tensor or three");
    for (int i = 0; i < 3; ++i) {
      PyObject* item = PySequence_Fast_GET_ITEM(o, i);
      const at::Tensor& t = tensor(item, name);
      expect_size(t, {sh.s, sh.h, sh.d}, name);
      expect_type(item, sh.type, name);
      const int64_t ld = token_stride(t, row, name);
      if (i == 0) r.ld = ld;
      if (ld != r.ld)
        refuse(std::string(name) + ": expected one token stride, got " + std::to_string(r.ld) +
               " and " + std::to_string(ld));
      r.at[i] = t.data_ptr();
      dev.take(item, name);
    }
    return r;
  }
  const at::Tensor& t = tensor(o, name);
  expect_size(t, {sh.s, 3, sh.h, sh.d}, name);
  expect_type(o, sh.type, name);
  r.ld = token_stride(t, 3 * row, name);
  dev.take(o, name);
  for (int i = 0; i < 3; ++i)
    r.at[i] = static_cast<char*>(t.data_ptr()) + i * row * (int64_t)t.element_size();
  return r;
}

// ---- checkpoints ----

bool is_act8(PyObject* o) { return PyObject_TypeCheck(o, act8_type); }

struct Ckpt {
  int8_t* codes = nullptr;
  float* scales = nullptr;
  int group = 0;
};

Ckpt checkpoint(PyObject* o, at::IntArrayRef size, int64_t group, Device& dev, const char* name) {
  if (!is_act8(o)) refuse(std::string(name) + ": expected an Act8");
  Ref codes = attr(o, s_codes), scales = attr(o, s_scales), g = attr(o, s_group);
  Ckpt c;
  c.group = (int)to_int(g.p, "group");
  if (group && c.group != group)
    refuse(std::string(name) + ": expected groups of " + std::to_string(group) + ", got " +
           std::to_string(c.group));
  if (c.group != 64 && c.group != 128) refuse(std::string(name) + ": expected groups of 64 or 128");
  const at::Tensor &tc = tensor(codes.p, name), &ts = tensor(scales.p, name);
  c10::SmallVector<int64_t, 8> want(size.begin(), size.end());
  want.back() = (want.back() + c.group - 1) / c.group;
  const struct { const at::Tensor& t; PyObject* o; at::IntArrayRef size; at::ScalarType type;
                 const char* part; } both[2] = {{tc, codes.p, size, at::kChar, ".codes"},
                                                {ts, scales.p, want, at::kFloat, ".scales"}};
  for (const auto& x : both) {
    if (x.t.sizes() == x.size && x.t.scalar_type() == x.type && x.t.is_contiguous()) continue;
    const std::string part = std::string(name) + x.part;
    if (x.t.sizes() != x.size)
      refuse(part + ": expected shape " + text(x.size) + ", got " + text(x.t.sizes()));
    expect_type(x.o, x.type, part.c_str());
    refuse(part + ": expected a contiguous tensor");
  }
  dev.take(codes.p, name, ".codes");
  dev.take(scales.p, name, ".scales");
  c.codes = static_cast<int8_t*>(tc.data_ptr());
  c.scales = static_cast<float*>(ts.data_ptr());
  return c;
}

// ---- norm and rotation ----

vmoba_norm_rope norm_rope(const Shape& sh, PyObject* nr, Device& dev) {
  vmoba_norm_rope n{};
  Ref dims = attr(nr, s_dims);
  int64_t v[3] = {-1, -1, -1};
  if ((PyTuple_Check(dims.p) || PyList_Check(dims.p)) && PySequence_Fast_GET_SIZE(dims.p) == 3)
    for (int i = 0; i < 3; ++i) {
      PyObject* o = PySequence_Fast_GET_ITEM(dims.p, i);
      v[i] = PyLong_Check(o) ? PyLong_AsLongLong(o) : -1;
      if (v[i] < 0 || v[i] > sh.d || v[i] % 2) v[0] = v[i] = -1;
    }
  PyErr_Clear();
  if (v[0] < 0 || v[1] < 0 || v[2] < 0 || v[0] + v[1] + v[2] > sh.d) {
    Ref got(PyObject_Repr(dims.p));
    refuse("dims: expected three even numbers >= 0 of sum <= " + std::to_string(sh.d) + ", got " +
           PyUnicode_AsUTF8(got.p));
  }
  n.dim_t = (int)v[0]; n.dim_h = (int)v[1]; n.dim_w = (int)v[2];
  Ref gq = attr(nr, s_q_weight), gk = attr(nr, s_k_weight), table = attr(nr, s_table);
  Ref eps = attr(nr, s_eps);
  if (gq.p != Py_None)
    n.q_weight = static_cast<float*>(at_(gq.p, {sh.d}, at::kFloat, dev, "q_weight"));
  if (gk.p != Py_None)
    n.k_weight = static_cast<float*>(at_(gk.p, {sh.d}, at::kFloat, dev, "k_weight"));
  const double e = PyFloat_AsDouble(eps.p);
  if (e == -1.0 && PyErr_Occurred()) throw Refused{};
  n.eps = (float)e;
  const int64_t entries = (sh.c.T * v[0] + sh.c.H * v[1] + sh.c.W * v[2]) / 2;
  if (entries) {
    if (table.p == Py_None) refuse("table: expected a rotation table (rope_table)");
    n.table = static_cast<float*>(at_(table.p, {entries, 2}, at::kFloat, dev, "table"));
  }
  return n;
}

// ---- launches ----

cudaStream_t stream_of(PyObject* o, Device& dev) {
  dev.settle();
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev.index).stream();
  Ref device = attr(o, s_device), index = attr(device.p, s_index), raw = attr(o, s_cuda_stream);
  if (to_int(index.p, "stream") != dev.index)
    refuse("stream: expected one of cuda:" + std::to_string(dev.index));
  return reinterpret_cast<cudaStream_t>(PyLong_AsUnsignedLongLong(raw.p));
}

// The entry's status, called with the tensors' device current.
template <typename F>
PyObject* call(const Device& dev, F f) {
  int rc;
  {
    c10::cuda::OptionalCUDAGuard guard;
    if (c10::cuda::current_device() != dev.index) guard.set_index((c10::DeviceIndex)dev.index);
    PyThreadState* state = PyEval_SaveThread();
    rc = f();
    PyEval_RestoreThread(state);
  }
  return PyLong_FromLong(rc);
}

// A C++ exception (torch's own, for a device in error) becomes a Python one.
template <typename F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F f) {
  if (n != want || !p_vmoba_act8_unpack) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments, or not bound");
    return nullptr;
  }
  try {
    return f();
  } catch (const Refused&) {
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// forward(shape, norm, qkv, q, k, v, blocks or None, ckpt or None, stream or None)
PyObject* forward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 9, [&]() -> PyObject* {
    const Shape& sh = shape_of(a[0]);
    Device dev;
    const bool part = a[6] != Py_None, from8 = is_act8(a[2]);
    if (from8 && a[7] != Py_None) refuse("ckpt: the raw values already come from a checkpoint");
    const int64_t five[4] = {sh.s, 3, sh.h, sh.d};
    Raw raw{};
    Ckpt src, to;
    if (from8) src = checkpoint(a[2], five, sh.d, dev, "qkv");
    else raw = raw_rows(sh, a[2], dev, "qkv");
    if (a[7] != Py_None) to = checkpoint(a[7], five, sh.d, dev, "ckpt");
    void* q = at_(a[3], {sh.s, sh.h, sh.d}, sh.type, dev, "q");
    void *k, *v, *blocks = nullptr;
    if (part) {
      k = at_(a[4], {sh.h, sh.s, sh.d}, sh.type, dev, "k_perm");
      v = at_(a[5], {sh.h, sh.s, sh.d}, sh.type, dev, "v_perm");
      blocks = at_(a[6], {sh.h, sh.blocks, sh.d}, at::kFloat, dev, "blocks");
    } else {
      k = at_(a[4], {sh.s, sh.h, sh.d}, sh.type, dev, "k");
      v = at_(a[5], {sh.s, sh.h, sh.d}, sh.type, dev, "v");
    }
    const vmoba_norm_rope nr = norm_rope(sh, a[1], dev);
    const cudaStream_t st = stream_of(a[8], dev);
    float* b = static_cast<float*>(blocks);
    return call(dev, [&] {
      if (from8)
        return part ? p_vmoba_qk_norm_rope_partition_act8(&sh.c, &nr, src.codes, src.scales, q, k,
                                                          v, b, st)
                    : p_vmoba_qk_norm_rope_act8(&sh.c, &nr, src.codes, src.scales, q, k, v, st);
      return part ? p_vmoba_qk_norm_rope_partition(&sh.c, &nr, raw.at[0], raw.at[1], raw.at[2],
                                                   raw.ld, q, k, v, b, to.codes, to.scales, st)
                  : p_vmoba_qk_norm_rope(&sh.c, &nr, raw.at[0], raw.at[1], raw.at[2], raw.ld, q, k,
                                         v, to.codes, to.scales, st);
    });
  });
}

// backward(shape, norm, qkv, dq, dk, dv, dqkv, dweight or None, ws or None, stream or None)
PyObject* backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject* {
    const Shape& sh = shape_of(a[0]);
    Device dev;
    const bool from8 = is_act8(a[2]);
    const int64_t five[4] = {sh.s, 3, sh.h, sh.d};
    Raw raw{};
    Ckpt src;
    if (from8) src = checkpoint(a[2], five, sh.d, dev, "qkv");
    else raw = raw_rows(sh, a[2], dev, "qkv");
    const char* names[3] = {"dq", "dk", "dv"};
    void* g[3];
    for (int i = 0; i < 3; ++i)
      g[i] = at_(a[3 + i], {sh.s, sh.h, sh.d}, sh.type, dev, names[i]);
    const Raw out = raw_rows(sh, a[6], dev, "dqkv");
    const vmoba_norm_rope nr = norm_rope(sh, a[1], dev);
    float* dw = nullptr;
    void* ws = nullptr;
    size_t ws_bytes = 0;
    if (a[7] != Py_None) {
      dw = static_cast<float*>(at_(a[7], {2, sh.d}, at::kFloat, dev, "dweight"));
      const at::Tensor& t = tensor(a[8], "ws");
      if (!t.is_contiguous()) refuse("ws: expected a contiguous tensor");
      dev.take(a[8], "ws");
      ws = t.data_ptr();
      ws_bytes = t.nbytes();
    }
    const cudaStream_t st = stream_of(a[9], dev);
    return call(dev, [&] {
      return from8 ? p_vmoba_qk_norm_rope_bwd_act8(&sh.c, &nr, src.codes, src.scales, g[0], g[1],
                                                   g[2], out.at[0], out.at[1], out.at[2], out.ld,
                                                   dw, ws, ws_bytes, st)
                   : p_vmoba_qk_norm_rope_bwd(&sh.c, &nr, raw.at[0], raw.at[1], raw.ld, g[0],
                                              g[1], g[2], out.at[0], out.at[1], out.at[2], out.ld,
                                              dw, ws, ws_bytes, st);
    });
  });
}

// act8(pack, values, ckpt, stream or None)
PyObject* act8(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 4, [&]() -> PyObject* {
    const bool pack = a[0] == Py_True;
    const char* name = pack ? "x" : "out";
    const at::Tensor& t = tensor(a[1], name);
    int type;
    if (t.scalar_type() == at::kBFloat16) {
      type = VMOBA_BF16;
    } else if (t.scalar_type() == at::kFloat) {
      type = VMOBA_F32;
    } else {
      Ref got(PyObject_Str(attr(a[1], s_dtype).p));
      refuse(std::string(name) + ": expected dtype bfloat16 or float32, got " +
             PyUnicode_AsUTF8(got.p));
    }
    if (t.dim() < 2) refuse(std::string(name) + ": expected at least two axes");
    const int64_t cols = t.size(t.dim() - 1);
    int64_t rows = cols ? t.numel() / cols : 0, ld = cols;
    if (!t.is_contiguous()) {
      if (t.dim() != 2 || (cols > 1 && t.stride(1) != 1) || (rows > 1 && t.stride(0) < cols))
        refuse(std::string(name) + ": expected dense rows, got strides " + text(t.strides()));
      if (rows > 1) ld = t.stride(0);
    }
    if (cols > INT32_MAX) refuse(std::string(name) + ": too many columns");
    Device dev;
    dev.take(a[1], name);
    const Ckpt c = checkpoint(a[2], t.sizes(), 0, dev, "ckpt");
    const cudaStream_t st = stream_of(a[3], dev);
    return call(dev, [&] {
      return pack ? p_vmoba_act8_pack(type, t.data_ptr(), rows, (int)cols, ld, c.group, c.codes,
                                      c.scales, st)
                  : p_vmoba_act8_unpack(type, c.codes, c.scales, rows, (int)cols, c.group,
                                        t.data_ptr(), ld, st);
    });
  });
}

// shape(T, H, W, n_heads, head_dim, mode, bt, bh, bw, dtype, blocks) -> capsule
PyObject* shape(PyObject*, PyObject* args) {
  Shape s{};
  int blocks;
  if (!PyArg_ParseTuple(args, "iiiiiiiiiii", &s.c.T, &s.c.H, &s.c.W, &s.c.n_heads, &s.c.head_dim,
                        &s.c.mode, &s.c.bt, &s.c.bh, &s.c.bw, &s.c.dtype, &blocks))
    return nullptr;
  s.s = (int64_t)s.c.T * s.c.H * s.c.W;
  s.h = s.c.n_heads;
  s.d = s.c.head_dim;
  s.blocks = blocks;
  s.type = s.c.dtype == VMOBA_BF16 ? at::kBFloat16 : at::kFloat;
  return PyCapsule_New(new Shape(s), "vmoba_shape", free_shape);
}

// bind({entry name: address}, Act8)
PyObject* bind(PyObject*, PyObject* args) {
  PyObject *table, *type;
  if (!PyArg_ParseTuple(args, "O!O!", &PyDict_Type, &table, &PyType_Type, &type)) return nullptr;
#define TAKE(f)                                                    \
  {                                                                \
    PyObject* o = PyDict_GetItemString(table, #f);                 \
    void* p = o ? PyLong_AsVoidPtr(o) : nullptr;                   \
    if (!p) {                                                      \
      if (!PyErr_Occurred()) PyErr_SetString(PyExc_KeyError, #f);  \
      return nullptr;                                              \
    }                                                              \
    p_##f = reinterpret_cast<decltype(p_##f)>(p);                  \
  }
  ENTRIES(TAKE)
#undef TAKE
  Py_INCREF(type);
  Py_XDECREF(reinterpret_cast<PyObject*>(act8_type));
  act8_type = reinterpret_cast<PyTypeObject*>(type);
  Py_RETURN_NONE;
}

using Fast = PyObject* (*)(PyObject*, PyObject* const*, Py_ssize_t);
PyCFunction fast(Fast f) { return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)); }

}  // namespace

PyMODINIT_FUNC PyInit__calls(void) {
  static PyMethodDef methods[] = {{"bind", bind, METH_VARARGS, nullptr},
                                  {"shape", shape, METH_VARARGS, nullptr},
                                  {"forward", fast(forward), METH_FASTCALL, nullptr},
                                  {"backward", fast(backward), METH_FASTCALL, nullptr},
                                  {"act8", fast(act8), METH_FASTCALL, nullptr},
                                  {nullptr, nullptr, 0, nullptr}};
  static PyModuleDef module = {PyModuleDef_HEAD_INIT, "_calls", nullptr, -1, methods};
  const struct { PyObject** to; const char* name; } names[] = {
      {&s_q_weight, "q_weight"}, {&s_k_weight, "k_weight"}, {&s_eps, "eps"}, {&s_table, "table"},
      {&s_dims, "dims"}, {&s_codes, "codes"}, {&s_scales, "scales"}, {&s_group, "group"},
      {&s_cuda_stream, "cuda_stream"}, {&s_device, "device"}, {&s_index, "index"},
      {&s_dtype, "dtype"}};
  for (const auto& n : names)
    if (!(*n.to = PyUnicode_InternFromString(n.name))) return nullptr;
  return PyModule_Create(&module);
}
