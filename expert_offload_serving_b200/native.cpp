// The marshalling of the short calls (moe_linear_w4, moe_balance_loss,
// moe_router_backward, moe_combine_backward), in C++: torch tensors to the plain
// pointers of include/moe.h.
//
// These kernels take a few microseconds, and checking the tensors and passing
// the arguments through Python and ctypes took 5.8 of the 8.3 us that a call
// cost its host thread; here it is under 1.  Nothing is computed and nothing is
// kept from one call for the next.  Each function takes its arguments by
// position (the Python functions of the same names give them names, defaults and
// documentation), raises ValueError for a tensor that is not what the call
// documents, and returns the library's status.
#include <Python.h>

#include <string>

#include <ATen/core/Tensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../include/moe.h"

namespace {

struct Refused {};   // a Python error is set

[[noreturn]] void refuse(const std::string& what) {
  PyErr_SetString(PyExc_ValueError, what.c_str());
  throw Refused();
}

std::string describe(const at::Tensor& t) {
  std::string s = std::string(c10::toString(t.scalar_type())) + " [";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  s += "] strides [";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.stride(i));
  return s + "] on " + t.device().str();
}

// The tensor of an argument; nullptr for None.
const at::Tensor* tensor(const char* name, PyObject* o, bool optional = false) {
  if (o == Py_None && optional) return nullptr;
  if (!THPVariable_Check(o)) refuse(std::string(name) + ": expected a tensor");
  return &THPVariable_Unpack(o);
}

// Everything a call is given lives on the current device.
void on_device(const char* name, const at::Tensor& t, int dev) {
  if (!t.is_cuda() || t.get_device() != dev)
    refuse(std::string(name) + ": expected a tensor on the current device cuda:" + std::to_string(dev) + ", got " +
           describe(t));
}

// Address of a contiguous tensor of one of two types (the same for one) with at
// least n elements.
void* mem(const char* name, const at::Tensor* t, int64_t n, at::ScalarType type, int dev) {
  if (t == nullptr) return nullptr;
  on_device(name, *t, dev);
  if (t->scalar_type() != type || t->numel() < n || !t->is_contiguous())
    refuse(std::string(name) + ": expected a contiguous " + c10::toString(type) + " tensor of >= " + std::to_string(n) +
           " elements, got " + describe(*t));
  return t->data_ptr();
}

// Address of a contiguous [rows, cols].
void* matrix(const char* name, const at::Tensor* t, int64_t rows, int64_t cols, at::ScalarType type, int dev) {
  if (t == nullptr) return nullptr;
  if (t->dim() != 2 || t->size(0) != rows || t->size(1) != cols)
    refuse(std::string(name) + ": expected shape (" + std::to_string(rows) + ", " + std::to_string(cols) + "), got " +
           describe(*t));
  return mem(name, t, rows * cols, type, dev);
}

void two_dims(const char* name, const at::Tensor& t) {
  if (t.dim() != 2) refuse(std::string(name) + ": expected two dimensions, got " + describe(t));
}

// Distance between the rows of a [rows, cols] whose rows are contiguous and do
// not overlap (a single row has none: any valid value).
int64_t row_distance(const char* name, const at::Tensor& t, int64_t rows, int64_t cols, int dev) {
  on_device(name, t, dev);
  if (t.dim() != 2 || t.size(0) != rows || t.size(1) != cols || (cols > 1 && t.stride(1) != 1) ||
      (rows > 1 && t.stride(0) < cols))
    refuse(std::string(name) + ": expected (" + std::to_string(rows) + ", " + std::to_string(cols) +
           ") with contiguous rows, got " + describe(t));
  return rows > 1 ? t.stride(0) : (cols + 7) / 8 * 8;
}

int float_type(const char* name, at::ScalarType t) {
  if (t == at::kFloat) return MOE_DT_F32;
  if (t == at::kBFloat16) return MOE_DT_BF16;
  if (t == at::kHalf) return MOE_DT_F16;
  refuse(std::string(name) + ": expected float32, bfloat16 or float16, got " + c10::toString(t));
}

int current_device(const char* name, const at::Tensor& t) {
  if (!t.is_cuda()) refuse(std::string(name) + ": expected a CUDA tensor, got " + describe(t));
  const int dev = c10::cuda::current_device();
  on_device(name, t, dev);
  return dev;
}

// None: the current stream; else the cudaStream_t as a number.
cudaStream_t stream_of(PyObject* o, int dev) {
  if (o == Py_None) return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream();
  void* p = PyLong_AsVoidPtr(o);
  if (p == nullptr && PyErr_Occurred()) throw Refused();
  return static_cast<cudaStream_t>(p);
}

int64_t number(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused();
  return v;
}

int fits_int(const char* name, int64_t v) {
  if (v < -2147483647 || v > 2147483647) refuse(std::string(name) + ": " + std::to_string(v) + " is out of range");
  return static_cast<int>(v);
}

// The memory of a call's tensors: what it writes overlaps nothing else of it.
class Memory {
 public:
  void in(const char* name, const void* p, int64_t bytes) { add({name, reinterpret_cast<uintptr_t>(p), bytes, false}); }
  void out(const char* name, const void* p, int64_t bytes) { add({name, reinterpret_cast<uintptr_t>(p), bytes, true}); }

 private:
  struct Range {
    const char* name;
    uintptr_t at;
    int64_t bytes;
    bool written;
  };
  void add(const Range& r) {
    if (r.at == 0 || r.bytes <= 0) return;
    for (int i = 0; i < n_; ++i)
      if ((r.written || r_[i].written) && r.at < r_[i].at + r_[i].bytes && r_[i].at < r.at + r.bytes)
        refuse(std::string(r.name) + " overlaps " + r_[i].name);
    r_[n_++] = r;
  }
  Range r_[16];
  int n_ = 0;
};

// Runs a call with its arguments counted and C++ exceptions turned into Python's.
template <typename F>
PyObject* guarded(const char* name, Py_ssize_t n, Py_ssize_t want, F f) {
  if (n != want) {
    PyErr_Format(PyExc_TypeError, "%s takes %zd arguments (%zd given)", name, want, n);
    return nullptr;
  }
  try {
    return PyLong_FromLong(f());
  } catch (const Refused&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

#define MOE_CALL(status, call) \
  int status;                  \
  Py_BEGIN_ALLOW_THREADS       \
  status = call;               \
  Py_END_ALLOW_THREADS

// (x, codes, scales, out, zeros, fmt, group, tensor_scale, flags, dev_status, stream)
PyObject* linear_w4(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("linear_w4", n, 11, [&] {
    const at::Tensor &x = *tensor("x", a[0]), &codes = *tensor("codes", a[1]), &scales = *tensor("scales", a[2]),
                     &out = *tensor("out", a[3]);
    const at::Tensor* zeros = tensor("zeros", a[4], true);
    const int fmt = fits_int("fmt", number(a[5])), group = fits_int("group", number(a[6]));
    const double ts = PyFloat_AsDouble(a[7]);
    if (ts == -1.0 && PyErr_Occurred()) throw Refused();
    const int flags = fits_int("flags", number(a[8]));
    const int dev = current_device("x", x);
    two_dims("x", x);
    two_dims("codes", codes);
    if (group <= 0) refuse("group=" + std::to_string(group));
    const int64_t T = x.size(0), K = x.size(1), N = codes.size(0), G = (K + group - 1) / group;
    const at::ScalarType st = fmt == MOE_W_INT4 ? scales.scalar_type() : at::kByte;
    moe_linear_shape s;
    s.N = fits_int("N", N);
    s.K = fits_int("K", K);
    s.fmt = fmt;
    s.group = group;
    s.scale_type = fmt == MOE_W_INT4 ? float_type("scales", st) : MOE_DT_F32;
    const int xt = float_type("x", x.scalar_type()), yt = float_type("out", out.scalar_type());
    const void* pc = matrix("codes", &codes, N, K / 2, at::kByte, dev);
    const void* ps = matrix("scales", &scales, N, G, st, dev);
    const void* pz = matrix("zeros", zeros, N, G, at::kByte, dev);
    const int64_t ldx = row_distance("x", x, T, K, dev);
    const int64_t ldy = row_distance("out", out, T, flags & MOE_LINEAR_SWIGLU ? N / 2 : N, dev);
    int32_t* status = static_cast<int32_t*>(mem("dev_status", tensor("dev_status", a[9], true), 1, at::kInt, dev));
    const cudaStream_t stream = stream_of(a[10], dev);
    const int t = fits_int("T", T);
    // x and out may be columns of one buffer, the same distance between their rows
    const int64_t xe = x.element_size(), ye = out.element_size(), yw = out.size(1) * ye, pitch = ldx * xe;
    const int64_t xb = T > 0 ? (T - 1) * pitch + K * xe : 0, yb = T > 0 ? (T - 1) * ldy * ye + yw : 0;
    const int64_t gap = static_cast<char*>(out.data_ptr()) - static_cast<char*>(x.data_ptr());
    const int64_t col = T > 1 && pitch > 0 && pitch == ldy * ye ? (gap % pitch + pitch) % pitch : -1;
    Memory m;
    m.out("out", out.data_ptr(), yb);
    if (!(col >= K * xe && col + yw <= pitch)) m.in("x", x.data_ptr(), xb);
    m.in("codes", pc, codes.numel());
    m.in("scales", ps, scales.numel() * scales.element_size());
    if (zeros != nullptr) m.in("zeros", pz, zeros->numel());
    // the status word may lie between the rows of x and out
    auto in_rows = [&](const at::Tensor& r, int64_t bytes, int64_t step, int64_t width) {
      const int64_t at = reinterpret_cast<char*>(status) - static_cast<char*>(r.data_ptr());
      return at > -4 && at < bytes && (at < 0 || at % step < width || at % step + 4 > step);
    };
    if (status != nullptr && T > 0) {
      if (in_rows(out, yb, ldy * ye, yw)) refuse("dev_status overlaps out");
      if (in_rows(x, xb, pitch, K * xe)) refuse("dev_status overlaps x");
      Memory w;
      w.in("codes", pc, codes.numel());
      w.in("scales", ps, scales.numel() * scales.element_size());
      if (zeros != nullptr) w.in("zeros", pz, zeros->numel());
      w.out("dev_status", status, 4);
    }
    MOE_CALL(r, moe_linear_w4(s, pc, ps, static_cast<const uint8_t*>(pz), static_cast<float>(ts), x.data_ptr(), xt, ldx,
                              t, out.data_ptr(), yt, ldy, flags, status, stream))
    return r;
  });
}

// What the calls on a routed batch share: logits, idx, seq_offsets and mask.
struct Batch {
  int dev, T, E, k, S;
  const float* logits;
  const int32_t* idx;
  const int32_t* off;
  const uint8_t* mask;
  Batch(PyObject* l, PyObject* i, PyObject* o, PyObject* m) {
    const at::Tensor &lt = *tensor("logits", l), &it = *tensor("idx", i);
    const at::Tensor *ot = tensor("seq_offsets", o, true), *mt = tensor("mask", m, true);
    dev = current_device("logits", lt);
    two_dims("logits", lt);
    two_dims("idx", it);
    T = fits_int("T", lt.size(0));
    E = fits_int("E", lt.size(1));
    k = fits_int("k", it.size(1));
    S = ot == nullptr ? 1 : fits_int("S", ot->numel() - 1);
    logits = static_cast<const float*>(mem("logits", &lt, lt.numel(), at::kFloat, dev));
    idx = static_cast<const int32_t*>(matrix("idx", &it, T, k, at::kInt, dev));
    off = static_cast<const int32_t*>(mem("seq_offsets", ot, int64_t(S) + 1, at::kInt, dev));
    mask = nullptr;
    if (mt != nullptr) {
      if (mt->scalar_type() != at::kBool && mt->scalar_type() != at::kByte)
        refuse("mask: expected bool or uint8, got " + describe(*mt));
      mask = static_cast<const uint8_t*>(mem("mask", mt, T, mt->scalar_type(), dev));
    }
  }
  float* f32(const char* name, PyObject* o, int64_t n, bool optional = false) const {
    return static_cast<float*>(mem(name, tensor(name, o, optional), n, at::kFloat, dev));
  }
  int32_t* i32(const char* name, PyObject* o, int64_t n, bool optional = false) const {
    return static_cast<int32_t*>(mem(name, tensor(name, o, optional), n, at::kInt, dev));
  }
  void into(Memory& m) const {
    m.in("logits", logits, int64_t(T) * E * 4);
    m.in("idx", idx, int64_t(T) * k * 4);
    m.in("seq_offsets", off, (int64_t(S) + 1) * 4);
    m.in("mask", mask, T);
  }
};

// (logits, idx, loss, counts, prob, coef, workspace, seq_offsets, mask, dev_status, stream)
PyObject* balance_loss(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("balance_loss", n, 11, [&] {
    const Batch b(a[0], a[1], a[7], a[8]);
    const int64_t SE = static_cast<int64_t>(b.S) * b.E;
    float* loss = b.f32("loss", a[2], 2);
    int32_t* counts = b.i32("counts", a[3], SE);
    float* prob = b.f32("prob", a[4], SE);
    float* coef = b.f32("coef", a[5], int64_t(b.S) + 1);
    const at::Tensor& w = *tensor("workspace", a[6]);
    void* ws = mem("workspace", &w, 0, at::kByte, b.dev);
    const size_t bytes = static_cast<size_t>(w.numel());
    int32_t* status = b.i32("dev_status", a[9], 1, true);
    const cudaStream_t stream = stream_of(a[10], b.dev);
    Memory m;
    b.into(m);
    m.out("loss", loss, 8);
    m.out("counts", counts, SE * 4);
    m.out("prob", prob, SE * 4);
    m.out("coef", coef, (int64_t(b.S) + 1) * 4);
    m.out("workspace", ws, w.numel());
    m.out("dev_status", status, 4);
    MOE_CALL(r, moe_balance_loss(b.logits, b.T, b.E, b.idx, b.k, b.off, b.S, b.mask, loss, counts, prob, coef, ws, bytes,
                                 status, stream))
    return r;
  });
}

// (logits, idx, dlogits, gate, dgate, counts, coef, dloss, seq_offsets, mask, dev_status, stream)
PyObject* router_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("router_backward", n, 12, [&] {
    const Batch b(a[0], a[1], a[8], a[9]);
    const int64_t TE = static_cast<int64_t>(b.T) * b.E, Tk = static_cast<int64_t>(b.T) * b.k;
    float* dlogits = b.f32("dlogits", a[2], TE);
    const float* gate = b.f32("gate", a[3], Tk, true);
    const float* dgate = b.f32("dgate", a[4], Tk, true);
    const int32_t* counts = b.i32("counts", a[5], static_cast<int64_t>(b.S) * b.E, true);
    const float* coef = b.f32("coef", a[6], int64_t(b.S) + 1, true);
    const float* dloss = b.f32("dloss", a[7], 2, true);
    int32_t* status = b.i32("dev_status", a[10], 1, true);
    const cudaStream_t stream = stream_of(a[11], b.dev);
    Memory m;
    b.into(m);
    m.in("gate", gate, Tk * 4);
    m.in("dgate", dgate, Tk * 4);
    m.in("counts", counts, static_cast<int64_t>(b.S) * b.E * 4);
    m.in("coef", coef, (int64_t(b.S) + 1) * 4);
    m.in("dloss", dloss, 8);
    m.out("dlogits", dlogits, TE * 4);
    m.out("dev_status", status, 4);
    MOE_CALL(r, moe_router_backward(b.logits, b.T, b.E, b.idx, gate, dgate, b.k, b.off, b.S, b.mask, counts, coef, dloss,
                                    dlogits, status, stream))
    return r;
  });
}

// (y_perm, idx, gate, inv_perm, slot_of_expert, dout, E, dgate, dy_perm, stream)
PyObject* combine_backward(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded("combine_backward", n, 10, [&] {
    const at::Tensor &dout = *tensor("dout", a[5]), &idx = *tensor("idx", a[1]);
    const int dev = current_device("dout", dout);
    two_dims("dout", dout);
    two_dims("idx", idx);
    const int64_t T = idx.size(0), k = idx.size(1), d = dout.size(1), p = T * k;
    const int E = fits_int("E", number(a[6]));
    auto f32 = [&](const char* name, PyObject* o, int64_t m, bool optional = false) {
      return static_cast<float*>(mem(name, tensor(name, o, optional), m, at::kFloat, dev));
    };
    auto i32 = [&](const char* name, PyObject* o, int64_t m, bool optional = false) {
      return static_cast<int32_t*>(mem(name, tensor(name, o, optional), m, at::kInt, dev));
    };
    const float* y = f32("y_perm", a[0], p * d);
    const int32_t* id = i32("idx", a[1], p);
    const float* gate = f32("gate", a[2], p, true);
    const int32_t* inv = i32("inv_perm", a[3], p);
    const int32_t* slot = i32("slot_of_expert", a[4], E, true);
    const float* o = static_cast<const float*>(matrix("dout", &dout, T, d, at::kFloat, dev));
    float* dg = f32("dgate", a[7], p);
    float* dy = f32("dy_perm", a[8], p * d, true);
    const int t = fits_int("T", T), kk = fits_int("k", k), dd = fits_int("d", d);
    const cudaStream_t stream = stream_of(a[9], dev);
    Memory m;
    m.in("y_perm", y, p * d * 4);
    m.in("idx", id, p * 4);
    m.in("gate", gate, p * 4);
    m.in("inv_perm", inv, p * 4);
    m.in("slot_of_expert", slot, int64_t(E) * 4);
    m.in("dout", o, T * d * 4);
    m.out("dgate", dg, p * 4);
    m.out("dy_perm", dy, p * d * 4);
    MOE_CALL(r, moe_combine_backward(y, id, gate, inv, slot, o, t, kk, dd, E, dg, dy, stream))
    return r;
  });
}

// The library's message for this thread (the calls above run in it).
PyObject* last_error(PyObject*, PyObject*) { return PyUnicode_DecodeUTF8(moe_last_error(), strlen(moe_last_error()), "replace"); }

#define MOE_FAST(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr
PyMethodDef methods[] = {
    {"linear_w4", MOE_FAST(linear_w4)},
    {"balance_loss", MOE_FAST(balance_loss)},
    {"router_backward", MOE_FAST(router_backward)},
    {"combine_backward", MOE_FAST(combine_backward)},
    {"last_error", last_error, METH_NOARGS, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&module); }
