// The decoding calls for Python: arguments checked, outputs and workspaces
// allocated, the C-ABI called on the current stream of the tensors' device.
// In Python itself these steps take twice as long as the launch they prepare,
// which is most of a decoding step's short calls.
#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <cmath>
#include <initializer_list>
#include <string>

#include "../../include/qwha.h"

namespace {

PyObject* g_error = nullptr;     // QwhaError(status, where)

struct Refused {};               // a Python error is set

[[noreturn]] void refuse(PyObject* kind, const std::string& what) {
  PyErr_SetString(kind, what.c_str());
  throw Refused{};
}

using Shape = std::initializer_list<int64_t>;

template <typename It>
std::string text(It b, It e) {
  std::string s = "(";
  for (It i = b; i != e; ++i) s += (i == b ? "" : ", ") + std::to_string(*i);
  return s + (e - b == 1 ? ",)" : ")");
}

const at::Tensor& tensor(PyObject* o, const char* name) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, std::string(name) + " must be a tensor");
  return THPVariable_Unpack(o);
}

const char* type_name(at::ScalarType t) {
  return t == at::kInt ? "torch.int32" : t == at::kFloat ? "torch.float32"
         : t == at::kBFloat16 ? "torch.bfloat16" : t == at::kByte ? "torch.uint8" : "another type";
}

// The address of a contiguous tensor of this type and shape on device `dev` (an
// index; -1: the CPU). Empty tensors have none.
void* given(const at::Tensor& t, at::ScalarType type, Shape shape, int dev, const char* name) {
  if (t.scalar_type() != type)
    refuse(PyExc_TypeError, std::string(name) + " must be " + type_name(type));
  const auto sizes = t.sizes();
  if (sizes.size() != shape.size() || !std::equal(shape.begin(), shape.end(), sizes.begin()))
    refuse(PyExc_ValueError, std::string(name) + " must have shape " +
                                 text(shape.begin(), shape.end()) + ", got " +
                                 text(sizes.begin(), sizes.end()));
  if (t.get_device() != dev)
    refuse(PyExc_ValueError, std::string(name) + " is on " + t.device().str() +
                                 ", not on the call's device");
  if (!t.is_contiguous()) refuse(PyExc_ValueError, "tensors must be contiguous");
  return t.numel() ? t.data_ptr() : nullptr;
}
template <typename P>
P* given(PyObject* o, at::ScalarType type, Shape shape, int dev, const char* name) {
  return static_cast<P*>(given(tensor(o, name), type, shape, dev, name));
}

qwha_dtype dtype_of(const at::Tensor& t) {
  if (t.scalar_type() == at::kFloat) return QWHA_F32;
  if (t.scalar_type() == at::kBFloat16) return QWHA_BF16;
  refuse(PyExc_TypeError, std::string("unsupported dtype ") + toString(t.scalar_type()));
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused{};
  return v;
}
// An int32 argument of the C-ABI; what does not fit is refused there, as -1
int32_t integer32(PyObject* o) {
  const int64_t v = integer(o);
  return v < INT32_MIN || v > INT32_MAX ? -1 : static_cast<int32_t>(v);
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused{};
  return v;
}
int32_t truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Refused{};
  return v;
}

// Makes the tensors' device current for a call, if it is not.
struct OnDevice {
  int back = -1;
  explicit OnDevice(int dev) {
    if (dev < 0) refuse(PyExc_ValueError, "tensors must live on the GPU");
    const int now = c10::hip::current_device();
    if (now != dev) {
      c10::hip::set_device(static_cast<c10::DeviceIndex>(dev));
      back = now;
    }
  }
  ~OnDevice() {
    if (back >= 0) c10::hip::set_device(static_cast<c10::DeviceIndex>(back));
  }
};
hipStream_t stream_of(int dev) {
  return c10::hip::getCurrentHIPStream(static_cast<c10::DeviceIndex>(dev)).stream();
}

// The caller's workspace, or one of `need` bytes from torch's allocator
struct Workspace {
  at::Tensor own;
  void* ptr = nullptr;
  size_t bytes = 0;
  template <typename Need>
  Workspace(PyObject* given_ws, const at::Tensor& like, int dev, Need&& need) {
    if (given_ws != Py_None) {
      const at::Tensor& t = tensor(given_ws, "ws");
      ptr = given(t, at::kByte, {t.numel()}, dev, "ws");
      bytes = static_cast<size_t>(t.numel());
    } else if (const size_t n = need(); n > 0) {
      own = at::empty({static_cast<int64_t>(n)}, like.options().dtype(at::kByte));
      ptr = own.data_ptr();
      bytes = n;
    }
  }
};

void check(qwha_status status, const char* where) {
  if (status == QWHA_OK) return;
  PyObject* e = PyObject_CallFunction(g_error, "is", static_cast<int>(status), where);
  if (e != nullptr) {
    PyErr_SetObject(g_error, e);
    Py_DECREF(e);
  }
  throw Refused{};
}

template <typename Fn>
PyObject* guarded(Py_ssize_t have, Py_ssize_t want, Fn&& fn) {
  HANDLE_TH_ERRORS
  if (have != want) {
    PyErr_Format(PyExc_TypeError, "%zd arguments, not %zd", want, have);
    return nullptr;
  }
  try {
    return fn();
  } catch (const Refused&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

PyObject* same(PyObject* o) {
  Py_INCREF(o);
  return o;
}

// x, codes, scales, zeros, bits, group, row_ptr, E, c, alpha, y, ws
PyObject* layer_decode(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 12, [&]() -> PyObject* {
    const at::Tensor &x = tensor(a[0], "x"), &scales = tensor(a[2], "scales");
    if (x.dim() != 2 || scales.dim() != 2)
      refuse(PyExc_ValueError, "x must be [T][d_in], scales [d_out][groups]");
    const int64_t T = x.size(0), d_in = x.size(1), d_out = scales.size(0), groups = scales.size(1);
    const int dev = static_cast<int>(x.get_device());
    const qwha_dtype act = dtype_of(x);
    const int64_t bits = integer(a[4]), group = integer(a[5]);
    if (bits != 2 && bits != 3 && bits != 4 && bits != 8)
      refuse(PyExc_ValueError, "bits=" + std::to_string(bits) + " is not one of 2, 3, 4, 8");
    if (group < 1 || groups != d_in / group || d_in % group != 0)
      refuse(PyExc_ValueError, "scales " + text(scales.sizes().begin(), scales.sizes().end()) +
                                   " do not hold " + std::to_string(d_in) +
                                   " columns in groups of " + std::to_string(group));
    const int64_t cpw = 32 / bits;
    const auto* codes =
        given<uint32_t>(a[1], at::kInt, {d_out, (d_in + cpw - 1) / cpw}, dev, "codes");
    const auto* s = given<float>(a[2], at::kFloat, {d_out, groups}, dev, "scales");
    const auto* z = given<float>(a[3], at::kFloat, {d_out, groups}, dev, "zeros");
    const int64_t p = a[8] == Py_None ? 0 : tensor(a[8], "c").numel();
    const int32_t *row_ptr = nullptr, *E = nullptr;
    const float* c = nullptr;
    if (p > 0) {
      row_ptr = given<int32_t>(a[6], at::kInt, {d_out + 1}, dev, "row_ptr");
      E = given<int32_t>(a[7], at::kInt, {p, 2}, dev, "E");
      c = given<float>(a[8], at::kFloat, {p}, dev, "c");
    }
    const void* xp = given(x, x.scalar_type(), {T, d_in}, dev, "x");
    const float alpha = static_cast<float>(number(a[9]));
    const OnDevice on(dev);
    at::Tensor out;
    if (a[10] == Py_None) out = at::empty({T, d_out}, x.options());
    const at::Tensor& y = a[10] == Py_None ? out : tensor(a[10], "y");
    void* yp = given(y, x.scalar_type(), {T, d_out}, dev, "y");
    if (d_in > INT32_MAX || d_out > INT32_MAX) refuse(PyExc_ValueError, "layer too large");
    const int32_t k = static_cast<int32_t>(d_in), rows = static_cast<int32_t>(d_out);
    const Workspace ws(a[11], x, dev, [&] { return qwha_layer_decode_workspace_bytes(T, k, rows, p); });
    check(qwha_layer_decode(xp, act, T, k, rows, codes, s, z, static_cast<int32_t>(bits),
                            static_cast<int32_t>(group), p, row_ptr, E, c, alpha, yp, ws.ptr,
                            ws.bytes, stream_of(dev)),
          "qwha_layer_decode");
    return a[10] == Py_None ? THPVariable_Wrap(out) : same(a[10]);
  });
}

// A cache of rows of head_dim columns and `heads` heads: codes, scales, zeros
struct CacheArgs {
  uint32_t* codes;
  float *scales, *zeros;
  int64_t n_pages;
  int32_t page;
  CacheArgs(PyObject* c, PyObject* s, PyObject* z, int64_t heads, int64_t head_dim, int64_t bits,
            int dev) {
    const at::Tensor& t = tensor(c, "codes");
    if (t.dim() != 5)
      refuse(PyExc_ValueError, "codes must be [2][n_pages][heads][page][words]");
    n_pages = t.size(1);
    const int64_t p = t.size(3);
    codes = static_cast<uint32_t*>(
        given(t, at::kInt, {2, n_pages, heads, p, head_dim * bits / 32}, dev, "codes"));
    scales = given<float>(s, at::kFloat, {2, n_pages, heads, p}, dev, "scales");
    zeros = given<float>(z, at::kFloat, {2, n_pages, heads, p}, dev, "zeros");
    page = p > INT32_MAX ? -1 : static_cast<int32_t>(p);
  }
};

int32_t to32(int64_t v) { return v > INT32_MAX ? -1 : static_cast<int32_t>(v); }

// k, v, slots, codes, scales, zeros, bits, rotate
PyObject* cache_write(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> PyObject* {
    const at::Tensor& k = tensor(a[0], "k");
    if (k.dim() != 3) refuse(PyExc_ValueError, "k must be [T][heads][head_dim]");
    const int64_t T = k.size(0), heads = k.size(1), dim = k.size(2);
    const int dev = static_cast<int>(k.get_device());
    const qwha_dtype act = dtype_of(k);
    const int32_t bits = integer32(a[6]);
    const CacheArgs c(a[3], a[4], a[5], heads, dim, bits, dev);
    const void* kp = given(k, k.scalar_type(), {T, heads, dim}, dev, "k");
    const void* vp = given(tensor(a[1], "v"), k.scalar_type(), {T, heads, dim}, dev, "v");
    const auto* slots = given<int32_t>(a[2], at::kInt, {T}, dev, "slots");
    const int32_t rotate = truth(a[7]);
    const OnDevice on(dev);
    check(qwha_cache_write(kp, vp, act, T, slots, to32(heads), to32(dim), bits, rotate, c.n_pages,
                           c.page, c.codes, c.scales, c.zeros, stream_of(dev)),
          "qwha_cache_write");
    return same(Py_None);
  });
}

// codes, scales, zeros, slots, bits, head_dim, rotate, fp32 output, k, v
PyObject* cache_read(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 10, [&]() -> PyObject* {
    const at::Tensor &codes = tensor(a[0], "codes"), &slots = tensor(a[3], "slots");
    if (codes.dim() != 5)
      refuse(PyExc_ValueError, "codes must be [2][n_pages][heads][page][words]");
    const int64_t T = slots.numel(), heads = codes.size(2), dim = integer(a[5]);
    const int dev = static_cast<int>(codes.get_device());
    const int32_t bits = integer32(a[4]);
    const CacheArgs c(a[0], a[1], a[2], heads, dim, bits, dev);
    const auto* sp = given<int32_t>(a[3], at::kInt, {T}, dev, "slots");
    const int32_t rotate = truth(a[6]);
    const OnDevice on(dev);
    at::Tensor out[2];
    const auto type = truth(a[7]) ? at::kFloat : at::kBFloat16;
    const auto options = codes.options().dtype(
        a[8] != Py_None ? tensor(a[8], "k").scalar_type()
                        : a[9] != Py_None ? tensor(a[9], "v").scalar_type() : type);
    void* p[2];
    for (int i = 0; i < 2; ++i) {
      if (a[8 + i] == Py_None) out[i] = at::empty({T, heads, dim}, options);
      const at::Tensor& t = a[8 + i] == Py_None ? out[i] : tensor(a[8 + i], i ? "v" : "k");
      p[i] = given(t, options.dtype().toScalarType(), {T, heads, dim}, dev, i ? "v" : "k");
      if (i == 0) dtype_of(t);
    }
    const qwha_dtype act = options.dtype().toScalarType() == at::kFloat ? QWHA_F32 : QWHA_BF16;
    check(qwha_cache_read(c.codes, c.scales, c.zeros, to32(heads), to32(dim), bits, rotate,
                          c.n_pages, c.page, sp, T, act, p[0], p[1], stream_of(dev)),
          "qwha_cache_read");
    PyObject* k = a[8] == Py_None ? THPVariable_Wrap(out[0]) : same(a[8]);
    PyObject* v = a[9] == Py_None ? THPVariable_Wrap(out[1]) : same(a[9]);
    PyObject* both = PyTuple_Pack(2, k, v);
    Py_DECREF(k);
    Py_DECREF(v);
    return both;
  });
}

// q, codes, scales, zeros, table, lens, bits, rotate, scale, out, ws
PyObject* cache_attn(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> PyObject* {
    const at::Tensor &q = tensor(a[0], "q"), &codes = tensor(a[1], "codes"),
                     &table = tensor(a[4], "table");
    if (q.dim() != 3 || table.dim() != 2 || codes.dim() != 5)
      refuse(PyExc_ValueError,
             "q must be [B][q_heads][head_dim], table [B][width], codes "
             "[2][n_pages][heads][page][words]");
    const int64_t B = q.size(0), q_heads = q.size(1), dim = q.size(2), width = table.size(1);
    const int64_t heads = codes.size(2);
    const int dev = static_cast<int>(q.get_device());
    const qwha_dtype act = dtype_of(q);
    const int32_t bits = integer32(a[6]);
    const CacheArgs c(a[1], a[2], a[3], heads, dim, bits, dev);
    const void* qp = given(q, q.scalar_type(), {B, q_heads, dim}, dev, "q");
    const auto* tp = given<int32_t>(a[4], at::kInt, {B, width}, dev, "table");
    const auto* lp = given<int32_t>(a[5], at::kInt, {B}, dev, "lens");
    const int32_t rotate = truth(a[7]);
    const float scale = static_cast<float>(
        a[8] == Py_None ? 1.0 / std::sqrt(static_cast<double>(dim)) : number(a[8]));
    const OnDevice on(dev);
    at::Tensor own;
    if (a[9] == Py_None) own = at::empty({B, q_heads, dim}, q.options());
    const at::Tensor& out = a[9] == Py_None ? own : tensor(a[9], "out");
    void* op = given(out, q.scalar_type(), {B, q_heads, dim}, dev, "out");
    const Workspace ws(a[10], q, dev, [&] {
      return qwha_cache_attn_workspace_bytes(to32(B), to32(q_heads), to32(heads), to32(dim),
                                             to32(width), c.page);
    });
    check(qwha_cache_attn(qp, act, to32(B), to32(q_heads), c.codes, c.scales, c.zeros, to32(heads),
                          to32(dim), bits, rotate, c.n_pages, c.page, tp, to32(width), lp, scale,
                          op, ws.ptr, ws.bytes, stream_of(dev)),
          "qwha_cache_attn");
    return a[9] == Py_None ? THPVariable_Wrap(own) : same(a[9]);
  });
}

PyObject* set_error(PyObject*, PyObject* cls) {
  Py_INCREF(cls);
  Py_XSETREF(g_error, cls);
  Py_RETURN_NONE;
}

template <typename F>
PyCFunction fast(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f));
}

PyMethodDef methods[] = {
    {"layer_decode", fast(layer_decode), METH_FASTCALL, nullptr},
    {"cache_write", fast(cache_write), METH_FASTCALL, nullptr},
    {"cache_read", fast(cache_read), METH_FASTCALL, nullptr},
    {"cache_attn", fast(cache_attn), METH_FASTCALL, nullptr},
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
