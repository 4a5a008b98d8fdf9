// binding.cpp -- the short way into the calls around the attention: the checks
// and allocations of __init__.py's functions for the everyday call (no output
// or stream given, tensors on the current device; eps and theta floats, axes a
// tuple, flags truth values), without the interpreter.  A call that is anything else, or that the library refuses,
// answers None, and the Python function of the same name goes through its
// checks and says what is wrong; so every rule is stated there, and this file
// may only accept what it would accept.
//
// At one token the kernels take 2 to 5 us, this way 3.5 to 6 and the Python way
// 14 to 19.  Where this file is not built, or built for another torch or Python,
// the Python way serves alone (__init__.py, _CheckedWay).
#include <Python.h>

#include <dlfcn.h>

#include <cstdint>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/fqa.h"

namespace {

decltype(&fqa_mx_quantize) mx_quantize;
decltype(&fqa_mx_rms_norm) mx_rms_norm;
decltype(&fqa_mx_dequantize) mx_dequantize;
decltype(&fqa_mx_matmul) mx_matmul;
decltype(&fqa_rotary) rotary;
PyObject* microscaled_type;
PyObject* rotary_type;

constexpr int64_t kMaxRows = 1 << 24, kMaxCols = 1 << 20;

// A tensor on the current device, or nothing.
const at::Tensor* tensor(PyObject* o, int device) {
  if (device < 0 || !THPVariable_Check(o)) return nullptr;
  const at::Tensor& t = THPVariable_Unpack(o);
  return t.is_cuda() && t.layout() == at::kStrided && t.get_device() == device ? &t : nullptr;
}

// The device of a call's first tensor, if it is the current one, else -1 (which
// no tensor is on).
int device_of(PyObject* o) {
  if (!THPVariable_Check(o)) return -1;
  const at::Tensor& t = THPVariable_Unpack(o);
  if (!t.is_cuda()) return -1;
  const int d = t.get_device();
  return d == c10::cuda::current_device() ? d : -1;
}

int device_of_codes(PyObject* o) {
  return (PyObject*)Py_TYPE(o) == microscaled_type ? device_of(PyTuple_GET_ITEM(o, 0)) : -1;
}

int float_type(const at::Tensor& t) {
  switch (t.scalar_type()) {
    case at::kBFloat16: return FQA_DTYPE_BF16;
    case at::kFloat: return FQA_DTYPE_F32;
    case at::kHalf: return FQA_DTYPE_F16;
    default: return -1;
  }
}

int format(PyObject* o) {
  if (!PyUnicode_Check(o)) return -1;
  if (PyUnicode_CompareWithASCIIString(o, "mxfp8") == 0) return FQA_MXFP8;
  if (PyUnicode_CompareWithASCIIString(o, "mxfp4") == 0) return FQA_MXFP4;
  if (PyUnicode_CompareWithASCIIString(o, "nvfp4") == 0) return FQA_NVFP4;
  return -1;
}

bool small_int(PyObject* o, long long* v) {
  if (!PyLong_CheckExact(o)) return false;
  int over = 0;
  *v = PyLong_AsLongLongAndOverflow(o, &over);
  return over == 0 && !(*v == -1 && PyErr_Occurred());
}

at::Tensor empty(at::IntArrayRef shape, at::ScalarType type, int device) {
  return at::detail::empty_cuda(shape, type, at::Device(at::kCUDA, (at::DeviceIndex)device), std::nullopt);
}

void* stream(int device) { return c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream(); }

// [..., K] as M rows of K at a common stride.
bool rows(const at::Tensor& x, int64_t* M, int64_t* K, int64_t* ld) {
  const int64_t d = x.dim();
  if (d < 2) return false;
  *K = x.size(d - 1);
  if (*K < 1 || *K > kMaxCols) return false;
  if (d == 2) {
    *M = x.size(0);
    if (*K > 1 && x.stride(1) != 1) return false;
    *ld = *M > 1 ? x.stride(0) : *K;
  } else {
    if (!x.is_contiguous()) return false;
    *M = x.numel() / *K;
    *ld = *K;
  }
  return *M <= kMaxRows;
}

struct MxShape {
  int64_t codes[2], scales[5];
  MxShape(int64_t M, int64_t K, int fmt) {
    const int64_t kp = (K + 31) / 32 * 32, width = fmt == FQA_NVFP4 ? 64 : 128;
    codes[0] = M;
    codes[1] = fmt == FQA_MXFP8 ? kp : kp / 2;
    const int64_t s[5] = {(M + 127) / 128, (kp + width - 1) / width, 32, 4, 4};
    for (int i = 0; i < 5; ++i) scales[i] = s[i];
  }
};

bool plain(const at::Tensor& t, at::ScalarType type, at::IntArrayRef shape) {
  return t.scalar_type() == type && t.sizes() == shape && t.is_contiguous();
}

struct Mx {
  const at::Tensor *codes, *scales, *row_scale;
  int64_t M, K;
  int fmt;
};

bool microscaled(PyObject* o, int device, Mx* q) {
  if ((PyObject*)Py_TYPE(o) != microscaled_type) return false;
  long long K;
  q->fmt = format(PyTuple_GET_ITEM(o, 4));
  q->codes = tensor(PyTuple_GET_ITEM(o, 0), device);
  q->scales = tensor(PyTuple_GET_ITEM(o, 1), device);
  q->row_scale = nullptr;
  if (q->fmt < 0 || !q->codes || !q->scales || !small_int(PyTuple_GET_ITEM(o, 3), &K) || K < 1 || K > kMaxCols ||
      q->codes->dim() != 2 || q->codes->size(0) > kMaxRows)
    return false;
  q->M = q->codes->size(0);
  q->K = K;
  const MxShape s(q->M, K, q->fmt);
  if (!plain(*q->codes, at::kByte, s.codes) || !plain(*q->scales, at::kByte, s.scales)) return false;
  PyObject* r = PyTuple_GET_ITEM(o, 2);
  if (q->fmt != FQA_NVFP4) return r == Py_None;
  q->row_scale = tensor(r, device);
  return q->row_scale && plain(*q->row_scale, at::kFloat, {q->M});
}

float* row_scale(const Mx& q) { return q.row_scale ? q.row_scale->data_ptr<float>() : nullptr; }

// New microscaled rows and the tuple that holds them.
struct NewMx {
  at::Tensor codes, scales, row_scale;
  NewMx(int64_t M, int64_t K, int fmt, int device) {
    const MxShape s(M, K, fmt);
    codes = empty(s.codes, at::kByte, device);
    scales = empty(s.scales, at::kByte, device);
    if (fmt == FQA_NVFP4) row_scale = empty({M}, at::kFloat, device);
  }
  float* row_ptr() const { return row_scale.defined() ? row_scale.data_ptr<float>() : nullptr; }
  PyObject* wrap(int64_t K, PyObject* fmt) const {
    PyObject* c = THPVariable_Wrap(codes);
    PyObject* s = THPVariable_Wrap(scales);
    PyObject* r = row_scale.defined() ? THPVariable_Wrap(row_scale) : Py_NewRef(Py_None);
    PyObject* k = PyLong_FromLongLong(K);
    PyObject* out = c && s && r && k ? PyObject_CallFunctionObjArgs(microscaled_type, c, s, r, k, fmt, nullptr) : nullptr;
    Py_XDECREF(c);
    Py_XDECREF(s);
    Py_XDECREF(r);
    Py_XDECREF(k);
    return out;
  }
};

at::ScalarType out_type(long long t) {
  return t == FQA_DTYPE_BF16 ? at::kBFloat16 : t == FQA_DTYPE_F32 ? at::kFloat : at::kHalf;
}

// quantize(x, fmt)
PyObject* quantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 2) Py_RETURN_NONE;
  const int device = device_of(a[0]), fmt = format(a[1]);
  const at::Tensor* x = tensor(a[0], device);
  int64_t M, K, ld;
  if (fmt < 0 || !x || float_type(*x) < 0 || !rows(*x, &M, &K, &ld)) Py_RETURN_NONE;
  const NewMx out(M, K, fmt, device);
  if (mx_quantize(x->data_ptr(), (fqa_dtype)float_type(*x), (int)M, (int)K, ld, (fqa_mx_format)fmt,
                  out.codes.data_ptr<uint8_t>(), out.scales.data_ptr<uint8_t>(), out.row_ptr(), stream(device)) != FQA_OK)
    Py_RETURN_NONE;
  return out.wrap(K, a[1]);
  END_HANDLE_TH_ERRORS
}

// dequantize(q, out_dtype)
PyObject* dequantize(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  long long type;
  Mx q;
  if (n != 2) Py_RETURN_NONE;
  const int device = device_of_codes(a[0]);
  if ( !small_int(a[1], &type) || type < 0 || type > 2 || !microscaled(a[0], device, &q)) Py_RETURN_NONE;
  at::Tensor out = empty({q.M, q.K}, out_type(type), device);
  if (mx_dequantize(q.codes->data_ptr<uint8_t>(), q.scales->data_ptr<uint8_t>(), row_scale(q), (int)q.M, (int)q.K,
                    (fqa_mx_format)q.fmt, out.data_ptr(), (fqa_dtype)type, stream(device)) != FQA_OK)
    Py_RETURN_NONE;
  return THPVariable_Wrap(out);
  END_HANDLE_TH_ERRORS
}

// rms_norm(x, weight, fmt, residual, eps)
PyObject* rms_norm(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 5 || !PyFloat_CheckExact(a[4])) Py_RETURN_NONE;
  const int device = device_of(a[0]), fmt = format(a[2]);
  const at::Tensor *x = tensor(a[0], device), *w = tensor(a[1], device);
  int64_t M, K, ld;
  if (fmt < 0 || !x || !w || float_type(*x) < 0 || !rows(*x, &M, &K, &ld)) Py_RETURN_NONE;
  const int type = float_type(*x);
  if ((w->scalar_type() != x->scalar_type() && w->scalar_type() != at::kFloat) || w->dim() != 1 || w->size(0) != K ||
      !w->is_contiguous())
    Py_RETURN_NONE;
  const at::Tensor* r = nullptr;
  int64_t Mr, Kr, ldr = K;
  at::Tensor h;
  if (a[3] != Py_None) {
    r = tensor(a[3], device);
    if (!r || r->sizes() != x->sizes() || (r->scalar_type() != x->scalar_type() && r->scalar_type() != at::kFloat) ||
        !rows(*r, &Mr, &Kr, &ldr))
      Py_RETURN_NONE;
    h = empty(x->sizes(), r->scalar_type(), device);
  }
  const NewMx out(M, K, fmt, device);
  if (mx_rms_norm(x->data_ptr(), (fqa_dtype)type, (int)M, (int)K, ld, w->data_ptr(), (fqa_dtype)float_type(*w),
                  (float)PyFloat_AS_DOUBLE(a[4]), r ? r->data_ptr() : nullptr, (fqa_dtype)(r ? float_type(*r) : type), ldr,
                  (fqa_mx_format)fmt, out.codes.data_ptr<uint8_t>(), out.scales.data_ptr<uint8_t>(), out.row_ptr(),
                  r ? h.data_ptr() : nullptr, stream(device)) != FQA_OK)
    Py_RETURN_NONE;
  PyObject* y = out.wrap(K, a[2]);
  PyObject* hh = r ? THPVariable_Wrap(h) : Py_NewRef(Py_None);
  PyObject* both = y && hh ? PyTuple_Pack(2, y, hh) : nullptr;
  Py_XDECREF(y);
  Py_XDECREF(hh);
  return both;
  END_HANDLE_TH_ERRORS
}

// matmul(a, b, bias, out_dtype)
PyObject* matmul(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  long long type;
  Mx p, q;
  if (n != 4) Py_RETURN_NONE;
  const int device = device_of_codes(a[0]);
  if ( !small_int(a[3], &type) || type < 0 || type > 2 || !microscaled(a[0], device, &p) ||
      !microscaled(a[1], device, &q) || p.fmt != q.fmt || p.K != q.K)
    Py_RETURN_NONE;
  const at::Tensor* bias = nullptr;
  if (a[2] != Py_None) {
    bias = tensor(a[2], device);
    if (!bias || !plain(*bias, at::kFloat, {q.M})) Py_RETURN_NONE;
  }
  at::Tensor out = empty({p.M, q.M}, out_type(type), device);
  if (mx_matmul(p.codes->data_ptr<uint8_t>(), p.scales->data_ptr<uint8_t>(), row_scale(p), q.codes->data_ptr<uint8_t>(),
                q.scales->data_ptr<uint8_t>(), row_scale(q), bias ? bias->data_ptr<float>() : nullptr, (int)p.M, (int)q.M,
                (int)p.K, (fqa_mx_format)p.fmt, out.data_ptr(), (fqa_dtype)type, stream(device)) != FQA_OK)
    Py_RETURN_NONE;
  return THPVariable_Wrap(out);
  END_HANDLE_TH_ERRORS
}

// rotate(q, k, rot, inverse)
PyObject* rotate(PyObject*, PyObject* const* a, Py_ssize_t n) {
  HANDLE_TH_ERRORS
  if (n != 4 || (PyObject*)Py_TYPE(a[2]) != rotary_type) Py_RETURN_NONE;
  const int device = device_of(a[0]);
  PyObject* f[8];                      // positions, axes, theta, split, shared, q_weight, k_weight, eps
  for (int i = 0; i < 8; ++i) f[i] = PyTuple_GET_ITEM(a[2], i);
  const at::Tensor *q = tensor(a[0], device), *k = nullptr, *pos = tensor(f[0], device);
  if (!q || !pos || q->dim() != 4 || q->size(3) != 128 || q->stride(3) != 1 || float_type(*q) < 0) Py_RETURN_NONE;
  if (a[1] != Py_None) {
    k = tensor(a[1], device);
    if (!k || k->dim() != 4 || k->scalar_type() != q->scalar_type() || k->size(0) != q->size(0) ||
        k->size(2) != q->size(2) || k->size(3) != 128 || k->stride(3) != 1)
      Py_RETURN_NONE;
  }
  const int64_t B = q->size(0), Hq = q->size(1), N = q->size(2), Hk = k ? k->size(1) : 0;
  if (B > INT32_MAX || Hq > INT32_MAX || N > INT32_MAX || Hk > INT32_MAX) Py_RETURN_NONE;
  int axes[4];
  if (!PyTuple_CheckExact(f[1])) Py_RETURN_NONE;
  const int64_t A = PyTuple_GET_SIZE(f[1]);
  if (A < 1 || A > 4) Py_RETURN_NONE;
  for (int i = 0; i < A; ++i) {
    long long v;
    if (!small_int(PyTuple_GET_ITEM(f[1], i), &v) || v < 2 || v > 128) Py_RETURN_NONE;
    axes[i] = (int)v;
  }
  const bool pf = pos->scalar_type() == at::kFloat;
  if ((!pf && pos->scalar_type() != at::kInt) || !pos->is_contiguous()) Py_RETURN_NONE;
  int64_t psb = 0;
  if (pos->dim() == 3 && pos->size(1) == N && pos->size(2) == A && (pos->size(0) == B || pos->size(0) == 1))
    psb = pos->size(0) > 1 ? N * A : 0;
  else if (pos->dim() != 2 || pos->size(0) != N || pos->size(1) != A)
    Py_RETURN_NONE;
  if (!PyFloat_CheckExact(f[2]) || !PyFloat_CheckExact(f[7]) || !PyBool_Check(f[3]) || !PyBool_Check(f[4]) ||
      !PyBool_Check(a[3]))
    Py_RETURN_NONE;
  const at::Tensor* w[2] = {nullptr, nullptr};
  for (int i = 0; i < 2; ++i)
    if (f[5 + i] != Py_None) {
      w[i] = tensor(f[5 + i], device);
      if (!w[i] || !plain(*w[i], q->scalar_type(), {128})) Py_RETURN_NONE;
    }
  at::Tensor qo = empty(q->sizes(), q->scalar_type(), device), ko;
  if (k) ko = empty(k->sizes(), q->scalar_type(), device);
  const int flags = (f[3] == Py_True ? FQA_ROTARY_SPLIT : 0) | (f[4] == Py_True ? FQA_ROTARY_SHARED : 0) |
                    (a[3] == Py_True ? FQA_ROTARY_INVERSE : 0);
  if (rotary(q->data_ptr(), k ? k->data_ptr() : nullptr, (fqa_dtype)float_type(*q), (int)B, (int)Hq, (int)Hk, (int)N, 128,
             q->stride(0), q->stride(1), q->stride(2), k ? k->stride(0) : 0, k ? k->stride(1) : 0, k ? k->stride(2) : 0,
             pos->data_ptr(), pf ? FQA_DTYPE_F32 : FQA_DTYPE_I32, psb, (int)A, axes, PyFloat_AS_DOUBLE(f[2]), flags,
             w[0] ? w[0]->data_ptr() : nullptr, w[1] ? w[1]->data_ptr() : nullptr, (float)PyFloat_AS_DOUBLE(f[7]),
             qo.data_ptr(), k ? ko.data_ptr() : nullptr, stream(device)) != FQA_OK)
    Py_RETURN_NONE;
  PyObject* x = THPVariable_Wrap(qo);
  PyObject* y = k ? THPVariable_Wrap(ko) : Py_NewRef(Py_None);
  PyObject* both = x && y ? PyTuple_Pack(2, x, y) : nullptr;
  Py_XDECREF(x);
  Py_XDECREF(y);
  return both;
  END_HANDLE_TH_ERRORS
}

// init(path of libfqa.so, Microscaled, Rotary)
PyObject* init(PyObject*, PyObject* args) {
  const char* path;
  PyObject *m, *r;
  if (!PyArg_ParseTuple(args, "sOO", &path, &m, &r)) return nullptr;
  void* lib = dlopen(path, RTLD_NOW | RTLD_LOCAL);
  if (!lib) {
    PyErr_SetString(PyExc_ImportError, dlerror());
    return nullptr;
  }
  mx_quantize = reinterpret_cast<decltype(mx_quantize)>(dlsym(lib, "fqa_mx_quantize"));
  mx_rms_norm = reinterpret_cast<decltype(mx_rms_norm)>(dlsym(lib, "fqa_mx_rms_norm"));
  mx_dequantize = reinterpret_cast<decltype(mx_dequantize)>(dlsym(lib, "fqa_mx_dequantize"));
  mx_matmul = reinterpret_cast<decltype(mx_matmul)>(dlsym(lib, "fqa_mx_matmul"));
  rotary = reinterpret_cast<decltype(rotary)>(dlsym(lib, "fqa_rotary"));
  if (!mx_quantize || !mx_rms_norm || !mx_dequantize || !mx_matmul || !rotary) {
    PyErr_SetString(PyExc_ImportError, "libfqa.so lacks a call");
    return nullptr;
  }
  microscaled_type = Py_NewRef(m);
  rotary_type = Py_NewRef(r);
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {{"init", init, METH_VARARGS, nullptr},
                         {"quantize", (PyCFunction)(void (*)(void))quantize, METH_FASTCALL, nullptr},
                         {"dequantize", (PyCFunction)(void (*)(void))dequantize, METH_FASTCALL, nullptr},
                         {"rms_norm", (PyCFunction)(void (*)(void))rms_norm, METH_FASTCALL, nullptr},
                         {"matmul", (PyCFunction)(void (*)(void))matmul, METH_FASTCALL, nullptr},
                         {"rotate", (PyCFunction)(void (*)(void))rotate, METH_FASTCALL, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

extern "C" __attribute__((visibility("default"))) PyObject* PyInit__binding(void) { return PyModule_Create(&module); }
