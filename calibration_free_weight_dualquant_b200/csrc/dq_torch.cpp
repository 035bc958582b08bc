// dq_torch.cpp -- argument marshalling of the linear layer's calls for torch
// tensors: checks, output allocation and the C call of dq_matmul, dq_norm_quant
// and dq_glu_quant, as a CPython module (binding.py chooses device and stream
// and calls it).  A single token's kernel takes 2 to 6 us; the same marshalling
// in Python took 8 to 13 us a call, compiled it takes 2.  No arithmetic here.
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstring>
#include <string>

#include "dq.h"

namespace {

PyObject* g_error = nullptr;  // binding.DQError
PyObject *k_codes, *k_scales, *k_tensor, *k_residual, *k_workspace;

struct Fail {};  // a Python exception is set

[[noreturn]] void fail(int status, const char* where, const std::string& what = std::string()) {
  const std::string msg = what.empty() ? std::string(where) : std::string(where) + ": " + what;
  PyObject* args = Py_BuildValue("(is)", status, msg.c_str());
  if (args) {
    PyErr_SetObject(g_error, args);
    Py_DECREF(args);
  }
  throw Fail();
}

struct Format {
  int id, group, per_byte;
  bool tensor_scale;
};
Format format_of(PyObject* o) {
  const int id = (int)PyLong_AsLong(o);
  return Format{id, id == DQ_NVFP4 ? 16 : 32, id == DQ_MXFP8 ? 1 : 2, id == DQ_NVFP4};
}

int dtype_of(at::ScalarType t) {
  return t == at::kFloat ? DQ_F32 : (t == at::kBFloat16 ? DQ_BF16 : (t == at::kHalf ? DQ_F16 : -1));
}
bool is_half(at::ScalarType t) { return t == at::kBFloat16 || t == at::kHalf; }

at::Tensor tensor(PyObject* o, const char* where) {
  if (!THPVariable_Check(o)) fail(DQ_EINVAL, where, "a torch tensor is needed");
  return THPVariable_Unpack(o);
}
at::Tensor item(PyObject* dict, PyObject* key, const char* where) {
  PyObject* o = PyObject_GetItem(dict, key);
  if (!o) throw Fail();  // KeyError, as from the dict itself
  if (!THPVariable_Check(o)) {
    Py_DECREF(o);
    fail(DQ_EINVAL, where, "a torch tensor is needed");
  }
  at::Tensor t = THPVariable_Unpack(o);
  Py_DECREF(o);
  return t;
}

at::Tensor empty(at::IntArrayRef size, at::ScalarType t, at::Device dev) {
  return at::detail::empty_cuda(size, t, dev, c10::nullopt);
}

void set(PyObject* dict, PyObject* key, const at::Tensor& t) {
  PyObject* o = THPVariable_Wrap(t);
  const bool ok = o && PyDict_SetItem(dict, key, o) == 0;
  Py_XDECREF(o);
  if (!ok) throw Fail();
}

// A quantized matrix {"codes", "block_scales", "tensor_scale"} of the format.
struct Quantized {
  at::Tensor codes, scales, sT;
  int64_t rows, cols;
  dq_outputs out{};
};
void quantized(Quantized* q, PyObject* dict, const Format& f, at::Device dev, const char* where) {
  q->codes = item(dict, k_codes, where);
  q->scales = item(dict, k_scales, where);
  if (q->codes.dim() != 2 || q->codes.scalar_type() != at::kByte || !q->codes.is_contiguous() || q->codes.device() != dev)
    fail(DQ_EINVAL, where, "codes must be a contiguous 2-D uint8 tensor on the call's device");
  q->rows = q->codes.size(0);
  q->cols = q->codes.size(1) * f.per_byte;
  if (q->scales.scalar_type() != at::kByte || !q->scales.is_contiguous() || q->scales.device() != dev || q->scales.dim() != 2 ||
      q->scales.size(0) != q->rows || q->scales.size(1) != q->cols / f.group)
    fail(DQ_EINVAL, where, "block_scales must be contiguous uint8 [rows][cols/group] on the call's device");
  q->out.codes = q->codes.data_ptr();
  q->out.block_scales = q->scales.data_ptr();
  if (f.tensor_scale) {
    PyObject* o = PyObject_GetItem(dict, k_tensor);
    if (!o) PyErr_Clear();
    if (o && THPVariable_Check(o)) q->sT = THPVariable_Unpack(o);
    Py_XDECREF(o);
    if (!q->sT.defined() || q->sT.scalar_type() != at::kFloat || q->sT.numel() != 1 || q->sT.device() != dev)
      fail(DQ_EINVAL, where, "NVFP4 needs a one-element float32 tensor_scale on the call's device");
    q->out.tensor_scale = static_cast<float*>(q->sT.data_ptr());
  }
}

// The outputs of a row quantizer: the caller's dict or a new one.
PyObject* row_outputs(Quantized* q, PyObject* out, int64_t rows, int64_t cols, const Format& f, at::Device dev,
                      const char* where) {
  if (out != Py_None) {
    quantized(q, out, f, dev, where);
    if (q->rows != rows || q->cols != cols) fail(DQ_EINVAL, where, "codes of another shape than the call's");
    Py_INCREF(out);
    return out;
  }
  if (cols % f.group != 0) fail(DQ_EINVAL, where, "columns are not a multiple of the group");
  q->codes = empty({rows, cols / f.per_byte}, at::kByte, dev);
  q->scales = empty({rows, cols / f.group}, at::kByte, dev);
  q->out.codes = q->codes.data_ptr();
  q->out.block_scales = q->scales.data_ptr();
  PyObject* d = PyDict_New();
  if (!d) throw Fail();
  try {
    set(d, k_codes, q->codes);
    set(d, k_scales, q->scales);
    if (f.tensor_scale) {
      q->sT = empty({1}, at::kFloat, dev);
      q->out.tensor_scale = static_cast<float*>(q->sT.data_ptr());
      set(d, k_tensor, q->sT);
    }
  } catch (...) {
    Py_DECREF(d);
    throw;
  }
  return d;
}

// The caller's workspace, or a new one of `need` bytes (none for 0).
at::Tensor workspace_of(PyObject* o, int64_t need, at::Device dev, const char* where) {
  if (o == Py_None) return need ? empty({need}, at::kByte, dev) : at::Tensor();
  at::Tensor w = tensor(o, where);
  if (w.device() != dev || w.scalar_type() != at::kByte || !w.is_contiguous())
    fail(DQ_EINVAL, where, "workspace must be a contiguous uint8 tensor on the call's device");
  return w;
}
void* ptr(const at::Tensor& t) { return t.defined() ? t.data_ptr() : nullptr; }
size_t bytes(const at::Tensor& t) { return t.defined() ? (size_t)t.numel() : 0; }

// A [cols] vector of 16-bit floats, or nothing.
at::Tensor channels(PyObject* o, int64_t cols, at::Device dev, const char* where) {
  if (o == Py_None) return at::Tensor();
  at::Tensor t = tensor(o, where);
  if (!is_half(t.scalar_type()) || t.numel() != cols || !t.is_contiguous() || t.device() != dev)
    fail(DQ_EINVAL, where, "must be a contiguous 16-bit float [cols] tensor on the call's device");
  return t;
}

// Launches and, with `check`, waits: without the interpreter's lock.
template <class F>
void run(F&& f, bool check, const at::Tensor& ws, void* stream, const char* where) {
  int st, dev = DQ_OK;
  Py_BEGIN_ALLOW_THREADS;
  st = f();
  if (st == DQ_OK && check) dev = dq_sync_status(ptr(ws), stream);
  Py_END_ALLOW_THREADS;
  if (st != DQ_OK) fail(st, where);
  if (dev != DQ_OK) fail(dev, (std::string(where) + " (device)").c_str());
}

template <class F>
PyObject* guarded(Py_ssize_t n, Py_ssize_t want, F&& f) {
  if (n != want) {
    PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
    return nullptr;
  }
  HANDLE_TH_ERRORS  // torch's exceptions as torch raises them: an allocation that failed is its OutOfMemoryError
  try {
    return f();
  } catch (const Fail&) {
    return nullptr;
  }
  END_HANDLE_TH_ERRORS
}

// matmul(stream, X, W, format, out, out_dtype, workspace, check) -> Y
PyObject* matmul(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> PyObject* {
    void* stream = PyLong_AsVoidPtr(a[0]);
    const Format f = format_of(a[3]);
    const bool check = a[7] == Py_True;
    const at::Device dev = item(a[1], k_codes, "dq_matmul: X").device();
    Quantized x, w;
    quantized(&x, a[1], f, dev, "dq_matmul: X");
    quantized(&w, a[2], f, dev, "dq_matmul: W");
    if (x.cols != w.cols) fail(DQ_EINVAL, "dq_matmul", "X and W differ in their columns");
    at::Tensor y;
    if (a[4] == Py_None) {
      const int dt = (int)PyLong_AsLong(a[5]);
      y = empty({x.rows, w.rows}, dt == DQ_F32 ? at::kFloat : (dt == DQ_BF16 ? at::kBFloat16 : at::kHalf), dev);
    } else {
      y = tensor(a[4], "dq_matmul: out");
      if (dtype_of(y.scalar_type()) < 0 || y.dim() != 2 || y.size(0) != x.rows || y.size(1) != w.rows || !y.is_contiguous() ||
          y.device() != dev)
        fail(DQ_EINVAL, "dq_matmul: out", "must be contiguous f32/bf16/f16 [tokens, rows] on the call's device");
    }
    const at::Tensor ws = workspace_of(a[6], check ? DQ_MATMUL_WORKSPACE_BYTES : 0, dev, "dq_matmul");
    run(
        [&] {
          return dq_matmul(&x.out, x.rows, &w.out, w.rows, x.cols, f.id, f.group, y.data_ptr(), dtype_of(y.scalar_type()),
                           ptr(ws), bytes(ws), stream);
        },
        check, ws, stream, "dq_matmul");
    return THPVariable_Wrap(y);
  });
}

// norm_quant(stream, X, weight, col_scales, format, residual, eps, out, residual_out, workspace, check) -> dict
PyObject* norm_quant(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 11, [&]() -> PyObject* {
    const char* where = "dq_norm_quant";
    void* stream = PyLong_AsVoidPtr(a[0]);
    const Format f = format_of(a[4]);
    const double eps = PyFloat_AsDouble(a[6]);
    if (eps == -1.0 && PyErr_Occurred()) throw Fail();
    const bool check = a[10] == Py_True;
    const at::Tensor x = tensor(a[1], where);
    if (!x.is_cuda() || !is_half(x.scalar_type()) || !x.is_contiguous() || x.dim() != 2)
      fail(DQ_EINVAL, where, "X must be a contiguous 2-D bf16/f16 CUDA tensor");
    const at::Device dev = x.device();
    const int64_t rows = x.size(0), cols = x.size(1);
    auto like = [&](PyObject* o, const char* what) {
      const at::Tensor t = tensor(o, what);
      if (t.scalar_type() != x.scalar_type() || t.sizes() != x.sizes() || !t.is_contiguous() || t.device() != dev)
        fail(DQ_EINVAL, what, "must match X");
      return t;
    };
    at::Tensor r, h;
    if (a[5] != Py_None) {
      r = like(a[5], "dq_norm_quant: residual");
      h = a[8] != Py_None ? like(a[8], "dq_norm_quant: residual_out") : empty({rows, cols}, x.scalar_type(), dev);
    } else if (a[8] != Py_None) {
      fail(DQ_EINVAL, where, "residual_out without a residual");
    }
    const at::Tensor g = channels(a[2], cols, dev, "dq_norm_quant: weight");
    if (g.defined() && g.scalar_type() != x.scalar_type()) fail(DQ_EINVAL, "dq_norm_quant: weight", "must have X's dtype");
    const at::Tensor b = channels(a[3], cols, dev, "dq_norm_quant: col_scales");
    Quantized q;
    PyObject* out = row_outputs(&q, a[7], rows, cols, f, dev, "dq_norm_quant: out");
    try {
      const int64_t need = f.tensor_scale ? DQ_ACT_WORKSPACE_BYTES + 8 * rows : (check ? DQ_ACT_WORKSPACE_BYTES : 0);
      const at::Tensor ws = workspace_of(a[9], need, dev, where);
      run(
          [&] {
            return dq_norm_quant(x.data_ptr(), ptr(r), dtype_of(x.scalar_type()), rows, cols, ptr(g), (float)eps, ptr(b),
                                 b.defined() ? dtype_of(b.scalar_type()) : DQ_BF16, f.id, f.group, &q.out, ptr(h), ptr(ws),
                                 bytes(ws), stream);
          },
          check, ws, stream, where);
      if (r.defined()) set(out, k_residual, h);
      if (ws.defined()) set(out, k_workspace, ws);
    } catch (...) {
      Py_DECREF(out);
      throw;
    }
    return out;
  });
}

// glu_quant(stream, gate or both halves, up or None, col_scales, format, out, workspace, check) -> dict
PyObject* glu_quant(PyObject*, PyObject* const* a, Py_ssize_t n) {
  return guarded(n, 8, [&]() -> PyObject* {
    const char* where = "dq_glu_quant";
    void* stream = PyLong_AsVoidPtr(a[0]);
    const Format f = format_of(a[4]);
    const bool check = a[7] == Py_True, one = a[2] == Py_None;
    const at::Tensor gate = tensor(a[1], where), up = one ? gate : tensor(a[2], where);
    for (const at::Tensor* t : {&gate, &up})
      if (!t->is_cuda() || !is_half(t->scalar_type()) || t->dim() != 2 || t->stride(1) != 1)
        fail(DQ_EINVAL, where, "gate and up must be 2-D bf16/f16 CUDA tensors with adjacent columns");
    if (one && gate.size(1) % 2 != 0) fail(DQ_EINVAL, where, "X must have an even number of columns");
    if (gate.sizes() != up.sizes() || gate.scalar_type() != up.scalar_type() || gate.device() != up.device() ||
        (gate.size(0) > 1 && gate.stride(0) != up.stride(0)))
      fail(DQ_EINVAL, where, "gate and up must agree in shape, dtype, device and row stride");
    const at::Device dev = gate.device();
    const int64_t rows = gate.size(0), cols = one ? gate.size(1) / 2 : gate.size(1);
    const int64_t ld = rows > 1 ? gate.stride(0) : (cols + 7) / 8 * 8;
    const at::Tensor b = channels(a[3], cols, dev, "dq_glu_quant: col_scales");
    Quantized q;
    PyObject* out = row_outputs(&q, a[5], rows, cols, f, dev, "dq_glu_quant: out");
    try {
      const at::Tensor ws = workspace_of(a[6], check || f.tensor_scale ? DQ_ACT_WORKSPACE_BYTES : 0, dev, where);
      const char* up_ptr = static_cast<const char*>(up.data_ptr()) + (one ? 2 * cols : 0);
      run(
          [&] {
            return dq_glu_quant(gate.data_ptr(), up_ptr, dtype_of(gate.scalar_type()), rows, cols, ld, ptr(b),
                                b.defined() ? dtype_of(b.scalar_type()) : DQ_BF16, f.id, f.group, &q.out, ptr(ws), bytes(ws),
                                stream);
          },
          check, ws, stream, where);
      if (ws.defined()) set(out, k_workspace, ws);
    } catch (...) {
      Py_DECREF(out);
      throw;
    }
    return out;
  });
}

PyObject* set_error(PyObject*, PyObject* cls) {
  Py_INCREF(cls);
  Py_XSETREF(g_error, cls);
  Py_RETURN_NONE;
}

PyMethodDef methods[] = {
    {"matmul", (PyCFunction)(void*)matmul, METH_FASTCALL, nullptr},
    {"norm_quant", (PyCFunction)(void*)norm_quant, METH_FASTCALL, nullptr},
    {"glu_quant", (PyCFunction)(void*)glu_quant, METH_FASTCALL, nullptr},
    {"set_error", set_error, METH_O, nullptr},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_dq_torch", "Argument marshalling of the linear layer's calls.", -1, methods};

}  // namespace

PyMODINIT_FUNC PyInit__dq_torch() {
  k_codes = PyUnicode_InternFromString("codes");
  k_scales = PyUnicode_InternFromString("block_scales");
  k_tensor = PyUnicode_InternFromString("tensor_scale");
  k_residual = PyUnicode_InternFromString("residual");
  k_workspace = PyUnicode_InternFromString("workspace");
  g_error = PyExc_RuntimeError;
  Py_INCREF(g_error);
  return PyModule_Create(&module);
}
