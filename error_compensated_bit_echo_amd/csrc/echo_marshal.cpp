// Native marshalling of torch tensors into the layer operators of libecho's C ABI
// (CPython extension module, imported by binding.py).  Up to 16 ranks bring up to
// five tensors each: reading their shapes, strides, types, devices and pointers
// through Python attributes took 25-40 us a call at P = 8, longer than the kernels
// of a decode step.  Every check of what the C ABI cannot see (shapes, types, strides
// and devices that agree) is made here; a function returns None, or (status, text)
// for an EchoError.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <hip/hip_runtime_api.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "echo.h"

namespace {

// An EchoError in the making; thrown within this file only.
struct Refused {
  echo_status status;
  std::string text;
};
// A Python exception is set.
struct Raised {};

[[noreturn]] void refuse(echo_status s, std::string text) { throw Refused{s, std::move(text)}; }

// A sequence's items, borrowed from the list or tuple kept here.
class Items {
 public:
  Items(PyObject* o, const char* what) : fast_(PySequence_Fast(o, "expected a sequence")) {
    if (fast_ == nullptr) {
      PyErr_Clear();
      refuse(ECHO_ERR_ARG, std::string(what) + ": expected a sequence");
    }
  }
  ~Items() { Py_XDECREF(fast_); }
  Items(const Items&) = delete;
  Items& operator=(const Items&) = delete;
  Py_ssize_t size() const { return PySequence_Fast_GET_SIZE(fast_); }
  PyObject* operator[](Py_ssize_t i) const { return PySequence_Fast_GET_ITEM(fast_, i); }

 private:
  PyObject* fast_;
};

const at::Tensor& tensor(PyObject* o, const char* what) {
  if (!THPVariable_Check(o)) refuse(ECHO_ERR_ARG, std::string(what) + ": expected tensors");
  return THPVariable_Unpack(o);
}

// P matrices of one shape, type and layout on one GPU.
struct Mats {
  int64_t rows = 0, cols = 0, s0 = 0, s1 = 0;
  at::ScalarType type = at::ScalarType::Undefined;
  void* ptr[ECHO_MAX_RANKS] = {};
};

struct Device {
  int index = -1;
  void on(const at::Tensor& t, const char* what) {
    if (!t.device().is_cuda() || (index >= 0 && t.device().index() != index))
      refuse(ECHO_ERR_ARG, std::string(what) + ": every tensor must be on one GPU");
    index = t.device().index();
  }
};

void take(Mats* m, int r, const at::Tensor& t, Device* dev, const char* what) {
  if (t.layout() != at::kStrided || t.dim() != 2) refuse(ECHO_ERR_ARG, std::string(what) + " must be matrices");
  if (r == 0) {
    m->rows = t.size(0);
    m->cols = t.size(1);
    m->s0 = t.stride(0);
    m->s1 = t.stride(1);
    m->type = t.scalar_type();
  } else if (t.size(0) != m->rows || t.size(1) != m->cols || t.scalar_type() != m->type ||
             (m->rows > 1 && t.stride(0) != m->s0) || (m->cols > 1 && t.stride(1) != m->s1)) {
    refuse(ECHO_ERR_ARG, std::string(what) + " must be of one shape, type and layout");
  }
  dev->on(t, what);
  m->ptr[r] = t.data_ptr();
}

int ranks(const Items& x, const char* what) {
  if (x.size() < 1) refuse(ECHO_ERR_ARG, std::string(what) + ": at least one matrix");
  if (x.size() > ECHO_MAX_RANKS) refuse(ECHO_ERR_SHAPE, std::string(what) + ": at most 16 matrices");
  return static_cast<int>(x.size());
}

Mats matrices(const Items& x, int P, Device* dev, const char* what) {
  Mats m;
  if (x.size() != P) refuse(ECHO_ERR_ARG, std::string(what) + ": the same number of matrices everywhere");
  for (int r = 0; r < P; ++r) take(&m, r, tensor(x[r], what), dev, what);
  if (m.cols > 1 && m.s1 != 1) refuse(ECHO_ERR_ARG, std::string(what) + " must have contiguous rows");
  if (m.rows <= 1) m.s0 = m.cols;  // the pitch of a single row says nothing
  return m;
}

int32_t elem_type(at::ScalarType t, const char* what) {
  switch (t) {
    case at::kFloat: return ECHO_F32;
    case at::kBFloat16: return ECHO_BF16;
    case at::kHalf: return ECHO_F16;
    default: refuse(ECHO_ERR_DTYPE, std::string(what) + ": float32, bfloat16 or float16 expected");
  }
}

// P (codes, scales) pairs.
struct Fp8 {
  Mats codes, scales;
  echo_fp8 c{};
};

int64_t blocks(int64_t n) { return (n + ECHO_FP8_BLOCK - 1) / ECHO_FP8_BLOCK; }

void fp8_matrices(Fp8* f, const Items& x, int P, Device* dev, const char* what) {
  if (x.size() != P) refuse(ECHO_ERR_ARG, std::string(what) + ": the same number of matrices everywhere");
  for (int r = 0; r < P; ++r) {
    const Items pair(x[r], what);
    if (pair.size() != 2) refuse(ECHO_ERR_ARG, std::string(what) + ": (codes, scales) pairs expected");
    take(&f->codes, r, tensor(pair[0], what), dev, what);
    take(&f->scales, r, tensor(pair[1], what), dev, what);
  }
  const int64_t rows = f->codes.rows, k = f->codes.cols;
  if (k > 1 && f->codes.s1 != 1) refuse(ECHO_ERR_ARG, std::string(what) + ": k must be contiguous");
  if (f->codes.type == at::kFloat8_e4m3fn) f->c.format = ECHO_E4M3;
  else if (f->codes.type == at::kFloat8_e5m2) f->c.format = ECHO_E5M2;
  else refuse(ECHO_ERR_DTYPE, std::string(what) + ": codes must be float8_e4m3fn or float8_e5m2");
  if (f->scales.type == at::kFloat) f->c.scale_type = ECHO_SCALE_F32;
  else if (f->scales.type == at::ScalarType::Float8_e8m0fnu) f->c.scale_type = ECHO_SCALE_E8M0;
  else refuse(ECHO_ERR_DTYPE, std::string(what) + ": scales must be float32 or float8_e8m0fnu");
  if (f->scales.cols != blocks(k) || (f->scales.rows != rows && f->scales.rows != blocks(rows)))
    refuse(ECHO_ERR_ARG, std::string(what) + ": scales of [" + std::to_string(f->scales.rows) + ", " +
                             std::to_string(f->scales.cols) + "] for codes of [" + std::to_string(rows) + ", " +
                             std::to_string(k) + "]");
  f->c.block_rows = f->scales.rows == rows ? 1 : ECHO_FP8_BLOCK;
  f->c.ld = rows > 1 ? f->codes.s0 : (k + 15) / 16 * 16;  // the pitch of a single row says nothing
  f->c.scale_row_stride = f->scales.s0;
  f->c.scale_k_stride = f->scales.s1;
  f->c.codes = f->codes.ptr;
  f->c.scales = f->scales.ptr;
}

// The stream: an integer handle, or None for torch's current stream on the device,
// which `current` (device index -> handle) gives.
echo_stream_t stream_of(PyObject* stream, PyObject* current, int device) {
  PyObject* h = stream;
  Py_INCREF(h);
  if (stream == Py_None) {
    Py_DECREF(h);
    h = PyObject_CallFunction(current, "i", device);
    if (h == nullptr) throw Raised{};
  }
  void* p = PyLong_AsVoidPtr(h);
  Py_DECREF(h);
  if (p == nullptr && PyErr_Occurred()) throw Raised{};
  return p;
}

// Makes a device current for a call, where it is not already.
class OnDevice {
 public:
  explicit OnDevice(int index) {
    if (hipGetDevice(&before_) != hipSuccess || (before_ != index && hipSetDevice(index) != hipSuccess))
      refuse(ECHO_ERR_HIP, "the tensors' device");
    changed_ = before_ != index;
  }
  ~OnDevice() {
    if (changed_) (void)hipSetDevice(before_);
  }
  OnDevice(const OnDevice&) = delete;
  OnDevice& operator=(const OnDevice&) = delete;

 private:
  int before_ = -1;
  bool changed_ = false;
};

PyObject* answer(echo_status s, const char* what) {
  if (s == ECHO_OK) Py_RETURN_NONE;
  return Py_BuildValue("is", static_cast<int>(s), what);
}

// Runs `f`, whose refusals and C++ exceptions become answers and Python errors.
template <typename F>
PyObject* guarded(F f) {
  try {
    return f();
  } catch (const Refused& r) {
    return Py_BuildValue("is", static_cast<int>(r.status), r.text.c_str());
  } catch (const Raised&) {
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  } catch (...) {
    PyErr_SetString(PyExc_RuntimeError, "unknown C++ exception");
    return nullptr;
  }
}

bool arguments(Py_ssize_t n, Py_ssize_t want) {
  if (n == want) return true;
  PyErr_SetString(PyExc_TypeError, "wrong number of arguments");
  return false;
}

// (X, rows or None, cols or None, stream, current)
PyObject* quantize_fp8(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (!arguments(n, 5)) return nullptr;
  return guarded([&]() -> PyObject* {
    if (args[1] == Py_None && args[2] == Py_None)
      refuse(ECHO_ERR_ARG, "echo_quantize_fp8: at least one of rows and cols");
    const Items X(args[0], "X");
    const int P = ranks(X, "X");
    Device dev;
    const Mats x = matrices(X, P, &dev, "X");
    Fp8 rows, cols;
    if (args[1] != Py_None) {
      const Items o(args[1], "rows");
      fp8_matrices(&rows, o, P, &dev, "rows");
      if (rows.codes.rows != x.rows || rows.codes.cols != x.cols) refuse(ECHO_ERR_ARG, "rows: codes of X's shape expected");
    }
    if (args[2] != Py_None) {
      const Items o(args[2], "cols");
      fp8_matrices(&cols, o, P, &dev, "cols");
      if (cols.codes.rows != x.cols || cols.codes.cols != x.rows)
        refuse(ECHO_ERR_ARG, "cols: codes of the transposed shape expected");
      // one row is a row and a block of rows: it goes by the other orientation
      if (args[1] != Py_None) {
        if (x.rows == 1) rows.c.block_rows = cols.c.block_rows;
        else if (x.cols == 1) cols.c.block_rows = rows.c.block_rows;
      }
    }
    const OnDevice on(dev.index);
    return answer(echo_quantize_fp8(x.ptr, P, x.rows, x.cols, x.s0, elem_type(x.type, "X"),
                                    args[1] == Py_None ? nullptr : &rows.c, args[2] == Py_None ? nullptr : &cols.c,
                                    stream_of(args[3], args[4], dev.index)),
                  "echo_quantize_fp8");
  });
}

// (A, W, out, stream, current)
PyObject* gemm_fp8(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (!arguments(n, 5)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Items A(args[0], "A"), W(args[1], "W"), O(args[2], "out");
    const int P = ranks(A, "A");
    Device dev;
    Fp8 a, w;
    fp8_matrices(&a, A, P, &dev, "A");
    fp8_matrices(&w, W, P, &dev, "W");
    const Mats o = matrices(O, P, &dev, "out");
    if (a.codes.cols != w.codes.cols) refuse(ECHO_ERR_ARG, "A and W must have the same k");
    if (o.rows != a.codes.rows || o.cols != w.codes.rows)
      refuse(ECHO_ERR_ARG, "out must be [" + std::to_string(a.codes.rows) + ", " + std::to_string(w.codes.rows) + "]");
    const OnDevice on(dev.index);
    return answer(echo_gemm_fp8(&a.c, &w.c, o.ptr, P, o.rows, o.cols, a.codes.cols, o.s0, elem_type(o.type, "out"),
                                stream_of(args[3], args[4], dev.index)),
                  "echo_gemm_fp8");
  });
}

// Rows and pitch of a tensor: any contiguous one, or a matrix with contiguous rows.
void row_layout(const at::Tensor& t, const at::Tensor& like, int64_t* rows, int64_t* cols, int64_t* ld, const char* what) {
  if (t.layout() != at::kStrided || t.sizes() != like.sizes())
    refuse(ECHO_ERR_ARG, std::string(what) + ": the shape of x expected");
  *cols = t.dim() > 0 ? t.size(-1) : 1;
  *rows = *cols > 0 ? t.numel() / *cols : 0;
  if (t.is_contiguous()) {
    *ld = *cols;
    return;
  }
  if (t.dim() != 2 || (*cols > 1 && t.stride(1) != 1))
    refuse(ECHO_ERR_ARG, std::string(what) + " must be contiguous, or a matrix with contiguous rows");
  *ld = t.stride(0);
}

// (x, residual or None, out, p, rng, offset as int64, first, stream, current)
PyObject* dropout_add(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (!arguments(n, 9)) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor &x = tensor(args[0], "x"), &out = tensor(args[2], "out"), &rng = tensor(args[4], "rng");
    const double p = PyFloat_AsDouble(args[3]);
    if (p == -1.0 && PyErr_Occurred()) throw Raised{};
    const long long offset = PyLong_AsLongLong(args[5]), first = PyLong_AsLongLong(args[6]);
    if (PyErr_Occurred()) throw Raised{};
    Device dev;
    dev.on(x, "x");
    dev.on(out, "out");
    dev.on(rng, "rng");
    int64_t rows, cols, ldx, ldo, ldr = 0;
    row_layout(x, x, &rows, &cols, &ldx, "x");
    row_layout(out, x, &rows, &cols, &ldo, "out");
    const void* residual = nullptr;
    const int32_t out_type = elem_type(out.scalar_type(), "out");
    if (args[1] != Py_None) {
      const at::Tensor& r = tensor(args[1], "residual");
      dev.on(r, "residual");
      row_layout(r, x, &rows, &cols, &ldr, "residual");
      if (r.scalar_type() != out.scalar_type()) refuse(ECHO_ERR_DTYPE, "residual and out must be of one type");
      residual = r.data_ptr();
    }
    if (rng.scalar_type() != at::kLong || rng.numel() != 2 || !rng.is_contiguous())
      refuse(ECHO_ERR_ARG, "rng must be a contiguous int64 tensor of 2 elements");
    const OnDevice on(dev.index);
    return answer(echo_dropout_add(x.data_ptr(), residual, out.data_ptr(), rows, cols, ldx, ldr, ldo,
                                   elem_type(x.scalar_type(), "x"), out_type, p,
                                   static_cast<const int64_t*>(rng.data_ptr()), offset, first,
                                   stream_of(args[7], args[8], dev.index)),
                  "echo_dropout_add");
  });
}

PyMethodDef methods[] = {
    {"quantize_fp8", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(quantize_fp8)), METH_FASTCALL, nullptr},
    {"gemm_fp8", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(gemm_fp8)), METH_FASTCALL, nullptr},
    {"dropout_add", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(dropout_add)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_echo_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__echo_marshal() { return PyModule_Create(&module_def); }
