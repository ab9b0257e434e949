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
#include <ATen/ops/empty.h>
#include <torch/csrc/autograd/python_variable.h>

#include <optional>
#include <string>
#include <vector>

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

// ---- operators of a training step around the blocks -------------------------------

const at::Tensor* optional_tensor(PyObject* o, const char* what) { return o == Py_None ? nullptr : &tensor(o, what); }

// Where a tensor lies.  One without elements lies nowhere: an address that is never used
// says that it was given.
void* address(const at::Tensor& t) {
  alignas(16) static char given;
  return t.numel() > 0 ? t.data_ptr() : &given;
}

// A tensor of x's shape on the call's GPU, or none.
struct RowsOf {
  void* p = nullptr;
  int64_t ld = 0;
  int32_t type = ECHO_F32;
};

RowsOf rows_like(const at::Tensor* t, const at::Tensor& like, Device* dev, int64_t* rows, int64_t* cols, const char* what) {
  RowsOf r;
  if (t == nullptr) return r;
  dev->on(*t, what);
  row_layout(*t, like, rows, cols, &r.ld, what);
  r.p = address(*t);
  r.type = elem_type(t->scalar_type(), what);
  return r;
}

// A vector of `cols` elements of the parameters' type, or none.
void* weight(const at::Tensor* t, int64_t cols, at::ScalarType* type, Device* dev, const char* what) {
  if (t == nullptr) return nullptr;
  dev->on(*t, what);
  if (t->layout() != at::kStrided || t->dim() != 1 || t->size(0) != cols || !t->is_contiguous())
    refuse(ECHO_ERR_ARG, std::string(what) + ": a contiguous vector as long as the rows expected");
  if (*type != at::ScalarType::Undefined && *type != t->scalar_type())
    refuse(ECHO_ERR_DTYPE, "the gate, the weights and their gradients must be of one type");
  *type = t->scalar_type();
  return t->data_ptr();
}

// A gate [cols] or [gate_rows, cols] with contiguous rows, or none.  One without rows goes
// with no rows of the stream (`of`): a gate per token of no tokens.
void* gate_of(const at::Tensor* t, int64_t of, int64_t cols, int64_t* rows, int64_t* ld, at::ScalarType* type, Device* dev,
              const char* what) {
  if (t == nullptr) return nullptr;
  dev->on(*t, what);
  if (t->layout() != at::kStrided || t->dim() < 1 || t->dim() > 2 || t->size(-1) != cols || (cols > 1 && t->stride(-1) != 1))
    refuse(ECHO_ERR_ARG, std::string(what) + ": a vector or matrix with contiguous rows as long as x's expected");
  if (*type != at::ScalarType::Undefined && *type != t->scalar_type())
    refuse(ECHO_ERR_DTYPE, "the gate, the weights and their gradients must be of one type");
  *type = t->scalar_type();
  *rows = t->dim() == 2 ? t->size(0) : 1;
  *ld = t->dim() == 2 ? t->stride(0) : cols;
  if (*rows > 0) return address(*t);
  if (of > 0) refuse(ECHO_ERR_SHAPE, std::string(what) + ": no rows");
  return nullptr;
}

double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return v;
}

bool truth(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised{};
  return v != 0;
}

// The caller's workspace, or one from torch's allocator for this call (`owned`): freed to
// the stream that is current, so only for calls on that stream.
void* workspace_of(PyObject* given, PyObject* stream, size_t need, const Device& dev, at::Tensor* owned, size_t* bytes) {
  *bytes = 0;
  if (given != Py_None) {
    const at::Tensor& t = tensor(given, "workspace");
    if (t.scalar_type() != at::kByte || !t.is_contiguous() || !t.device().is_cuda() || t.device().index() != dev.index)
      refuse(ECHO_ERR_ARG, "workspace: a contiguous uint8 tensor on the tensors' GPU expected");
    *bytes = static_cast<size_t>(t.numel());
    return t.numel() > 0 ? t.data_ptr() : nullptr;
  }
  if (need == 0) return nullptr;
  if (stream != Py_None) refuse(ECHO_ERR_WORKSPACE, "a call on a stream of its own takes the caller's workspace");
  *owned = at::empty({static_cast<int64_t>(need)}, at::TensorOptions().dtype(at::kByte).device(
                                                       at::Device(at::kCUDA, static_cast<c10::DeviceIndex>(dev.index))));
  *bytes = need;
  return owned->data_ptr();
}

// Tells autograd that a call wrote into a tensor: a graph that saved it from before then
// refuses its backward pass rather than differentiate with the new values.  Inference
// tensors have no version to move.
void wrote(const at::Tensor& t) {
  if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

void wrote(PyObject* o) {
  if (o != Py_None) wrote(THPVariable_Unpack(o));
}

void wrote(const Items& x) {
  for (Py_ssize_t i = 0; i < x.size(); ++i) wrote(x[i]);
}

struct Block {
  echo_block c{};
  int64_t rows = 0, cols = 0;
  at::ScalarType params = at::ScalarType::Undefined;
};

// args: gate, w_post, w_pre, post_norm, residual_scale, weight_offset, eps
void block_params(Block* b, PyObject* const* args, Device* dev) {
  b->c.gate = gate_of(optional_tensor(args[0], "gate"), b->rows, b->cols, &b->c.gate_rows, &b->c.ld_gate, &b->params, dev, "gate");
  b->c.w_post = weight(optional_tensor(args[1], "w_post"), b->cols, &b->params, dev, "w_post");
  b->c.w_pre = weight(optional_tensor(args[2], "w_pre"), b->cols, &b->params, dev, "w_pre");
  b->c.post_norm = truth(args[3]);
  b->c.residual_scale = number(args[4]);
  b->c.weight_offset = number(args[5]);
  b->c.eps = number(args[6]);
  b->c.rows = b->rows;
  b->c.cols = b->cols;
  b->c.param_dtype = b->params == at::ScalarType::Undefined ? ECHO_F32 : elem_type(b->params, "weights");
}

// (x, out or None, a or None, y or None, gate, w_post, w_pre, post_norm, residual_scale, weight_offset, eps, stream, current)
PyObject* block_norm(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (!arguments(n, 13)) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor& x = tensor(args[0], "x");
    Device dev;
    Block b;
    const RowsOf mx = rows_like(&x, x, &dev, &b.rows, &b.cols, "x");
    const RowsOf mo = rows_like(optional_tensor(args[1], "out"), x, &dev, &b.rows, &b.cols, "out");
    const RowsOf ma = rows_like(optional_tensor(args[2], "a"), x, &dev, &b.rows, &b.cols, "a");
    const RowsOf my = rows_like(optional_tensor(args[3], "y"), x, &dev, &b.rows, &b.cols, "y");
    if (args[1] != Py_None && mo.type != mx.type) refuse(ECHO_ERR_DTYPE, "x and out must be of one type");
    block_params(&b, args + 4, &dev);
    b.c.x_dtype = mx.type;
    b.c.y_dtype = args[3] != Py_None ? my.type : mx.type;
    b.c.a_dtype = args[2] != Py_None ? ma.type : mx.type;
    const OnDevice on(dev.index);
    const echo_status s = echo_block_norm(&b.c, mx.p, mx.ld, my.p, my.ld, mo.p, mo.ld, ma.p, ma.ld,
                                          stream_of(args[11], args[12], dev.index));
    if (s == ECHO_OK)
      for (int i : {1, 2}) wrote(args[i]);
    return answer(s, "echo_block_norm");
  });
}

// (out, dout, da, dx, y, dy, dgate, dw_post, dw_pre, gate, w_post, w_pre, post_norm, residual_scale, weight_offset, eps,
// workspace, stream, current)
PyObject* block_norm_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (!arguments(n, 19)) return nullptr;
  return guarded([&]() -> PyObject* {
    const at::Tensor& out = tensor(args[0], "out");
    Device dev;
    Block b;
    const auto rows = [&](int i, const char* what) {
      return rows_like(optional_tensor(args[i], what), out, &dev, &b.rows, &b.cols, what);
    };
    const RowsOf mo = rows(0, "out"), mdo = rows(1, "dout"), mda = rows(2, "da"), mdx = rows(3, "dx"), my = rows(4, "y"),
                 mdy = rows(5, "dy");
    if ((mdo.p != nullptr && mdo.type != mo.type) || (mdx.p != nullptr && mdx.type != mo.type) ||
        (mdy.p != nullptr && my.p != nullptr && mdy.type != my.type))
      refuse(ECHO_ERR_DTYPE, "a gradient must be of the type of what it is the gradient of");
    block_params(&b, args + 9, &dev);
    int64_t gate_rows = b.c.gate_rows, ldg = 0;
    void* dgate = gate_of(optional_tensor(args[6], "dgate"), b.rows, b.cols, &gate_rows, &ldg, &b.params, &dev, "dgate");
    if (dgate != nullptr && gate_rows != b.c.gate_rows) refuse(ECHO_ERR_ARG, "dgate: the gate's shape expected");
    void* dw_post = weight(optional_tensor(args[7], "dw_post"), b.cols, &b.params, &dev, "dw_post");
    void* dw_pre = weight(optional_tensor(args[8], "dw_pre"), b.cols, &b.params, &dev, "dw_pre");
    b.c.x_dtype = mo.type;
    b.c.y_dtype = args[4] != Py_None ? my.type : mo.type;
    b.c.a_dtype = args[2] != Py_None ? mda.type : mo.type;
    const OnDevice on(dev.index);
    at::Tensor owned;
    size_t bytes = 0;
    const size_t need = echo_block_norm_workspace(b.rows, b.cols, b.c.gate != nullptr ? b.c.gate_rows : 0);
    void* ws = workspace_of(args[16], args[17], need, dev, &owned, &bytes);
    const echo_status s = echo_block_norm_backward(&b.c, mo.p, mo.ld, my.p, my.ld, mdo.p, mdo.ld, mda.p, mda.ld, mdx.p, mdx.ld,
                                                   mdy.p, mdy.ld, dgate, ldg, dw_post, dw_pre, ws, bytes,
                                                   stream_of(args[17], args[18], dev.index));
    if (s == ECHO_OK)
      for (int i : {3, 5, 6, 7, 8}) wrote(args[i]);
    return answer(s, "echo_block_norm_backward");
  });
}

// Pointers, lengths and types of a list of tensors.
struct Tensors {
  std::vector<void*> p;
  std::vector<int64_t> n;
  std::vector<int32_t> type;
};

void tensor_list(Tensors* l, const Items& x, Device* dev, const char* what) {
  const size_t n = static_cast<size_t>(x.size());
  l->p.reserve(n);
  l->n.reserve(n);
  l->type.reserve(n);
  for (size_t i = 0; i < n; ++i) {
    const at::Tensor& t = tensor(x[static_cast<Py_ssize_t>(i)], what);
    dev->on(t, what);
    if (t.layout() != at::kStrided || !t.is_non_overlapping_and_dense())
      refuse(ECHO_ERR_ARG, std::string(what) + " must be tensors whose elements lie together");
    l->p.push_back(t.data_ptr());
    l->n.push_back(t.numel());
    l->type.push_back(elem_type(t.scalar_type(), what));
  }
}

// (grads, norm, workspace, stream, current), or (grads, norm, workspace, out or None, max_norm, stream, current)
PyObject* clip(PyObject* const* args, bool scale) {
  return guarded([&]() -> PyObject* {
    const Items G(args[0], "grads");
    const at::Tensor& norm = tensor(args[1], "norm");
    PyObject *stream = args[scale ? 5 : 3], *current = args[scale ? 6 : 4];
    Device dev;
    dev.on(norm, "norm");
    if (norm.scalar_type() != at::kFloat || norm.numel() != 1) refuse(ECHO_ERR_ARG, "norm: one element of float32 expected");
    Tensors g, o;
    std::optional<Items> to_items;
    tensor_list(&g, G, &dev, "grads");
    const int64_t count = static_cast<int64_t>(g.p.size());
    if (scale && args[3] != Py_None) {
      const Items& O = to_items.emplace(args[3], "out");
      if (O.size() != G.size()) refuse(ECHO_ERR_ARG, "out: as many tensors as gradients expected");
      tensor_list(&o, O, &dev, "out");
      for (Py_ssize_t i = 0; i < O.size(); ++i) {
        const at::Tensor &a = tensor(G[i], "grads"), &b = tensor(O[i], "out");
        if (a.scalar_type() != b.scalar_type() || a.sizes() != b.sizes() || (a.numel() > 1 && a.strides() != b.strides()))
          refuse(ECHO_ERR_ARG, "out: tensors like the gradients expected");
      }
    }
    const OnDevice on(dev.index);
    at::Tensor owned;
    size_t bytes = 0;
    void* ws = workspace_of(args[2], stream, echo_clip_workspace(count), dev, &owned, &bytes);
    float* to = static_cast<float*>(norm.data_ptr());
    const echo_stream_t s = stream_of(stream, current, dev.index);
    if (!scale) {
      const echo_status e = echo_grad_norm(g.p.data(), g.n.data(), g.type.data(), count, to, ws, bytes, s);
      if (e == ECHO_OK) wrote(norm);
      return answer(e, "echo_grad_norm");
    }
    const echo_status e = echo_clip_grads(g.p.data(), (args[3] != Py_None ? o : g).p.data(), g.n.data(), g.type.data(), count,
                                          number(args[4]), to, ws, bytes, s);
    if (e == ECHO_OK) {
      wrote(norm);
      wrote(to_items ? *to_items : G);
    }
    return answer(e, "echo_clip_grads");
  });
}

PyObject* grad_norm(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return arguments(n, 5) ? clip(args, false) : nullptr;
}

PyObject* clip_grads(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return arguments(n, 7) ? clip(args, true) : nullptr;
}

// Token ids of any shape, contiguous.
int32_t token_bytes(const at::Tensor& t, Device* dev) {
  dev->on(t, "tokens");
  if (t.scalar_type() != at::kLong && t.scalar_type() != at::kInt) refuse(ECHO_ERR_DTYPE, "tokens: int64 or int32 expected");
  if (t.layout() != at::kStrided || !t.is_contiguous()) refuse(ECHO_ERR_ARG, "tokens must be contiguous");
  return t.scalar_type() == at::kLong ? 8 : 4;
}

int64_t whole(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  return v;
}

// (tables, tokens, out, scale, first, stream, current)
PyObject* embed(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (!arguments(n, 7)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Items E(args[0], "tables"), O(args[2], "out");
    const int P = ranks(E, "tables");
    const at::Tensor& tokens = tensor(args[1], "tokens");
    Device dev;
    const Mats e = matrices(E, P, &dev, "tables"), o = matrices(O, P, &dev, "out");
    const int32_t wide = token_bytes(tokens, &dev);
    if (o.rows != tokens.numel() || o.cols != e.cols)
      refuse(ECHO_ERR_ARG, "out must be [" + std::to_string(tokens.numel()) + ", " + std::to_string(e.cols) + "]");
    const OnDevice on(dev.index);
    const echo_status s = echo_embed(e.ptr, tokens.data_ptr(), o.ptr, P, e.rows, e.cols, e.s0, o.rows, o.s0,
                                     elem_type(e.type, "tables"), elem_type(o.type, "out"), wide, whole(args[4]), number(args[3]),
                                     stream_of(args[5], args[6], dev.index));
    if (s == ECHO_OK) wrote(O);
    return answer(s, "echo_embed");
  });
}

// (dout, tokens, dtables, scale, first, workspace, stream, current)
PyObject* embed_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (!arguments(n, 8)) return nullptr;
  return guarded([&]() -> PyObject* {
    const Items E(args[2], "dtables");
    const int P = ranks(E, "dtables");
    const at::Tensor &dout = tensor(args[0], "dout"), &tokens = tensor(args[1], "tokens");
    Device dev;
    const Mats e = matrices(E, P, &dev, "dtables");
    const int32_t wide = token_bytes(tokens, &dev);
    Mats d;
    take(&d, 0, dout, &dev, "dout");
    // the strides of no rows say nothing (those of an expanded gradient are 0)
    if (d.rows > 0 && d.cols > 1 && d.s1 != 1) refuse(ECHO_ERR_ARG, "dout must have contiguous rows");
    if (d.rows != tokens.numel() || d.cols != e.cols)
      refuse(ECHO_ERR_ARG, "dout must be [" + std::to_string(tokens.numel()) + ", " + std::to_string(e.cols) + "]");
    const OnDevice on(dev.index);
    at::Tensor owned;
    size_t bytes = 0;
    void* ws = workspace_of(args[5], args[6], echo_embed_workspace(d.rows, d.cols), dev, &owned, &bytes);
    const echo_status s = echo_embed_backward(d.ptr[0], tokens.data_ptr(), e.ptr, P, e.rows, e.cols, e.s0, d.rows, d.s0,
                                              elem_type(d.type, "dout"), elem_type(e.type, "dtables"), wide, whole(args[4]),
                                              number(args[3]), ws, bytes, stream_of(args[6], args[7], dev.index));
    if (s == ECHO_OK) wrote(E);
    return answer(s, "echo_embed_backward");
  });
}

template <PyObject* (*F)(PyObject*, PyObject* const*, Py_ssize_t)>
PyMethodDef method(const char* name) {
  return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {
    method<quantize_fp8>("quantize_fp8"),
    method<gemm_fp8>("gemm_fp8"),
    method<dropout_add>("dropout_add"),
    method<block_norm>("block_norm"),
    method<block_norm_backward>("block_norm_backward"),
    method<grad_norm>("grad_norm"),
    method<clip_grads>("clip_grads"),
    method<embed>("embed"),
    method<embed_backward>("embed_backward"),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_echo_marshal", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__echo_marshal() { return PyModule_Create(&module_def); }
