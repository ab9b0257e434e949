// C-ABI host side of the operators of a training step around the tensor-parallel blocks:
// argument validation and launches on the caller's stream.  See include/echo.h for the
// contract of every entry point.
#include <math.h>

#include <algorithm>
#include <new>

#include "echo.h"
#include "echo_layer_check.h"
#include "echo_step_internal.h"

namespace {

constexpr int64_t kMaxRows = (int64_t{1} << 31) - 1;
constexpr int64_t kMaxElems = int64_t{1} << 40;

bool known(int32_t dtype) {
  int64_t es;
  return elem_bytes(dtype, &es);
}

// Kernels exist for fp32 with one of the 16-bit types.
bool types_mix(int32_t a, int32_t b) {
  return !((a == ECHO_BF16 && b == ECHO_F16) || (a == ECHO_F16 && b == ECHO_BF16));
}

int64_t bytes_of(int32_t dtype) { return dtype == ECHO_F32 ? 4 : 2; }

// A matrix [rows, cols] of one type, or none (nullptr).
struct Mat {
  const void* p;
  int64_t rows, ld;
  int32_t dtype;
};

// Pitch and alignment of a matrix of `cols` columns; its pitch is set where there is one row.
echo_status check_mat(Mat* m, int64_t cols) {
  if (m->p == nullptr) return ECHO_OK;
  m->ld = pitch_of(m->rows, cols, m->ld);
  if (!pitch_fits(m->rows, cols, m->ld, bytes_of(m->dtype))) return ECHO_ERR_SHAPE;
  return aligned(m->p, static_cast<uintptr_t>(bytes_of(m->dtype))) ? ECHO_OK : ECHO_ERR_ARG;
}

Area area_of(const Mat& m, int64_t cols) {
  const int64_t es = bytes_of(m.dtype);
  return area(m.p, m.rows, cols * es, m.ld * es);
}

// No written matrix shares memory with another one; `same` (of the written one at
// `same_of`) may be the very same matrix.
bool apart(const Mat* outs, int n_out, const Mat* ins, int n_in, int64_t cols, int same_of, int same) {
  for (int i = 0; i < n_out; ++i) {
    if (outs[i].p == nullptr || outs[i].rows == 0) continue;
    const Area a = area_of(outs[i], cols);
    for (int j = i + 1; j < n_out; ++j)
      if (outs[j].p != nullptr && outs[j].rows != 0 && overlap(a, area_of(outs[j], cols))) return false;
    for (int j = 0; j < n_in; ++j) {
      if (ins[j].p == nullptr || ins[j].rows == 0) continue;
      if (i == same_of && j == same && outs[i].p == ins[j].p && outs[i].ld == ins[j].ld) continue;
      if (overlap(a, area_of(ins[j], cols))) return false;
    }
  }
  return true;
}

bool is_finite(double v) { return v - v == 0.0; }

echo_status check_block(const echo_block* b, bool has_y) {
  if (b == nullptr) return ECHO_ERR_ARG;
  if (!known(b->x_dtype) || !known(b->y_dtype) || !known(b->a_dtype) || !known(b->param_dtype)) return ECHO_ERR_DTYPE;
  if (!types_mix(b->x_dtype, b->y_dtype) || !types_mix(b->x_dtype, b->a_dtype) || !types_mix(b->y_dtype, b->a_dtype))
    return ECHO_ERR_DTYPE;
  if (b->rows < 0 || b->cols < 0 || b->rows > kMaxRows || b->cols > echo::kStepMaxCols) return ECHO_ERR_SHAPE;
  if (b->cols > 0 && b->rows > kMaxElems / b->cols) return ECHO_ERR_SHAPE;
  if (b->post_norm != 0 && b->post_norm != 1) return ECHO_ERR_ARG;
  if (b->gate != nullptr && (b->gate_rows < 1 || b->rows % b->gate_rows != 0)) return ECHO_ERR_SHAPE;
  const float alpha = static_cast<float>(b->residual_scale), offset = static_cast<float>(b->weight_offset);
  if (!is_finite(alpha) || !is_finite(offset)) return ECHO_ERR_ARG;
  if (!(b->eps >= 0x1p-126) || !is_finite(static_cast<float>(b->eps))) return ECHO_ERR_ARG;  // also refuses NaN
  // what belongs to the block's output needs one
  if (!has_y && (b->post_norm != 0 || b->gate != nullptr || alpha != 1.0f)) return ECHO_ERR_ARG;
  if (b->w_post != nullptr && b->post_norm == 0) return ECHO_ERR_ARG;
  const uintptr_t es = static_cast<uintptr_t>(bytes_of(b->param_dtype));
  if (!aligned(b->gate, es) || !aligned(b->w_post, es) || !aligned(b->w_pre, es)) return ECHO_ERR_ARG;
  return ECHO_OK;
}

echo::BlockParams params_of(const echo_block& b, const Mat& gate) {
  echo::BlockParams p{};
  p.gate = b.gate;
  p.w_post = b.w_post;
  p.w_pre = b.w_pre;
  p.ldg = gate.ld;
  p.n_gates = b.gate != nullptr ? b.gate_rows : 1;
  p.rows_per_gate = b.rows / p.n_gates;
  p.R = b.rows;
  p.C = b.cols;
  p.alpha = static_cast<float>(b.residual_scale);
  p.offset = static_cast<float>(b.weight_offset);
  p.eps = static_cast<float>(b.eps);
  p.inv_cols = static_cast<float>(1.0 / static_cast<double>(b.cols));
  p.elem = b.param_dtype;
  p.post = b.post_norm;
  return p;
}

echo_status status_of(hipError_t e) { return e == hipSuccess ? ECHO_OK : ECHO_ERR_HIP; }

echo::Elem elem(int32_t dtype) { return static_cast<echo::Elem>(dtype); }

// ---- clipping ----

// The tensors' types, lengths and pointers.
echo_status check_tensors(const void* const* src, void* const* dst, const int64_t* n, const int32_t* dtypes, int64_t count) {
  if (count < 0 || count > (int64_t{1} << 24)) return ECHO_ERR_SHAPE;
  if (count > 0 && (src == nullptr || n == nullptr || dtypes == nullptr)) return ECHO_ERR_ARG;
  int64_t chunks = 0;
  for (int64_t i = 0; i < count; ++i) {
    if (!known(dtypes[i])) return ECHO_ERR_DTYPE;
    if (n[i] < 0 || n[i] > kMaxElems) return ECHO_ERR_SHAPE;
    chunks += echo::clip_chunks(n[i] * bytes_of(dtypes[i]));
    if (chunks >= int64_t{1} << 31) return ECHO_ERR_SHAPE;
    if (n[i] == 0) continue;
    const uintptr_t es = static_cast<uintptr_t>(bytes_of(dtypes[i]));
    if (src[i] == nullptr || !aligned(src[i], es)) return ECHO_ERR_ARG;
    if (dst != nullptr && (dst[i] == nullptr || !aligned(dst[i], es))) return ECHO_ERR_ARG;
  }
  return ECHO_OK;
}

// One stretch of memory of a clipping call.
struct Stretch {
  uintptr_t lo, hi;
  bool written;
};

// Whether what is written (results, the norm, the workspace) lies apart from all else, a
// result's own input aside where that
// is the very same memory.  In order of their starts, a stretch meets an earlier one iff
// it starts before the furthest end so far: of the written ones, and of any if it is written.
echo_status tensors_apart(const void* const* src, void* const* dst, const int64_t* n, const int32_t* dtypes,
                          int64_t count, const float* norm, const void* workspace) {
  Stretch* all = new (std::nothrow) Stretch[static_cast<size_t>(2 * count + 2)];
  if (all == nullptr) return ECHO_ERR_WORKSPACE;
  int64_t m = 0;
  for (int64_t i = 0; i < count; ++i) {
    if (n[i] == 0) continue;
    const uintptr_t s = reinterpret_cast<uintptr_t>(src[i]), d = dst != nullptr ? reinterpret_cast<uintptr_t>(dst[i]) : 0;
    const uintptr_t bytes = static_cast<uintptr_t>(n[i] * bytes_of(dtypes[i]));
    if (dst != nullptr) all[m++] = Stretch{d, d + bytes, true};
    if (dst == nullptr || s != d) all[m++] = Stretch{s, s + bytes, false};
  }
  const uintptr_t at = reinterpret_cast<uintptr_t>(norm), w = reinterpret_cast<uintptr_t>(workspace);
  all[m++] = Stretch{at, at + sizeof(float), true};
  if (count > 0) all[m++] = Stretch{w, w + echo_clip_workspace(count), true};
  std::sort(all, all + m, [](const Stretch& a, const Stretch& b) { return a.lo < b.lo; });
  uintptr_t end = 0, written_end = 0;
  bool ok = true;
  for (int64_t i = 0; i < m && ok; ++i) {
    ok = all[i].lo >= (all[i].written ? end : written_end);
    end = std::max(end, all[i].hi);
    if (all[i].written) written_end = std::max(written_end, all[i].hi);
  }
  delete[] all;
  return ok ? ECHO_OK : ECHO_ERR_ARG;
}

// Fills the arguments of one launch after the other and hands each to f.
template <typename Args, typename F>
echo_status for_launches(const void* const* src, void* const* dst, const int64_t* n, const int32_t* dtypes, int64_t count,
                         F f) {
  Args a;
  a.tensors = 0;
  uint32_t chunks = 0;
  for (int64_t i = 0; i <= count; ++i) {
    if (a.tensors == Args::kTensors || (i == count && a.tensors > 0)) {
      a.first[a.tensors] = chunks;
      if (f(a) != hipSuccess) return ECHO_ERR_HIP;
      a.tensors = 0;
      chunks = 0;
    }
    if (i == count || n[i] == 0) continue;
    const int64_t bytes = n[i] * bytes_of(dtypes[i]);
    a.src[a.tensors] = src[i];
    if (sizeof(a.dst) > sizeof(void*)) a.dst[a.tensors] = dst[i];
    a.tail[a.tensors] = echo::clip_tail(bytes, dtypes[i]);
    a.first[a.tensors++] = chunks;
    chunks += static_cast<uint32_t>(echo::clip_chunks(bytes));
  }
  return ECHO_OK;
}

// The tensors' squares, as *n_part partial sums.
echo_status launch_sums(const void* const* src, const int64_t* n, const int32_t* dtypes, int64_t count, double* part,
                        int64_t* n_part, hipStream_t s) {
  *n_part = 0;
  return for_launches<echo::ClipInPlace>(src, nullptr, n, dtypes, count, [&](const echo::ClipInPlace& a) {
    const hipError_t e = echo::launch_clip_sum(a, part + *n_part, s);
    *n_part += echo::clip_grid(a.first[a.tensors]);
    return e;
  });
}

template <typename Args>
echo_status launch_scales(const void* const* src, void* const* dst, const int64_t* n, const int32_t* dtypes, int64_t count,
                          const double* part, int64_t n_part, double max_norm, float* norm, hipStream_t s) {
  int64_t bytes = 0;
  for (int64_t i = 0; i < count; ++i) bytes += n[i] * bytes_of(dtypes[i]);
  const bool stream = bytes >= echo::kClipStream;
  return for_launches<Args>(src, dst, n, dtypes, count, [&](const Args& a) {
    const hipError_t e = echo::launch_clip_scale(a, part, n_part, max_norm, norm, stream, s);
    norm = nullptr;  // the first launch writes it
    return e;
  });
}

echo_status check_clip_workspace(int64_t count, const void* workspace, size_t bytes) {
  if (count > 0 && (workspace == nullptr || bytes < echo_clip_workspace(count))) return ECHO_ERR_WORKSPACE;
  return aligned(workspace, 8) ? ECHO_OK : ECHO_ERR_ARG;
}

// ---- embedding ----

// Sizes that both directions share.
echo_status check_embed(int32_t P, int64_t rows, int64_t cols, int64_t n_tokens, int32_t t_dtype, int32_t o_dtype,
                        int32_t token_bytes, int64_t first, double scale) {
  if (!known(t_dtype) || !known(o_dtype) || !types_mix(t_dtype, o_dtype)) return ECHO_ERR_DTYPE;
  if (token_bytes != 4 && token_bytes != 8) return ECHO_ERR_DTYPE;
  if (P < 1 || P > ECHO_MAX_RANKS || rows < 0 || cols < 0 || n_tokens < 0 || cols > echo::kStepMaxCols ||
      n_tokens > (int64_t{1} << 27) || rows > (int64_t{1} << 31) - 2 || P * rows > (int64_t{1} << 31) - 2)
    return ECHO_ERR_SHAPE;
  if (first < 0 || first > int64_t{1} << 62 || !is_finite(static_cast<float>(scale))) return ECHO_ERR_ARG;
  return ECHO_OK;
}


}  // namespace

extern "C" {

echo_status echo_block_norm(const echo_block* b, const void* x, int64_t ldx, const void* y, int64_t ldy, void* out,
                            int64_t ldo, void* a, int64_t lda, echo_stream_t stream) {
  echo_status e = check_block(b, y != nullptr);
  if (e != ECHO_OK) return e;
  if ((y != nullptr) != (out != nullptr) && b->rows > 0 && b->cols > 0) return ECHO_ERR_ARG;
  if (a == nullptr && b->w_pre != nullptr) return ECHO_ERR_ARG;
  if (b->rows == 0 || b->cols == 0) return ECHO_OK;
  if (x == nullptr || (out == nullptr && a == nullptr)) return ECHO_ERR_ARG;
  const int64_t C = b->cols;
  Mat gate{b->gate, b->gate != nullptr ? b->gate_rows : 0, b->ld_gate, b->param_dtype};
  Mat mats[] = {{x, b->rows, ldx, b->x_dtype}, {y, b->rows, ldy, b->y_dtype}, {out, b->rows, ldo, b->x_dtype},
                {a, b->rows, lda, b->a_dtype}};
  for (Mat& m : mats)
    if ((e = check_mat(&m, C)) != ECHO_OK) return e;
  if ((e = check_mat(&gate, C)) != ECHO_OK) return e;
  const Mat ins[] = {mats[0], mats[1], gate, {b->w_post, 1, C, b->param_dtype}, {b->w_pre, 1, C, b->param_dtype}};
  // out may be x itself: a thread reads an element before it writes it
  if (!apart(mats + 2, 2, ins, 5, C, 0, 0)) return ECHO_ERR_ARG;
  echo::BlockNormArgs n{};
  n.p = params_of(*b, gate);
  n.x = x;
  n.y = y;
  n.out = out;
  n.a = a;
  n.ldx = mats[0].ld;
  n.ldy = mats[1].ld;
  n.ldo = mats[2].ld;
  n.lda = mats[3].ld;
  // a type that no operand has would only ask for another kernel
  const int32_t yt = y != nullptr ? b->y_dtype : b->x_dtype, at = a != nullptr ? b->a_dtype : b->x_dtype;
  return status_of(echo::launch_block_norm(n, elem(b->x_dtype), elem(yt), elem(at), static_cast<hipStream_t>(stream)));
}

size_t echo_block_norm_workspace(int64_t rows, int64_t cols, int64_t gate_rows) {
  if (rows < 1 || cols < 1 || rows > kMaxRows || cols > echo::kStepMaxCols || gate_rows < 0 ||
      (gate_rows > 0 && rows % gate_rows != 0))
    return 0;
  return echo::block_norm_workspace(rows, cols, gate_rows > 0 ? gate_rows : 1);
}

echo_status echo_block_norm_backward(const echo_block* b, const void* out, int64_t ldo, const void* y, int64_t ldy,
                                     const void* dout, int64_t lddo, const void* da, int64_t ldda, void* dx, int64_t lddx,
                                     void* dy, int64_t lddy, void* dgate, int64_t ld_dgate, void* dw_post, void* dw_pre,
                                     void* workspace, size_t workspace_bytes, echo_stream_t stream) {
  echo_status e = check_block(b, y != nullptr);
  if (e != ECHO_OK) return e;
  if ((dy != nullptr && y == nullptr) || (dgate != nullptr && b->gate == nullptr) ||
      (dw_post != nullptr && b->w_post == nullptr) || (dw_pre != nullptr && b->w_pre == nullptr))
    return ECHO_ERR_ARG;
  if (b->w_pre != nullptr && da == nullptr) return ECHO_ERR_ARG;
  if (b->cols == 0) return ECHO_OK;
  if (dx == nullptr && dy == nullptr && dgate == nullptr && dw_post == nullptr && dw_pre == nullptr) return ECHO_ERR_ARG;
  if (b->rows > 0 && (out == nullptr || (dout == nullptr && da == nullptr))) return ECHO_ERR_ARG;
  const int64_t C = b->cols;
  const int64_t n_gates = b->gate != nullptr ? b->gate_rows : 0;
  Mat gate{b->gate, n_gates, b->ld_gate, b->param_dtype};
  Mat ins[] = {{dout, b->rows, lddo, b->x_dtype}, {out, b->rows, ldo, b->x_dtype}, {y, b->rows, ldy, b->y_dtype},
               {da, b->rows, ldda, b->a_dtype}, gate, {b->w_post, 1, C, b->param_dtype}, {b->w_pre, 1, C, b->param_dtype}};
  Mat outs[] = {{dx, b->rows, lddx, b->x_dtype}, {dy, b->rows, lddy, b->y_dtype}, {dgate, n_gates, ld_dgate, b->param_dtype},
                {dw_post, 1, C, b->param_dtype}, {dw_pre, 1, C, b->param_dtype}};
  for (Mat& m : ins)
    if ((e = check_mat(&m, C)) != ECHO_OK) return e;
  for (Mat& m : outs)
    if ((e = check_mat(&m, C)) != ECHO_OK) return e;
  const size_t need = echo_block_norm_workspace(b->rows, C, n_gates);
  const bool sums = dgate != nullptr || dw_post != nullptr || dw_pre != nullptr;
  if (need > 0) {
    if (workspace == nullptr || workspace_bytes < need) return ECHO_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return ECHO_ERR_ARG;
    const Area w = area(workspace, 1, static_cast<int64_t>(need), 0);
    for (const Mat& m : ins)
      if (m.p != nullptr && m.rows != 0 && overlap(w, area_of(m, C))) return ECHO_ERR_ARG;
    for (const Mat& m : outs)
      if (m.p != nullptr && m.rows != 0 && overlap(w, area_of(m, C))) return ECHO_ERR_ARG;
  }
  // dx may be dout itself: a thread reads an element before it writes it
  if (!apart(outs, 5, ins, 7, C, 0, 0)) return ECHO_ERR_ARG;
  if (b->rows == 0 && !sums) return ECHO_OK;
  echo::BlockNormBwdArgs n{};
  n.p = params_of(*b, ins[4]);
  n.out = out;
  n.y = y;
  n.dout = dout;
  n.da = da;
  n.dx = dx;
  n.dy = dy;
  n.dgate = dgate;
  n.dw_post = dw_post;
  n.dw_pre = dw_pre;
  n.ldo = ins[1].ld;
  n.ldy = ins[2].ld;
  n.lddo = ins[0].ld;
  n.ldda = ins[3].ld;
  n.lddx = outs[0].ld;
  n.lddy = outs[1].ld;
  n.lddg = outs[2].ld;
  n.part = static_cast<float*>(workspace);
  n.stats = reinterpret_cast<float4*>(static_cast<char*>(workspace) +
                                      (echo::block_norm_part(b->rows, C, n.p.n_gates) + 15) / 16 * 16);
  const int32_t yt = y != nullptr ? b->y_dtype : b->x_dtype, at = da != nullptr ? b->a_dtype : b->x_dtype;
  return status_of(echo::launch_block_norm_bwd(n, elem(b->x_dtype), elem(yt), elem(at), static_cast<hipStream_t>(stream)));
}

size_t echo_clip_workspace(int64_t n_tensors) {
  if (n_tensors < 1 || n_tensors > (int64_t{1} << 24)) return 0;
  const int64_t launches = (n_tensors + echo::ClipInPlace::kTensors - 1) / echo::ClipInPlace::kTensors;
  return static_cast<size_t>(launches) * echo::kClipGroups * sizeof(double);
}

echo_status echo_grad_norm(const void* const* grads, const int64_t* numel, const int32_t* dtypes, int64_t n_tensors,
                           float* norm, void* workspace, size_t workspace_bytes, echo_stream_t stream) {
  echo_status e = check_tensors(grads, nullptr, numel, dtypes, n_tensors);
  if (e != ECHO_OK) return e;
  if (norm == nullptr || !aligned(norm, 4)) return ECHO_ERR_ARG;
  if ((e = check_clip_workspace(n_tensors, workspace, workspace_bytes)) != ECHO_OK) return e;
  if ((e = tensors_apart(grads, nullptr, numel, dtypes, n_tensors, norm, workspace)) != ECHO_OK) return e;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  double* part = static_cast<double*>(workspace);
  int64_t n_part;
  if ((e = launch_sums(grads, numel, dtypes, n_tensors, part, &n_part, s)) != ECHO_OK) return e;
  return status_of(echo::launch_clip_norm(part, n_part, norm, s));
}

echo_status echo_clip_grads(const void* const* grads, void* const* out, const int64_t* numel, const int32_t* dtypes,
                            int64_t n_tensors, double max_norm, float* norm, void* workspace, size_t workspace_bytes,
                            echo_stream_t stream) {
  echo_status e = check_tensors(grads, out, numel, dtypes, n_tensors);
  if (e != ECHO_OK) return e;
  if (n_tensors > 0 && out == nullptr) return ECHO_ERR_ARG;
  if (!(max_norm >= 0.0) || !is_finite(max_norm)) return ECHO_ERR_ARG;  // also refuses NaN
  if (norm == nullptr || !aligned(norm, 4)) return ECHO_ERR_ARG;
  if ((e = check_clip_workspace(n_tensors, workspace, workspace_bytes)) != ECHO_OK) return e;
  if ((e = tensors_apart(grads, out, numel, dtypes, n_tensors, norm, workspace)) != ECHO_OK) return e;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  double* part = static_cast<double*>(workspace);
  int64_t n_part;
  if ((e = launch_sums(grads, numel, dtypes, n_tensors, part, &n_part, s)) != ECHO_OK) return e;
  if (n_part == 0) return status_of(echo::launch_clip_norm(part, 0, norm, s));
  if (n_part > echo::kClipGroups) {
    if ((e = status_of(echo::launch_clip_join(part, n_part, s))) != ECHO_OK) return e;
    n_part = 1;
  }
  bool in_place = true;
  for (int64_t i = 0; i < n_tensors && in_place; ++i) in_place = numel[i] == 0 || grads[i] == out[i];
  return in_place ? launch_scales<echo::ClipInPlace>(grads, out, numel, dtypes, n_tensors, part, n_part, max_norm, norm, s)
                  : launch_scales<echo::ClipApart>(grads, out, numel, dtypes, n_tensors, part, n_part, max_norm, norm, s);
}

echo_status echo_embed(const void* const* tables, const void* tokens, void* const* out, int32_t P, int64_t rows,
                       int64_t cols, int64_t ldt, int64_t n_tokens, int64_t ldo, int32_t table_dtype, int32_t out_dtype,
                       int32_t token_bytes, int64_t first, double scale, echo_stream_t stream) {
  echo_status e = check_embed(P, rows, cols, n_tokens, table_dtype, out_dtype, token_bytes, first, scale);
  if (e != ECHO_OK) return e;
  if (cols == 0 || n_tokens == 0) return ECHO_OK;
  if (tokens == nullptr || out == nullptr || (tables == nullptr && rows > 0)) return ECHO_ERR_ARG;
  if (!aligned(tokens, static_cast<uintptr_t>(token_bytes))) return ECHO_ERR_ARG;
  echo::EmbedArgs a{};
  Mat ins[ECHO_MAX_RANKS], outs[ECHO_MAX_RANKS];
  for (int r = 0; r < P; ++r) {
    ins[r] = Mat{rows > 0 ? tables[r] : nullptr, rows, ldt, table_dtype};
    outs[r] = Mat{out[r], n_tokens, ldo, out_dtype};
    if ((ins[r].p == nullptr && rows > 0) || outs[r].p == nullptr) return ECHO_ERR_ARG;
    if ((e = check_mat(&ins[r], cols)) != ECHO_OK || (e = check_mat(&outs[r], cols)) != ECHO_OK) return e;
    a.table[r] = ins[r].p;
    a.out[r] = out[r];
  }
  if (!apart(outs, P, ins, P, cols, -1, -1)) return ECHO_ERR_ARG;
  const Area t = area(tokens, 1, n_tokens * token_bytes, 0);
  for (int r = 0; r < P; ++r)
    if (overlap(area_of(outs[r], cols), t)) return ECHO_ERR_ARG;
  a.tokens = tokens;
  a.V = rows;
  a.C = cols;
  a.ldt = ins[0].ld;
  a.T = n_tokens;
  a.ldo = outs[0].ld;
  a.first = first;
  a.scale = static_cast<float>(scale);
  a.P = P;
  a.wide = token_bytes == 8;
  return status_of(echo::launch_embed(a, elem(table_dtype), elem(out_dtype), static_cast<hipStream_t>(stream)));
}

size_t echo_embed_workspace(int64_t n_tokens, int64_t cols) {
  if (n_tokens < 1 || cols < 1 || n_tokens > (int64_t{1} << 27) || cols > echo::kStepMaxCols) return 0;
  return echo::embed_layout(n_tokens, cols).bytes;
}

echo_status echo_embed_backward(const void* dout, const void* tokens, void* const* dtables, int32_t P, int64_t rows,
                                int64_t cols, int64_t ldt, int64_t n_tokens, int64_t lddo, int32_t out_dtype,
                                int32_t table_dtype, int32_t token_bytes, int64_t first, double scale, void* workspace,
                                size_t workspace_bytes, echo_stream_t stream) {
  echo_status e = check_embed(P, rows, cols, n_tokens, table_dtype, out_dtype, token_bytes, first, scale);
  if (e != ECHO_OK) return e;
  if (cols == 0 || rows == 0) return ECHO_OK;
  if (dtables == nullptr || (n_tokens > 0 && (tokens == nullptr || dout == nullptr))) return ECHO_ERR_ARG;
  if (!aligned(tokens, static_cast<uintptr_t>(token_bytes))) return ECHO_ERR_ARG;
  const size_t need = echo_embed_workspace(n_tokens, cols);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return ECHO_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return ECHO_ERR_ARG;
  echo::EmbedBwdArgs a{};
  Mat in{dout, n_tokens, lddo, out_dtype}, outs[ECHO_MAX_RANKS];
  if ((e = check_mat(&in, cols)) != ECHO_OK) return e;
  for (int r = 0; r < P; ++r) {
    outs[r] = Mat{dtables[r], rows, ldt, table_dtype};
    if (outs[r].p == nullptr) return ECHO_ERR_ARG;
    if ((e = check_mat(&outs[r], cols)) != ECHO_OK) return e;
    a.dtable[r] = dtables[r];
  }
  if (!apart(outs, P, &in, 1, cols, -1, -1)) return ECHO_ERR_ARG;
  if (n_tokens > 0) {
    const Area t = area(tokens, 1, n_tokens * token_bytes, 0), w = area(workspace, 1, static_cast<int64_t>(need), 0);
    if (overlap(w, t) || overlap(w, area_of(in, cols))) return ECHO_ERR_ARG;
    for (int r = 0; r < P; ++r)
      if (overlap(area_of(outs[r], cols), t) || overlap(area_of(outs[r], cols), w)) return ECHO_ERR_ARG;
  }
  a.dout = dout;
  a.tokens = tokens;
  a.V = rows;
  a.C = cols;
  a.ldt = outs[0].ld;
  a.T = n_tokens;
  a.lddo = in.ld;
  a.first = first;
  a.scale = static_cast<float>(scale);
  a.P = P;
  a.wide = token_bytes == 8;
  a.workspace = workspace;
  return status_of(echo::launch_embed_bwd(a, elem(out_dtype), elem(table_dtype), static_cast<hipStream_t>(stream)));
}

}  // extern "C"
