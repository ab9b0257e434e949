// C-ABI host side of the operators of the layer around the all-reduce: argument
// validation and one launch each on the caller's stream.  See include/echo.h for
// the contract of every entry point.
#include <math.h>

#include "echo.h"
#include "echo_layer_check.h"
#include "echo_layer_internal.h"

namespace {

int64_t blocks(int64_t n) { return (n + ECHO_FP8_BLOCK - 1) / ECHO_FP8_BLOCK; }

// Tiles of 128 x 128 over all ranks: a launch numbers its threads in 32 bits, 256
// (quantizer) or 512 (product) to a tile, a quarter of a tile at the smallest.
constexpr int64_t kMaxTiles = (int64_t{1} << 21) - 1;

// The scales of [rows, k] codes as an area.
Area scale_area(const echo_fp8& f, int r, int64_t rows, int64_t k) {
  const int64_t n0 = f.block_rows == 1 ? rows : blocks(rows), n1 = blocks(k);
  const int64_t es = f.scale_type == ECHO_SCALE_F32 ? 4 : 1;
  const bool by_row = f.scale_row_stride >= f.scale_k_stride;  // the wider stride
  const int64_t no = by_row ? n0 : n1, so = by_row ? f.scale_row_stride : f.scale_k_stride;
  const int64_t ni = by_row ? n1 : n0, si = by_row ? f.scale_k_stride : f.scale_row_stride;
  return area(f.scales[r], no, ((ni - 1) * si + 1) * es, so * es);
}

// Formats, layouts and pointers of P matrices [rows, k] (both at least 1).
echo_status check_fp8(const echo_fp8& f, int32_t P, int64_t rows, int64_t k, bool output) {
  if (f.format != ECHO_E4M3 && f.format != ECHO_E5M2) return ECHO_ERR_ARG;
  if (f.scale_type != ECHO_SCALE_F32 && f.scale_type != ECHO_SCALE_E8M0) return ECHO_ERR_ARG;
  if (f.block_rows != 1 && f.block_rows != ECHO_FP8_BLOCK) return ECHO_ERR_ARG;
  if (f.codes == nullptr || f.scales == nullptr) return ECHO_ERR_ARG;
  if (f.ld < k || f.ld % 16 != 0 || f.ld > echo::kFp8MaxDim) return ECHO_ERR_SHAPE;
  const int64_t n0 = f.block_rows == 1 ? rows : blocks(rows), n1 = blocks(k);
  if (f.scale_row_stride < 0 || f.scale_k_stride < 0) return ECHO_ERR_SHAPE;
  // the kernels address the scales of a block along k through 32-bit offsets
  constexpr int64_t kMaxExtent = int64_t{1} << 29;
  if ((n0 > 1 && f.scale_row_stride > kMaxExtent / n0) || (n1 > 1 && f.scale_k_stride > kMaxExtent / n1))
    return ECHO_ERR_SHAPE;
  if (output) {
    // distinct elements: one stride steps over the whole extent of the other dimension
    const bool rows_inside = n1 == 1 || (f.scale_row_stride >= 1 && f.scale_k_stride >= (n0 - 1) * f.scale_row_stride + 1);
    const bool k_inside = n0 == 1 || (f.scale_k_stride >= 1 && f.scale_row_stride >= (n1 - 1) * f.scale_k_stride + 1);
    const bool one_row = n0 == 1 && (n1 == 1 || f.scale_k_stride >= 1);
    const bool one_col = n1 == 1 && (n0 == 1 || f.scale_row_stride >= 1);
    if (!(n0 == 1 ? one_row : n1 == 1 ? one_col : (rows_inside || k_inside))) return ECHO_ERR_SHAPE;
  }
  const uintptr_t sa = f.scale_type == ECHO_SCALE_F32 ? 4 : 1;
  for (int r = 0; r < P; ++r)
    if (f.codes[r] == nullptr || f.scales[r] == nullptr || !aligned(f.codes[r], 16) || !aligned(f.scales[r], sa))
      return ECHO_ERR_ARG;
  return ECHO_OK;
}

}  // namespace

extern "C" {

echo_status echo_quantize_fp8(const void* const* X, int32_t P, int64_t rows, int64_t cols, int64_t ldx,
                              int32_t dtype, const echo_fp8* along_rows, const echo_fp8* along_cols,
                              echo_stream_t stream) {
  int64_t es = 0;
  if (!elem_bytes(dtype, &es)) return ECHO_ERR_DTYPE;
  if (P < 1 || P > ECHO_MAX_RANKS || rows < 0 || cols < 0 || rows > echo::kFp8MaxDim || cols > echo::kFp8MaxDim)
    return ECHO_ERR_SHAPE;
  if (along_rows == nullptr && along_cols == nullptr) return ECHO_ERR_ARG;
  if (along_rows != nullptr && along_cols != nullptr &&
      (along_rows->format != along_cols->format || along_rows->scale_type != along_cols->scale_type ||
       along_rows->block_rows != along_cols->block_rows))
    return ECHO_ERR_ARG;
  if (rows == 0 || cols == 0) return ECHO_OK;
  if (P * blocks(rows) * blocks(cols) > kMaxTiles) return ECHO_ERR_SHAPE;
  if (X == nullptr) return ECHO_ERR_ARG;
  ldx = pitch_of(rows, cols, ldx);
  if (!pitch_fits(rows, cols, ldx, es)) return ECHO_ERR_SHAPE;
  echo_status e;
  if (along_rows != nullptr && (e = check_fp8(*along_rows, P, rows, cols, true)) != ECHO_OK) return e;
  if (along_cols != nullptr && (e = check_fp8(*along_cols, P, cols, rows, true)) != ECHO_OK) return e;
  Area ins[ECHO_MAX_RANKS], outs[4 * ECHO_MAX_RANKS];
  int n_out = 0;
  for (int r = 0; r < P; ++r) {
    if (X[r] == nullptr || !aligned(X[r], static_cast<uintptr_t>(es))) return ECHO_ERR_ARG;
    ins[r] = area(X[r], rows, cols * es, ldx * es);
    if (along_rows != nullptr) {
      outs[n_out++] = area(along_rows->codes[r], rows, cols, along_rows->ld);
      outs[n_out++] = scale_area(*along_rows, r, rows, cols);
    }
    if (along_cols != nullptr) {
      outs[n_out++] = area(along_cols->codes[r], cols, rows, along_cols->ld);
      outs[n_out++] = scale_area(*along_cols, r, cols, rows);
    }
  }
  if (!outputs_apart(outs, n_out, ins, P)) return ECHO_ERR_ARG;
  echo::QuantFp8Args a{};
  a.R = rows;
  a.C = cols;
  a.ldx = ldx;
  const echo_fp8& any = along_rows != nullptr ? *along_rows : *along_cols;
  a.e5m2 = any.format == ECHO_E5M2;
  a.e8m0 = any.scale_type == ECHO_SCALE_E8M0;
  for (int r = 0; r < P; ++r) a.X[r] = X[r];
  const auto fill = [P](echo::Fp8Out* o, const echo_fp8* f) {
    if (f == nullptr) return;
    for (int r = 0; r < P; ++r) {
      o->codes[r] = static_cast<uint8_t*>(f->codes[r]);
      o->scales[r] = f->scales[r];
    }
    o->ld = f->ld;
    o->srs = f->scale_row_stride;
    o->sks = f->scale_k_stride;
  };
  fill(&a.rows, along_rows);
  fill(&a.cols, along_cols);
  return echo::launch_quantize_fp8(a, P, static_cast<echo::Elem>(dtype), any.block_rows == ECHO_FP8_BLOCK,
                                   static_cast<hipStream_t>(stream)) == hipSuccess
             ? ECHO_OK
             : ECHO_ERR_HIP;
}

echo_status echo_gemm_fp8(const echo_fp8* A, const echo_fp8* W, void* const* out, int32_t P, int64_t M,
                          int64_t N, int64_t K, int64_t ldo, int32_t out_dtype, echo_stream_t stream) {
  int64_t es = 0;
  if (!elem_bytes(out_dtype, &es)) return ECHO_ERR_DTYPE;
  if (P < 1 || P > ECHO_MAX_RANKS || M < 0 || N < 0 || K < 0 || M > echo::kFp8MaxDim || N > echo::kFp8MaxDim ||
      K > echo::kFp8MaxDim)
    return ECHO_ERR_SHAPE;
  if (A == nullptr || W == nullptr) return ECHO_ERR_ARG;
  if (A->scale_type != W->scale_type) return ECHO_ERR_ARG;
  if (M == 0 || N == 0) return ECHO_OK;
  if (P * blocks(M) * blocks(N) > kMaxTiles) return ECHO_ERR_SHAPE;
  if (out == nullptr) return ECHO_ERR_ARG;
  ldo = pitch_of(M, N, ldo);
  if (!pitch_fits(M, N, ldo, es)) return ECHO_ERR_SHAPE;
  echo_status e;
  if (K > 0) {
    if ((e = check_fp8(*A, P, M, K, false)) != ECHO_OK) return e;
    if ((e = check_fp8(*W, P, N, K, false)) != ECHO_OK) return e;
  }
  Area ins[4 * ECHO_MAX_RANKS], outs[ECHO_MAX_RANKS];
  int n_in = 0;
  for (int r = 0; r < P; ++r) {
    if (out[r] == nullptr || !aligned(out[r], static_cast<uintptr_t>(es))) return ECHO_ERR_ARG;
    outs[r] = area(out[r], M, N * es, ldo * es);
    if (K > 0) {
      ins[n_in++] = area(A->codes[r], M, K, A->ld);
      ins[n_in++] = area(W->codes[r], N, K, W->ld);
      ins[n_in++] = scale_area(*A, r, M, K);
      ins[n_in++] = scale_area(*W, r, N, K);
    }
  }
  if (!outputs_apart(outs, P, ins, n_in)) return ECHO_ERR_ARG;
  echo::GemmFp8Args a{};
  for (int r = 0; r < P; ++r) {
    if (K > 0) {
      a.A[r] = static_cast<const uint8_t*>(A->codes[r]);
      a.W[r] = static_cast<const uint8_t*>(W->codes[r]);
      a.sA[r] = A->scales[r];
      a.sW[r] = W->scales[r];
    }
    a.out[r] = out[r];
  }
  a.M = M;
  a.N = N;
  a.K = K;
  a.lda = A->ld;
  a.ldw = W->ld;
  a.ldo = ldo;
  a.sa_row = A->scale_row_stride;
  a.sa_k = A->scale_k_stride;
  a.sw_row = W->scale_row_stride;
  a.sw_k = W->scale_k_stride;
  a.sa_shift = A->block_rows == 1 ? 0 : 7;
  a.sw_shift = W->block_rows == 1 ? 0 : 7;
  a.out_elem = out_dtype;
  return echo::launch_gemm_fp8(a, P, A->format == ECHO_E5M2, W->format == ECHO_E5M2,
                               A->scale_type == ECHO_SCALE_E8M0, static_cast<hipStream_t>(stream)) == hipSuccess
             ? ECHO_OK
             : ECHO_ERR_HIP;
}

echo_status echo_dropout_add(const void* x, const void* residual, void* out, int64_t rows, int64_t cols,
                             int64_t ldx, int64_t ldr, int64_t ldo, int32_t x_dtype, int32_t out_dtype,
                             double p, const int64_t* rng, int64_t offset, int64_t first,
                             echo_stream_t stream) {
  int64_t ex = 0, eo = 0;
  if (!elem_bytes(x_dtype, &ex) || !elem_bytes(out_dtype, &eo)) return ECHO_ERR_DTYPE;
  constexpr int64_t kMaxSide = (int64_t{1} << 31) - 1, kMaxElems = int64_t{1} << 40;
  if (rows < 0 || cols < 0 || rows > kMaxSide || cols > kMaxSide) return ECHO_ERR_SHAPE;
  if (cols > 0 && rows > kMaxElems / cols) return ECHO_ERR_SHAPE;
  if (!(p >= 0.0) || p > 1.0 - 1.0 / 65536.0) return ECHO_ERR_ARG;  // also refuses NaN
  const int64_t n = rows * cols;
  if (first < 0 || first > (int64_t{1} << 62) - n) return ECHO_ERR_ARG;
  if (n == 0) return ECHO_OK;
  ldx = pitch_of(rows, cols, ldx);
  ldo = pitch_of(rows, cols, ldo);
  ldr = residual != nullptr ? pitch_of(rows, cols, ldr) : cols;
  if (!pitch_fits(rows, cols, ldx, ex) || !pitch_fits(rows, cols, ldo, eo) || !pitch_fits(rows, cols, ldr, eo))
    return ECHO_ERR_SHAPE;
  if (x == nullptr || out == nullptr || rng == nullptr) return ECHO_ERR_ARG;
  if (!aligned(x, static_cast<uintptr_t>(ex)) || !aligned(out, static_cast<uintptr_t>(eo)) ||
      !aligned(residual, static_cast<uintptr_t>(eo)) || !aligned(rng, 8))
    return ECHO_ERR_ARG;
  const Area ao = area(out, rows, cols * eo, ldo * eo), ax = area(x, rows, cols * ex, ldx * ex);
  const Area ag = area(rng, 1, 16, 0);
  // in place: every element is read and written by one thread, the read first
  const bool on_x = out == x && ex == eo && ldx == ldo;
  const bool on_r = out == residual && ldr == ldo;
  if ((!on_x && overlap(ao, ax)) || overlap(ao, ag)) return ECHO_ERR_ARG;
  if (residual != nullptr && !on_r && overlap(ao, area(residual, rows, cols * eo, ldr * eo))) return ECHO_ERR_ARG;
  echo::DropoutArgs a{};
  a.x = x;
  a.residual = residual;
  a.out = out;
  a.R = rows;
  a.C = cols;
  a.ldx = ldx;
  a.ldr = ldr;
  a.ldo = ldo;
  a.rng = rng;
  a.offset = offset;
  a.first = first;
  const double t = nearbyint(p * 65536.0);  // at most 65535
  a.threshold = static_cast<uint32_t>(t);
  a.scale = static_cast<float>(65536.0 / (65536.0 - t));
  return echo::launch_dropout(a, static_cast<echo::Elem>(x_dtype), static_cast<echo::Elem>(out_dtype),
                              static_cast<hipStream_t>(stream)) == hipSuccess
             ? ECHO_OK
             : ECHO_ERR_HIP;
}

}  // extern "C"
