// The end of one block and the start of the next in one pass over a row:
//   out = alpha x + gate * n,  n = y rs(y) (offset + w_post), or y without a post-norm
//   a   = out rs(out) (offset + w_pre),  rs(v) = 1 / sqrt(mean(v^2) + eps)
// A workgroup takes a row at a time and holds it in registers, 8 columns to a thread and
// run, so that x and y are read once and the statistics cost no second pass.  The next
// block's norm starts from the stream as it is stored, so that a call on the stored
// stream, and the backward pass, see the same row.
#include <type_traits>

#include "echo_row.h"

namespace echo {
namespace {

template <int X, int Y, int A, int RUNS>
__global__ __launch_bounds__(kMaxThreads) void echo_block_norm_k(const BlockNormArgs a) {
  __shared__ Slots<1> lds;
  int turn = 0;
  const int64_t C = a.p.C;
  for (int64_t row = blockIdx.x; row < a.p.R; row += gridDim.x) {
    float v[RUNS][8];
#pragma unroll
    for (int k = 0; k < RUNS; ++k) {
      const int64_t at = run_at(k);
      load_run<X>(a.x, row * a.ldx + at, run_length(at, C), v[k]);
    }
    if (a.y != nullptr) {
      float y[RUNS][8];
#pragma unroll
      for (int k = 0; k < RUNS; ++k) {
        const int64_t at = run_at(k);
        load_run<Y>(a.y, row * a.ldy + at, run_length(at, C), y[k]);
      }
      if (a.p.post) {
        float s[1] = {0.0f};
#pragma unroll
        for (int k = 0; k < RUNS; ++k)
#pragma unroll
          for (int i = 0; i < 8; ++i) s[0] = s[0] + y[k][i] * y[k][i];
        block_sums(s, &lds, &turn);
        const float rs = reciprocal_rms(s[0], a.p);
#pragma unroll
        for (int k = 0; k < RUNS; ++k) {
          const int64_t at = run_at(k);
          float w[8];
          load_weight(a.p, a.p.w_post, at, run_length(at, C), w);
#pragma unroll
          for (int i = 0; i < 8; ++i) y[k][i] = y[k][i] * rs * w[i];
        }
      }
      if (a.p.gate != nullptr) {
        const int64_t g = row / a.p.rows_per_gate * a.p.ldg;
#pragma unroll
        for (int k = 0; k < RUNS; ++k) {
          const int64_t at = run_at(k);
          float w[8];
          load_run(a.p.elem, a.p.gate, g + at, run_length(at, C), w);
#pragma unroll
          for (int i = 0; i < 8; ++i) y[k][i] = y[k][i] * w[i];
        }
      }
#pragma unroll
      for (int k = 0; k < RUNS; ++k) {
        const int64_t at = run_at(k);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[k][i] = stored<X>(a.p.alpha * v[k][i] + y[k][i]);
        store_run<X>(a.out, row * a.ldo + at, run_length(at, C), v[k]);
      }
    }
    if (a.a != nullptr) {
      float s[1] = {0.0f};
#pragma unroll
      for (int k = 0; k < RUNS; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) s[0] = s[0] + v[k][i] * v[k][i];
      block_sums(s, &lds, &turn);
      const float rs = reciprocal_rms(s[0], a.p);
#pragma unroll
      for (int k = 0; k < RUNS; ++k) {
        const int64_t at = run_at(k);
        float w[8];
        load_weight(a.p, a.p.w_pre, at, run_length(at, C), w);
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = v[k][i] * rs * w[i];
        store_run<A>(a.a, row * a.lda + at, run_length(at, C), w);
      }
    }
  }
}

// Rows longer than the registers hold: the row is read again (from the caches) for each
// statistic.  A thread reads back only what it wrote itself.
template <int X, int Y, int A>
__global__ __launch_bounds__(kMaxThreads) void echo_block_norm_long_k(const BlockNormArgs a) {
  __shared__ Slots<1> lds;
  int turn = 0;
  const int64_t C = a.p.C, runs = (C + 8 * kMaxThreads - 1) / (8 * kMaxThreads);
  for (int64_t row = blockIdx.x; row < a.p.R; row += gridDim.x) {
    float rs = 1.0f;
    if (a.y != nullptr && a.p.post) {
      float s[1] = {0.0f};
      for (int64_t k = 0; k < runs; ++k) {
        const int64_t at = run_at(k);
        float y[8];
        load_run<Y>(a.y, row * a.ldy + at, run_length(at, C), y);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = y[i] * y[i];
        s[0] = s[0] + sum8(y);
      }
      block_sums(s, &lds, &turn);
      rs = reciprocal_rms(s[0], a.p);
    }
    float s[1] = {0.0f};
    for (int64_t k = 0; k < runs; ++k) {
      const int64_t at = run_at(k);
      const int n = run_length(at, C);
      float v[8];
      load_run<X>(a.x, row * a.ldx + at, n, v);
      if (a.y != nullptr) {
        float y[8], w[8];
        load_run<Y>(a.y, row * a.ldy + at, n, y);
        if (a.p.post) {
          load_weight(a.p, a.p.w_post, at, n, w);
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = y[i] * rs * w[i];
        }
        if (a.p.gate != nullptr) {
          load_run(a.p.elem, a.p.gate, row / a.p.rows_per_gate * a.p.ldg + at, n, w);
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = y[i] * w[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = stored<X>(a.p.alpha * v[i] + y[i]);
        store_run<X>(a.out, row * a.ldo + at, n, v);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = v[i] * v[i];
      s[0] = s[0] + sum8(v);
    }
    if (a.a == nullptr) continue;
    block_sums(s, &lds, &turn);
    const float ra = reciprocal_rms(s[0], a.p);
    const void* in = a.y != nullptr ? a.out : a.x;
    const int64_t ld = a.y != nullptr ? a.ldo : a.ldx;
    for (int64_t k = 0; k < runs; ++k) {
      const int64_t at = run_at(k);
      const int n = run_length(at, C);
      float v[8], w[8];
      load_run<X>(in, row * ld + at, n, v);
      load_weight(a.p, a.p.w_pre, at, n, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = v[i] * ra * w[i];
      store_run<A>(a.a, row * a.lda + at, n, v);
    }
  }
}

template <int X, int Y, int A, int RUNS>
hipError_t launch_runs(const BlockNormArgs& a, unsigned grid, hipStream_t s) {
  hipLaunchKernelGGL((echo_block_norm_k<X, Y, A, RUNS>), dim3(grid), dim3(row_threads(a.p.C, RUNS)), 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_block_norm(const BlockNormArgs& a, Elem x, Elem y, Elem out_a, hipStream_t s) {
  const unsigned grid = static_cast<unsigned>(a.p.R < (int64_t{1} << 20) ? a.p.R : (int64_t{1} << 20));
  return with_types(x, y, out_a, [&](auto X, auto Y, auto A) {
    const int64_t per = 8 * kMaxThreads;
    if (a.p.C <= per) return launch_runs<X(), Y(), A(), 1>(a, grid, s);
    if (a.p.C <= 2 * per) return launch_runs<X(), Y(), A(), 2>(a, grid, s);
    hipLaunchKernelGGL((echo_block_norm_long_k<X(), Y(), A()>), dim3(grid), dim3(kMaxThreads), 0, s, a);
    return hipGetLastError();
  });
}

}  // namespace echo
