// The end of one block and the start of the next in one pass over a row:
//   out = alpha x + gate * n,  n = y rs(y) (offset + w_post), or y without a post-norm
//   a   = out rs(out) (offset + w_pre),  rs(v) = 1 / sqrt(mean(v^2) + eps)
// A workgroup takes a row at a time and holds it in registers, 8 columns to a thread and
// run, so that x and y are read once and the statistics cost no second pass.  The next
// block's norm starts from the stream as it is stored, so that a call on the stored
// stream, and the backward pass, see the same row.
//
// Bound by the memory: 16384 x 8192 bfloat16 with a post-norm, a gate and two weights takes
// 196 us, 5.5 TB/s of what it has to move (an elementwise product of two tensors reaches 6.2),
// and fetches and writes no byte twice; 8192 x 4096 39 us, 2048 x 4096 fp32 22. One row of 8192
// takes 3 us of kernel, one trip to memory and two reductions.
#include <type_traits>

#include "echo_row.h"

namespace echo {
namespace {

// The sum over a row of a thread's runs' sums.  Rows of up to 8192 columns are added up the
// same way with one run to a thread as with two.
template <int RUNS, int MAXT>
__device__ __forceinline__ float row_sum(float (&v)[RUNS], Slots<1>* lds, int* turn) {
  if constexpr (RUNS * MAXT <= kMaxThreads && RUNS > 1) {
    return block_sum_of_runs(v, lds, turn);
  } else {
    float s[1] = {v[0]};
#pragma unroll
    for (int k = 1; k < RUNS; ++k) s[0] = s[0] + v[k];
    block_sums(s, lds, turn);
    return s[0];
  }
}

// EARLY: the parameters are loaded with the row.  Behind the row's statistics they come from
// the L2 cache a workgroup at a time, which costs 3 to 8 %, but their registers would leave
// one workgroup of 1024 threads and two runs to a CU (8192 x 12288 bfloat16: 196 us, against
// 147 with two).
template <int X, int Y, int A, int RUNS, int MAXT, bool EARLY, bool STREAM>
__global__ __launch_bounds__(MAXT) void echo_block_norm_k(const BlockNormArgs a, int64_t row0) {
  __shared__ Slots<1> lds;
  int turn = 0;
  const int64_t C = a.p.C;
  const int e = a.p.elem;
  const int64_t row = row0 + blockIdx.x;
  const int64_t gate_row = a.p.gate != nullptr ? gate_of(a.p, row) * a.p.ldg : 0;
  Run run[RUNS];
  Raw<X> rx[RUNS];
  Raw<Y> ry[RUNS];
  RawParam rpost[RUNS], rgate[RUNS], rpre[RUNS];
#pragma unroll
  for (int k = 0; k < RUNS; ++k) {
    run[k] = run_of(k, C);
    if (a.y != nullptr) load_raw<Y>(a.y, row * a.ldy, run[k].at, &ry[k]);
    load_raw<X>(a.x, row * a.ldx, run[k].at, &rx[k]);
  }
#pragma unroll
  for (int k = 0; k < RUNS; ++k) {
    if (EARLY && a.p.w_post != nullptr) load_raw(e, a.p.w_post, 0, run[k].at, &rpost[k]);
    if (EARLY && a.p.gate != nullptr) load_raw(e, a.p.gate, gate_row, run[k].at, &rgate[k]);
    if (EARLY && a.p.w_pre != nullptr) load_raw(e, a.p.w_pre, 0, run[k].at, &rpre[k]);
  }
  float v[RUNS][8];
  float s[RUNS];
  if (a.y != nullptr) {
    float rs = 1.0f;
    if (a.p.post) {
#pragma unroll
      for (int k = 0; k < RUNS; ++k) {
        float y[8];
        widen<Y>(ry[k], y);
        clear_below(run[k].lo, y);
        s[k] = dot8(y, y, 0.0f);
      }
      rs = reciprocal_rms(row_sum<RUNS, MAXT>(s, &lds, &turn), a.p);
    }
#pragma unroll
    for (int k = 0; k < RUNS; ++k) {
      float y[8], w[8];
      widen<Y>(ry[k], y);
      if (a.p.post) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = y[i] * rs;
        if (a.p.w_post != nullptr) {
          if (!EARLY) load_raw(e, a.p.w_post, 0, run[k].at, &rpost[k]);
          widen(e, rpost[k], w);
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = y[i] * (w[i] + a.p.offset);
        }
      }
      if (a.p.gate != nullptr) {
        if (!EARLY) load_raw(e, a.p.gate, gate_row, run[k].at, &rgate[k]);
        widen(e, rgate[k], w);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = y[i] * w[i];
      }
      widen<X>(rx[k], v[k]);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[k][i] = stored<X>(a.p.alpha * v[k][i] + y[i]);
      store_from<X, STREAM>(a.out, row * a.ldo, run[k], v[k]);
    }
  } else {
#pragma unroll
    for (int k = 0; k < RUNS; ++k) widen<X>(rx[k], v[k]);
  }
  if (a.a == nullptr) return;
#pragma unroll
  for (int k = 0; k < RUNS; ++k) {
    clear_below(run[k].lo, v[k]);
    s[k] = dot8(v[k], v[k], 0.0f);
  }
  const float rs = reciprocal_rms(row_sum<RUNS, MAXT>(s, &lds, &turn), a.p);
#pragma unroll
  for (int k = 0; k < RUNS; ++k) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[k][i] = v[k][i] * rs;
    if (a.p.w_pre != nullptr) {
      float w[8];
      if (!EARLY) load_raw(e, a.p.w_pre, 0, run[k].at, &rpre[k]);
      widen(e, rpre[k], w);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[k][i] = v[k][i] * (w[i] + a.p.offset);
    }
    store_from<A, STREAM>(a.a, row * a.lda, run[k], v[k]);
  }
}

// Rows longer than the registers hold, and rows of fewer than 8 columns: the row is read again
// (from the caches) for each statistic.  A thread reads back only what it wrote itself.
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
          load_run(a.p.elem, a.p.gate, gate_of(a.p, row) * a.p.ldg + at, n, w);
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

template <int X, int Y, int A, int RUNS, int MAXT, bool EARLY, bool STREAM = false>
hipError_t launch_runs(const BlockNormArgs& a, hipStream_t s) {
  const int threads = row_threads(a.p.C, RUNS);
  const int64_t most = ((int64_t{1} << 32) - 1) / threads;  // a launch numbers its threads in 32 bits
  for (int64_t row = 0; row < a.p.R; row += most) {
    const int64_t rows = a.p.R - row < most ? a.p.R - row : most;
    hipLaunchKernelGGL((echo_block_norm_k<X, Y, A, RUNS, MAXT, EARLY, STREAM>), dim3(static_cast<unsigned>(rows)), dim3(threads), 0, s, a, row);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_block_norm(const BlockNormArgs& a, Elem x, Elem y, Elem out_a, hipStream_t s) {
  return with_types(x, y, out_a, [&](auto X, auto Y, auto A) {
    const int64_t per = 8 * kMaxThreads;
    // two runs to a thread where there are rows for several workgroups to a CU (16384 x 8192
    // bfloat16: 195 us, one run 199, and 197 and 204 with results that stay in the caches; 65536 x
    // 2048: 182 and 186), one where there are few (2048 x 4096: 12.8 us, two runs 13.1), or where a
    // row is short (262144 x 512: 171 and 206)
    if (a.p.C >= 8 && a.p.C <= per) {
      if (a.p.C <= 1024 || a.p.R <= 2048) return launch_runs<X(), Y(), A(), 1, 1024, true>(a, s);
      const int64_t x = elem_size(X()), y = a.y != nullptr ? x + elem_size(Y()) : 0;
      constexpr bool kAny = X() != kElemF32 || A() != kElemF32;  // 16-bit results
      if (kAny && block_streams(a.p.R, a.p.C, x + y + elem_size(A()))) return launch_runs<X(), Y(), A(), 2, 512, true, kAny>(a, s);
      return launch_runs<X(), Y(), A(), 2, 512, true>(a, s);
    }
    if (a.p.C >= 8 && a.p.C <= 2 * per) return launch_runs<X(), Y(), A(), 2, 1024, false>(a, s);
    const unsigned grid = static_cast<unsigned>(a.p.R < (int64_t{1} << 20) ? a.p.R : (int64_t{1} << 20));
    hipLaunchKernelGGL((echo_block_norm_long_k<X(), Y(), A()>), dim3(grid), dim3(kMaxThreads), 0, s, a);
    return hipGetLastError();
  });
}

}  // namespace echo
