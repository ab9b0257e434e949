// Gradients of the block norm (see echo_block_norm.hip).  With s the stream as stored,
// rs = rs(s), u = da (offset + w_pre) and t the whole gradient of s,
//   t  = dout + rs u - s rs^3 mean(u s),           dx = alpha t
//   dn = gate t,  v = dn (offset + w_post),        dy = ry v - y ry^3 mean(v y)  (ry = rs(y); dn without a post-norm)
//   dw_pre = sum over rows of da s rs,  dw_post = sum of dn y ry,  dgate = sum over the gate's rows of t n.
// sum s^2, sum u s and sum y^2 need nothing but the inputs, so they are one reduction and
// no statistics of the forward pass are kept; sum v y needs t, which is the second.  A
// workgroup takes consecutive rows and sums its columns in registers; the workgroups' sums
// go to the workspace and are added in order by a second kernel, so the result does not
// depend on timing.
#include <type_traits>

#include "echo_row.h"

namespace echo {

// 512 workgroups where the rows suffice: two to a CU.
constexpr int64_t kBwdGroups = 512;

BlockSplit block_split(int64_t R, int64_t n_gates) {
  BlockSplit s{};
  if (R == 0) return s;
  const int64_t per_gate = R / n_gates;
  if (n_gates < kBwdGroups) {
    const int64_t most = kBwdGroups / n_gates;  // workgroups to a gate
    s.rows = (per_gate + most - 1) / most;
    s.chunks = (per_gate + s.rows - 1) / s.rows;
    s.groups = n_gates * s.chunks;
  } else {
    s.gates = (n_gates + kBwdGroups - 1) / kBwdGroups;
    s.groups = (n_gates + s.gates - 1) / s.gates;
    s.rows = s.gates * per_gate;
  }
  return s;
}

namespace {

enum Sum { kSumPre = 0, kSumPost = 1, kSumGate = 2, kSums = 3 };

__device__ __forceinline__ float* part_at(const BlockNormBwdArgs& a, int64_t group, int sum) {
  return a.part + (group * kSums + sum) * a.p.C;
}

// The rows of workgroup blockIdx.x.
__device__ __forceinline__ void rows_of(const BlockNormBwdArgs& a, const BlockSplit& sp, int64_t* lo, int64_t* hi) {
  if (sp.chunks != 0) {
    const int64_t g = blockIdx.x / sp.chunks, c = blockIdx.x % sp.chunks;
    *lo = g * a.p.rows_per_gate + c * sp.rows;
    const int64_t end = (g + 1) * a.p.rows_per_gate;
    *hi = *lo + sp.rows < end ? *lo + sp.rows : end;
  } else {
    *lo = blockIdx.x * sp.rows;
    *hi = *lo + sp.rows < a.p.R ? *lo + sp.rows : a.p.R;
  }
}

template <int X, int Y, int A>
__global__ __launch_bounds__(kMaxThreads) void echo_block_norm_bwd_k(const BlockNormBwdArgs a, const BlockSplit sp) {
  __shared__ Slots<3> lds;
  int turn = 0;
  const int64_t C = a.p.C, at = run_at(0);
  const int n = run_length(at, C);
  const float cols = static_cast<float>(C);
  float wp[8], wq[8], acc[kSums][8];
  load_weight(a.p, a.p.w_pre, at, n, wp);
  load_weight(a.p, a.p.w_post, at, n, wq);
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[kSumPre][i] = acc[kSumPost][i] = acc[kSumGate][i] = 0.0f;
  int64_t lo, hi;
  rows_of(a, sp, &lo, &hi);
  for (int64_t row = lo; row < hi; ++row) {
    float s[8], da[8], t[8], y[8];
    load_run<X>(a.out, row * a.ldo + at, n, s);
#pragma unroll
    for (int i = 0; i < 8; ++i) da[i] = t[i] = y[i] = 0.0f;
    if (a.da != nullptr) load_run<A>(a.da, row * a.ldda + at, n, da);
    if (a.dout != nullptr) load_run<X>(a.dout, row * a.lddo + at, n, t);
    if (a.y != nullptr) load_run<Y>(a.y, row * a.ldy + at, n, y);
    float m[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      m[0] = m[0] + s[i] * s[i];
      m[1] = m[1] + da[i] * wp[i] * s[i];
      m[2] = m[2] + y[i] * y[i];
    }
    block_sums(m, &lds, &turn);
    if (a.da != nullptr) {
      const float rs = reciprocal_rms(m[0], a.p), k = rs * rs * (m[1] / cols);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        t[i] = t[i] + rs * (da[i] * wp[i] - s[i] * k);
        acc[kSumPre][i] = acc[kSumPre][i] + da[i] * (s[i] * rs);
      }
    }
    if (a.dx != nullptr) {
      float dx[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) dx[i] = a.p.alpha * t[i];
      store_run<X>(a.dx, row * a.lddx + at, n, dx);
    }
    if (a.y == nullptr) continue;
    float gate[8];
    if (a.p.gate != nullptr) {
      load_run(a.p.elem, a.p.gate, row / a.p.rows_per_gate * a.p.ldg + at, n, gate);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) gate[i] = 1.0f;
    }
    float dy[8];
    if (a.p.post) {
      const float ry = reciprocal_rms(m[2], a.p);
      float q[1] = {0.0f};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float yh = y[i] * ry, dn = gate[i] * t[i];
        acc[kSumGate][i] = acc[kSumGate][i] + t[i] * (yh * wq[i]);
        acc[kSumPost][i] = acc[kSumPost][i] + dn * yh;
        dy[i] = dn * wq[i];
        q[0] = q[0] + dy[i] * y[i];
      }
      block_sums(q, &lds, &turn);
      const float k = ry * ry * (q[0] / cols);
#pragma unroll
      for (int i = 0; i < 8; ++i) dy[i] = ry * (dy[i] - y[i] * k);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        acc[kSumGate][i] = acc[kSumGate][i] + t[i] * y[i];
        dy[i] = gate[i] * t[i];
      }
    }
    if (a.dy != nullptr) store_run<Y>(a.dy, row * a.lddy + at, n, dy);
    if (sp.chunks == 0 && a.dgate != nullptr && (row + 1) % a.p.rows_per_gate == 0) {
      // the last row of a gate that is this workgroup's alone
      store_run(a.p.elem, a.dgate, row / a.p.rows_per_gate * a.lddg + at, n, acc[kSumGate]);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[kSumGate][i] = 0.0f;
    }
  }
  if (a.dw_pre != nullptr) store_run<kElemF32>(part_at(a, blockIdx.x, kSumPre), at, n, acc[kSumPre]);
  if (a.dw_post != nullptr) store_run<kElemF32>(part_at(a, blockIdx.x, kSumPost), at, n, acc[kSumPost]);
  if (a.dgate != nullptr && sp.chunks != 0)
    store_run<kElemF32>(part_at(a, blockIdx.x, kSumGate), at, n, acc[kSumGate]);
}

__device__ __forceinline__ void add_to(float* p, int64_t at, int n, bool first, const float v[8]) {
  float o[8];
  if (first) {
    store_run<kElemF32>(p, at, n, v);
    return;
  }
  load_run<kElemF32>(p, at, n, o);
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = o[i] + v[i];
  store_run<kElemF32>(p, at, n, o);
}

// Rows of more than 8 * kMaxThreads columns: the inputs are read again for each statistic
// and the column sums are kept in the workspace, each by the thread that owns its columns.
template <int X, int Y, int A>
__global__ __launch_bounds__(kMaxThreads) void echo_block_norm_bwd_long_k(const BlockNormBwdArgs a, const BlockSplit sp) {
  __shared__ Slots<3> lds;
  int turn = 0;
  const int64_t C = a.p.C, runs = (C + 8 * kMaxThreads - 1) / (8 * kMaxThreads);
  const float cols = static_cast<float>(C);
  int64_t lo, hi;
  rows_of(a, sp, &lo, &hi);
  for (int64_t row = lo; row < hi; ++row) {
    const int64_t gate_row = row / a.p.rows_per_gate;
    float m[3] = {0.0f, 0.0f, 0.0f};
    for (int64_t j = 0; j < runs; ++j) {
      const int64_t at = run_at(j);
      const int n = run_length(at, C);
      float s[8], v[8], w[8];
      load_run<X>(a.out, row * a.ldo + at, n, s);
      if (a.da != nullptr) {
        load_run<A>(a.da, row * a.ldda + at, n, v);
        load_weight(a.p, a.p.w_pre, at, n, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = v[i] * w[i] * s[i];
        m[1] = m[1] + sum8(v);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] = s[i] * s[i];
      m[0] = m[0] + sum8(s);
      if (a.y != nullptr) {
        load_run<Y>(a.y, row * a.ldy + at, n, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = v[i] * v[i];
        m[2] = m[2] + sum8(v);
      }
    }
    block_sums(m, &lds, &turn);
    const float rs = reciprocal_rms(m[0], a.p), k = rs * rs * (m[1] / cols);
    const float ry = a.p.post ? reciprocal_rms(m[2], a.p) : 1.0f;
    float ky = 0.0f;
    // two rounds: the statistic of the post-norm's gradient, then the gradients
    for (int round = a.y != nullptr && a.p.post ? 0 : 1; round < 2; ++round) {
      float q[1] = {0.0f};
      for (int64_t j = 0; j < runs; ++j) {
        const int64_t at = run_at(j);
        const int n = run_length(at, C);
        float t[8], s[8], v[8], w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = 0.0f;
        if (a.dout != nullptr) load_run<X>(a.dout, row * a.lddo + at, n, t);
        if (a.da != nullptr) {
          load_run<X>(a.out, row * a.ldo + at, n, s);
          load_run<A>(a.da, row * a.ldda + at, n, v);
          load_weight(a.p, a.p.w_pre, at, n, w);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            t[i] = t[i] + rs * (v[i] * w[i] - s[i] * k);
            v[i] = v[i] * (s[i] * rs);
          }
          if (round == 1 && a.dw_pre != nullptr) add_to(part_at(a, blockIdx.x, kSumPre), at, n, row == lo, v);
        }
        if (a.y != nullptr) {
          float y[8], gate[8];
          load_run<Y>(a.y, row * a.ldy + at, n, y);
          if (a.p.gate != nullptr) {
            load_run(a.p.elem, a.p.gate, gate_row * a.p.ldg + at, n, gate);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) gate[i] = 1.0f;
          }
          load_weight(a.p, a.p.post ? a.p.w_post : nullptr, at, n, w);
          if (round == 0) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = gate[i] * t[i] * w[i] * y[i];
            q[0] = q[0] + sum8(v);
          } else {
            float dy[8], dw[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float dn = gate[i] * t[i], yh = y[i] * ry;
              dy[i] = ry * (dn * w[i] - y[i] * ky);
              dw[i] = dn * yh;
              v[i] = t[i] * (yh * w[i]);
            }
            if (a.dy != nullptr) store_run<Y>(a.dy, row * a.lddy + at, n, dy);
            if (a.dw_post != nullptr) add_to(part_at(a, blockIdx.x, kSumPost), at, n, row == lo, dw);
            if (a.dgate != nullptr) {
              float* p = part_at(a, blockIdx.x, kSumGate);
              add_to(p, at, n, row == lo || (sp.chunks == 0 && row % a.p.rows_per_gate == 0), v);
              if (sp.chunks == 0 && (row + 1) % a.p.rows_per_gate == 0) {
                load_run<kElemF32>(p, at, n, v);
                store_run(a.p.elem, a.dgate, gate_row * a.lddg + at, n, v);
              }
            }
          }
        }
        if (round == 1 && a.dx != nullptr) {
#pragma unroll
          for (int i = 0; i < 8; ++i) t[i] = a.p.alpha * t[i];
          store_run<X>(a.dx, row * a.lddx + at, n, t);
        }
      }
      if (round == 0) {
        block_sums(q, &lds, &turn);
        ky = ry * ry * (q[0] / cols);
      }
    }
  }
}

// The workgroups' column sums added in order: 64 columns to a workgroup, whose four
// wavefronts take a quarter of the sums each.  blockIdx.y: w_pre, w_post, then the gates.
__global__ __launch_bounds__(256) void echo_block_norm_join_k(const BlockNormBwdArgs a, const BlockSplit sp, int64_t n_gates) {
  __shared__ float lds[4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 64 + lane;
  for (int64_t job = blockIdx.y; job < 2 + n_gates; job += gridDim.y) {
    const int sum = job < kSumGate ? static_cast<int>(job) : kSumGate;
    void* to = sum == kSumPre ? a.dw_pre : sum == kSumPost ? a.dw_post : a.dgate;
    if (to == nullptr) continue;
    const int64_t first = sum == kSumGate ? (job - kSumGate) * sp.chunks : 0;
    const int64_t count = sum == kSumGate ? sp.chunks : sp.groups;
    const int64_t lo = first + count * wave / 4, hi = first + count * (wave + 1) / 4;
    float v = 0.0f;
    if (col < a.p.C)
      for (int64_t g = lo; g < hi; ++g) v = v + part_at(a, g, sum)[col];
    __syncthreads();
    lds[wave][lane] = v;
    __syncthreads();
    if (wave == 0 && col < a.p.C) {
      v = (lds[0][lane] + lds[1][lane]) + (lds[2][lane] + lds[3][lane]);
      const int64_t at = (sum == kSumGate ? (job - kSumGate) * a.lddg : 0) + col;
      if (a.p.elem == kElemF32) store1<kElemF32>(to, at, v);
      else if (a.p.elem == kElemBf16) store1<kElemBf16>(to, at, v);
      else store1<kElemF16>(to, at, v);
    }
  }
}

}  // namespace

hipError_t launch_block_norm_bwd(const BlockNormBwdArgs& a, Elem x, Elem y, Elem out_a, hipStream_t s) {
  const BlockSplit sp = block_split(a.p.R, a.p.n_gates);
  const dim3 grid(static_cast<unsigned>(sp.groups));
  // without rows only the sums are written: zeros
  const hipError_t e = a.p.R == 0 ? hipSuccess : with_types(x, y, out_a, [&](auto X, auto Y, auto A) {
    if (a.p.C <= 8 * kMaxThreads)
      hipLaunchKernelGGL((echo_block_norm_bwd_k<X(), Y(), A()>), grid, dim3(row_threads(a.p.C, 1)), 0, s, a, sp);
    else
      hipLaunchKernelGGL((echo_block_norm_bwd_long_k<X(), Y(), A()>), grid, dim3(kMaxThreads), 0, s, a, sp);
    return hipGetLastError();
  });
  if (e != hipSuccess) return e;
  const int64_t gates = a.dgate != nullptr && (sp.chunks != 0 || a.p.R == 0) ? a.p.n_gates : 0;
  if (a.dw_pre == nullptr && a.dw_post == nullptr && gates == 0) return hipSuccess;
  hipLaunchKernelGGL(echo_block_norm_join_k, dim3(static_cast<unsigned>((a.p.C + 63) / 64), static_cast<unsigned>(2 + (gates < 1024 ? gates : 1024))),
                     dim3(256), 0, s, a, sp, gates);
  return hipGetLastError();
}

}  // namespace echo
