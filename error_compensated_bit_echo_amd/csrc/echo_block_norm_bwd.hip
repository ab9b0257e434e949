// Gradients of the block norm (see echo_block_norm.hip).  With s the stream as stored,
// rs = rs(s), u = da (offset + w_pre) and t the whole gradient of s,
//   t  = dout + rs u - s rs^3 mean(u s),           dx = alpha t
//   dn = gate t,  v = dn (offset + w_post),        dy = ry v - y ry^3 mean(v y)  (ry = rs(y); dn without a post-norm)
//   dw_pre = sum over rows of da s rs,  dw_post = sum of dn y ry,  dgate = sum over the gate's rows of t n.
// sum s^2, sum u s and sum y^2 need nothing but the inputs, so they are one reduction and
// no statistics of the forward pass are kept; sum v y needs t, which is the second.  A
// workgroup takes every n-th row of a gate's (all rows without one), or the rows of whole
// gates, and sums its columns in registers; the workgroups' sums go to the workspace and are
// added in order by a second kernel, so the result does not depend on timing.
//
// As many workgroups as the CUs hold, each with its next row's inputs in flight while it works
// on one; the parameters' factors wait in LDS, which leaves the registers (127 of 128) to the
// sums and the inputs. 16384 x 8192 bfloat16 takes 296 us (5.4 TB/s of what it has to move), the
// kernel 286 and the join 6; the vector units issue in 56 % of its cycles, so that every
// instruction a row counts: with the exact root and division it took 345, with a 64-bit
// division a row 309. 2048 x 4096 fp32: 57 us, 10 of them the column sums' way through memory.
#include <type_traits>

#include "echo_row.h"

namespace echo {

namespace {

enum Sum { kSumPre = 0, kSumPost = 1, kSumGate = 2, kSums = 3 };

__device__ __forceinline__ float* part_at(const BlockNormBwdArgs& a, int64_t group, int sum) {
  return a.part + (group * kSums + sum) * a.p.C;
}

// The rows of workgroup blockIdx.x, and the gate of the first.  Row numbers fit 32 bits, whose
// divisions are a quarter of those in 64.
struct Rows {
  int64_t lo, hi, step, gate;
};
__device__ __forceinline__ Rows rows_of(const BlockNormBwdArgs& a, const BlockSplit& sp) {
  if (sp.chunks != 0) {
    const uint32_t chunks = static_cast<uint32_t>(sp.chunks), g = blockIdx.x / chunks;
    return Rows{g * a.p.rows_per_gate + (blockIdx.x - g * chunks), (g + 1) * a.p.rows_per_gate, sp.chunks, g};
  }
  const int64_t lo = blockIdx.x * sp.rows, hi = lo + sp.rows;
  return Rows{lo, hi < a.p.R ? hi : a.p.R, 1, blockIdx.x * sp.gates};
}

// A row's inputs as they are loaded.
template <int X, int Y, int A>
struct RawRow {
  Raw<X> s, dout;
  Raw<A> da;
  Raw<Y> y;
  __device__ __forceinline__ void load(const BlockNormBwdArgs& a, int64_t row, uint32_t at) {
    load_raw<X>(a.out, row * a.ldo, at, &s);
    if (a.da != nullptr) load_raw<A>(a.da, row * a.ldda, at, &da);
    if (a.y != nullptr) load_raw<Y>(a.y, row * a.ldy, at, &y);
    if (a.dout != nullptr) load_raw<X>(a.dout, row * a.lddo, at, &dout);
  }
  __device__ __forceinline__ void load_any(const BlockNormBwdArgs& a, int64_t row, Run run) {
    echo::load_any<X>(a.out, row * a.ldo, run, &s);
    if (a.da != nullptr) echo::load_any<A>(a.da, row * a.ldda, run, &da);
    if (a.y != nullptr) echo::load_any<Y>(a.y, row * a.ldy, run, &y);
    if (a.dout != nullptr) echo::load_any<X>(a.dout, row * a.lddo, run, &dout);
  }
};

// A thread's 8 factors of a weight or gate in LDS, which only it reads: 32 bytes a thread.
struct Factors {
  float4* v;
  __device__ __forceinline__ void put(const float w[8]) const {
    v[threadIdx.x] = make_float4(w[0], w[1], w[2], w[3]);
    v[blockDim.x + threadIdx.x] = make_float4(w[4], w[5], w[6], w[7]);
  }
  __device__ __forceinline__ void get(float w[8]) const {
    const float4 a = v[threadIdx.x], b = v[blockDim.x + threadIdx.x];
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
    w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
  }
};

__device__ __forceinline__ void factor_of(int e, bool given, float offset, const RawParam& r, int lo, float w[8]) {
  if (given) {
    widen(e, r, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = w[i] + offset;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 1.0f;
  }
  clear_below(lo, w);
}

template <int X, int Y, int A, bool STREAM>
__global__ __launch_bounds__(kMaxThreads) void echo_block_norm_bwd_k(const BlockNormBwdArgs a, const BlockSplit sp) {
  __shared__ Slots<3> lds;
  extern __shared__ float4 factors[];
  const Factors pre{factors}, post{factors + 2 * blockDim.x}, gates{factors + 4 * blockDim.x};
  int turn = 0;
  const int64_t C = a.p.C;
  const Run run = run_of(0, C);
  const uint32_t at = run.at;
  const int e = a.p.elem;
  const Rows rows = rows_of(a, sp);
  RawRow<X, Y, A> next;
  next.load(a, rows.lo, at);
  float acc[kSums][8];
  {
    RawParam r[3];
    float w[8];
    if (a.p.w_pre != nullptr) load_raw(e, a.p.w_pre, 0, at, &r[0]);
    if (a.p.w_post != nullptr) load_raw(e, a.p.w_post, 0, at, &r[1]);
    if (a.p.gate != nullptr) load_raw(e, a.p.gate, rows.gate * a.p.ldg, at, &r[2]);
    factor_of(e, a.p.w_pre != nullptr, a.p.offset, r[0], run.lo, w);
    pre.put(w);
    factor_of(e, a.p.w_post != nullptr, a.p.offset, r[1], run.lo, w);
    post.put(w);
    factor_of(e, a.p.gate != nullptr, 0.0f, r[2], run.lo, w);
    gates.put(w);
  }
  int64_t gate_row = rows.gate, gate_left = a.p.rows_per_gate;  // of whole gates
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[kSumPre][i] = acc[kSumPost][i] = acc[kSumGate][i] = 0.0f;
  for (int64_t row = rows.lo; row < rows.hi; row += rows.step) {
    const RawRow<X, Y, A> raw = next;
    if (row + rows.step < rows.hi) next.load(a, row + rows.step, at);  // in flight while this row is worked on
    float s[8], t[8], y[8], w[8];
    widen<X>(raw.s, s);
    clear_below(run.lo, s);
    float m[3] = {0.0f, 0.0f, 0.0f};
    m[0] = dot8(s, s, 0.0f);
    if (a.da != nullptr) {
      float da[8];
      widen<A>(raw.da, da);
      clear_below(run.lo, da);
      pre.get(w);
#pragma unroll
      for (int i = 0; i < 8; ++i) m[1] = __builtin_fmaf(da[i] * w[i], s[i], m[1]);
    }
    if (a.y != nullptr) {
      widen<Y>(raw.y, y);
      clear_below(run.lo, y);
      m[2] = dot8(y, y, 0.0f);
    }
    block_sums(m, &lds, &turn);
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = 0.0f;
    if (a.dout != nullptr) {
      widen<X>(raw.dout, t);
      clear_below(run.lo, t);
    }
    if (a.da != nullptr) {
      float da[8];
      widen<A>(raw.da, da);
      clear_below(run.lo, da);
      pre.get(w);
      const float rs = reciprocal_rms(m[0], a.p), k = rs * rs * (m[1] * a.p.inv_cols);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        t[i] = __builtin_fmaf(rs, __builtin_fmaf(da[i], w[i], -(s[i] * k)), t[i]);
        acc[kSumPre][i] = __builtin_fmaf(da[i], s[i] * rs, acc[kSumPre][i]);
      }
    }
    if (a.dx != nullptr) {
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] = a.p.alpha * t[i];
      store_from<X, STREAM>(a.dx, row * a.lddx, run, s);
    }
    if (a.y == nullptr) continue;
    float gate[8];
    gates.get(gate);
    if (a.p.post) {
      const float ry = reciprocal_rms(m[2], a.p);
      float q[1] = {0.0f};
      post.get(w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float yh = y[i] * ry, dn = gate[i] * t[i];
        acc[kSumGate][i] = __builtin_fmaf(t[i], yh * w[i], acc[kSumGate][i]);
        acc[kSumPost][i] = __builtin_fmaf(dn, yh, acc[kSumPost][i]);
        t[i] = dn * w[i];
        q[0] = __builtin_fmaf(t[i], y[i], q[0]);
      }
      block_sums(q, &lds, &turn);
      const float k = ry * ry * (q[0] * a.p.inv_cols);
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] = ry * __builtin_fmaf(-y[i], k, t[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        acc[kSumGate][i] = __builtin_fmaf(t[i], y[i], acc[kSumGate][i]);
        t[i] = gate[i] * t[i];
      }
    }
    if (a.dy != nullptr) store_from<Y, STREAM>(a.dy, row * a.lddy, run, t);
    if (sp.chunks == 0 && --gate_left == 0) {
      // the last row of a gate that is this workgroup's alone
      if (a.dgate != nullptr) store_from(e, a.dgate, gate_row * a.lddg, run, acc[kSumGate]);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[kSumGate][i] = 0.0f;
      ++gate_row;
      gate_left = a.p.rows_per_gate;
      if (a.p.gate != nullptr && row + 1 < rows.hi) {
        RawParam r;
        load_raw(e, a.p.gate, gate_row * a.p.ldg, at, &r);
        factor_of(e, true, 0.0f, r, run.lo, gate);
        gates.put(gate);
      }
    }
  }
  if (a.dw_pre != nullptr) store_from<kElemF32>(part_at(a, blockIdx.x, kSumPre), 0, run, acc[kSumPre]);
  if (a.dw_post != nullptr) store_from<kElemF32>(part_at(a, blockIdx.x, kSumPost), 0, run, acc[kSumPost]);
  if (a.dgate != nullptr && sp.chunks != 0)
    store_from<kElemF32>(part_at(a, blockIdx.x, kSumGate), 0, run, acc[kSumGate]);
}

// ---- rows that do not fit: statistics, then a pass by columns -------------------------------
//
// 8192 x 12288 bfloat16: 447 us, of which the statistics 214 (3.8 TB/s, a workgroup to a CU)
// and the columns 223 (5.4 TB/s). One pass with two runs to a thread needs more registers than
// there are: 920 us, spilled; three passes over each row from the caches took 860.

// rs(out), its square times mean(u out), rs(y), its square times mean(v y)
__device__ __forceinline__ float4 stats_of(const BlockNormBwdArgs& a, const float m[3]) {
  const float rs = reciprocal_rms(m[0], a.p), ry = a.p.post ? reciprocal_rms(m[2], a.p) : 1.0f;
  return make_float4(rs, rs * rs * (m[1] * a.p.inv_cols), ry, 0.0f);
}

// A thread's share of the three sums, from its 8 columns.
template <int X, int Y, int A>
__device__ __forceinline__ void add_squares(const BlockNormBwdArgs& a, const RawRow<X, Y, A>& raw, const RawParam& pre, int lo,
                                            float m[3]) {
  float s[8], v[8], w[8];
  widen<X>(raw.s, s);
  clear_below(lo, s);
  if (a.da != nullptr) {
    widen<A>(raw.da, v);
    clear_below(lo, v);
    factor_of(a.p.elem, a.p.w_pre != nullptr, a.p.offset, pre, lo, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = v[i] * w[i] * s[i];
    m[1] = m[1] + sum8(v);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) s[i] = s[i] * s[i];
  m[0] = m[0] + sum8(s);
  if (a.y != nullptr) {
    widen<Y>(raw.y, v);
    clear_below(lo, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = v[i] * v[i];
    m[2] = m[2] + sum8(v);
  }
}

// The whole gradient of the stream's 8 columns.
template <int X, int Y, int A>
__device__ __forceinline__ void stream_gradient(const BlockNormBwdArgs& a, const RawRow<X, Y, A>& raw, const float pre[8], int lo,
                                                float4 st, float t[8], float dw[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) t[i] = dw[i] = 0.0f;
  if (a.dout != nullptr) {
    widen<X>(raw.dout, t);
    clear_below(lo, t);
  }
  if (a.da != nullptr) {
    float s[8], da[8];
    widen<X>(raw.s, s);
    clear_below(lo, s);
    widen<A>(raw.da, da);
    clear_below(lo, da);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      t[i] = __builtin_fmaf(st.x, __builtin_fmaf(da[i], pre[i], -(s[i] * st.y)), t[i]);
      dw[i] = da[i] * (s[i] * st.x);
    }
  }
}

// sum v y over 8 columns.
template <int X, int Y, int A>
__device__ __forceinline__ float post_product(const BlockNormBwdArgs& a, const RawRow<X, Y, A>& raw, const RawParam (&r)[3], int lo,
                                              float4 st) {
  const int e = a.p.elem;
  float t[8], y[8], w[8], unused[8];
  factor_of(e, a.p.w_pre != nullptr, a.p.offset, r[0], lo, w);
  stream_gradient<X, Y, A>(a, raw, w, lo, st, t, unused);
  widen<Y>(raw.y, y);
  clear_below(lo, y);
  factor_of(e, a.p.w_post != nullptr, a.p.offset, r[1], lo, w);
#pragma unroll
  for (int i = 0; i < 8; ++i) t[i] = t[i] * w[i] * y[i];
  if (a.p.gate != nullptr) {
    factor_of(e, true, 0.0f, r[2], lo, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = t[i] * w[i];
  }
  return sum8(t);
}

__device__ __forceinline__ void load_params(const BlockNormBwdArgs& a, int64_t gate_row, uint32_t at, RawParam (&r)[3]) {
  if (a.p.w_pre != nullptr) load_raw(a.p.elem, a.p.w_pre, 0, at, &r[0]);
  if (a.p.w_post != nullptr) load_raw(a.p.elem, a.p.w_post, 0, at, &r[1]);
  if (a.p.gate != nullptr) load_raw(a.p.elem, a.p.gate, gate_row * a.p.ldg, at, &r[2]);
}

__device__ __forceinline__ void load_any_params(const BlockNormBwdArgs& a, int64_t gate_row, Run run, RawParam (&r)[3]) {
  if (a.p.w_pre != nullptr) load_any(a.p.elem, a.p.w_pre, 0, run, &r[0]);
  if (a.p.w_post != nullptr) load_any(a.p.elem, a.p.w_post, 0, run, &r[1]);
  if (a.p.gate != nullptr) load_any(a.p.elem, a.p.gate, gate_row * a.p.ldg, run, &r[2]);
}

// Rows of up to 16 * kMaxThreads columns in the registers.
template <int X, int Y, int A>
__global__ __launch_bounds__(kMaxThreads) void echo_block_norm_stats_k(const BlockNormBwdArgs a, int64_t row0) {
  constexpr int kRuns = 2;
  __shared__ Slots<3> lds;
  int turn = 0;
  const int64_t C = a.p.C, row = row0 + blockIdx.x;
  RawRow<X, Y, A> raw[kRuns];
  RawParam r[kRuns][3];
#pragma unroll
  for (int k = 0; k < kRuns; ++k) {
    const Run run = run_of(k, C);
    raw[k].load(a, row, run.at);
    if (a.p.w_pre != nullptr) load_raw(a.p.elem, a.p.w_pre, 0, run.at, &r[k][0]);
  }
  float m[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int k = 0; k < kRuns; ++k) add_squares<X, Y, A>(a, raw[k], r[k][0], run_of(k, C).lo, m);
  block_sums(m, &lds, &turn);
  float4 st = stats_of(a, m);
  if (a.y != nullptr && a.p.post) {
    float q[1] = {0.0f};
#pragma unroll
    for (int k = 0; k < kRuns; ++k) {
      const Run run = run_of(k, C);
      load_params(a, gate_of(a.p, row), run.at, r[k]);
      q[0] = q[0] + post_product<X, Y, A>(a, raw[k], r[k], run.lo, st);
    }
    block_sums(q, &lds, &turn);
    st.w = st.z * st.z * (q[0] * a.p.inv_cols);
  }
  if (threadIdx.x == 0) a.stats[row] = st;
}

// Rows of any length: the inputs are read again for the second statistic.
template <int X, int Y, int A>
__global__ __launch_bounds__(kMaxThreads) void echo_block_norm_stats_long_k(const BlockNormBwdArgs a) {
  __shared__ Slots<3> lds;
  int turn = 0;
  const int64_t C = a.p.C;
  const int runs = static_cast<int>((C + 8 * kMaxThreads - 1) / (8 * kMaxThreads));
  for (int64_t row = blockIdx.x; row < a.p.R; row += gridDim.x) {
    float m[3] = {0.0f, 0.0f, 0.0f};
    RawRow<X, Y, A> raw;
    RawParam r[3];
    for (int k = 0; k < runs; ++k) {
      const Run run = any_run_of(k, C);
      raw.load_any(a, row, run);
      if (a.p.w_pre != nullptr) load_any(a.p.elem, a.p.w_pre, 0, run, &r[0]);
      add_squares<X, Y, A>(a, raw, r[0], run.lo, m);
    }
    block_sums(m, &lds, &turn);
    float4 st = stats_of(a, m);
    if (a.y != nullptr && a.p.post) {
      float q[1] = {0.0f};
      for (int k = 0; k < runs; ++k) {
        const Run run = any_run_of(k, C);
        raw.load_any(a, row, run);
        load_any_params(a, gate_of(a.p, row), run, r);
        q[0] = q[0] + post_product<X, Y, A>(a, raw, r, run.lo, st);
      }
      block_sums(q, &lds, &turn);
      st.w = st.z * st.z * (q[0] * a.p.inv_cols);
    }
    if (threadIdx.x == 0) a.stats[row] = st;
  }
}

// The gradients of kColumnTile columns of a workgroup's rows, whose statistics are known: no
// sums over a row are left, so rows pass without a barrier.
template <int X, int Y, int A, bool STREAM>
__global__ __launch_bounds__(kColumnTile / 8) void echo_block_norm_cols_k(const BlockNormBwdArgs a, const BlockSplit sp) {
  const int64_t C = a.p.C;
  const Run run = any_run_of(blockIdx.y, C);
  const int e = a.p.elem;
  const Rows rows = rows_of(a, sp);
  RawRow<X, Y, A> next;
  next.load_any(a, rows.lo, run);
  float4 next_st = a.stats[rows.lo];
  RawParam r[3];
  load_any_params(a, rows.gate, run, r);
  int64_t gate_row = rows.gate, gate_left = a.p.rows_per_gate;  // of whole gates
  float pre[8], post[8], gate[8], acc[kSums][8];
  factor_of(e, a.p.w_pre != nullptr, a.p.offset, r[0], run.lo, pre);
  factor_of(e, a.p.w_post != nullptr, a.p.offset, r[1], run.lo, post);
  factor_of(e, a.p.gate != nullptr, 0.0f, r[2], run.lo, gate);
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[kSumPre][i] = acc[kSumPost][i] = acc[kSumGate][i] = 0.0f;
  for (int64_t row = rows.lo; row < rows.hi; row += rows.step) {
    const RawRow<X, Y, A> raw = next;
    const float4 st = next_st;
    if (row + rows.step < rows.hi) {
      next.load_any(a, row + rows.step, run);
      next_st = a.stats[row + rows.step];
    }
    float t[8], w[8];
    stream_gradient<X, Y, A>(a, raw, pre, run.lo, st, t, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[kSumPre][i] = acc[kSumPre][i] + w[i];
    if (a.dx != nullptr) {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = a.p.alpha * t[i];
      store_from<X, STREAM>(a.dx, row * a.lddx, run, w);
    }
    if (a.y == nullptr) continue;
    float y[8];
    widen<Y>(raw.y, y);
    clear_below(run.lo, y);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float yh = y[i] * st.z, dn = gate[i] * t[i];
      acc[kSumGate][i] = __builtin_fmaf(t[i], yh * post[i], acc[kSumGate][i]);
      acc[kSumPost][i] = __builtin_fmaf(dn, yh, acc[kSumPost][i]);
      // an infinite y times the 0 that stands for no post-norm would be no number
      w[i] = a.p.post ? st.z * __builtin_fmaf(dn, post[i], -(y[i] * st.w)) : dn;
    }
    if (a.dy != nullptr) store_from<Y, STREAM>(a.dy, row * a.lddy, run, w);
    if (sp.chunks == 0 && --gate_left == 0) {
      // the last row of a gate that is this workgroup's alone
      if (a.dgate != nullptr) store_from(e, a.dgate, gate_row * a.lddg, run, acc[kSumGate]);
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[kSumGate][i] = 0.0f;
      ++gate_row;
      gate_left = a.p.rows_per_gate;
      if (a.p.gate != nullptr && row + 1 < rows.hi) {
        load_any(e, a.p.gate, gate_row * a.p.ldg, run, &r[2]);
        factor_of(e, true, 0.0f, r[2], run.lo, gate);
      }
    }
  }
  if (a.dw_pre != nullptr) store_from<kElemF32>(part_at(a, blockIdx.x, kSumPre), 0, run, acc[kSumPre]);
  if (a.dw_post != nullptr) store_from<kElemF32>(part_at(a, blockIdx.x, kSumPost), 0, run, acc[kSumPost]);
  if (a.dgate != nullptr && sp.chunks != 0)
    store_from<kElemF32>(part_at(a, blockIdx.x, kSumGate), 0, run, acc[kSumGate]);
}

// The workgroups' column sums added in an order of their own: 64 columns to a workgroup,
// whose 16 wavefronts take every 16th sum each, four loads at a time.  blockIdx.y: w_pre,
// w_post, then the gates.
__global__ __launch_bounds__(kMaxThreads) void echo_block_norm_join_k(const BlockNormBwdArgs a, const BlockSplit sp,
                                                                      int64_t n_gates) {
  __shared__ float lds[kMaxWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t col = static_cast<int64_t>(blockIdx.x) * 64 + lane;
  for (int64_t job = blockIdx.y; job < 2 + n_gates; job += gridDim.y) {
    const int sum = job < kSumGate ? static_cast<int>(job) : kSumGate;
    void* to = sum == kSumPre ? a.dw_pre : sum == kSumPost ? a.dw_post : a.dgate;
    if (to == nullptr) continue;
    const int64_t first = sum == kSumGate ? (job - kSumGate) * sp.chunks : 0;
    const int count = static_cast<int>(sum == kSumGate ? sp.chunks : sp.groups);
    const int64_t step = kMaxWaves * kSums * a.p.C;
    float v = 0.0f;
    if (col < a.p.C) {
      const float* p = part_at(a, first + wave, sum) + col;
      int g = wave;
      for (; g + 3 * kMaxWaves < count; g += 4 * kMaxWaves, p += 4 * step) {
        const float v0 = p[0], v1 = p[step], v2 = p[2 * step], v3 = p[3 * step];
        v = v + ((v0 + v1) + (v2 + v3));
      }
      for (; g < count; g += kMaxWaves, p += step) v = v + p[0];
    }
    __syncthreads();
    lds[wave][lane] = v;
    __syncthreads();
    if (wave == 0 && col < a.p.C) {
      v = 0.0f;
#pragma unroll
      for (int i = 0; i < kMaxWaves; ++i) v = v + lds[i][lane];
      const int64_t at = (sum == kSumGate ? (job - kSumGate) * a.lddg : 0) + col;
      if (a.p.elem == kElemF32) store1<kElemF32>(to, at, v);
      else if (a.p.elem == kElemBf16) store1<kElemBf16>(to, at, v);
      else store1<kElemF16>(to, at, v);
    }
  }
}

}  // namespace

hipError_t launch_block_norm_bwd(const BlockNormBwdArgs& a, Elem x, Elem y, Elem out_a, hipStream_t s) {
  const BlockSplit sp = block_split(a.p.R, a.p.n_gates, a.p.C);
  const unsigned groups = static_cast<unsigned>(sp.groups);
  // without rows only the sums are written: zeros
  const hipError_t e = a.p.R == 0 ? hipSuccess : with_types(x, y, out_a, [&](auto X, auto Y, auto A) -> hipError_t {
    constexpr bool kAny = X() != kElemF32 || Y() != kElemF32;  // 16-bit results
    const int64_t bytes = 3 * elem_size(X()) + elem_size(A()) + (a.y != nullptr ? 2 * elem_size(Y()) : 0);
    const bool stream = kAny && block_streams(a.p.R, a.p.C, bytes);
    if (block_fits(a.p.C)) {
      const int threads = row_threads(a.p.C, 1);
      const auto launch = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(groups), dim3(threads), threads * 6 * sizeof(float4), s, a, sp);
        return hipGetLastError();
      };
      return stream ? launch(echo_block_norm_bwd_k<X(), Y(), A(), kAny>) : launch(echo_block_norm_bwd_k<X(), Y(), A(), false>);
    }
    if (a.p.C > 8 * kMaxThreads && a.p.C <= 16 * kMaxThreads) {
      const int threads = row_threads(a.p.C, 2);
      const int64_t most = ((int64_t{1} << 32) - 1) / threads;  // a launch numbers its threads in 32 bits
      for (int64_t row = 0; row < a.p.R; row += most) {
        const int64_t rows = a.p.R - row < most ? a.p.R - row : most;
        hipLaunchKernelGGL((echo_block_norm_stats_k<X(), Y(), A()>), dim3(static_cast<unsigned>(rows)), dim3(threads), 0, s, a,
                           row);
        const hipError_t r = hipGetLastError();
        if (r != hipSuccess) return r;
      }
    } else {
      const unsigned rows = static_cast<unsigned>(a.p.R < (1 << 20) ? a.p.R : (1 << 20));
      hipLaunchKernelGGL((echo_block_norm_stats_long_k<X(), Y(), A()>), dim3(rows), dim3(kMaxThreads), 0, s, a);
      const hipError_t r = hipGetLastError();
      if (r != hipSuccess) return r;
    }
    const unsigned tiles = static_cast<unsigned>((a.p.C + kColumnTile - 1) / kColumnTile);
    const auto launch = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, dim3(groups, tiles), dim3(kColumnTile / 8), 0, s, a, sp);
      return hipGetLastError();
    };
    return stream ? launch(echo_block_norm_cols_k<X(), Y(), A(), kAny>) : launch(echo_block_norm_cols_k<X(), Y(), A(), false>);
  });
  if (e != hipSuccess) return e;
  const int64_t gates = a.dgate != nullptr && (sp.chunks != 0 || a.p.R == 0) ? a.p.n_gates : 0;
  if (a.dw_pre == nullptr && a.dw_post == nullptr && gates == 0) return hipSuccess;
  hipLaunchKernelGGL(echo_block_norm_join_k, dim3(static_cast<unsigned>((a.p.C + 63) / 64), static_cast<unsigned>(2 + (gates < 1024 ? gates : 1024))),
                     dim3(kMaxThreads), 0, s, a, sp, gates);
  return hipGetLastError();
}

}  // namespace echo
