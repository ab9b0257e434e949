// What the row-wise kernels of the training step share: sums over a wavefront and a
// workgroup, rows cut into chunks of 8 columns, element types known at run time.
#pragma once

#pragma clang fp contract(off)

#include "echo_elem.h"
#include "echo_step_internal.h"

namespace echo {
namespace {

constexpr int kMaxWaves = kMaxThreads / 64;

// Another lane's value; 0 in the rows that ROWS leaves out.
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, ROWS, 0xF, ROWS == 0xF));
}

// The sum over the wavefront's 64 lanes, in lane 63: four exchanges within rows of 16 lanes,
// then row to row.  All lanes are active.
__device__ __forceinline__ float wave_sum(float v) {
  v = v + dpp<0xB1>(v);   // quad_perm [1, 0, 3, 2]
  v = v + dpp<0x4E>(v);   // quad_perm [2, 3, 0, 1]
  v = v + dpp<0x141>(v);  // row_half_mirror
  v = v + dpp<0x140>(v);  // row_mirror
  v = v + dpp<0x142, 0xA>(v);  // row_bcast:15 into rows 1 and 3
  return v + dpp<0x143, 0xC>(v);  // row_bcast:31 into rows 2 and 3
}

// Sums of N values over the workgroup, in every thread.  Consecutive calls alternate
// between two slots: a slot is written again only behind the barrier of the call between,
// which every thread reaches after it has read it.
template <int N>
struct Slots {
  float v[2][N][kMaxWaves];
};

template <int N, int M>
__device__ __forceinline__ void block_sums(float (&v)[N], Slots<M>* lds, int* turn) {
  static_assert(N <= M, "slots");
  const int waves = static_cast<int>(blockDim.x) >> 6;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  if (waves == 1) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v[i]), 63));
    return;
  }
  const int slot = *turn;
  *turn ^= 1;
  const int wave = static_cast<int>(threadIdx.x) >> 6, lane = static_cast<int>(threadIdx.x) & 63;
  if (lane == 63) {
#pragma unroll
    for (int i = 0; i < N; ++i) lds->v[slot][i][wave] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    // up to 16 wavefronts: a row of 16 lanes holds their sums, every row the same
    float w = (lane & 15) < waves ? lds->v[slot][i][lane & 15] : 0.0f;
    w = w + dpp<0xB1>(w);
    w = w + dpp<0x4E>(w);
    w = w + dpp<0x141>(w);
    v[i] = w + dpp<0x140>(w);
  }
}

// The sum over the workgroup and a thread's RUNS runs, in the order in which a workgroup of
// RUNS times as many threads with a run each adds them up: a row's sum does not depend on
// which of the two works on it.  More than one wavefront, 16 of runs at most.
template <int RUNS>
__device__ __forceinline__ float block_sum_of_runs(float (&v)[RUNS], Slots<1>* lds, int* turn) {
  const int waves = static_cast<int>(blockDim.x) >> 6, slot = *turn;
  *turn ^= 1;
  const int wave = static_cast<int>(threadIdx.x) >> 6, lane = static_cast<int>(threadIdx.x) & 63;
#pragma unroll
  for (int k = 0; k < RUNS; ++k) {
    v[k] = wave_sum(v[k]);
    if (lane == 63) lds->v[slot][0][k * waves + wave] = v[k];
  }
  __syncthreads();
  float w = (lane & 15) < RUNS * waves ? lds->v[slot][0][lane & 15] : 0.0f;
  w = w + dpp<0xB1>(w);
  w = w + dpp<0x4E>(w);
  w = w + dpp<0x141>(w);
  return w + dpp<0x140>(w);
}

// A run of up to 8 columns: n of them lie in the row.
template <int E>
__device__ __forceinline__ void load_run(const void* base, int64_t at, int n, float v[8]) {
  if (n >= 8) {
    load8<E>(base, at, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? load1<E>(base, at + i) : 0.0f;
  }
}

template <int E>
__device__ __forceinline__ void store_run(void* base, int64_t at, int n, const float v[8]) {
  if (n >= 8) {
    store8<E>(base, at, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) store1<E>(base, at + i, v[i]);
  }
}

// The same where the type is an argument of the launch.
__device__ __forceinline__ void load_run(int elem, const void* base, int64_t at, int n, float v[8]) {
  if (elem == kElemF32) load_run<kElemF32>(base, at, n, v);
  else if (elem == kElemBf16) load_run<kElemBf16>(base, at, n, v);
  else load_run<kElemF16>(base, at, n, v);
}

// v as it reads back from an element of the type.
template <int E>
__device__ __forceinline__ float stored(float v) {
  return static_cast<float>(narrow<E>(v));
}

// s plus the products of 8 pairs.
__device__ __forceinline__ float dot8(const float a[8], const float b[8], float s) {
#pragma unroll
  for (int i = 0; i < 8; ++i) s = __builtin_fmaf(a[i], b[i], s);
  return s;
}

__device__ __forceinline__ float sum8(const float v[8]) {
  return ((v[0] + v[1]) + (v[2] + v[3])) + ((v[4] + v[5]) + (v[6] + v[7]));
}

// The columns of a row that a thread's run i of `runs` holds: consecutive threads take
// consecutive runs of 8.
__device__ __forceinline__ int64_t run_at(int64_t i) {
  return (i * blockDim.x + threadIdx.x) * 8;
}
__device__ __forceinline__ int run_length(int64_t at, int64_t C) {
  const int64_t n = C - at;
  return n >= 8 ? 8 : n > 0 ? static_cast<int>(n) : 0;
}

// A run of 8 columns as the register kernels take it.  All of a kernel's loads are issued
// before the first is used, so they may not hang on branches: a run that would reach past
// the row starts at the row's last 8 columns instead, and its elements below `lo` are other
// threads' (all 8 where the whole run lies behind the row).  Rows have 8 columns at least.
struct Run {
  uint32_t at;  // 32 bits beside a row's uniform start: one register, not two, for an address
  int lo;
};

__device__ __forceinline__ Run run_of(int k, int64_t C) {
  const uint32_t at = (k * blockDim.x + threadIdx.x) * 8, last = static_cast<uint32_t>(C) - 8;
  return at <= last ? Run{at, 0} : Run{last, at - last < 8 ? static_cast<int>(at - last) : 8};
}

// Elements as they are loaded.
template <int E>
struct Raw {
  typename ElemOf<E>::T v __attribute__((ext_vector_type(8)));
};

template <int E>
__device__ __forceinline__ void load_raw(const void* base, int64_t row, uint32_t at, Raw<E>* r) {
  const typename ElemOf<E>::T* p = static_cast<const typename ElemOf<E>::T*>(base) + row;
  __builtin_memcpy(&r->v, p + at, sizeof(r->v));
}

template <int E>
__device__ __forceinline__ void widen(const Raw<E>& r, float v[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = static_cast<float>(r.v[i]);
}

// Parameters, whose type is an argument of the launch.
struct RawParam {
  uint32_t w[8];
};

__device__ __forceinline__ void load_raw(int elem, const void* base, int64_t row, uint32_t at, RawParam* r) {
  if (elem == kElemF32) {
    const float* p = static_cast<const float*>(base) + row;
    __builtin_memcpy(r->w, p + at, 32);
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(base) + row;
    __builtin_memcpy(r->w, p + at, 16);
  }
}

__device__ __forceinline__ void widen(int elem, const RawParam& r, float v[8]) {
  if (elem == kElemF32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r.w[i]);
  } else if (elem == kElemBf16) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(i & 1 ? r.w[i >> 1] & 0xFFFF0000u : r.w[i >> 1] << 16);
  } else {
    Raw<kElemF16> h;
    __builtin_memcpy(&h.v, r.w, 16);
    widen<kElemF16>(h, v);
  }
}

// The same for rows of fewer than 8 columns too: the first run starts before the row then
// (`at` wraps), and its elements from `lo` on are the row's.
__device__ __forceinline__ Run any_run_of(int k, int64_t C) {
  if (C >= 8) return run_of(k, C);
  const uint32_t at = static_cast<uint32_t>(C) - 8;
  return Run{at, k == 0 && threadIdx.x == 0 ? 8 - static_cast<int>(C) : 8};
}

template <int E>
__device__ __forceinline__ void load_any(const void* base, int64_t row, Run run, Raw<E>* r) {
  if (static_cast<int>(run.at) >= 0) {
    load_raw<E>(base, row, run.at, r);
  } else {
    const typename ElemOf<E>::T* p = static_cast<const typename ElemOf<E>::T*>(base) + row;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int j = static_cast<int>(run.at) + i;
      r->v[i] = p[j > 0 ? j : 0];
    }
  }
}

__device__ __forceinline__ void load_any(int elem, const void* base, int64_t row, Run run, RawParam* r) {
  if (elem == kElemF32) {
    Raw<kElemF32> f;
    load_any<kElemF32>(base, row, run, &f);
    __builtin_memcpy(r->w, &f.v, 32);
  } else {  // either 16-bit type: its bits
    Raw<kElemF16> h;
    load_any<kElemF16>(base, row, run, &h);
    __builtin_memcpy(r->w, &h.v, 16);
  }
}

// Zeros in place of the elements that are other threads'.  The branch is the wavefront's, on
// a scalar: most hold whole runs alone.
__device__ __forceinline__ void clear_below(int lo, float v[8]) {
  if (__ballot(lo > 0) != 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < lo ? 0.0f : v[i];
  }
}

// STREAM: 16-bit elements go past the caches (fp32 ones do not: a run of them is two stores,
// which only a cache makes one line of).
template <int E, bool STREAM = false>
__device__ __forceinline__ void store_from(void* base, int64_t row, Run run, const float v[8]) {
  typedef typename ElemOf<E>::T T;
  T* p = static_cast<T*>(base) + row;
  if (run.lo == 0) {
    if constexpr (STREAM && E != kElemF32) {
      typedef uint32_t u4 __attribute__((ext_vector_type(4), aligned(2)));
      Raw<E> x;
#pragma unroll
      for (int i = 0; i < 8; ++i) x.v[i] = narrow<E>(v[i]);
      u4 w;
      __builtin_memcpy(&w, &x.v, 16);
      __builtin_nontemporal_store(w, reinterpret_cast<u4*>(p + run.at));
    } else {
      store8<E>(p, run.at, v);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i >= run.lo) store1<E>(p, run.at + i, v[i]);
  }
}

__device__ __forceinline__ void store_from(int elem, void* base, int64_t row, Run run, const float v[8]) {
  if (elem == kElemF32) store_from<kElemF32>(base, row, run, v);
  else if (elem == kElemBf16) store_from<kElemBf16>(base, row, run, v);
  else store_from<kElemF16>(base, row, run, v);
}

// The factor of a norm's weight: offset + w, 1 without a weight.
__device__ __forceinline__ void load_weight(const BlockParams& p, const void* w, int64_t at, int n, float v[8]) {
  if (w == nullptr) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 1.0f;
    return;
  }
  load_run(p.elem, w, at, n, v);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = v[i] + p.offset;
}

// The row of the gate for a row of the stream; both fit 32 bits, whose division is a quarter
// of that in 64.
__device__ __forceinline__ int64_t gate_of(const BlockParams& p, int64_t row) {
  return static_cast<uint32_t>(row) / static_cast<uint32_t>(p.rows_per_gate);
}

// 1 / sqrt(mean of the squares + eps), by the reciprocal root's instruction (1 ulp; what is
// under the root is at least 2^-126): the exact division and root are 60 instructions, as
// many as a row's 8 columns take.
__device__ __forceinline__ float reciprocal_rms(float squares, const BlockParams& p) {
#if defined(__HIP_DEVICE_COMPILE__)
  return __builtin_amdgcn_rsqf(__builtin_fmaf(squares, p.inv_cols, p.eps));
#else
  return 0.0f;
#endif
}

}  // namespace

// Calls f with the three types as constants; bfloat16 and fp16 do not come together.
template <typename F>
hipError_t with_types(Elem x, Elem y, Elem a, F f) {
#define ECHO_TYPES(X, Y, A)                                            \
  if (x == X && y == Y && a == A)                                      \
    return f(std::integral_constant<int, X>{}, std::integral_constant<int, Y>{}, std::integral_constant<int, A>{});
#define ECHO_TYPES_WITH(H)                                                                              \
  ECHO_TYPES(H, H, H) ECHO_TYPES(H, H, kElemF32) ECHO_TYPES(H, kElemF32, H) ECHO_TYPES(H, kElemF32, kElemF32) \
  ECHO_TYPES(kElemF32, H, H) ECHO_TYPES(kElemF32, H, kElemF32) ECHO_TYPES(kElemF32, kElemF32, H)
  ECHO_TYPES_WITH(kElemBf16)
  ECHO_TYPES_WITH(kElemF16)
  ECHO_TYPES(kElemF32, kElemF32, kElemF32)
#undef ECHO_TYPES_WITH
#undef ECHO_TYPES
  return hipErrorInvalidValue;
}

}  // namespace echo
