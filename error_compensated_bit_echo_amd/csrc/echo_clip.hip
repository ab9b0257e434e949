// The norm of many tensors together, and the tensors scaled by min(1, max_norm / (norm +
// 1e-6)).  Two launches for up to 176 tensors (280 in place): the first adds squares, a
// partial sum per workgroup; in the second every workgroup adds the partial sums, in the same
// order (one workgroup beforehand, where several launches left some), and scales its chunks.
// Tensors come in the launch's arguments, so nothing is kept between calls and a captured call
// needs no table in device memory.
//
// Squares are formed and added in 64 bits, so that neither a gradient of 1e30 nor one of
// 1e-30 is lost; the memory hides it.
//
// Bound by the memory: 64 tensors of 16 Mi fp32 take 2.22 ms, the squares 0.69 (6.2 TB/s) and
// the scaling 1.54 (5.6 TB/s); 24 tensors of 4096 take 9 to 11 us, 3.4 and 4.3 of them the
// kernels; 331 mixed ones of 26 M elements 47 us in five launches.
#include "echo_row.h"

namespace echo {
namespace {

constexpr int kThreads = 256;
constexpr int kUnits = static_cast<int>(kClipChunk) / 16 / kThreads;  // 16-byte units of a chunk to a thread
constexpr int kHalf = kUnits / 2;

__device__ __forceinline__ double wave_sum64(double v) {
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) v = v + __shfl_xor(v, m);
  return v;
}

// The sum over the workgroup, in every thread.
__device__ __forceinline__ double block_sum64(double v, double* lds) {
  v = wave_sum64(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  return (lds[0] + lds[1]) + (lds[2] + lds[3]);
}

// Chunks of 8 next to each other, where a tensor has them whole, share their 256 KB page by page: a
// chunk is 8 pages of 4 KB, 32 KB apart.  The 8 lie with workgroups of the 8 XCDs, each of which so
// keeps to one remainder of 32 KB in a large tensor (a copy of 1 GiB in chunks: 5.99 TB/s, with
// chunks of 32 KB in a row 5.37).
constexpr int kPage = kThreads * 16, kSpan = 8;
static_assert(kPage * kSpan == kClipChunk, "a page to a round of the threads");

// A launch's chunks: where each lies.  Every lane keeps a few of the tensors' first chunks, so
// that finding a chunk's tensor is a count of those not behind it, with no chain of loads.
template <typename Args>
struct Tensors {
  static constexpr int kEach = (Args::kTensors + 63) / 64;
  uint32_t first[kEach];

  template <typename A>
  __device__ __forceinline__ void load(const A* a) {
    const int lane = threadIdx.x & 63, n = a->tensors;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int t = i * 64 + lane;
      first[i] = t < n ? a->first[t] : ~0u;
    }
  }
  __device__ __forceinline__ int tensor_of(uint32_t chunk) const {
    int t = -1;
#pragma unroll
    for (int i = 0; i < kEach; ++i) t += __popcll(__ballot(first[i] <= chunk));
    return t;
  }
};

struct Chunk {
  int64_t at;      // its first byte in the tensor
  int tensor, elem;
  int bytes;       // of it
  int step;        // bytes from a thread's unit to its next
};

template <typename Args, typename A>
__device__ __forceinline__ Chunk chunk_of(const A* a, const Tensors<Args>& ts, uint32_t c) {
  const int t = ts.tensor_of(c);
  const uint32_t tail = a->tail[t], first = a->first[t], end = a->first[t + 1], in = c - first;
  const int elem = static_cast<int>(tail >> 14), last = static_cast<int>(((tail & 0x3FFF) + 1) * 2);
  if ((in | (kSpan - 1)) < end - first - (last < kClipChunk ? 1 : 0))
    return Chunk{static_cast<int64_t>(in / kSpan) * (kSpan * kClipChunk) + in % kSpan * kPage, t, elem, static_cast<int>(kClipChunk),
                 kSpan * kPage};
  return Chunk{static_cast<int64_t>(in) * kClipChunk, t, elem, c + 1 == end ? last : static_cast<int>(kClipChunk), kPage};
}

// 16 bytes of a chunk.  One that would reach past the tensor's end starts 16 bytes before it
// instead, and its first `lo` bytes are another thread's (16: all of them).  All of a
// chunk's loads are issued before the first is used.
struct Unit {
  uint32_t w[4];
};

struct Spot {
  int64_t at;
  int lo;
};

__device__ __forceinline__ Spot spot_of(const Chunk& c, int k) {
  const int at = (k * kThreads + static_cast<int>(threadIdx.x)) * 16, last = c.bytes - 16;
  return at <= last ? Spot{c.at + k * c.step + static_cast<int>(threadIdx.x) * 16, 0} : Spot{c.at + last, at - last < 16 ? at - last : 16};
}

template <int N>
__device__ __forceinline__ void load_units(const Chunk& c, const char* p, Unit (&u)[N]) {
  if (c.at + c.bytes >= 16) {
#pragma unroll
    for (int k = 0; k < N; ++k) __builtin_memcpy(u[k].w, p + spot_of(c, k).at, 16);
  } else {
    // a tensor of fewer than 16 bytes: its elements are the unit's last ones
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t at = static_cast<int64_t>(c.bytes) - 16 + i * 4;  // of a dword of the unit
      const uint32_t low = at >= 0 ? *reinterpret_cast<const uint16_t*>(p + at) : 0;
      const uint32_t high = at + 2 >= 0 ? *reinterpret_cast<const uint16_t*>(p + at + 2) : 0;
      u[0].w[i] = low | high << 16;
    }
#pragma unroll
    for (int k = 1; k < N; ++k) u[k] = u[0];
  }
}

template <int E>
__device__ __forceinline__ double unit_squares(const Unit& u, int lo) {
  typedef typename ElemOf<E>::T T;
  constexpr int kN = 16 / sizeof(T);
  T x[kN];
  __builtin_memcpy(x, u.w, 16);
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const double v = static_cast<double>(i * static_cast<int>(sizeof(T)) >= lo ? static_cast<float>(x[i]) : 0.0f);
    s = __builtin_fma(v, v, s);
  }
  return s;
}

template <int E, int N>
__device__ __forceinline__ double squares_of(const Chunk& c, const char* p) {
  Unit u[N];
  load_units(c, p, u);
  double s = 0.0;
#pragma unroll
  for (int k = 0; k < N; ++k) s = s + unit_squares<E>(u[k], spot_of(c, k).lo);
  return s;
}

// A chunk that half the units cover, and so a short tensor, is loaded by halves.
template <int E>
__device__ __forceinline__ double squares(const Chunk& c, const char* p) {
  return c.bytes <= kHalf * kThreads * 16 ? squares_of<E, kHalf>(c, p) : squares_of<E, kUnits>(c, p);
}

__global__ __launch_bounds__(kThreads) void echo_clip_sum_k(const ClipInPlace given, double* part) {
  __shared__ double lds[4];
  const auto* a = kernel_args<ClipInPlace>();
  Tensors<ClipInPlace> ts;
  ts.load(a);
  const uint32_t chunks = a->first[a->tensors];
  double s = 0.0;
  for (uint32_t i = blockIdx.x; i < chunks; i += gridDim.x) {
    const Chunk c = chunk_of(a, ts, i);
    const char* p = static_cast<const char*>(a->src[c.tensor]);
    if (c.elem == kElemF32) s = s + squares<kElemF32>(c, p);
    else if (c.elem == kElemBf16) s = s + squares<kElemBf16>(c, p);
    else s = s + squares<kElemF16>(c, p);
  }
  s = block_sum64(s, lds);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
}

__device__ __forceinline__ double sum_of(const double* part, int64_t n_part, double* lds) {
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < n_part; i += kThreads) s = s + part[i];
  return block_sum64(s, lds);
}

__device__ __forceinline__ double norm_of(const double* part, int64_t n_part, double* lds) {
  return sqrt(sum_of(part, n_part, lds));
}

// STREAM: past the caches, so that what the first launch read and the cache still holds is not
// replaced by the results.
template <int E, bool STREAM>
__device__ __forceinline__ void scale_unit(const Unit& u, char* o, Spot at, float f) {
  typedef typename ElemOf<E>::T T;
  constexpr int kN = 16 / sizeof(T);
  T x[kN];
  __builtin_memcpy(x, u.w, 16);
#pragma unroll
  for (int i = 0; i < kN; ++i) x[i] = narrow<E>(static_cast<float>(x[i]) * f);
  if (at.lo == 0) {
    typedef uint32_t u4 __attribute__((ext_vector_type(4), aligned(2)));
    u4 w;
    __builtin_memcpy(&w, x, 16);
    u4* to = reinterpret_cast<u4*>(o + at.at);
    if constexpr (STREAM) __builtin_nontemporal_store(w, to);
    else *to = w;
  } else {
#pragma unroll
    for (int i = 0; i < kN; ++i)
      if (i * static_cast<int>(sizeof(T)) >= at.lo) reinterpret_cast<T*>(o + at.at)[i] = x[i];
  }
}

template <int E, bool STREAM, int N>
__device__ __forceinline__ void scale_units(const Chunk& c, const char* p, char* o, float f) {
  Unit u[N];
  load_units(c, p, u);
#pragma unroll
  for (int k = 0; k < N; ++k) scale_unit<E, STREAM>(u[k], o, spot_of(c, k), f);
}

template <int E, bool STREAM>
__device__ __forceinline__ void scale(const Chunk& c, const char* p, char* o, float f) {
  if (c.bytes <= kHalf * kThreads * 16) scale_units<E, STREAM, kHalf>(c, p, o, f);
  else scale_units<E, STREAM, kUnits>(c, p, o, f);
}

template <typename Args, bool STREAM>
__global__ __launch_bounds__(kThreads) void echo_clip_scale_k(const Args given, const double* part, int64_t n_part,
                                                              double max_norm, float* norm) {
  __shared__ double lds[4];
  const auto* a = kernel_args<Args>();
  Tensors<Args> ts;
  ts.load(a);
  const double total = norm_of(part, n_part, lds);
  if (norm != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *norm = static_cast<float>(total);
  // a norm that is not a number makes every element one; an infinite norm gives 0
  const double f64 = max_norm / (total + 1e-6);
  const float f = f64 >= 1.0 ? 1.0f : static_cast<float>(f64);
  constexpr bool kApart = sizeof(a->dst) > sizeof(void*);
  if (!kApart && f == 1.0f) return;
  const uint32_t chunks = a->first[a->tensors];
  // from the last chunk on: the first launch read it last, so it is likeliest to be cached
  for (uint32_t i = blockIdx.x; i < chunks; i += gridDim.x) {
    const Chunk c = chunk_of(a, ts, chunks - 1 - i);
    const char* p = static_cast<const char*>(a->src[c.tensor]);
    char* o = kApart ? static_cast<char*>(a->dst[c.tensor]) : const_cast<char*>(p);
    if (f == 1.0f && p == o) continue;
    if (c.elem == kElemF32) scale<kElemF32, STREAM>(c, p, o, f);
    else if (c.elem == kElemBf16) scale<kElemBf16, STREAM>(c, p, o, f);
    else scale<kElemF16, STREAM>(c, p, o, f);
  }
}

__global__ __launch_bounds__(kThreads) void echo_clip_norm_k(const double* part, int64_t n_part, float* norm) {
  __shared__ double lds[4];
  const double total = norm_of(part, n_part, lds);
  if (threadIdx.x == 0) *norm = static_cast<float>(total);
}

// One partial sum in place of all, the same that norm_of adds up.
__global__ __launch_bounds__(kThreads) void echo_clip_join_k(double* part, int64_t n_part) {
  __shared__ double lds[4];
  const double total = sum_of(part, n_part, lds);
  if (threadIdx.x == 0) part[0] = total;
}

template <typename Args>
hipError_t launch_scale(const Args& a, const double* part, int64_t n_part, double max_norm, float* norm, bool stream, hipStream_t s) {
  const dim3 grid(clip_grid(a.first[a.tensors]));
  if (stream)
    hipLaunchKernelGGL((echo_clip_scale_k<Args, true>), grid, dim3(kThreads), 0, s, a, part, n_part, max_norm, norm);
  else
    hipLaunchKernelGGL((echo_clip_scale_k<Args, false>), grid, dim3(kThreads), 0, s, a, part, n_part, max_norm, norm);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_clip_sum(const ClipInPlace& a, double* part, hipStream_t s) {
  hipLaunchKernelGGL(echo_clip_sum_k, dim3(clip_grid(a.first[a.tensors])), dim3(kThreads), 0, s, a, part);
  return hipGetLastError();
}

hipError_t launch_clip_scale(const ClipInPlace& a, const double* part, int64_t n_part, double max_norm, float* norm,
                             bool stream, hipStream_t s) {
  return launch_scale(a, part, n_part, max_norm, norm, stream, s);
}

hipError_t launch_clip_scale(const ClipApart& a, const double* part, int64_t n_part, double max_norm, float* norm,
                             bool stream, hipStream_t s) {
  return launch_scale(a, part, n_part, max_norm, norm, stream, s);
}

hipError_t launch_clip_join(double* part, int64_t n_part, hipStream_t s) {
  hipLaunchKernelGGL(echo_clip_join_k, dim3(1), dim3(kThreads), 0, s, part, n_part);
  return hipGetLastError();
}

hipError_t launch_clip_norm(const double* part, int64_t n_part, float* norm, hipStream_t s) {
  hipLaunchKernelGGL(echo_clip_norm_k, dim3(1), dim3(kThreads), 0, s, part, n_part, norm);
  return hipGetLastError();
}

}  // namespace echo
