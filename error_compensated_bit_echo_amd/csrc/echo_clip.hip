// The norm of many tensors together, and the tensors scaled by min(1, max_norm / (norm +
// 1e-6)).  Two launches for up to kClipTensors tensors: the first adds squares, a partial
// sum per workgroup; in the second every workgroup adds the partial sums, in the same
// order, and scales its chunks.  Tensors come in the launch's arguments, so nothing is kept
// between calls and a captured call needs no table in device memory.
//
// Squares are formed and added in 64 bits, so that neither a gradient of 1e30 nor one of
// 1e-30 is lost; the memory hides it.
#include "echo_row.h"

namespace echo {
namespace {

constexpr int kThreads = 256;
constexpr int kRuns = 8;                            // runs of 8 elements to a thread and chunk
constexpr int64_t kChunk = kThreads * kRuns * 8;    // elements

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

// The tensor that holds a chunk: the last one whose first chunk is not behind it.
template <typename Args>
__device__ __forceinline__ int tensor_of(const Args* a, uint32_t chunk) {
  int lo = 0, hi = a->tensors;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a->first[mid] <= chunk) lo = mid;
    else hi = mid;
  }
  return lo;
}

template <int E>
__device__ __forceinline__ double chunk_squares(const void* p, int64_t at, int64_t n) {
  double s = 0.0;
  if (at + kChunk <= n) {
    float v[kRuns][8];
#pragma unroll
    for (int k = 0; k < kRuns; ++k) load8<E>(p, at + (k * kThreads + threadIdx.x) * 8, v[k]);
#pragma unroll
    for (int k = 0; k < kRuns; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) s = s + static_cast<double>(v[k][i]) * static_cast<double>(v[k][i]);
  } else {
    for (int k = 0; k < kRuns; ++k) {
      const int64_t j = at + (k * kThreads + threadIdx.x) * 8;
      float v[8];
      load_run<E>(p, j, run_length(j, n), v);
#pragma unroll
      for (int i = 0; i < 8; ++i) s = s + static_cast<double>(v[i]) * static_cast<double>(v[i]);
    }
  }
  return s;
}

__global__ __launch_bounds__(kThreads) void echo_clip_sum_k(const ClipArgs given, double* part) {
  __shared__ double lds[4];
  const auto* a = kernel_args<ClipArgs>();
  const uint32_t chunks = a->first[a->tensors];
  double s = 0.0;
  for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int t = tensor_of(a, c);
    const int64_t at = static_cast<int64_t>(c - a->first[t]) * kChunk, n = a->n[t];
    const void* p = a->src[t];
    const int e = a->elem[t];
    if (e == kElemF32) s = s + chunk_squares<kElemF32>(p, at, n);
    else if (e == kElemBf16) s = s + chunk_squares<kElemBf16>(p, at, n);
    else s = s + chunk_squares<kElemF16>(p, at, n);
  }
  s = block_sum64(s, lds);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
}

__device__ __forceinline__ double norm_of(const double* part, int64_t n_part, double* lds) {
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < n_part; i += kThreads) s = s + part[i];
  return sqrt(block_sum64(s, lds));
}

template <int E>
__device__ __forceinline__ void scale_chunk(const void* p, void* o, int64_t at, int64_t n, float f) {
  if (at + kChunk <= n) {
    float v[kRuns][8];
#pragma unroll
    for (int k = 0; k < kRuns; ++k) load8<E>(p, at + (k * kThreads + threadIdx.x) * 8, v[k]);
#pragma unroll
    for (int k = 0; k < kRuns; ++k) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[k][i] = v[k][i] * f;
      store8<E>(o, at + (k * kThreads + threadIdx.x) * 8, v[k]);
    }
  } else {
    for (int k = 0; k < kRuns; ++k) {
      const int64_t j = at + (k * kThreads + threadIdx.x) * 8;
      const int m = run_length(j, n);
      float v[8];
      load_run<E>(p, j, m, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = v[i] * f;
      store_run<E>(o, j, m, v);
    }
  }
}

__global__ __launch_bounds__(kThreads) void echo_clip_scale_k(const ClipArgs given, const double* part, int64_t n_part,
                                                              double max_norm, float* norm) {
  __shared__ double lds[4];
  const auto* a = kernel_args<ClipArgs>();
  const double total = norm_of(part, n_part, lds);
  if (norm != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *norm = static_cast<float>(total);
  // a norm that is not a number makes every element one; an infinite norm gives 0
  const double f64 = max_norm / (total + 1e-6);
  const float f = f64 >= 1.0 ? 1.0f : static_cast<float>(f64);
  const uint32_t chunks = a->first[a->tensors];
  // from the last chunk on: the first launch read it last, so it is likeliest to be cached
  for (uint32_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    const uint32_t chunk = chunks - 1 - c;
    const int t = tensor_of(a, chunk);
    const int64_t at = static_cast<int64_t>(chunk - a->first[t]) * kChunk, n = a->n[t];
    const void* p = a->src[t];
    void* o = a->dst[t];
    if (f == 1.0f && p == o) continue;
    const int e = a->elem[t];
    if (e == kElemF32) scale_chunk<kElemF32>(p, o, at, n, f);
    else if (e == kElemBf16) scale_chunk<kElemBf16>(p, o, at, n, f);
    else scale_chunk<kElemF16>(p, o, at, n, f);
  }
}

__global__ __launch_bounds__(kThreads) void echo_clip_norm_k(const double* part, int64_t n_part, float* norm) {
  __shared__ double lds[4];
  const double total = norm_of(part, n_part, lds);
  if (threadIdx.x == 0) *norm = static_cast<float>(total);
}

unsigned clip_grid(uint32_t chunks) {
  return chunks < static_cast<uint32_t>(kClipGroups) ? chunks : static_cast<unsigned>(kClipGroups);
}

}  // namespace

int64_t clip_chunks(int64_t n) { return (n + kChunk - 1) / kChunk; }

hipError_t launch_clip_sum(const ClipArgs& a, double* part, int64_t at, int64_t* used, hipStream_t s) {
  const unsigned grid = clip_grid(a.first[a.tensors]);
  *used = grid;
  hipLaunchKernelGGL(echo_clip_sum_k, dim3(grid), dim3(kThreads), 0, s, a, part + at);
  return hipGetLastError();
}

hipError_t launch_clip_scale(const ClipArgs& a, const double* part, int64_t n_part, double max_norm, float* norm,
                             hipStream_t s) {
  hipLaunchKernelGGL(echo_clip_scale_k, dim3(clip_grid(a.first[a.tensors])), dim3(kThreads), 0, s, a, part, n_part,
                     max_norm, norm);
  return hipGetLastError();
}

hipError_t launch_clip_norm(const double* part, int64_t n_part, float* norm, hipStream_t s) {
  hipLaunchKernelGGL(echo_clip_norm_k, dim3(1), dim3(kThreads), 0, s, part, n_part, norm);
  return hipGetLastError();
}

}  // namespace echo
