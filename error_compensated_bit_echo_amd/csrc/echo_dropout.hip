// Residual dropout with a mask from a counter-based generator: out = residual +
// keep(e) * x * scale per element, and without a residual its backward pass.
//
// The mask: element index e = first + i * cols + j belongs to chunk e / 8; the
// four 32-bit words of Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel
// random numbers: as easy as 1, 2, 3", SC 2011) with counter (chunk, step) and
// key rng[0] give the chunk's eight 16-bit draws, and e is kept iff its draw is
// at least the threshold.  A thread owns the part of one chunk that lies in one
// row: eight elements share one generator call, which costs 20 32 x 32 -> 64-bit
// products and 40 exclusive ors, five 32-bit operations per element.  (With
// 32-bit draws, four elements a call, the arithmetic rather than memory would
// bound the bfloat16 forms.)  Nothing is stored but the output, and the result
// does not depend on how the elements are split over threads.
#pragma clang fp contract(off)

#include "echo_elem.h"

namespace echo {
namespace {

constexpr int kThreads = 256;

struct Draws {
  uint32_t w[4];
};

__device__ __forceinline__ Draws philox10(uint64_t chunk, uint64_t step, uint64_t key) {
  uint32_t c0 = static_cast<uint32_t>(chunk), c1 = static_cast<uint32_t>(chunk >> 32);
  uint32_t c2 = static_cast<uint32_t>(step), c3 = static_cast<uint32_t>(step >> 32);
  uint32_t k0 = static_cast<uint32_t>(key), k1 = static_cast<uint32_t>(key >> 32);
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t p0 = static_cast<uint64_t>(c0) * 0xD2511F53u;
    const uint64_t p1 = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
    c0 = static_cast<uint32_t>(p1 >> 32) ^ c1 ^ k0;
    c1 = static_cast<uint32_t>(p1);
    c2 = static_cast<uint32_t>(p0 >> 32) ^ c3 ^ k1;
    c3 = static_cast<uint32_t>(p0);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return Draws{{c0, c1, c2, c3}};
}

__device__ __forceinline__ bool kept(const Draws& d, int lane, uint32_t threshold) {
  const uint32_t w = d.w[lane >> 1];
  return ((lane & 1) ? w >> 16 : w & 0xFFFFu) >= threshold;
}

// Rows are blocks of blockIdx.y (and every gridDim.y rows after), chunks of a row
// are threads of the x dimension (and every grid width after).
template <int X, int O, bool RES>
__global__ __launch_bounds__(kThreads) void echo_dropout_k(const DropoutArgs a) {
  const uint64_t key = static_cast<uint64_t>(a.rng[0]);
  const uint64_t step = static_cast<uint64_t>(a.rng[1]) + static_cast<uint64_t>(a.offset);
  for (int64_t row = blockIdx.y; row < a.R; row += gridDim.y) {
    const int64_t e0 = a.first + row * a.C;        // index of the row's first element
    const int64_t q0 = e0 >> 3;                    // its chunk
    const int64_t nq = ((e0 + a.C + 7) >> 3) - q0;  // chunks the row touches
    const int64_t ox = row * a.ldx, orr = row * a.ldr, oo = row * a.ldo;
    for (int64_t q = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; q < nq;
         q += static_cast<int64_t>(gridDim.x) * kThreads) {
      const int64_t j = ((q0 + q) << 3) - e0;  // column of the chunk's first element (may lie before the row)
      const Draws d = philox10(static_cast<uint64_t>(q0 + q), step, key);
      if (j >= 0 && j + 8 <= a.C) {
        float v[8];
        load8<X>(a.x, ox + j, v);
        float r[8];
        if constexpr (RES) load8<O>(a.residual, orr + j, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[i] = kept(d, i, a.threshold) ? v[i] * a.scale : 0.0f;
          if constexpr (RES) v[i] = v[i] + r[i];
        }
        store8<O>(a.out, oo + j, v);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (j + i >= 0 && j + i < a.C) {
            float y = kept(d, i, a.threshold) ? load1<X>(a.x, ox + j + i) * a.scale : 0.0f;
            if constexpr (RES) y = y + load1<O>(a.residual, orr + j + i);
            store1<O>(a.out, oo + j + i, y);
          }
      }
    }
  }
}

template <int X, int O>
hipError_t launch(const DropoutArgs& a, dim3 grid, hipStream_t s) {
  if (a.residual != nullptr)
    hipLaunchKernelGGL((echo_dropout_k<X, O, true>), grid, dim3(kThreads), 0, s, a);
  else
    hipLaunchKernelGGL((echo_dropout_k<X, O, false>), grid, dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

template <int X>
hipError_t launch_x(const DropoutArgs& a, Elem out, dim3 grid, hipStream_t s) {
  switch (out) {
    case kElemF32: return launch<X, kElemF32>(a, grid, s);
    case kElemBf16: return launch<X, kElemBf16>(a, grid, s);
    default: return launch<X, kElemF16>(a, grid, s);
  }
}

}  // namespace

hipError_t launch_dropout(const DropoutArgs& given, Elem x, Elem out, hipStream_t s) {
  DropoutArgs a = given;
  // rows that follow each other without a gap are one row: no chunk is drawn twice
  // and none is cut
  if (a.R > 1 && a.ldx == a.C && a.ldo == a.C && (a.residual == nullptr || a.ldr == a.C)) {
    a.C *= a.R;
    a.R = 1;
  }
  const int64_t per_row = (a.C / 8 + 2 + kThreads - 1) / kThreads;  // a row of C touches at most C/8 + 2 chunks
  const dim3 grid(static_cast<unsigned>(per_row < (1 << 20) ? per_row : (1 << 20)),
                  static_cast<unsigned>(a.R < 65535 ? a.R : 65535));
  switch (x) {
    case kElemF32: return launch_x<kElemF32>(a, out, grid, s);
    case kElemBf16: return launch_x<kElemBf16>(a, out, grid, s);
    default: return launch_x<kElemF16>(a, out, grid, s);
  }
}

}  // namespace echo
