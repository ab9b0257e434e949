// Residual dropout with a mask from a counter-based generator: out = residual +
// keep(e) * x * scale per element, and without a residual its backward pass.
//
// The mask: element index e = first + i * cols + j belongs to chunk e / 8; the
// four 32-bit words of Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel
// random numbers: as easy as 1, 2, 3", SC 2011) with counter (chunk, step) and
// key rng[0] give the chunk's eight 16-bit draws, and e is kept iff its draw is
// at least the threshold.  A thread owns the part of one chunk that lies in one
// row: eight elements share one generator call, which costs 20 products of 32 x 32
// to 64 bits and 40 exclusive ors, an instruction each: seven and a half an element,
// the key's additions being scalar.  Nothing is stored but the output, and the result
// does not depend on how the elements are split over threads.
//
// Bound by the memory: 16384 x 8192 bfloat16 with a residual takes 140 us, 5.75
// TB/s of what it has to move (a plain elementwise copy reaches 6.2 on this card);
// non-temporal loads or stores change nothing there.  Rows of odd lengths: 4095 x
// 4097 bfloat16 without a residual takes 13.4 us (5.0 TB/s) with the chunks of all
// rows numbered through, 16.1 us with rows as blocks of the grid's second axis,
// where the last workgroup of every row is mostly idle.
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

// The part of chunk q0 + q that lies in row `row`.
template <int X, int O, bool RES>
__device__ __forceinline__ void dropout_chunk(const DropoutArgs& a, uint64_t key, uint64_t step, int64_t row, int64_t q) {
  const int64_t e0 = a.first + row * a.C;  // index of the row's first element
  const int64_t chunk = (e0 >> 3) + q;
  const int64_t j = (chunk << 3) - e0;  // column of the chunk's first element (may lie before the row)
  if (j >= a.C) return;
  const int64_t ox = row * a.ldx, orr = row * a.ldr, oo = row * a.ldo;
  const Draws d = philox10(static_cast<uint64_t>(chunk), step, key);
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

// A thread a chunk of a row, `per_row` chunks to a row.  FLAT: all rows' chunks are
// numbered through (their number fits 32 bits), so that rows of any length fill the
// workgroups; otherwise rows are blocks of blockIdx.y and every gridDim.y rows after.
template <int X, int O, bool RES, bool FLAT>
__global__ __launch_bounds__(kThreads) void echo_dropout_k(const DropoutArgs a, int64_t per_row) {
  const uint64_t key = static_cast<uint64_t>(a.rng[0]);
  const uint64_t step = static_cast<uint64_t>(a.rng[1]) + static_cast<uint64_t>(a.offset);
  if constexpr (FLAT) {
    const uint32_t n = static_cast<uint32_t>(per_row), id = blockIdx.x * kThreads + threadIdx.x;
    const uint32_t row = id / n;
    if (row < a.R) dropout_chunk<X, O, RES>(a, key, step, row, id - row * n);
  } else {
    for (int64_t row = blockIdx.y; row < a.R; row += gridDim.y)
      for (int64_t q = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; q < per_row;
           q += static_cast<int64_t>(gridDim.x) * kThreads)
        dropout_chunk<X, O, RES>(a, key, step, row, q);
  }
}

template <int X, int O, bool RES>
hipError_t launch_as(const DropoutArgs& a, hipStream_t s) {
  // a row of C touches at most (C + 7) / 8 + 1 chunks, one less where all start at a chunk's start
  const bool whole = a.first % 8 == 0 && (a.R == 1 || a.C % 8 == 0);
  const int64_t per_row = (a.C + 7) / 8 + (whole ? 0 : 1);
  const int64_t blocks = (per_row + kThreads - 1) / kThreads;
  if (a.R > 1 && a.R <= ((int64_t{1} << 32) - kThreads) / per_row) {
    const int64_t all = (a.R * per_row + kThreads - 1) / kThreads;
    hipLaunchKernelGGL((echo_dropout_k<X, O, RES, true>), dim3(static_cast<unsigned>(all)), dim3(kThreads), 0, s, a,
                       per_row);
  } else {
    const dim3 grid(static_cast<unsigned>(blocks < (1 << 20) ? blocks : (1 << 20)),
                    static_cast<unsigned>(a.R < 65535 ? a.R : 65535));
    hipLaunchKernelGGL((echo_dropout_k<X, O, RES, false>), grid, dim3(kThreads), 0, s, a, per_row);
  }
  return hipGetLastError();
}

template <int X, int O>
hipError_t launch(const DropoutArgs& a, hipStream_t s) {
  return a.residual != nullptr ? launch_as<X, O, true>(a, s) : launch_as<X, O, false>(a, s);
}

template <int X>
hipError_t launch_x(const DropoutArgs& a, Elem out, hipStream_t s) {
  switch (out) {
    case kElemF32: return launch<X, kElemF32>(a, s);
    case kElemBf16: return launch<X, kElemBf16>(a, s);
    default: return launch<X, kElemF16>(a, s);
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
  switch (x) {
    case kElemF32: return launch_x<kElemF32>(a, out, s);
    case kElemBf16: return launch_x<kElemBf16>(a, out, s);
    default: return launch_x<kElemF16>(a, out, s);
  }
}

}  // namespace echo
