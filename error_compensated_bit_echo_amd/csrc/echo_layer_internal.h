// Internal interface of the operators of the layer around the all-reduce (8-bit
// quantizer and product, residual dropout): launch arguments.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "echo_internal.h"

namespace echo {

constexpr int kFp8Block = 128;                  // elements of k per scale
constexpr int64_t kFp8MaxDim = int64_t{1} << 22;  // rows, k and the pitch of codes

enum Elem { kElemF32 = 0, kElemBf16 = 1, kElemF16 = 2 };  // echo_dtype

// One orientation of the quantizer's output.
struct Fp8Out {
  uint8_t* codes[kMaxRanks];
  void* scales[kMaxRanks];
  int64_t ld;        // bytes between rows of codes
  int64_t srs, sks;  // scale strides, elements: (block of) rows, blocks along k
};

struct QuantFp8Args {
  const void* X[kMaxRanks];
  int64_t R, C, ldx;  // rows, columns, elements between rows
  Fp8Out rows, cols;  // codes[0] == nullptr: not wanted
  int32_t e5m2, e8m0;
  int32_t stream;  // set by the launcher: the codes along the rows go past the caches
};
// block128: one scale per 128 x 128 block instead of per row and 128 elements
hipError_t launch_quantize_fp8(const QuantFp8Args& a, int P, Elem x, bool block128, hipStream_t s);

struct GemmFp8Args {
  const uint8_t* A[kMaxRanks];
  const uint8_t* W[kMaxRanks];
  const void* sA[kMaxRanks];
  const void* sW[kMaxRanks];
  void* out[kMaxRanks];
  int64_t M, N, K;
  int64_t lda, ldw, ldo;  // bytes, bytes, elements between rows
  int64_t sa_row, sa_k, sw_row, sw_k;  // scale strides, elements
  int32_t sa_shift, sw_shift;          // scale row of matrix row i: i >> shift (0 or 7)
  int32_t out_elem;                    // Elem
};
hipError_t launch_gemm_fp8(const GemmFp8Args& a, int P, bool a_e5m2, bool w_e5m2, bool e8m0, hipStream_t s);

struct DropoutArgs {
  const void* x;
  const void* residual;  // nullptr: none
  void* out;
  int64_t R, C, ldx, ldr, ldo;
  const int64_t* rng;  // key, step
  int64_t offset, first;
  uint32_t threshold;  // kept iff the 16-bit draw is at least this
  float scale;
};
hipError_t launch_dropout(const DropoutArgs& a, Elem x, Elem out, hipStream_t s);

}  // namespace echo
