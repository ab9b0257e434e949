// The product of matrices in 8-bit floating point with a scale per 128 elements of
// k, on the matrix cores: out[m, n] = sum_b sA[m, b] sW[n, b] sum_{k in b} A[m, k] W[n, k].
//
// The codes are widened to bfloat16, which holds every value of both formats, and
// multiplied with v_mfma_f32_16x16x32_bf16, whose fp32 sums are precise; a block's
// sum is scaled and added in fp32.  (The 8-bit instructions align the products of
// each run of 8 consecutive k to the largest of them and drop what lies below 2^-13
// of it: measured 1.5e-5 of the result against 6e-9 for normal e4m3 data.)
// The product is computed transposed (W supplies the instruction's first operand),
// so a lane holds four consecutive columns n of one row m.
#pragma clang fp contract(off)

#include "echo_elem.h"

namespace echo {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;

// 32 bytes of a row from byte k on, zeros from K on.  The 16-byte runs that hold a
// valid byte lie within the row's pitch (a multiple of 16).
__device__ __forceinline__ i32x8 load_frag(const uint8_t* row, int64_t k, int64_t K) {
  i32x8 f{};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int64_t at = k + 16 * h;
    const int64_t left = K - at;
    if (left <= 0) continue;
    i32x4 x = *reinterpret_cast<const i32x4*>(row + at);
    if (left < 16) {
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        const int64_t n = left - 4 * d;  // valid bytes of this dword
        if (n <= 0) x[d] = 0;
        else if (n < 4) x[d] &= (1 << (8 * n)) - 1;
      }
    }
#pragma unroll
    for (int d = 0; d < 4; ++d) f[4 * h + d] = x[d];
  }
  return f;
}

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// 8 codes (two dwords) as bfloat16, exactly.
template <bool E5>
__device__ __forceinline__ bf16x8 widen8(int lo, int hi) {
  bf16x8 x{};
#if defined(__HIP_DEVICE_COMPILE__)
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t w = static_cast<uint32_t>(i ? hi : lo);
    const bf16x2 p = E5 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w, 1.0f, false)
                        : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false);
    const bf16x2 q = E5 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w, 1.0f, true)
                        : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true);
    x[4 * i] = p[0];
    x[4 * i + 1] = p[1];
    x[4 * i + 2] = q[0];
    x[4 * i + 3] = q[1];
  }
#endif
  return x;
}

// The sum over a block: lane l supplies 32 codes of row l % 16 of W and of A (any
// assignment of k to lanes does, as both operands use the same).
template <bool A5, bool W5>
__device__ __forceinline__ f32x4 block_sum(i32x8 w, i32x8 a) {
  f32x4 c{};
#if defined(__HIP_DEVICE_COMPILE__)
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen8<W5>(w[2 * i], w[2 * i + 1]), widen8<A5>(a[2 * i], a[2 * i + 1]),
                                                c, 0, 0, 0);
#endif
  return c;
}

// A scale as fp32.
template <bool E8>
__device__ __forceinline__ float scale_at(const void* s, int64_t at) {
  if constexpr (E8) {
    const uint32_t b = static_cast<const uint8_t*>(s)[at];
    return __uint_as_float(b == 255 ? 0x7FC00000u : b == 0 ? 0x00400000u : b << 23);  // 0: 2^-127, subnormal
  } else {
    return static_cast<const float*>(s)[at];
  }
}

// 64 x 64 tiles, four wavefronts of 32 x 32, fragments straight from memory.
template <bool A5, bool W5, bool E8>
__global__ __launch_bounds__(kThreads) void echo_gemm_fp8_k(const GemmFp8Args a, int64_t tiles_n) {
  const int r = blockIdx.y;
  const uint8_t *A = a.A[0], *W = a.W[0];
  const void *sA = a.sA[0], *sW = a.sW[0];
  void* out = a.out[0];
#pragma unroll
  for (int i = 1; i < kMaxRanks; ++i)
    if (r == i) {
      A = a.A[i];
      W = a.W[i];
      sA = a.sA[i];
      sW = a.sW[i];
      out = a.out[i];
    }
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t tm = blockIdx.x / tiles_n, tn = blockIdx.x - tm * tiles_n;
  const int64_t m0 = tm * 64 + 32 * (wave >> 1), n0 = tn * 64 + 32 * (wave & 1);
  const int sub = lane & 15, g = lane >> 4;
  int64_t m[2], n[2];  // the rows this lane supplies, clamped: what lies past the edge is not stored
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    m[i] = m0 + 16 * i + sub < a.M ? m0 + 16 * i + sub : a.M - 1;
    n[i] = n0 + 16 * i + sub < a.N ? n0 + 16 * i + sub : a.N - 1;
  }
  f32x4 acc[2][2] = {};
  const int64_t nb = (a.K + kFp8Block - 1) / kFp8Block;
  for (int64_t b = 0; b < nb; ++b) {
    i32x8 fa[2], fw[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      fa[i] = load_frag(A + m[i] * a.lda, b * kFp8Block + 32 * g, a.K);
      fw[i] = load_frag(W + n[i] * a.ldw, b * kFp8Block + 32 * g, a.K);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float ca = scale_at<E8>(sA, (m[i] >> a.sa_shift) * a.sa_row + b * a.sa_k);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const f32x4 p = block_sum<A5, W5>(fw[j], fa[i]);
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          int64_t nn = n0 + 16 * j + 4 * g + v;
          nn = nn < a.N ? nn : a.N - 1;
          const float cw = scale_at<E8>(sW, (nn >> a.sw_shift) * a.sw_row + b * a.sw_k);
          acc[i][j][v] = __builtin_fmaf(p[v], ca * cw, acc[i][j][v]);
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int64_t mm = m0 + 16 * i + sub, nn = n0 + 16 * j + 4 * g + v;
        if (mm < a.M && nn < a.N) {
          const int64_t at = mm * a.ldo + nn;
          if (a.out_elem == kElemF32) store1<kElemF32>(out, at, acc[i][j][v]);
          else if (a.out_elem == kElemBf16) store1<kElemBf16>(out, at, acc[i][j][v]);
          else store1<kElemF16>(out, at, acc[i][j][v]);
        }
      }
}

template <bool A5, bool W5, bool E8>
hipError_t launch(const GemmFp8Args& a, int P, hipStream_t s) {
  const int64_t tm = (a.M + 63) / 64, tn = (a.N + 63) / 64;
  const dim3 grid(static_cast<unsigned>(tm * tn), static_cast<unsigned>(P));
  hipLaunchKernelGGL((echo_gemm_fp8_k<A5, W5, E8>), grid, dim3(kThreads), 0, s, a, tn);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm_fp8(const GemmFp8Args& a, int P, bool a_e5m2, bool w_e5m2, bool e8m0, hipStream_t s) {
  if (e8m0)
    return a_e5m2 ? (w_e5m2 ? launch<true, true, true>(a, P, s) : launch<true, false, true>(a, P, s))
                  : (w_e5m2 ? launch<false, true, true>(a, P, s) : launch<false, false, true>(a, P, s));
  return a_e5m2 ? (w_e5m2 ? launch<true, true, false>(a, P, s) : launch<true, false, false>(a, P, s))
                : (w_e5m2 ? launch<false, true, false>(a, P, s) : launch<false, false, false>(a, P, s));
}

}  // namespace echo
