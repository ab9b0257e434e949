// Quantizer to 8-bit floating point with a power-of-two scale per 128 elements.
//
// For a block with the largest finite magnitude a = (1 + m) 2^(e-127) (e, m from
// the bits of a), the largest finite value of both formats is 0.875 * 2^top
// (top = 9 for e4m3, 16 for e5m2), so the smallest power of two s with a / s in
// range has the biased exponent e + 1 - top, plus one where (1 + m) / 2 > 0.875,
// at least 1 (2^-126), and s = 1 for a = 0.  Multiplying by 1 / s is exact, so the
// hardware conversion (nearest, ties to even) is the only rounding.
//
// A workgroup of 256 threads takes a 128 x 128 tile: thread t holds rows
// 8 (t / 16) .. + 7 and columns 8 (t % 16) .. + 7, so a load instruction covers
// whole 256-byte row segments (bfloat16), a row block's maximum is a reduction over
// 16 lanes in registers, and the transposed codes leave each thread as 8 bytes
// along the rows.  Those go through an LDS tile of 128 x 128 bytes whose 8-byte
// chunks are swizzled by the column group and come back as 16-byte runs: X is read
// once and every code is written once, in full 128-byte lines.
// Without the transpose, and with a scale per row, a unit of 16 lanes quantizes one
// block of 128 elements on its own (rows of few tokens spread over all CUs).
#pragma clang fp contract(off)

#include "echo_elem.h"

namespace echo {
namespace {

constexpr int kThreads = 256;
constexpr uint32_t kInfBits = 0x7F800000u;

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// The larger of x and of what the lane `CTRL` away holds (a DPP move within 16 lanes).
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t x) {
  return umax(x, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(static_cast<int>(x), static_cast<int>(x), CTRL, 0xF,
                                                                   0xF, false)));
}
// Maximum over the 16 lanes of a row: quad swaps, then the half-row and row mirrors.
__device__ __forceinline__ uint32_t row16_max(uint32_t x) {
  x = dpp_max<0xB1>(x);
  x = dpp_max<0x4E>(x);
  x = dpp_max<0x141>(x);
  return dpp_max<0x140>(x);
}
// Maximum over the four 16-lane rows of a wavefront.
__device__ __forceinline__ uint32_t across_rows_max(uint32_t x) {
  x = umax(x, static_cast<uint32_t>(__shfl_xor(static_cast<int>(x), 16)));
  return umax(x, static_cast<uint32_t>(__shfl_xor(static_cast<int>(x), 32)));
}

__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }
// the magnitude of a finite value, 0 for infinities and NaN
__device__ __forceinline__ uint32_t finite_magnitude(float v) {
  const uint32_t u = magnitude(v);
  return u < kInfBits ? u : 0u;
}

// The biased exponent of the block's scale from the bits of its largest magnitude.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax, bool e5m2) {
  const int e = static_cast<int>(amax >> 23) + (e5m2 ? 1 - 16 : 1 - 9) + ((amax & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return amax == 0 ? 127u : static_cast<uint32_t>(e < 1 ? 1 : e);
}
// 1 / 2^(b - 127), 1 <= b <= 253: the exponent 254 - b
__device__ __forceinline__ float inverse_scale(uint32_t b) { return __uint_as_float((254u - b) << 23); }

__device__ __forceinline__ void store_scale(void* s, int64_t at, uint32_t b, bool e8m0) {
  if (e8m0) static_cast<uint8_t*>(s)[at] = static_cast<uint8_t>(b);
  else static_cast<float*>(s)[at] = __uint_as_float(b << 23);
}

// Four scaled values to four codes.
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, bool e5m2) {
  int w = 0;
  if (e5m2) {
    w = __builtin_amdgcn_cvt_pk_bf8_f32(a, b, w, false);
    w = __builtin_amdgcn_cvt_pk_bf8_f32(c, d, w, true);
  } else {
    w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, w, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
  }
  return static_cast<uint32_t>(w);
}

// A value that is not finite becomes NaN (e5m2 would keep an infinity).
__device__ __forceinline__ float nan_if_not_finite(float v) { return magnitude(v) < kInfBits ? v : __uint_as_float(0x7FC00000u); }

// Row r0 .. of X, columns c .. c + 7, zeros outside the matrix.
template <int X>
__device__ __forceinline__ void load_row8(const void* x, int64_t ldx, int64_t row, int64_t c, int64_t R, int64_t C,
                                          float v[8]) {
  if (row < R && c + 8 <= C)
    load8<X>(x, row * ldx + c, v);
  else
    load_part<X>(x, row * ldx + c, row < R && c < C ? static_cast<int>(C - c) : 0, v);
}

// The codes of columns c .. c + 7 of a row, at most n of them.
__device__ __forceinline__ void store_codes8(uint8_t* p, uint2 w, int n) {
  if (n >= 8) {
    *reinterpret_cast<uint2*>(p) = w;
  } else {
    const uint64_t b = (static_cast<uint64_t>(w.y) << 32) | w.x;
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < n) p[i] = static_cast<uint8_t>(b >> (8 * i));
  }
}

// A scale per row and block, no transpose: unit u of a rank is row u / nb, block u % nb.
template <int X>
__global__ __launch_bounds__(kThreads) void echo_quant_rows_k(const QuantFp8Args a) {
  const int r = blockIdx.y;
  const auto* k = kernel_args<QuantFp8Args>();
  const void* x = k->X[r];
  uint8_t* q = k->rows.codes[r];
  void* sc = k->rows.scales[r];
  const bool e5m2 = a.e5m2 != 0;
  const int64_t nb = (a.C + kFp8Block - 1) / kFp8Block, units = a.R * nb;
  const int l = threadIdx.x & 15;
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * (kThreads / 16) + (threadIdx.x >> 4); u < units;
       u += static_cast<int64_t>(gridDim.x) * (kThreads / 16)) {
    const int64_t row = u / nb, b = u - row * nb, c = b * kFp8Block + 8 * l;
    float v[8];
    load_row8<X>(x, a.ldx, row, c, a.R, a.C, v);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = umax(m, magnitude(v[i]));
    m = row16_max(m);
    if (m >= kInfBits) {  // the block holds a value that is not finite
      m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        m = umax(m, finite_magnitude(v[i]));
        v[i] = nan_if_not_finite(v[i]);
      }
      m = row16_max(m);
    }
    const uint32_t sb = scale_byte(m, e5m2);
    const float inv = inverse_scale(sb);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = v[i] * inv;
    const uint2 w = make_uint2(codes4(v[0], v[1], v[2], v[3], e5m2), codes4(v[4], v[5], v[6], v[7], e5m2));
    const int64_t left = a.C - c;
    if (left > 0) store_codes8(q + row * a.rows.ld + c, w, left < 8 ? static_cast<int>(left) : 8);
    if (l == 0) store_scale(sc, row * a.rows.srs + b * a.rows.sks, sb, a.e8m0 != 0);
  }
}

// A 128 x 128 tile; COLS: the transposed codes are wanted too (or only); B128: one
// scale for the tile.
template <int X, bool COLS, bool B128>
__global__ __launch_bounds__(kThreads) void echo_quant_tile_k(const QuantFp8Args a) {
  __shared__ __attribute__((aligned(16))) uint8_t tile[COLS ? 128 * 128 : 16];
  __shared__ uint32_t part[4][128];  // per wavefront: column maxima (or the tile's)
  const int64_t nbc = (a.C + kFp8Block - 1) / kFp8Block, nbr = (a.R + kFp8Block - 1) / kFp8Block;
  const int64_t per = nbc * nbr;
  const int r = static_cast<int>(blockIdx.x / per);
  const int64_t at = blockIdx.x - r * per;
  const int64_t br = at / nbc, bc = at - br * nbc;
  const auto* k = kernel_args<QuantFp8Args>();
  const void* x = k->X[r];
  uint8_t *qr = k->rows.codes[r], *qc = k->cols.codes[r];
  void *sr = k->rows.scales[r], *sc = k->cols.scales[r];
  const bool e5m2 = a.e5m2 != 0, e8m0 = a.e8m0 != 0;
  const int t = threadIdx.x, cg = t & 15, rg = t >> 4, wave = t >> 6;
  const int64_t row0 = br * kFp8Block + 8 * rg, col0 = bc * kFp8Block + 8 * cg;
  float v[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) load_row8<X>(x, a.ldx, row0 + i, col0, a.R, a.C, v[i]);

  // A value that is not finite turns into NaN and does not count; the whole
  // workgroup takes this pass or none of it does.
  uint32_t any = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) any = umax(any, magnitude(v[i][j]));
  const bool clean = __syncthreads_and(any < kInfBits);
  if (!clean) {
    any = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        any = umax(any, finite_magnitude(v[i][j]));
        v[i][j] = nan_if_not_finite(v[i][j]);
      }
  }
  const auto counted = [&](float f) { return clean ? magnitude(f) : finite_magnitude(f); };

  uint32_t tile_byte = 0;
  if constexpr (B128) {
    const uint32_t m = across_rows_max(row16_max(any));
    if ((t & 63) == 0) part[wave][0] = m;
    __syncthreads();
    tile_byte = scale_byte(umax(umax(part[0][0], part[1][0]), umax(part[2][0], part[3][0])), e5m2);
    if (t == 0) {
      if (qr != nullptr) store_scale(sr, br * a.rows.srs + bc * a.rows.sks, tile_byte, e8m0);
      if (qc != nullptr) store_scale(sc, bc * a.cols.srs + br * a.cols.sks, tile_byte, e8m0);
    }
  }
  if (qr != nullptr) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t sb = tile_byte;
      if constexpr (!B128) {
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = umax(m, counted(v[i][j]));
        sb = scale_byte(row16_max(m), e5m2);
      }
      const float inv = inverse_scale(sb);
      const uint2 w = make_uint2(codes4(v[i][0] * inv, v[i][1] * inv, v[i][2] * inv, v[i][3] * inv, e5m2),
                                 codes4(v[i][4] * inv, v[i][5] * inv, v[i][6] * inv, v[i][7] * inv, e5m2));
      const int64_t row = row0 + i, left = a.C - col0;
      if (row < a.R) {
        if (left > 0) store_codes8(qr + row * a.rows.ld + col0, w, left < 8 ? static_cast<int>(left) : 8);
        if (!B128 && cg == 0) store_scale(sr, row * a.rows.srs + bc * a.rows.sks, sb, e8m0);
      }
    }
  }
  if constexpr (COLS) {
    uint32_t sbc[8];
    if constexpr (!B128) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = umax(m, counted(v[i][j]));
        m = across_rows_max(m);
        if ((t & 63) < 16) part[wave][8 * cg + j] = m;
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int c = 8 * cg + j;
        sbc[j] = scale_byte(umax(umax(part[0][c], part[1][c]), umax(part[2][c], part[3][c])), e5m2);
      }
      if (rg == 0) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (col0 + j < a.C) store_scale(sc, (col0 + j) * a.cols.srs + br * a.cols.sks, sbc[j], e8m0);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) sbc[j] = tile_byte;
    }
    // column 8 cg + j of the tile: 128 bytes of codes, 8-byte chunk rg (this thread's
    // rows) at slot rg ^ cg
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float inv = inverse_scale(sbc[j]);
      const uint2 w = make_uint2(codes4(v[0][j] * inv, v[1][j] * inv, v[2][j] * inv, v[3][j] * inv, e5m2),
                                 codes4(v[4][j] * inv, v[5][j] * inv, v[6][j] * inv, v[7][j] * inv, e5m2));
      *reinterpret_cast<uint2*>(tile + (8 * cg + j) * 128 + 8 * (rg ^ cg)) = w;
    }
    __syncthreads();
    // out in 16-byte runs: 8 lanes cover a column's 128 rows
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int c = 32 * u + (t >> 3), run = t & 7, f = (c >> 3) & 15;
      // chunks 2 run and 2 run + 1 sit in one 16-byte slot, swapped where f is odd
      const uint4 w = *reinterpret_cast<const uint4*>(tile + c * 128 + 16 * (run ^ (f >> 1)));
      const uint2 lo = (f & 1) ? make_uint2(w.z, w.w) : make_uint2(w.x, w.y);
      const uint2 hi = (f & 1) ? make_uint2(w.x, w.y) : make_uint2(w.z, w.w);
      const int64_t col = bc * kFp8Block + c, row = br * kFp8Block + 16 * run, left = a.R - row;
      if (col < a.C && left > 0) {
        uint8_t* p = qc + col * a.cols.ld + row;
        if (left >= 16) {
          *reinterpret_cast<uint4*>(p) = make_uint4(lo.x, lo.y, hi.x, hi.y);
        } else {
          store_codes8(p, lo, static_cast<int>(left));
          if (left > 8) store_codes8(p + 8, hi, static_cast<int>(left - 8));
        }
      }
    }
  }
}

template <int X>
hipError_t launch(const QuantFp8Args& a, int P, bool block128, hipStream_t s) {
  const int64_t nbc = (a.C + kFp8Block - 1) / kFp8Block, nbr = (a.R + kFp8Block - 1) / kFp8Block;
  const bool cols = a.cols.codes[0] != nullptr;
  if (!cols && !block128) {
    const int64_t blocks = (a.R * nbc + kThreads / 16 - 1) / (kThreads / 16);
    const dim3 grid(static_cast<unsigned>(blocks < (1 << 20) ? blocks : (1 << 20)), static_cast<unsigned>(P));
    hipLaunchKernelGGL((echo_quant_rows_k<X>), grid, dim3(kThreads), 0, s, a);
    return hipGetLastError();
  }
  const dim3 grid(static_cast<unsigned>(P * nbc * nbr));
  if (cols && block128)
    hipLaunchKernelGGL((echo_quant_tile_k<X, true, true>), grid, dim3(kThreads), 0, s, a);
  else if (cols)
    hipLaunchKernelGGL((echo_quant_tile_k<X, true, false>), grid, dim3(kThreads), 0, s, a);
  else
    hipLaunchKernelGGL((echo_quant_tile_k<X, false, true>), grid, dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_fp8(const QuantFp8Args& a, int P, Elem x, bool block128, hipStream_t s) {
  switch (x) {
    case kElemF32: return launch<kElemF32>(a, P, block128, s);
    case kElemBf16: return launch<kElemBf16>(a, P, block128, s);
    default: return launch<kElemF16>(a, P, block128, s);
  }
}

}  // namespace echo
