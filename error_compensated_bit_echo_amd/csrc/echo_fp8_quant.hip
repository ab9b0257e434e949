// Quantizer to 8-bit floating point with a power-of-two scale per 128 elements.
//
// For a block with the largest finite magnitude a = (1 + m) 2^(e-127) (e, m from
// the bits of a), the largest finite value of both formats is 0.875 * 2^top
// (top = 9 for e4m3, 16 for e5m2), so the smallest power of two s with a / s in
// range has the biased exponent e + 1 - top, plus one where (1 + m) / 2 > 0.875,
// at least 1 (2^-126), and s = 1 for a = 0.  x / s is exact, and the hardware's
// scaled conversions (nearest, ties to even; checked on the device for every 16-bit
// value) divide and round at once: the only rounding.
//
// A workgroup of 256 threads takes a 128 x 128 tile: thread t holds rows
// 8 (t / 16) .. + 7 and columns 8 (t % 16) .. + 7, so a load instruction covers
// whole 256-byte row segments (16-bit elements), a row block's maximum is a reduction
// over 16 lanes in registers, and the transposed codes leave each thread as 8 bytes
// along the rows.  Those go through an LDS tile of 128 x 128 bytes whose 8-byte
// chunks are swizzled by the column group and come back as 16-byte runs: X is read
// once and every code is written once, in full 128-byte lines.  16-bit elements stay
// packed: maxima two at a time on their magnitudes' bits, conversions two at a time
// from the packed pair, three instructions per element for both orientations.
// Measured, 8192 x 8192 both ways: bfloat16 55 us (4.9 TB/s; with every element in fp32,
// at twelve instructions, the kernel took half as long again), fp32 75 us (5.35 TB/s).  The
// memory bounds it: of a copy that writes every line once this card does 5.1 (the
// library's) to 6.2 TB/s, and the order in which tiles are taken moves the time by up to
// 15 % (down the columns 68 us; contiguous runs of tiles per XCD 66; one tile after the
// other 59; side by side in pairs on an XCD, as here, 57, and 55 past the caches).
// Without the transpose, with a scale per row and fewer than 512 tiles, a unit of 16
// lanes quantizes one block of 128 elements on its own, so that few tokens spread over
// all CUs (8 ranks of 64 x 1024: 4.9 us, which is the launch; with 512 tiles and more the
// tile kernel is faster: 8 x 512 x 2048 7.1 against 7.8 us, 8192 x 8192 39.9 against 48.6).
#pragma clang fp contract(off)

#include <type_traits>

#include "echo_elem.h"

namespace echo {
namespace {

constexpr int kThreads = 256;

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
typedef int16_t i16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }
// the larger of each half
__device__ __forceinline__ uint32_t umax2(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t,
                            __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}

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
// MAX over the four 16-lane rows of a wavefront (lanes l, l ^ 16, l ^ 32, l ^ 48).
template <typename Max>
__device__ __forceinline__ uint32_t across_rows(uint32_t x, Max max) {
#if defined(__HIP_DEVICE_COMPILE__)
  const auto a = __builtin_amdgcn_permlane16_swap(x, x, false, false);
  x = max(a[0], a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(x, x, false, false);
  x = max(b[0], b[1]);
#endif
  return x;
}

// The biased exponent of the block's scale from the fp32 bits of its largest magnitude.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax, bool e5m2) {
  const int e = static_cast<int>(amax >> 23) + (e5m2 ? 1 - 16 : 1 - 9) + ((amax & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return amax == 0 ? 127u : static_cast<uint32_t>(e < 1 ? 1 : e);
}
__device__ __forceinline__ float scale_of(uint32_t byte) { return __uint_as_float(byte << 23); }

__device__ __forceinline__ void store_scale(void* s, int64_t at, uint32_t b, bool e8m0) {
  if (e8m0) static_cast<uint8_t*>(s)[at] = static_cast<uint8_t>(b);
  else static_cast<uint32_t*>(s)[at] = b << 23;
}

// n (at most 8) of the codes of 8 consecutive elements.
__device__ __forceinline__ void store_codes8(uint8_t* p, uint2 w, int n) {
  if (n >= 8) {
    *reinterpret_cast<uint2*>(p) = w;
  } else {
    uint64_t b = (static_cast<uint64_t>(w.y) << 32) | w.x;
#pragma unroll 1
    for (int i = 0; i < n; ++i, b >>= 8) p[i] = static_cast<uint8_t>(b);
  }
}

// ROWS x 8 elements of a thread, 16-bit elements as packed pairs.
template <int X, int ROWS>
struct Part {
  static constexpr bool kF16 = X == kElemF16;
  static constexpr uint32_t kInf = kF16 ? 0x7C00u : 0x7F80u;
  static constexpr int kColWords = 4;  // words of column maxima: two columns each
  uint32_t d[ROWS][4];

  // Row i from row `row`, columns c .. c + 7 of X.
  __device__ __forceinline__ void load(int i, const void* x, int64_t at) {
    __builtin_memcpy(d[i], static_cast<const uint16_t*>(x) + at, 16);
  }
  // Moves row i down by `shift` elements (0 .. 7), zeros behind; `keep` false: all zeros.
  __device__ __forceinline__ void shift(int i, int shift, bool keep) {
    uint32_t* w = d[i];
    const bool s4 = shift & 4, s2 = shift & 2, s1 = shift & 1;
    w[0] = s4 ? w[2] : w[0];
    w[1] = s4 ? w[3] : w[1];
    w[2] = s4 ? 0u : w[2];
    w[3] = s4 ? 0u : w[3];
#pragma unroll
    for (int q = 0; q < 4; ++q) w[q] = s2 ? (q < 3 ? w[q < 3 ? q + 1 : 3] : 0u) : w[q];
#pragma unroll
    for (int q = 0; q < 4; ++q) w[q] = s1 ? (w[q] >> 16) | (q < 3 ? w[q < 3 ? q + 1 : 3] << 16 : 0u) : w[q];
#pragma unroll
    for (int q = 0; q < 4; ++q) w[q] = keep ? w[q] : 0u;
  }
  __device__ __forceinline__ void set(int i, int j, const void* x, int64_t at, bool keep) {
    const uint32_t v = static_cast<const uint16_t*>(x)[at];
    const uint32_t w = (j & 1) ? d[i][j >> 1] : 0u;
    d[i][j >> 1] = w | (keep ? v << (16 * (j & 1)) : 0u);
  }
  // Magnitudes of a pair.  FINITE: 0 for infinities and NaN.
  template <bool FINITE>
  static __device__ __forceinline__ uint32_t magnitudes(uint32_t w) {
    w &= 0x7FFF7FFFu;
    if constexpr (FINITE) w = ((w & 0xFFFFu) < kInf ? w & 0xFFFFu : 0u) | ((w >> 16) < kInf ? w & 0xFFFF0000u : 0u);
    return w;
  }
  template <bool FINITE>
  __device__ __forceinline__ uint32_t row_word(int i) const {
    return umax2(umax2(magnitudes<FINITE>(d[i][0]), magnitudes<FINITE>(d[i][1])),
                 umax2(magnitudes<FINITE>(d[i][2]), magnitudes<FINITE>(d[i][3])));
  }
  static __device__ __forceinline__ uint32_t halves_max(uint32_t w) { return umax(w & 0xFFFFu, w >> 16); }
  // the fp32 bits of a magnitude
  static __device__ __forceinline__ uint32_t to_f32(uint32_t m) {
    if constexpr (kF16) return __float_as_uint(static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(m))));
    else return m << 16;
  }
  // Largest magnitudes (of this thread): of a row, of all rows, of columns 2 q and 2 q + 1.
  template <bool FINITE>
  __device__ __forceinline__ uint32_t row_max(int i) const {
    return halves_max(row_word<FINITE>(i));
  }
  template <bool FINITE>
  __device__ __forceinline__ uint32_t all_max() const {
    uint32_t m = row_word<FINITE>(0);
#pragma unroll
    for (int i = 1; i < ROWS; ++i) m = umax2(m, row_word<FINITE>(i));
    return halves_max(m);
  }
  template <bool FINITE>
  __device__ __forceinline__ uint32_t col_word(int q) const {
    uint32_t m = magnitudes<FINITE>(d[0][q]);
#pragma unroll
    for (int i = 1; i < ROWS; ++i) m = umax2(m, magnitudes<FINITE>(d[i][q]));
    return m;
  }
  static __device__ __forceinline__ uint32_t col_across(uint32_t w) {
    return across_rows(w, [](uint32_t a, uint32_t b) { return umax2(a, b); });
  }
  static __device__ __forceinline__ uint32_t col_join(uint32_t a, uint32_t b) { return umax2(a, b); }
  // column j's magnitude in the words of 8 columns
  static __device__ __forceinline__ uint32_t col_of(const uint32_t* w, int j) {
    return (j & 1) ? w[j >> 1] >> 16 : w[j >> 1] & 0xFFFFu;
  }
  // Infinities become NaN.
  __device__ __forceinline__ void no_infinities() {
#pragma unroll
    for (int i = 0; i < ROWS; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t w = d[i][q];
        d[i][q] = ((w & 0x7FFFu) < kInf ? w & 0xFFFFu : 0x7FFFu) | ((w & 0x7FFF0000u) < (kInf << 16) ? w & 0xFFFF0000u : 0x7FFF0000u);
      }
  }
  // Two elements to the low or high half of a word of codes.
  template <bool HI>
  static __device__ __forceinline__ i16x2 two(i16x2 w, uint32_t pair, float s, bool e5m2) {
#if defined(__HIP_DEVICE_COMPILE__)
    if constexpr (kF16) {
      const f16x2 v = __builtin_bit_cast(f16x2, pair);
      return e5m2 ? __builtin_amdgcn_cvt_scalef32_pk_bf8_f16(w, v, s, HI) : __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(w, v, s, HI);
    } else {
      const bf16x2 v = __builtin_bit_cast(bf16x2, pair);
      return e5m2 ? __builtin_amdgcn_cvt_scalef32_pk_bf8_bf16(w, v, s, HI) : __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(w, v, s, HI);
    }
#else
    return w;
#endif
  }
  static __device__ __forceinline__ uint32_t four(uint32_t a, uint32_t b, float s, bool e5m2) {
    i16x2 w{};
    w = two<false>(w, a, s, e5m2);
    return __builtin_bit_cast(uint32_t, two<true>(w, b, s, e5m2));
  }
  __device__ __forceinline__ uint2 row_codes(int i, float s, bool e5m2) const {
    return make_uint2(four(d[i][0], d[i][1], s, e5m2), four(d[i][2], d[i][3], s, e5m2));
  }
  // column j's elements of rows i and i + 1
  __device__ __forceinline__ uint32_t pair(int i, int j) const {
    return __builtin_amdgcn_perm(d[i + 1][j >> 1], d[i][j >> 1], (j & 1) ? 0x07060302u : 0x05040100u);
  }
  __device__ __forceinline__ uint2 col_codes(int j, float s, bool e5m2) const {
    return make_uint2(four(pair(0, j), pair(2, j), s, e5m2), four(pair(4, j), pair(6, j), s, e5m2));
  }
};

// The same for fp32 elements.
template <int ROWS>
struct Part<kElemF32, ROWS> {
  static constexpr uint32_t kInf = 0x7F800000u;
  static constexpr int kColWords = 8;
  float d[ROWS][8];

  __device__ __forceinline__ void load(int i, const void* x, int64_t at) {
    __builtin_memcpy(d[i], static_cast<const float*>(x) + at, 32);
  }
  __device__ __forceinline__ void shift(int i, int shift, bool keep) {
    float* w = d[i];
#pragma unroll
    for (int by = 4; by > 0; by >>= 1) {
      const bool s = shift & by;
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = s ? (j + by < 8 ? w[j + by < 8 ? j + by : 7] : 0.0f) : w[j];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = keep ? w[j] : 0.0f;
  }
  __device__ __forceinline__ void set(int i, int j, const void* x, int64_t at, bool keep) {
    const float v = static_cast<const float*>(x)[at];
    d[i][j] = keep ? v : 0.0f;
  }
  template <bool FINITE>
  static __device__ __forceinline__ uint32_t magnitude(float v) {
    const uint32_t u = __float_as_uint(v) & 0x7FFFFFFFu;
    return !FINITE || u < kInf ? u : 0u;
  }
  static __device__ __forceinline__ uint32_t to_f32(uint32_t m) { return m; }
  template <bool FINITE>
  __device__ __forceinline__ uint32_t row_max(int i) const {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = umax(m, magnitude<FINITE>(d[i][j]));
    return m;
  }
  template <bool FINITE>
  __device__ __forceinline__ uint32_t all_max() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) m = umax(m, row_max<FINITE>(i));
    return m;
  }
  template <bool FINITE>
  __device__ __forceinline__ uint32_t col_word(int j) const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) m = umax(m, magnitude<FINITE>(d[i][j]));
    return m;
  }
  static __device__ __forceinline__ uint32_t col_across(uint32_t w) {
    return across_rows(w, [](uint32_t a, uint32_t b) { return umax(a, b); });
  }
  static __device__ __forceinline__ uint32_t col_join(uint32_t a, uint32_t b) { return umax(a, b); }
  static __device__ __forceinline__ uint32_t col_of(const uint32_t* w, int j) { return w[j]; }
  __device__ __forceinline__ void no_infinities() {
#pragma unroll
    for (int i = 0; i < ROWS; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (magnitude<false>(d[i][j]) >= kInf) d[i][j] = __uint_as_float(0x7FC00000u);
  }
  static __device__ __forceinline__ uint32_t four(float a, float b, float c, float e, float s, bool e5m2) {
    i16x2 w{};
#if defined(__HIP_DEVICE_COMPILE__)
    if (e5m2) {
      w = __builtin_amdgcn_cvt_scalef32_pk_bf8_f32(w, a, b, s, false);
      w = __builtin_amdgcn_cvt_scalef32_pk_bf8_f32(w, c, e, s, true);
    } else {
      w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, a, b, s, false);
      w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, c, e, s, true);
    }
#endif
    return __builtin_bit_cast(uint32_t, w);
  }
  __device__ __forceinline__ uint2 row_codes(int i, float s, bool e5m2) const {
    return make_uint2(four(d[i][0], d[i][1], d[i][2], d[i][3], s, e5m2), four(d[i][4], d[i][5], d[i][6], d[i][7], s, e5m2));
  }
  __device__ __forceinline__ uint2 col_codes(int j, float s, bool e5m2) const {
    return make_uint2(four(d[0][j], d[1][j], d[2][j], d[3][j], s, e5m2), four(d[4][j], d[5][j], d[6][j], d[7][j], s, e5m2));
  }
};

// Rows row .. + ROWS - 1, columns c .. c + 7 of X [R, C], zeros outside.  INSIDE: none is.
// Otherwise a row is read as the 8 elements that end with its last at the latest, and
// moved down; only matrices of fewer than 8 columns are read one by one.
template <bool INSIDE, typename Part, int ROWS>
__device__ __forceinline__ void load_rows(Part& v, const void* x, int64_t ldx, int64_t row, int64_t c, int64_t R, int64_t C) {
  if constexpr (INSIDE) {
#pragma unroll
    for (int i = 0; i < ROWS; ++i) v.load(i, x, (row + i) * ldx + c);
  } else if (C >= 8) {
    const int64_t from = c + 8 <= C ? c : C - 8;
    const int by = static_cast<int>(c - from);  // 8 and more: nothing of it is inside
#pragma unroll
    for (int i = 0; i < ROWS; ++i) v.load(i, x, (row + i < R ? row + i : R - 1) * ldx + from);
#pragma unroll
    for (int i = 0; i < ROWS; ++i) v.shift(i, by & 7, row + i < R && by < 8);
  } else {
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        v.set(i, j, x, (row + i < R ? row + i : R - 1) * ldx + (j < C ? j : C - 1), row + i < R && c == 0 && j < C);
      __builtin_amdgcn_sched_barrier(0);  // not all rows' loads at once: they would not fit the registers
    }
  }
}

// A scale per row and block, no transpose: unit u of a rank is row u / nb, block u % nb.
template <int X>
__global__ __launch_bounds__(kThreads) void echo_quant_rows_k(const QuantFp8Args a) {
  typedef Part<X, 1> P;
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
    P v;
    if (c + 8 <= a.C) load_rows<true, P, 1>(v, x, a.ldx, row, c, a.R, a.C);
    else load_rows<false, P, 1>(v, x, a.ldx, row, c, a.R, a.C);
    uint32_t m = row16_max(v.template row_max<false>(0));
    if (m >= P::kInf) {  // the block holds a value that is not finite
      m = row16_max(v.template row_max<true>(0));
      v.no_infinities();
    }
    const uint32_t sb = scale_byte(P::to_f32(m), e5m2);
    const int64_t left = a.C - c;
    if (left > 0) store_codes8(q + row * a.rows.ld + c, v.row_codes(0, scale_of(sb), e5m2), left < 8 ? static_cast<int>(left) : 8);
    if (l == 0) store_scale(sc, row * a.rows.srs + b * a.rows.sks, sb, a.e8m0 != 0);
  }
}

// A 128 x 128 tile; COLS: the transposed codes are wanted too (or only); B128: one
// scale for the tile; INSIDE: no row or column of it lies outside the matrix.
struct TileOf {
  const void* x;
  uint8_t *qr, *qc;
  void *sr, *sc;
  int64_t br, bc;
};
template <int X, bool COLS, bool B128, bool INSIDE>
__device__ __forceinline__ void quant_tile(const QuantFp8Args& a, const TileOf& o, uint8_t* tile,
                                           uint32_t (*part)[16 * Part<X, 8>::kColWords]) {
  typedef Part<X, 8> P;
  constexpr int kWords = P::kColWords;
  const int64_t br = o.br, bc = o.bc;
  uint8_t *const qr = o.qr, *const qc = o.qc;
  void *const sr = o.sr, *const sc = o.sc;
  const bool e5m2 = a.e5m2 != 0, e8m0 = a.e8m0 != 0;
  const int t = threadIdx.x, cg = t & 15, rg = t >> 4, wave = t >> 6;
  const int64_t row0 = br * kFp8Block + 8 * rg, col0 = bc * kFp8Block + 8 * cg;
  P v;
  load_rows<INSIDE, P, 8>(v, o.x, a.ldx, row0, col0, a.R, a.C);

  // The maxima, of what counts: with a value that is not finite anywhere in the tile,
  // the whole workgroup takes them again without such values.
  uint32_t row_max[8], col_max[kWords], all = 0;
  const auto maxima = [&](auto finite) {
    constexpr bool FINITE = decltype(finite)::value;
    if constexpr (B128) {
      all = v.template all_max<FINITE>();
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) row_max[i] = v.template row_max<FINITE>(i);
      if constexpr (COLS) {
#pragma unroll
        for (int q = 0; q < kWords; ++q) col_max[q] = v.template col_word<FINITE>(q);
      }
    }
  };
  maxima(std::false_type{});
  if constexpr (!B128) {
#pragma unroll
    for (int i = 0; i < 8; ++i) all = umax(all, row_max[i]);
  }
  if (__syncthreads_or(all >= P::kInf)) {
    maxima(std::true_type{});
    v.no_infinities();
  }

  uint32_t tile_byte = 0;
  if constexpr (B128) {
    const uint32_t m = across_rows(row16_max(all), [](uint32_t p, uint32_t q) { return umax(p, q); });
    if ((t & 63) == 0) part[wave][0] = m;
    __syncthreads();
    tile_byte = scale_byte(P::to_f32(umax(umax(part[0][0], part[1][0]), umax(part[2][0], part[3][0]))), e5m2);
    if (t == 0) {
      if (qr != nullptr) store_scale(sr, br * a.rows.srs + bc * a.rows.sks, tile_byte, e8m0);
      if (qc != nullptr) store_scale(sc, bc * a.cols.srs + br * a.cols.sks, tile_byte, e8m0);
    }
  } else if constexpr (COLS) {
#pragma unroll
    for (int q = 0; q < kWords; ++q) {
      col_max[q] = P::col_across(col_max[q]);
      if ((t & 63) < 16) part[wave][kWords * cg + q] = col_max[q];
    }
  }
  if (qr != nullptr) {
    const int left = INSIDE || a.C - col0 >= 8 ? 8 : static_cast<int>(a.C - col0);
    uint32_t mine = 0;  // lane cg < 8 of the 16 keeps row cg's scale
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t sb = tile_byte;
      if constexpr (!B128) sb = scale_byte(P::to_f32(row16_max(row_max[i])), e5m2);
      if (cg == i) mine = sb;
      const uint2 w = v.row_codes(i, scale_of(sb), e5m2);
      uint8_t* const p = qr + (row0 + i) * a.rows.ld + col0;
      if (INSIDE && a.stream) __builtin_nontemporal_store(__builtin_bit_cast(u32x2, w), reinterpret_cast<u32x2*>(p));
      else if (INSIDE || (row0 + i < a.R && left > 0)) store_codes8(p, w, left);
    }
    if (!B128 && cg < 8 && (INSIDE || row0 + cg < a.R)) store_scale(sr, (row0 + cg) * a.rows.srs + bc * a.rows.sks, mine, e8m0);
  }
  if constexpr (COLS) {
    uint32_t words[kWords];
    if constexpr (!B128) {
      __syncthreads();
#pragma unroll
      for (int q = 0; q < kWords; ++q) {
        const int c = kWords * cg + q;
        words[q] = P::col_join(P::col_join(part[0][c], part[1][c]), P::col_join(part[2][c], part[3][c]));
      }
    }
    // column 8 cg + j of the tile: 128 bytes of codes, 8-byte chunk rg (this thread's
    // rows) at slot rg ^ cg
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      uint32_t sb = tile_byte;
      if constexpr (!B128) {
        sb = scale_byte(P::to_f32(P::col_of(words, j)), e5m2);
        if (rg == j && (INSIDE || col0 + j < a.C)) store_scale(sc, (col0 + j) * a.cols.srs + br * a.cols.sks, sb, e8m0);
      }
      *reinterpret_cast<uint2*>(tile + (8 * cg + j) * 128 + 8 * (rg ^ cg)) = v.col_codes(j, scale_of(sb), e5m2);
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
      if (INSIDE || (col < a.C && left > 0)) {
        uint8_t* p = qc + col * a.cols.ld + row;
        if (INSIDE || left >= 16) {
          *reinterpret_cast<uint4*>(p) = make_uint4(lo.x, lo.y, hi.x, hi.y);
        } else {
          store_codes8(p, lo, static_cast<int>(left));
          if (left > 8) store_codes8(p + 8, hi, static_cast<int>(left - 8));
        }
      }
    }
  }
}

template <int X, bool COLS, bool B128>
__global__ __launch_bounds__(kThreads) void echo_quant_tile_k(const QuantFp8Args a) {
  __shared__ __attribute__((aligned(16))) uint8_t tile[COLS ? 128 * 128 : 16];
  __shared__ __attribute__((aligned(16))) uint32_t part[4][16 * Part<X, 8>::kColWords];  // per wavefront: maxima
  const int64_t nbc = (a.C + kFp8Block - 1) / kFp8Block, nbr = (a.R + kFp8Block - 1) / kFp8Block;
  const uint32_t per = static_cast<uint32_t>(nbc * nbr);
  // The hardware hands workgroups to the eight XCDs in turn: of every 16, an XCD gets two
  // tiles that lie side by side, so that one L2 holds 256 bytes of a row's codes.
  const uint32_t i = blockIdx.x, id = (i | 15) < gridDim.x ? (i & ~15u) + 2 * (i & 7) + ((i >> 3) & 1) : i;
  const uint32_t r = id / per, at = id - r * per;
  const int64_t br = at / static_cast<uint32_t>(nbc), bc = at - br * nbc;
  const auto* k = kernel_args<QuantFp8Args>();
  const TileOf o{k->X[r], k->rows.codes[r], k->cols.codes[r], k->rows.scales[r], k->cols.scales[r], br, bc};
  if ((br + 1) * kFp8Block <= a.R && (bc + 1) * kFp8Block <= a.C) quant_tile<X, COLS, B128, true>(a, o, tile, part);
  else quant_tile<X, COLS, B128, false>(a, o, tile, part);
}

// A call that reads and writes more than the 256 MB last-level cache leaves nothing useful
// in it: the codes along the rows, in pieces of 128 bytes, then go past the caches.
// With the products that read them next, us: 8192 x 8192 bfloat16 both ways 54.7 against
// 56.4 (169 against 174 with both products), 16384 x 16384 215 against 219 (447 against
// 456); in a smaller call the product would miss them: 2048 x 4096 9.8 against 10.9, but
// 50.1 against 45.8 with one product.  (The codes along the columns: slower from 16384 x
// 16384 on, 243 against 219.)
constexpr int64_t kCache = int64_t{1} << 28;

template <int X>
hipError_t launch(const QuantFp8Args& given, int P, bool block128, hipStream_t s) {
  const int64_t nbc = (given.C + kFp8Block - 1) / kFp8Block, nbr = (given.R + kFp8Block - 1) / kFp8Block;
  const bool cols = given.cols.codes[0] != nullptr;
  if (!cols && !block128 && P * nbc * nbr < 512) {
    const int64_t blocks = (given.R * nbc + kThreads / 16 - 1) / (kThreads / 16);
    const dim3 grid(static_cast<unsigned>(blocks < (1 << 20) ? blocks : (1 << 20)), static_cast<unsigned>(P));
    hipLaunchKernelGGL((echo_quant_rows_k<X>), grid, dim3(kThreads), 0, s, given);
    return hipGetLastError();
  }
  const dim3 grid(static_cast<unsigned>(P * nbc * nbr));
  QuantFp8Args a = given;
  const int64_t per = (X == kElemF32 ? 4 : 2) + (a.rows.codes[0] != nullptr) + cols;
  a.stream = P * a.R * a.C * per >= kCache;
  if (cols && block128)
    hipLaunchKernelGGL((echo_quant_tile_k<X, true, true>), grid, dim3(kThreads), 0, s, a);
  else if (cols)
    hipLaunchKernelGGL((echo_quant_tile_k<X, true, false>), grid, dim3(kThreads), 0, s, a);
  else if (!block128)
    hipLaunchKernelGGL((echo_quant_tile_k<X, false, false>), grid, dim3(kThreads), 0, s, a);
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
