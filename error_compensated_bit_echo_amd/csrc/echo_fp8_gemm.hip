// The product of matrices in 8-bit floating point with a scale per 128 elements of
// k, on the matrix cores: out[m, n] = sum_b sA[m, b] sW[n, b] sum_{k in b} A[m, k] W[n, k].
//
// Two ways to a block's sum.
//   * The 8-bit instruction v_mfma_scale_f32_32x32x64_f8f6f4, with exponent-byte
//     scales applied by the instruction itself.  It aligns the products of each run
//     of 8 consecutive k to the largest of them and drops what lies below 2^-13 of it
//     (measured: 1.5e-5 of the result for normal e4m3 data, whatever K), so it serves
//     outputs of 16 bits, whose own rounding is 2^-9 or 2^-12.
//   * Codes widened to bfloat16, which holds every value of both formats, and
//     v_mfma_f32_32x32x16_bf16, whose fp32 sums are precise (measured 6e-9 per
//     block), at half the rate: fp32 outputs.
// The product is computed transposed (W supplies the instruction's first operand),
// so a lane holds runs of four consecutive columns n of one row m.
#pragma clang fp contract(off)

#include <type_traits>

#include "echo_elem.h"
#include "echo_slab.h"

namespace echo {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// 8 codes (two dwords), times a power of two, as bfloat16: exact where the product is
// a normal bfloat16.
template <bool E5>
__device__ __forceinline__ bf16x8 widen8(int lo, int hi, float scale = 1.0f) {
  bf16x8 x{};
#if defined(__HIP_DEVICE_COMPILE__)
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t w = static_cast<uint32_t>(i ? hi : lo);
    const bf16x2 p = E5 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w, scale, false)
                        : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, false);
    const bf16x2 q = E5 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8(w, scale, true)
                        : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, true);
    x[4 * i] = p[0];
    x[4 * i + 1] = p[1];
    x[4 * i + 2] = q[0];
    x[4 * i + 3] = q[1];
  }
#endif
  return x;
}

// A scale's bits: fp32 bits, or the exponent byte.
template <bool E8>
__device__ __forceinline__ uint32_t scale_bits(const void* s, int64_t at) {
  if constexpr (E8) return static_cast<const uint8_t*>(s)[at];
  else return static_cast<const uint32_t*>(s)[at];
}
// ... and its value in fp32 (exponent byte 0 is 2^-127, subnormal, and 255 NaN).
template <bool E8>
__device__ __forceinline__ float scale_value(uint32_t b) {
  if constexpr (E8) return __uint_as_float(b == 255 ? 0x7FC00000u : b == 0 ? 0x00400000u : b << 23);
  else return __uint_as_float(b);
}

struct RankPtrs {
  const uint8_t *A, *W;
  const void *sA, *sW;
  void* out;
};
__device__ __forceinline__ RankPtrs rank_ptrs(int r) {
  const auto* k = kernel_args<GemmFp8Args>();
  return RankPtrs{k->A[r], k->W[r], k->sA[r], k->sW[r], k->out[r]};
}

// Stores n (at most 4) consecutive columns of a row one by one.
__device__ __forceinline__ void store_each(void* out, int64_t at, int64_t left, const float* v, int n, int elem) {
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (e < n && e < left) {
      if (elem == kElemF32) store1<kElemF32>(out, at + e, v[e]);
      else if (elem == kElemBf16) store1<kElemBf16>(out, at + e, v[e]);
      else store1<kElemF16>(out, at + e, v[e]);
    }
}

// ---- few rows of A -------------------------------------------------------------
//
// 16 CT columns of the output (rows of W) per workgroup of NW wavefronts, which share
// k: wavefront w takes the blocks w, w + NW, ... of 128 and reads its codes of W and A
// straight from memory (W is read once in all), and the sums meet in LDS in a fixed
// order.  Codes are widened to bfloat16 (the matrix cores idle anyway); exponent-byte
// scales are applied as they are widened.  One token against N = K = 8192: the kernel takes
// 14.9 us (16.0 over weights that no cache holds), 4.5 TB/s of codes, where reading alone
// reaches 7.1; from call to call 14.5, so the launch is hidden behind the kernel before it.
// The wavefronts wait for 53 % of their cycles: each has two rounds of loads, the second
// issued when the first has been multiplied.

// A lane's 32 bytes of a block of 128: 16-byte chunks g and g + 4, so that the four
// lanes of a row read 64 contiguous bytes at a time.  TAIL: the block is cut off by K,
// and reads as zeros from there.  (The 16-byte runs that hold a valid byte lie within
// the row's pitch, a multiple of 16.)
template <bool TAIL>
__device__ __forceinline__ i32x8 load_frag(const uint8_t* block, int g, int left) {
  i32x4 x[2] = {};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int at = 16 * (g + 4 * h);
    if constexpr (!TAIL) {
      x[h] = *reinterpret_cast<const i32x4*>(block + at);
    } else if (at < left) {
      x[h] = *reinterpret_cast<const i32x4*>(block + at);
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        const int n = left - at - 4 * d;  // valid bytes of this dword
        if (n <= 0) x[h][d] = 0;
        else if (n < 4) x[h][d] &= (1 << (8 * n)) - 1;
      }
    }
  }
  return __builtin_shufflevector(x[0], x[1], 0, 1, 2, 3, 4, 5, 6, 7);
}

// MT tiles of 16 rows of A, CT of 16 rows of W; U blocks' loads go out at a time.
// WB: fp32 scales of blocks of 128 rows of W, one for a tile's 16 columns.
template <int MT, int CT, int U, int NW, bool WB, bool A5, bool W5, bool E8>
__global__ __launch_bounds__(64 * NW) void echo_gemm_fp8_thin_k(const GemmFp8Args a) {
  __shared__ f32x4 part[NW][MT][CT][64];
  const RankPtrs p = rank_ptrs(blockIdx.z);
  const int lane = threadIdx.x & 63, sub = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m0 = static_cast<int>(blockIdx.y) * (16 * MT), n0 = static_cast<int>(blockIdx.x) * (16 * CT);
  const int M = static_cast<int>(a.M), N = static_cast<int>(a.N), K = static_cast<int>(a.K);
  // The rows this lane supplies, clamped (what lies past the edge is not stored), and
  // where their scales are: with exponent bytes those of the same rows, with fp32 scales
  // W's of the four columns the lane holds.
  constexpr int kScalesW = E8 || WB ? 1 : 4;
  const uint8_t *rowA[MT], *rowW[CT];
  uint32_t sa[MT], sw[CT][kScalesW];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int m = m0 + 16 * i + sub < M ? m0 + 16 * i + sub : M - 1;
    rowA[i] = p.A + m * a.lda;
    sa[i] = static_cast<uint32_t>((m >> a.sa_shift) * a.sa_row);
  }
#pragma unroll
  for (int j = 0; j < CT; ++j) {
    const int n = n0 + 16 * j + sub < N ? n0 + 16 * j + sub : N - 1;
    rowW[j] = p.W + n * a.ldw;
#pragma unroll
    for (int v = 0; v < kScalesW; ++v) {
      const int c = E8 ? n : n0 + 16 * j + 4 * g + v < N ? n0 + 16 * j + 4 * g + v : N - 1;
      sw[j][v] = static_cast<uint32_t>((c >> a.sw_shift) * a.sw_row);
    }
  }
  f32x4 acc[MT][CT] = {};
  struct Block {
    i32x8 fa[MT], fw[CT];
    uint32_t ca[MT], cw[CT][kScalesW];
  };
  auto load = [&](Block& x, int b, auto tail) {
    constexpr bool TAIL = decltype(tail)::value;
    const int left = K - b * kFp8Block;
#pragma unroll
    for (int j = 0; j < CT; ++j) x.fw[j] = load_frag<TAIL>(rowW[j] + b * kFp8Block, g, left);
#pragma unroll
    for (int i = 0; i < MT; ++i) x.fa[i] = load_frag<TAIL>(rowA[i] + b * kFp8Block, g, left);
    constexpr int kBytes = E8 ? 1 : 4;
    const uint8_t* const pa = static_cast<const uint8_t*>(p.sA) + b * a.sa_k * kBytes;
    const uint8_t* const pw = static_cast<const uint8_t*>(p.sW) + b * a.sw_k * kBytes;
#pragma unroll
    for (int i = 0; i < MT; ++i) x.ca[i] = scale_bits<E8>(pa, sa[i]);
#pragma unroll
    for (int j = 0; j < CT; ++j)
#pragma unroll
      for (int v = 0; v < kScalesW; ++v) x.cw[j][v] = scale_bits<E8>(pw, sw[j][v]);
  };
  auto multiply = [&](const Block& x) {
    f32x4 t[MT][CT] = {};
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      bf16x8 wa[CT];
#pragma unroll
      for (int j = 0; j < CT; ++j)
        wa[j] = widen8<W5>(x.fw[j][2 * s], x.fw[j][2 * s + 1], E8 ? scale_value<E8>(x.cw[j][0]) : 1.0f);
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const bf16x8 aa = widen8<A5>(x.fa[i][2 * s], x.fa[i][2 * s + 1], E8 ? scale_value<E8>(x.ca[i]) : 1.0f);
#if defined(__HIP_DEVICE_COMPILE__)
#pragma unroll
        for (int j = 0; j < CT; ++j) {
          f32x4& c = E8 ? acc[i][j] : t[i][j];
          c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wa[j], aa, c, 0, 0, 0);
        }
#endif
      }
    }
    if constexpr (!E8) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < CT; ++j)
#pragma unroll
          for (int v = 0; v < 4; ++v)
            acc[i][j][v] = __builtin_fmaf(t[i][j][v], __uint_as_float(x.ca[i]) * __uint_as_float(x.cw[j][WB ? 0 : v]),
                                          acc[i][j][v]);
    }
  };
  const int full = K / kFp8Block;
  int b = wave;
  for (; b + (U - 1) * NW < full; b += U * NW) {
    Block x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) load(x[u], b + u * NW, std::false_type{});
#pragma unroll
    for (int u = 0; u < U; ++u) multiply(x[u]);
  }
  for (; b < full; b += NW) {
    Block x;
    load(x, b, std::false_type{});
    multiply(x);
  }
  if (b == full && K % kFp8Block != 0) {
    Block x;
    load(x, b, std::true_type{});
    multiply(x);
  }
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < CT; ++j) part[wave][i][j][lane] = acc[i][j];
  __syncthreads();
  // wavefront w sums and writes the sub-tiles w, w + NW, ...
  for (int u = wave; u < MT * CT; u += NW) {
    const int i = u / CT, j = u - i * CT;
    f32x4 s = part[0][i][j][lane];
#pragma unroll
    for (int w = 1; w < NW; ++w) {
      const f32x4 x = part[w][i][j][lane];
#pragma unroll
      for (int v = 0; v < 4; ++v) s[v] = s[v] + x[v];
    }
    const int mm = m0 + 16 * i + sub, nn = n0 + 16 * j + 4 * g;
    if (mm < M) {
      const float v[4] = {s[0], s[1], s[2], s[3]};
      store_each(p.out, mm * a.ldo + nn, N - nn, v, 4, a.out_elem);
    }
  }
}

// The product over nothing: zeros.
__global__ __launch_bounds__(256) void echo_gemm_fp8_zero_k(const GemmFp8Args a) {
  const RankPtrs p = rank_ptrs(blockIdx.z);
  for (int64_t m = blockIdx.y; m < a.M; m += gridDim.y)
    for (int64_t n = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; n < a.N; n += static_cast<int64_t>(gridDim.x) * 256) {
      if (a.out_elem == kElemF32) store1<kElemF32>(p.out, m * a.ldo + n, 0.0f);
      else store1<kElemBf16>(p.out, m * a.ldo + n, 0.0f);  // the same bits in fp16
    }
}

// ---- tiles through LDS -----------------------------------------------------------
//
// A workgroup of WM x WN wavefronts computes a BM x BN tile, each wavefront BM / WM
// rows and BN / WN columns in 32 x 32 sub-tiles.  k advances one block of 128 (128
// bytes of each row) at a time through a ring of S LDS slabs, filled straight from
// memory while earlier slabs are multiplied; each K step needs one barrier.  16-byte
// chunk c of row r lies at slot c ^ ((r / 2) % 8) of its 128-byte row, so a fragment
// read covers all LDS banks.  Lane l supplies row l % 32 of a sub-tile and the bytes
// 64 (l / 32) .. + 63 of the K step: which k a lane and instruction covers does not
// matter, as both operands use the same assignment and a scale covers all 128.
// Accumulator v of lane l is row l % 32 of the tile's A rows and column
// 8 (v / 4) + 4 (l / 32) + v % 4 of its W rows.
// The scales of a K step's rows are staged in LDS by one load per thread, a step
// ahead, in a ring of three (a wavefront may still read step it's while another
// writes step it + 2's).
// Rows past the edge read as zeros (the buffer resources end with the matrix), and
// so does what lies past K in the last step: 16-byte chunks by an offset out of
// range, the bytes behind K in the last chunk by one pass over the slab.
// Measured: M = N = K = 8192 402 us (2.74 PFLOP/s; the library's product without block
// scales 339) and, with fp32 outputs, 738 (1.49; the library's bfloat16 product reaches
// 1.44); P = 4, M = 2048, N = K = 4096 108-125 us on three machines (2.2-2.5).  The matrix
// cores are busy 74 % of the CUs' busy cycles at 8192 (80 % with fp32 outputs) and 67 % at
// the shorter k, where a tile's first loads and its store weigh more; the clock falls to
// 1.7 GHz at 8192 and 1.9 at the shorter k.

// An offset past the end of every buffer resource here (they stay below 2^31 bytes).
constexpr uint32_t kPastEnd = 0x80000000u;

// Which tile a workgroup takes.  The hardware hands the workgroups of a launch to the
// eight XCDs in turn, and each XCD has its own L2: workgroup i takes a tile of the
// (i % 8)-th contiguous run, and tiles are ordered in bands of 8 row tiles, so the
// tiles an XCD works on at a time share their panels of A and of W.
struct TileAt {
  int rank, m0, n0;
};
template <int BM, int BN>
__device__ __forceinline__ TileAt tile_at(uint32_t gm, uint32_t gn) {
  const uint32_t T = gridDim.x, x = blockIdx.x % 8, q = T / 8, rem = T % 8;
  uint32_t id = x * q + (x < rem ? x : rem) + blockIdx.x / 8;
  const uint32_t rank = id / (gm * gn);
  id -= rank * gm * gn;
  const uint32_t band = id / (8 * gn), in_band = id - band * 8 * gn;
  const uint32_t high = gm - 8 * band < 8 ? gm - 8 * band : 8;  // row tiles of this band
  return TileAt{static_cast<int>(rank), static_cast<int>(8 * band + in_band % high) * BM,
                static_cast<int>(in_band / high) * BN};
}

// The slabs and scales of a tile's K steps.  BYTES: scales are staged as exponent
// bytes, else as fp32.  G: groups of NW wavefronts that share k, each with slabs of its
// own: step `it` of group g is block G it + g, and all groups take as many steps (past
// the last block they multiply zeros).
template <int BM, int BN, int NW, int S, int G, bool BYTES, bool E8>
struct Slabs {
  static constexpr int kThreads = 64 * NW;
  static constexpr int JA = BM / (8 * NW), JW = BN / (8 * NW), kLoads = JA + JW;  // 1 KiB slab blocks per wavefront
  static constexpr int kSlabA = BM * 128, kSlab = (BM + BN) * 128;
  static constexpr int kPer = (BM + BN + kThreads - 1) / kThreads;  // scales per thread
  static constexpr int kRows = kPer * kThreads;                     // rows with a scale, rounded up to whole threads
  static constexpr int kBytes = S * kSlab + 3 * 4 * kRows;          // of a group
  static_assert(JA * 8 * NW == BM && JW * 8 * NW == BN, "slab blocks split evenly");
  static_assert(BM % 64 == 0 && BN % 64 == 0, "a wavefront stages scales of one operand");

  // One array for slabs and scales: with two, the compiler tells the accesses of each
  // apart and then waits for every load into LDS before the next fragment read.
  uint8_t* lds;
  BufRsrc rA, rW;
  uint32_t offA[JA], offW[JW];
  const uint8_t* sp[kPer];
  int64_t sk[kPer];
  uint32_t sreg[kPer];
  int K, K16, blocks, steps, t, lane, wave, group, sblock;

  __device__ __forceinline__ int chunk_of(int row) const { return (lane & 7) ^ ((row >> 1) & 7); }
  __device__ __forceinline__ uint32_t* scales(int ring) const {
    return reinterpret_cast<uint32_t*>(lds + S * kSlab) + ring * kRows;
  }

  __device__ __forceinline__ void init(uint8_t* l, const GemmFp8Args& a, const RankPtrs& p, const TileAt& at) {
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    group = G == 1 ? 0 : wave / NW;
    wave -= group * NW;
    lds = l + group * kBytes;
    t = threadIdx.x - group * kThreads;
    lane = t & 63;
    K = static_cast<int>(a.K);
    K16 = (K + 15) / 16 * 16;
    blocks = (K + 127) / 128;
    steps = (blocks + G - 1) / G;
    sblock = group;
    const int M = static_cast<int>(a.M), N = static_cast<int>(a.N);
    const int rows_a = M - at.m0 < BM ? M - at.m0 : BM, rows_w = N - at.n0 < BN ? N - at.n0 : BN;
    rA = buffer_rsrc(p.A + at.m0 * a.lda, static_cast<int32_t>((rows_a - 1) * a.lda + K16));
    rW = buffer_rsrc(p.W + at.n0 * a.ldw, static_cast<int32_t>((rows_w - 1) * a.ldw + K16));
    // Lane l fills slot l of each 1 KiB block: row 8 i + l / 8, slot l % 8.
#pragma unroll
    for (int j = 0; j < JA; ++j) {
      const int row = 8 * (JA * wave + j) + (lane >> 3);
      offA[j] = static_cast<uint32_t>(row * static_cast<int>(a.lda) + 16 * chunk_of(row));
    }
#pragma unroll
    for (int j = 0; j < JW; ++j) {
      const int row = 8 * (JW * wave + j) + (lane >> 3);
      offW[j] = static_cast<uint32_t>(row * static_cast<int>(a.ldw) + 16 * chunk_of(row));
    }
    // Thread t stages the scales of rows t, t + kThreads, ... of A's then W's.
    constexpr int kScaleBytes = E8 ? 1 : 4;
#pragma unroll
    for (int u = 0; u < kPer; ++u) {
      const bool of_a = 64 * (wave + u * NW) < BM;
      int i = t + u * kThreads + (of_a ? at.m0 : at.n0 - BM);
      const int end = of_a ? M : N;
      i = i < end ? i : end - 1;  // past the edge: any scale does
      sp[u] = static_cast<const uint8_t*>(of_a ? p.sA : p.sW) +
              (of_a ? (i >> a.sa_shift) * a.sa_row : (i >> a.sw_shift) * a.sw_row) * kScaleBytes;
      sk[u] = (of_a ? a.sa_k : a.sw_k) * kScaleBytes;
    }
  }

  // The loads of K step `it` into slab `buf`.  LAST: of the last step, whose chunks
  // past K16 read as zeros.
  template <bool LAST>
  __device__ __forceinline__ void issue(int buf, int it) {
    uint8_t* As = lds + buf * kSlab + 1024 * JA * wave;
    uint8_t* Ws = lds + buf * kSlab + kSlabA + 1024 * JW * wave;
    int from = (it * G + group) * 128;
    const int chunks = (K16 - from) / 16;
    if constexpr (G > 1 && LAST) from = chunks > 0 ? from : 0;  // past K: every chunk is out of range by itself
#pragma unroll
    for (int j = 0; j < JA; ++j) {
      uint32_t off = offA[j];
      if constexpr (LAST) off = chunk_of(8 * (JA * wave + j) + (lane >> 3)) < chunks ? off : kPastEnd;
      buffer_load_lds16<0>(rA, As + 1024 * j, off, static_cast<uint32_t>(from));
    }
#pragma unroll
    for (int j = 0; j < JW; ++j) {
      uint32_t off = offW[j];
      if constexpr (LAST) off = chunk_of(8 * (JW * wave + j) + (lane >> 3)) < chunks ? off : kPastEnd;
      buffer_load_lds16<0>(rW, Ws + 1024 * j, off, static_cast<uint32_t>(from));
    }
  }

  __device__ __forceinline__ void load_scales() {  // the next K step's
    const int b = G == 1 || sblock < blocks ? sblock : blocks - 1;  // past the last block: not used
#pragma unroll
    for (int u = 0; u < kPer; ++u) sreg[u] = scale_bits<E8>(sp[u] + b * sk[u], 0);
    sblock += G;
  }
  // The scales of step `it`.  Past the last block they are zeros too: the products there
  // are, and an infinite scale would make NaN of them.
  __device__ __forceinline__ void stage_scales(int ring, int it, const uint32_t* from) {
    const bool past = G > 1 && it * G + group >= blocks;
#pragma unroll
    for (int u = 0; u < kPer; ++u)
      scales(ring)[t + u * kThreads] = past ? 0u : BYTES ? from[u] : __float_as_uint(scale_value<E8>(from[u]));
  }

  // Zeros behind K in the last chunk of the last slab, on both sides (a NaN there
  // would survive a product with zero).
  __device__ __forceinline__ void clear_tail(int buf) {
    const int c = K % 128 / 16, n = K % 16;
    for (int row = (blocks - 1) % G == group ? t : BM + BN; row < BM + BN; row += kThreads) {
      const int in = row < BM ? row : row - BM;
      uint8_t* b = lds + buf * kSlab + row * 128 + 16 * (c ^ ((in >> 1) & 7));
      for (int i = n; i < 16; ++i) b[i] = 0;
    }
    __syncthreads();
  }

  // Step 0's scales staged, step 1's on their way, the loads of the first S steps out and
  // the first slab landed.
  __device__ __forceinline__ void start() {
    uint32_t first[kPer];  // staged once everything is on its way
    load_scales();
#pragma unroll
    for (int u = 0; u < kPer; ++u) first[u] = sreg[u];
    if (steps > 1) load_scales();
    for (int s = 0; s < S && s < steps; ++s) {
      if (s + 1 < steps) issue<false>(s, s);
      else issue<true>(s, s);
    }
    stage_scales(0, 0, first);
    if (steps >= S)
      __builtin_amdgcn_s_waitcnt(vmcnt_at_most_lds_drained((S - 1) * kLoads));
    else
      __builtin_amdgcn_s_waitcnt(vmcnt_at_most_lds_drained(0));
    slab_barrier();
    if (steps == 1 && K % 16 != 0) clear_tail(0);
  }

  // Between the reads of step it's slab `cur` and those of the next one `next`: the next
  // step's scales are staged, this wavefront's reads are done, the next slab has landed,
  // and the barrier; then slab `cur` is free and the loads of step it + S go out into
  // it (ISSUE 1; 2: they are the last step's; 0: none are left), so a slab has S - 1
  // whole steps to arrive.  The scales of step it + 2 are loaded before them: waiting
  // for those waits for everything issued earlier.
  template <int ISSUE>
  __device__ __forceinline__ void wait_next(int it, int next, int ring1) {
    stage_scales(ring1, it + 1, sreg);
    __builtin_amdgcn_s_waitcnt(vmcnt_at_most_lds_drained(ISSUE != 0 ? (S - 2) * kLoads : 0));
    __builtin_amdgcn_sched_barrier(0);
    slab_barrier();
    if constexpr (ISSUE == 0) {
      if (it + 2 == steps && K % 16 != 0) clear_tail(next);
      if (it + 2 < steps) load_scales();
    } else {
      load_scales();
    }
  }
  template <int ISSUE>
  __device__ __forceinline__ void refill(int it, int cur) {
    if constexpr (ISSUE == 1) issue<false>(cur, it + S);
    if constexpr (ISSUE == 2) issue<true>(cur, it + S);
  }

  // Runs step(it, ISSUE, LAST) for every K step.  The steps of the main loop contain no
  // branch: the compiler would move a step's instructions past it, behind the barrier.
  template <typename Step>
  __device__ __forceinline__ void run(Step step) {
    int it = 0;
    for (; it < steps - S - 1; ++it) step(it, std::integral_constant<int, 1>{}, std::false_type{});
    if (it == steps - S - 1) step(it++, std::integral_constant<int, 2>{}, std::false_type{});
    for (; it < steps - 1; ++it) step(it, std::integral_constant<int, 0>{}, std::false_type{});
    step(it, std::integral_constant<int, 0>{}, std::true_type{});
  }
};

// Adds the groups' accumulators (N runs of four per lane) in group 0, in a fixed order:
// the others leave theirs in their own part of LDS.  False: this wavefront is done.
template <typename SL, int G, int N>
__device__ __forceinline__ bool join_groups(uint8_t* lds, const SL& sl, f32x4 (&acc)[N]) {
  static_assert(SL::kThreads * N * 16 <= SL::kBytes, "a group's accumulators fit its part of LDS");
  if (sl.group != 0) {
    f32x4* mine = reinterpret_cast<f32x4*>(lds + sl.group * SL::kBytes) + sl.wave * (64 * N) + sl.lane;
#pragma unroll
    for (int i = 0; i < N; ++i) mine[64 * i] = acc[i];
  }
  __syncthreads();
  if (sl.group != 0) return false;
#pragma unroll
  for (int g = 1; g < G; ++g) {
    const f32x4* theirs = reinterpret_cast<const f32x4*>(lds + g * SL::kBytes) + sl.wave * (64 * N) + sl.lane;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int v = 0; v < 4; ++v) acc[i][v] = acc[i][v] + theirs[64 * i][v];
  }
  return true;
}

// Writes RW x CW of the tile out of a wavefront's registers, 32 rows at a time, through
// its own region of LDS (the slabs are free once every wavefront is here): `put(region,
// pitch, i)` lays rows 32 i .. 32 i + 31 out row-major, and they come back as 16 bytes
// of a row per lane, so the stores cover whole lines.  (Straight from the
// accumulators, in 32-byte pieces, the stores of a 256 x 256 tile on every CU took
// 10 us.)
template <int E, int RW, int CW, int REGION, typename Put>
__device__ __forceinline__ void store_tile(uint8_t* region, const GemmFp8Args& a, void* out, int row0, int col0, Put put) {
  typedef typename ElemOf<E>::T T;
  constexpr int kPitch = CW * sizeof(T) + 16, kPerLane = 16 / sizeof(T);
  static_assert(32 * kPitch <= REGION, "a region of LDS per wavefront");
  constexpr int kLanes = CW / kPerLane, kStep = 64 / kLanes;  // lanes per row, rows per instruction
  const int lane = threadIdx.x & 63, sr = lane / kLanes, scol = lane % kLanes * kPerLane;
  const int n = col0 + scol, M = static_cast<int>(a.M), N = static_cast<int>(a.N);
#pragma unroll
  for (int i = 0; i < RW / 32; ++i) {
    put(region, kPitch, i);
    T* row = static_cast<T*>(out) + (row0 + 32 * i + sr) * a.ldo + n;
#pragma unroll
    for (int u = 0; u < 32 / kStep; ++u) {
      const u32x4 o = *reinterpret_cast<const u32x4*>(region + (sr + u * kStep) * kPitch + scol * sizeof(T));
      if (row0 + 32 * i + sr + u * kStep < M) {
        if (n + kPerLane <= N) {
          __builtin_memcpy(row, &o, 16);
        } else {
          T each[kPerLane];
          __builtin_memcpy(each, &o, 16);
#pragma unroll
          for (int e = 0; e < kPerLane; ++e)
            if (n + e < N) row[e] = each[e];
        }
      }
      row += kStep * a.ldo;
    }
  }
}

// Four values to consecutive elements of a row in LDS.
template <int E>
__device__ __forceinline__ void put4(uint8_t* at, float a, float b, float c, float d) {
  typedef typename ElemOf<E>::T T4 __attribute__((ext_vector_type(4)));
  *reinterpret_cast<T4*>(at) = T4{narrow<E>(a), narrow<E>(b), narrow<E>(c), narrow<E>(d)};
}

enum TileMode {
  kScaled8 = 0,     // the 8-bit instruction applies exponent-byte scales
  kWide = 1,        // bfloat16, a block's sum scaled in fp32
  kWideScaled = 2,  // bfloat16, exponent-byte scales applied as the codes are widened
};

// 32 x 32 sub-tiles.  Lane l supplies row l % 32 of a sub-tile and the bytes
// 64 (l / 32) .. + 63 of the K step, in two half steps.  Accumulator v of lane l is
// row l % 32 of the tile's A rows and column 8 (v / 4) + 4 (l / 32) + v % 4 of its W
// rows.
template <int BM, int BN, int WM, int WN, int S, int G, int MODE, bool A5, bool W5, bool E8>
__global__ __launch_bounds__(64 * WM * WN * G) void echo_gemm_fp8_tile_k(const GemmFp8Args a, uint32_t gm, uint32_t gn) {
  constexpr bool kBf16 = MODE == kWide || MODE == kWideScaled;       // else the 8-bit instruction
  constexpr bool kFolded = MODE == kScaled8 || MODE == kWideScaled;  // scales applied with the products
  static_assert(!kFolded || E8, "only exponent bytes fold into the products");
  constexpr int NW = WM * WN, RW = BM / WM, CW = BN / WN, MI = RW / 32, NJ = CW / 32;
  static_assert(MI * 32 * WM == BM && NJ * 32 * WN == BN, "even splits");
  typedef Slabs<BM, BN, NW, S, G, MODE == kScaled8, E8> SL;
  constexpr int kSlab = SL::kSlab, kSlabA = SL::kSlabA;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[G * SL::kBytes];
  const TileAt tile = tile_at<BM, BN>(gm, gn);
  const RankPtrs p = rank_ptrs(tile.rank);
  SL sl;
  sl.init(lds, a, p, tile);
  const int lane = sl.lane, half = lane >> 5, wm = sl.wave / WN, wn = sl.wave % WN;

  f32x16 acc[MI][NJ];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;
  [[maybe_unused]] f32x16 blk[MI][NJ];

  // Fragments of a half step: 32 bytes per lane of each sub-tile, as two 16-byte
  // chunks.  They roll: as soon as the instructions that use a fragment are issued,
  // the next half step's is read in its place (A's, used until the end, alternate
  // between two sets with the 8-bit instruction).
  constexpr int kSetsA = kBf16 ? 1 : 2;
  i32x4 fa[kSetsA][MI][2], fw[NJ][2];
  int at[2][2];  // byte offset of this lane's chunk c of half step hs in a 32-row sub-tile
#pragma unroll
  for (int hs = 0; hs < 2; ++hs)
#pragma unroll
    for (int c = 0; c < 2; ++c) at[hs][c] = (lane & 31) * 128 + 16 * ((4 * half + 2 * hs + c) ^ ((lane >> 1) & 7));
  auto read_a = [&](int set, int slab, int hs, int c) {
    const uint8_t* b = sl.lds + slab * kSlab + RW * wm * 128 + at[hs][c];
#pragma unroll
    for (int i = 0; i < MI; ++i) fa[set][i][c] = *reinterpret_cast<const i32x4*>(b + 4096 * i);
  };
  auto read_w = [&](int j, int slab, int hs, int c) {
    const uint8_t* b = sl.lds + slab * kSlab + kSlabA + CW * wn * 128 + at[hs][c];
    fw[j][c] = *reinterpret_cast<const i32x4*>(b + 4096 * j);
  };
  // kFolded: the scales of the rows this lane supplies, this step's and the next's
  uint32_t ea[MI], ew[NJ], ea1[MI], ew1[NJ];
  auto read_scales = [&](int ring, uint32_t* sa, uint32_t* sw) {
#pragma unroll
    for (int i = 0; i < MI; ++i) sa[i] = sl.scales(ring)[RW * wm + 32 * i + (lane & 31)];
#pragma unroll
    for (int j = 0; j < NJ; ++j) sw[j] = sl.scales(ring)[BM + CW * wn + 32 * j + (lane & 31)];
  };
  // The instructions of half step HS, reading the next one's fragments (READ) from
  // slab `slab`.
  auto half_step = [&](auto hs, auto read, int slab) {
    constexpr int HS = decltype(hs)::value;
    constexpr bool READ = decltype(read)::value;
    [[maybe_unused]] const f32x16 zero{};
#if defined(__HIP_DEVICE_COMPILE__)
    if constexpr (!kBf16) {
      if constexpr (READ) {
        read_a(HS ^ 1, slab, HS ^ 1, 0);
        read_a(HS ^ 1, slab, HS ^ 1, 1);
      }
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const i32x8 w = __builtin_shufflevector(fw[j][0], fw[j][1], 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
        for (int i = 0; i < MI; ++i) {
          const i32x8 x8 = __builtin_shufflevector(fa[HS][i][0], fa[HS][i][1], 0, 1, 2, 3, 4, 5, 6, 7);
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
              w, x8, acc[i][j], W5 ? 1 : 0, A5 ? 1 : 0, 0, static_cast<int>(ew[j]), 0, static_cast<int>(ea[i]));
        }
        if constexpr (READ) {
          read_w(j, slab, HS ^ 1, 0);
          read_w(j, slab, HS ^ 1, 1);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    } else {
#pragma unroll
      for (int s = 0; s < 4; ++s) {  // 16 k each
        const int c = s >> 1, d = 2 * (s & 1);
        const auto scale = [](uint32_t e) { return MODE == kWideScaled ? __uint_as_float(e) : 1.0f; };
        bf16x8 wb[NJ];
#pragma unroll
        for (int j = 0; j < NJ; ++j) wb[j] = widen8<W5>(fw[j][c][d], fw[j][c][d + 1], scale(ew[j]));
#pragma unroll
        for (int i = 0; i < MI; ++i) {
          const bf16x8 ab = widen8<A5>(fa[0][i][c][d], fa[0][i][c][d + 1], scale(ea[i]));
#pragma unroll
          for (int j = 0; j < NJ; ++j) {
            if constexpr (MODE == kWideScaled)
              acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(wb[j], ab, acc[i][j], 0, 0, 0);
            else
              blk[i][j] =
                  __builtin_amdgcn_mfma_f32_32x32x16_bf16(wb[j], ab, HS == 0 && s == 0 ? zero : blk[i][j], 0, 0, 0);
          }
        }
        if constexpr (READ) {
          if (s & 1) {
            read_a(0, slab, HS ^ 1, c);
#pragma unroll
            for (int j = 0; j < NJ; ++j) read_w(j, slab, HS ^ 1, c);
          }
        }
      }
    }
#endif
  };
  constexpr std::integral_constant<int, 0> H0{};
  constexpr std::integral_constant<int, 1> H1{};
  constexpr std::true_type kYes{};
  constexpr std::false_type kNo{};

  sl.start();
  if constexpr (kFolded) read_scales(0, ea, ew);
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    read_a(0, 0, 0, c);
#pragma unroll
    for (int j = 0; j < NJ; ++j) read_w(j, 0, 0, c);
  }
  int cur = 0, ring = 0;  // slab and scales of the step
  auto step = [&](int it, auto issues, auto last) {
    constexpr int ISSUE = decltype(issues)::value;
    const int next = cur + 1 == S ? 0 : cur + 1, ring1 = ring == 2 ? 0 : ring + 1;
    half_step(H0, kYes, cur);
    if constexpr (!decltype(last)::value) {
      sl.template wait_next<ISSUE>(it, next, ring1);
      if constexpr (kFolded) read_scales(ring1, ea1, ew1);
      sl.template refill<ISSUE>(it, cur);
      half_step(H1, kYes, next);
    } else {
      half_step(H1, kNo, 0);
    }
    if constexpr (!kFolded) {
      float ca[MI];
#pragma unroll
      for (int i = 0; i < MI; ++i) ca[i] = __uint_as_float(sl.scales(ring)[RW * wm + 32 * i + (lane & 31)]);
      if (a.sw_shift != 0) {  // one scale for a sub-tile's 32 columns
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          const float cw = __uint_as_float(sl.scales(ring)[BM + CW * wn + 32 * j]);
#pragma unroll
          for (int i = 0; i < MI; ++i) {
            const float c = ca[i] * cw;
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][j][v] = __builtin_fmaf(blk[i][j][v], c, acc[i][j][v]);
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          f32x4 cw[4];
#pragma unroll
          for (int v4 = 0; v4 < 4; ++v4)
            cw[v4] = *reinterpret_cast<const f32x4*>(&sl.scales(ring)[BM + CW * wn + 32 * j + 8 * v4 + 4 * half]);
#pragma unroll
          for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int v = 0; v < 16; ++v)
              acc[i][j][v] = __builtin_fmaf(blk[i][j][v], ca[i] * cw[v >> 2][v & 3], acc[i][j][v]);
        }
      }
    } else if constexpr (!decltype(last)::value) {
#pragma unroll
      for (int i = 0; i < MI; ++i) ea[i] = ea1[i];
#pragma unroll
      for (int j = 0; j < NJ; ++j) ew[j] = ew1[j];
    }
    cur = next;
    ring = ring1;
  };
  sl.run(step);

  __syncthreads();
  if constexpr (G > 1) {
    f32x4 flat[MI * NJ * 4];
#pragma unroll
    for (int i = 0; i < MI * NJ * 16; ++i) flat[i / 4][i % 4] = acc[i / 16 / NJ][i / 16 % NJ][i % 16];
    if (!join_groups<SL, G>(lds, sl, flat)) return;
#pragma unroll
    for (int i = 0; i < MI * NJ * 16; ++i) acc[i / 16 / NJ][i / 16 % NJ][i % 16] = flat[i / 4][i % 4];
  }
  const auto store = [&](auto elem) {
    constexpr int E = decltype(elem)::value;
    constexpr int kRegion = SL::kBytes / NW / 16 * 16;
    store_tile<E, RW, CW, kRegion>(
        lds + sl.wave * kRegion, a, p.out, tile.m0 + RW * wm, tile.n0 + CW * wn, [&](uint8_t* region, int pitch, int i) {
#pragma unroll
          for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int v = 0; v < 16; v += 4)
              put4<E>(region + (lane & 31) * pitch + (32 * j + 2 * v + 4 * half) * sizeof(typename ElemOf<E>::T),
                      acc[i][j][v], acc[i][j][v + 1], acc[i][j][v + 2], acc[i][j][v + 3]);
        });
  };
  if constexpr (kBf16) {
    store(std::integral_constant<int, kElemF32>{});
  } else {
    if (a.out_elem == kElemBf16) store(std::integral_constant<int, kElemBf16>{});
    else store(std::integral_constant<int, kElemF16>{});
  }
}

// fp32 scales on the 8-bit instruction: 16 x 16 sub-tiles, whose v_mfma_..._16x16x128
// sums a whole block of 128 at once into four registers, so that the scaling (four
// multiply-adds per instruction, half its time) follows two instructions behind and
// runs beside the matrix cores, with no second set of accumulators.  Lane l supplies
// row l % 16 of a sub-tile and the bytes 32 (l / 16) .. + 31 of the K step, and holds
// row l % 16 of the A rows, columns 4 (l / 16) .. + 3 of the W rows.  A step's fragments
// of A stay in registers; those of W come one sub-tile ahead.
// WB: W's scales are of blocks of 128 rows, one for all of a wavefront's columns.
// Measured: P = 2, M = N = K = 4096 130 us, 150 with a scale per row of W (2.1 and 1.8
// PFLOP/s; exponent bytes, which the instruction applies, 107).  The matrix cores are busy
// 49 and 42 % of the cycles: 47 and 42 % of the LDS's active cycles are bank conflicts of the
// fragment reads, and the 256 x 256 tile spills 64 and 104 bytes of registers a lane.
template <int BM, int BN, int WM, int WN, int S, int G, bool WB, bool A5, bool W5>
__global__ __launch_bounds__(64 * WM * WN * G) void echo_gemm_fp8_fma_k(const GemmFp8Args a, uint32_t gm, uint32_t gn) {
  constexpr int NW = WM * WN, RW = BM / WM, CW = BN / WN, MI = RW / 16, NJ = CW / 16;
  static_assert(MI * 16 * WM == BM && NJ * 16 * WN == BN && CW <= 128 && 128 % CW == 0, "even splits");
  static_assert(NJ % 2 == 0 && NJ >= 4, "fragments of W alternate between two sets");
  typedef Slabs<BM, BN, NW, S, G, false, false> SL;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[G * SL::kBytes];
  const TileAt tile = tile_at<BM, BN>(gm, gn);
  const RankPtrs p = rank_ptrs(tile.rank);
  SL sl;
  sl.init(lds, a, p, tile);
  const int lane = sl.lane, sub = lane & 15, g = lane >> 4, wm = sl.wave / WN, wn = sl.wave % WN;

  f32x4 acc[MI][NJ] = {};
  i32x8 fa[MI], fw[2];
  int at[2];  // byte offset of this lane's chunk c in a 16-row sub-tile
#pragma unroll
  for (int c = 0; c < 2; ++c) at[c] = sub * 128 + 16 * ((2 * g + c) ^ (sub >> 1));
  auto frag = [&](const uint8_t* b) {
    const i32x4 lo = *reinterpret_cast<const i32x4*>(b + at[0]), hi = *reinterpret_cast<const i32x4*>(b + at[1]);
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  };
  auto read_a = [&](int slab, int i) { fa[i] = frag(sl.lds + slab * SL::kSlab + (RW * wm + 16 * i) * 128); };
  auto read_w = [&](int slab, int j) {
    fw[j & 1] = frag(sl.lds + slab * SL::kSlab + SL::kSlabA + (CW * wn + 16 * j) * 128);
  };
  // this step's scales: of the lane's rows of A (times W's where one covers all its
  // columns), and of its columns of the sub-tiles at hand (the previous column's last sums are still to come)
  float ca[MI];
  f32x4 cw[3];
  auto read_ca = [&](int ring) {
#pragma unroll
    for (int i = 0; i < MI; ++i) ca[i] = __uint_as_float(sl.scales(ring)[RW * wm + 16 * i + sub]);
    if constexpr (WB) {
      const float w = __uint_as_float(sl.scales(ring)[BM + CW * wn]);
#pragma unroll
      for (int i = 0; i < MI; ++i) ca[i] = ca[i] * w;
    }
  };
  auto read_cw = [&](int ring, int j) {
    if constexpr (!WB) cw[j % 3] = *reinterpret_cast<const f32x4*>(sl.scales(ring) + BM + CW * wn + 16 * j + 4 * g);
  };
  f32x4 sum[2];  // the last two block sums
  auto add = [&](int k) {  // the k-th, of sub-tile (k % MI, k / MI)
    const int i = k % MI, j = k / MI;
#pragma unroll
    for (int v = 0; v < 4; ++v)
      acc[i][j][v] = __builtin_fmaf(sum[k & 1][v], WB ? ca[i] : ca[i] * cw[j % 3][v], acc[i][j][v]);
  };
  // the instructions of sub-tile column j
  auto column = [&](int j) {
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const int k = j * MI + i;
      if (k >= 2) add(k - 2);
#if defined(__HIP_DEVICE_COMPILE__)
      sum[k & 1] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fw[j & 1], fa[i], f32x4{}, W5 ? 1 : 0, A5 ? 1 : 0, 0,
                                                                    127, 0, 127);
#endif
    }
  };

  sl.start();
#pragma unroll
  for (int i = 0; i < MI; ++i) read_a(0, i);
  read_w(0, 0);
  read_w(0, 1);
  read_ca(0);
  read_cw(0, 0);
  int cur = 0, ring = 0;
  auto step = [&](int it, auto issues, auto last) {
    constexpr int ISSUE = decltype(issues)::value;
    constexpr bool LAST = decltype(last)::value;
    const int next = cur + 1 == S ? 0 : cur + 1, ring1 = ring == 2 ? 0 : ring + 1;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      if (j + 1 < NJ) read_cw(ring, j + 1);
      column(j);
      if (j + 2 < NJ) read_w(cur, j + 2);
      __builtin_amdgcn_sched_barrier(0);
      if (j + 3 == NJ) {
        // the slab's last fragments are on their way
        if constexpr (!LAST) {
          sl.template wait_next<ISSUE>(it, next, ring1);
          sl.template refill<ISSUE>(it, cur);
        }
      }
      if constexpr (!LAST) {
        if (j + 2 >= NJ) read_w(next, j + 2 - NJ);
      }
    }
    if constexpr (!LAST) {
#pragma unroll
      for (int i = 0; i < MI; ++i) read_a(next, i);
    }
    add(MI * NJ - 2);
    add(MI * NJ - 1);
    if constexpr (!LAST) {
      read_ca(ring1);
      read_cw(ring1, 0);
    }
    cur = next;
    ring = ring1;
  };
  sl.run(step);

  __syncthreads();
  if constexpr (G > 1) {
    f32x4 flat[MI * NJ];
#pragma unroll
    for (int i = 0; i < MI * NJ; ++i) flat[i] = acc[i / NJ][i % NJ];
    if (!join_groups<SL, G>(lds, sl, flat)) return;
#pragma unroll
    for (int i = 0; i < MI * NJ; ++i) acc[i / NJ][i % NJ] = flat[i];
  }
  const auto store = [&](auto elem) {
    constexpr int E = decltype(elem)::value;
    constexpr int kRegion = SL::kBytes / NW / 16 * 16;
    store_tile<E, RW, CW, kRegion>(
        lds + sl.wave * kRegion, a, p.out, tile.m0 + RW * wm, tile.n0 + CW * wn, [&](uint8_t* region, int pitch, int i) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < NJ; ++j) {
              const f32x4 o = acc[2 * i + h][j];
              put4<E>(region + (16 * h + sub) * pitch + (16 * j + 4 * g) * sizeof(typename ElemOf<E>::T), o[0], o[1], o[2],
                      o[3]);
            }
        });
  };
  if (a.out_elem == kElemBf16) store(std::integral_constant<int, kElemBf16>{});
  else store(std::integral_constant<int, kElemF16>{});
}

template <int BM, int BN, int WM, int WN, int S, int G, int MODE, bool A5, bool W5, bool E8>
hipError_t tile(const GemmFp8Args& a, int P, hipStream_t s) {
  const uint32_t gm = static_cast<uint32_t>((a.M + BM - 1) / BM), gn = static_cast<uint32_t>((a.N + BN - 1) / BN);
  hipLaunchKernelGGL((echo_gemm_fp8_tile_k<BM, BN, WM, WN, S, G, MODE, A5, W5, E8>), dim3(gm * gn * P),
                     dim3(64 * WM * WN * G), 0, s, a, gm, gn);
  return hipGetLastError();
}

template <int BM, int BN, int WM, int WN, int S, int G, bool WB, bool A5, bool W5>
hipError_t fma_tile(const GemmFp8Args& a, int P, hipStream_t s) {
  const uint32_t gm = static_cast<uint32_t>((a.M + BM - 1) / BM), gn = static_cast<uint32_t>((a.N + BN - 1) / BN);
  hipLaunchKernelGGL((echo_gemm_fp8_fma_k<BM, BN, WM, WN, S, G, WB, A5, W5>), dim3(gm * gn * P), dim3(64 * WM * WN * G), 0, s,
                     a, gm, gn);
  return hipGetLastError();
}

template <int MT, int CT, int U, int NW, bool WB, bool A5, bool W5, bool E8>
hipError_t thin(const GemmFp8Args& a, int P, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>((a.N + 16 * CT - 1) / (16 * CT)),
                  static_cast<unsigned>((a.M + 16 * MT - 1) / (16 * MT)), static_cast<unsigned>(P));
  hipLaunchKernelGGL((echo_gemm_fp8_thin_k<MT, CT, U, NW, WB, A5, W5, E8>), grid, dim3(64 * NW), 0, s, a);
  return hipGetLastError();
}

// E8: exponent-byte scales.  WB: fp32 scales, W's of blocks of 128 rows.
//
// Up to 32 rows of A: the kernel that shares k, by the number of 16-row tiles of W over
// all ranks, so that there are enough workgroups to fill the chip and as much in flight
// as possible.  Measured with cold weights, us: P = 8, M = 16, N = 4096, K = 1024:
// 9.9 with 4 tiles per workgroup of 8 wavefronts, 12.2 with 2 of 16, 15.3 with 1 of 8;
// P = 8, N = 1024, K = 4096: 10.3 with 2 tiles of 16 wavefronts, 12.5 with 1 of 16; one
// token against N = K = 8192, where A costs nothing: 19.0 and 15.8.
// Above that, tiles by the number t of 64 x 64 tiles over all ranks and b of 128 x 128
// ones; us for bfloat16 outputs with exponent bytes, then fp32 outputs:
//   t <= 256, the CUs, and K over 1024: a K step of a lone workgroup is bound by its own
//     chain of waits (0.5 us; more slabs alone changed nothing, as a step's scales are
//     loaded one step ahead whatever the number of slabs), so four groups of four
//     wavefronts share k (M = 64, N = K = 8192: 19.9 against 23.8 with two groups and
//     31.8 with one; M = 500, N = 640, K = 7552, fp32 output: 20.7, 23.9 and 31.9);
//   t <= 512: two groups, two workgroups per CU (P = 4, M = 128, N = K = 4096: 18.7, 26.5
//     against 22.2, 28.9 with one and 24.1 with four; P = 8, M = 64: 26.4, 30.7 against
//     34, 46 with 128 x 128 tiles; P = 4, M = 128, N = 4096, K = 512: 5.9 against 6.2);
//   b <= 256, M over 64 and K over 1024: 128 x 128, two groups (M = 1024, N = K = 4096:
//     23.3, 40.1 against 26.0, 40.8 with one; M = 600: 20.9, 32.0 against 24.3, 35.4 with
//     64 x 128 tiles; at K = 1024 one group is faster, 9.3 against 10.1);
//   b < 192, or M <= 64, where more rows would multiply zeros: 64 x 128, 2 slabs (P = 16,
//     M = 64, N = 4096, K = 1024: 13.5, 16.2 against 15.1, 19.4 with 128 x 128 tiles and
//     16.2, 19.9 with 64 x 64 ones in two groups);
//   b < 384, or M <= 128: 128 x 128, four wavefronts, 2 slabs, two workgroups per CU
//     (M = 1024, N = 4096, K = 1024: 9.6, 14.5 against 12.1, 17.2 with 256 x 128 tiles and
//     10.0, 14.3 with 64 x 128; M = 1280, N = K = 4096: 29.5, 48.3 against 30.1, 44.5 and
//     30.8, 46.4; M = 128, N = 65536, K = 4096: 70.2, 77.9 against 74.7, 99.9 with
//     256 x 256 and 87, 96 with 64 x 128);
//   256 x 256 where those number at least 192, three quarters of the CUs (P = 4,
//     M = 2048, N = K = 4096: 130 against 168 with 128 x 128 tiles);
//   else 256 x 128, 3 slabs (P = 2, M = 1024, N = K = 4096: 37.3 against 38.5 with
//     128 x 128 and 76 with 64 x 64).
// The same with fp32 scales and 16-bit outputs, where tiles have 128 columns at least and
// two groups are the most that fits LDS (P = 4, M = 64, N = K = 4096: 18.6 against 22.2
// with one; M = 1024, N = K = 4096 27.5 with two groups against 33.8).
// (b < 384: M = 1024, N = 4096, K = 1024 11.4 against 13.6 with 256 x 128 and 10.7 with
// 64 x 128; M = 1280, N = K = 4096 39.5 against 36.6 and 36.4.)
// fp32 scales and fp32 outputs take 256 x 128 tiles at most: a block's sum has
// accumulators of its own (b < 384, same sizes: 15.9 against 20.0 and 15.6; 78.7 against
// 58.8 and 61.7, where the rule made for the other forms loses).
// The rules count tiles and look at M; they do not see how the last round of tiles fills
// the CUs or how much of a tile lies past N: M = 2304, N = 8192, K = 4096 (288 tiles of
// 256 x 256) takes 92 us where M = 2048 takes 55, and M = 65536, N = 64, K = 4096 58,
// reading its operands 38.
template <bool A5, bool W5, bool E8, bool WB>
hipError_t launch(const GemmFp8Args& a, int P, hipStream_t s) {
  const int64_t columns = (a.N + 15) / 16 * P;  // 16 rows of W each
  if (a.M <= 16) {
    if (columns >= 1024) return thin<1, 4, 1, 8, WB, A5, W5, E8>(a, P, s);
    if (columns >= 512 && a.M > 4) return thin<1, 2, 1, 16, WB, A5, W5, E8>(a, P, s);
    return thin<1, 1, 2, 16, WB, A5, W5, E8>(a, P, s);
  }
  if (a.M <= 32) return thin<2, 2, 2, 8, WB, A5, W5, E8>(a, P, s);
  const int64_t b = (a.M + 127) / 128 * ((a.N + 127) / 128) * P;
  const int64_t t = (a.M + 63) / 64 * ((a.N + 63) / 64) * P;
  const bool four = t <= 256 && a.K > 1024, two = t <= 512, low = b < 192 || a.M <= 64, medium = b < 384 || a.M <= 128;
  const bool pair = b <= 256 && a.M > 64 && a.K > 1024;
  const bool large = (a.M + 255) / 256 * ((a.N + 255) / 256) * P >= 192;
  if (a.out_elem == kElemF32) {
    constexpr TileMode MODE = E8 ? kWideScaled : kWide;
    if (four) return tile<64, 64, 2, 2, 2, 4, MODE, A5, W5, E8>(a, P, s);
    if (two) return tile<64, 64, 2, 2, 2, 2, MODE, A5, W5, E8>(a, P, s);
    if (pair) return tile<128, 128, 2, 2, 2, 2, MODE, A5, W5, E8>(a, P, s);
    if (low) return tile<64, 128, 2, 2, 2, 1, MODE, A5, W5, E8>(a, P, s);
    if (medium) return tile<128, 128, 2, 2, 2, 1, MODE, A5, W5, E8>(a, P, s);
    if constexpr (E8) {
      if (large) return tile<256, 256, 4, 2, 2, 1, MODE, A5, W5, E8>(a, P, s);
    }
    return tile<256, 128, 4, 2, 3, 1, MODE, A5, W5, E8>(a, P, s);
  }
  if constexpr (E8) {
    if (four) return tile<64, 64, 2, 2, 2, 4, kScaled8, A5, W5, true>(a, P, s);
    if (two) return tile<64, 64, 2, 2, 2, 2, kScaled8, A5, W5, true>(a, P, s);
    if (pair) return tile<128, 128, 2, 2, 2, 2, kScaled8, A5, W5, true>(a, P, s);
    if (low) return tile<64, 128, 2, 2, 2, 1, kScaled8, A5, W5, true>(a, P, s);
    if (medium) return tile<128, 128, 2, 2, 2, 1, kScaled8, A5, W5, true>(a, P, s);
    if (large) return tile<256, 256, 4, 2, 2, 1, kScaled8, A5, W5, true>(a, P, s);
    return tile<256, 128, 4, 2, 3, 1, kScaled8, A5, W5, true>(a, P, s);
  } else {
    if (two) return fma_tile<64, 128, 2, 2, 3, 2, WB, A5, W5>(a, P, s);
    if (pair) return fma_tile<128, 128, 2, 2, 2, 2, WB, A5, W5>(a, P, s);
    if (low) return fma_tile<64, 128, 2, 2, 2, 1, WB, A5, W5>(a, P, s);
    if (medium) return fma_tile<128, 128, 2, 2, 2, 1, WB, A5, W5>(a, P, s);
    if (large) return fma_tile<256, 256, 4, 2, 2, 1, WB, A5, W5>(a, P, s);
    return fma_tile<256, 128, 4, 2, 3, 1, WB, A5, W5>(a, P, s);
  }
}

template <bool A5, bool W5>
hipError_t launch_formats(const GemmFp8Args& a, int P, bool e8m0, hipStream_t s) {
  if (e8m0) return launch<A5, W5, true, false>(a, P, s);
  return a.sw_shift != 0 ? launch<A5, W5, false, true>(a, P, s) : launch<A5, W5, false, false>(a, P, s);
}

}  // namespace

hipError_t launch_gemm_fp8(const GemmFp8Args& a, int P, bool a_e5m2, bool w_e5m2, bool e8m0, hipStream_t s) {
  if (a.K == 0) {
    const dim3 grid(static_cast<unsigned>((a.N + 255) / 256 < 64 ? (a.N + 255) / 256 : 64),
                    static_cast<unsigned>(a.M < 4096 ? a.M : 4096), static_cast<unsigned>(P));
    hipLaunchKernelGGL(echo_gemm_fp8_zero_k, grid, dim3(256), 0, s, a);
    return hipGetLastError();
  }
  if (a_e5m2) return w_e5m2 ? launch_formats<true, true>(a, P, e8m0, s) : launch_formats<true, false>(a, P, e8m0, s);
  return w_e5m2 ? launch_formats<false, true>(a, P, e8m0, s) : launch_formats<false, false>(a, P, e8m0, s);
}

}  // namespace echo
