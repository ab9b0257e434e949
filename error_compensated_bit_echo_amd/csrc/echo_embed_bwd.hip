// Gradient of the embedding: dtable_r[v] = scale * (sum of dout[t] over the tokens t with
// row r V + v, in rising order of t), zeros for rows without a token.
//
// The tokens are sorted by row (stable, so equal tokens stay in order), then runs of equal
// tokens are summed: no atomics on sums, so the result is the same from call to call.  The
// sort is a radix sort of 9-bit digits: two for vocabularies of up to 2^18 - 1 rows.  Up to
// kSmall tokens one workgroup holds them all in LDS; more take three launches a digit: counts
// per tile, their prefix sums, placement.  Either way the launches' other workgroups clear the
// tables meanwhile, which takes longer than the sort where tables are large.
//
// The sorted tokens are cut into chunks of equal length, whatever the runs: a chunk writes
// the rows of runs that lie inside it, and puts the sum of a run that crosses its start or
// its end into the workspace; a last launch adds those up along the chunks.  So a token
// that comes up ten thousand times costs as much as ten thousand different ones.
//
// Bound by the memory: 16384 tokens, 4 tables of 16384 x 4096 fp32, take 259 us on inputs that change from
// call to call, 5.2 TB/s, and 238 on the same again: the zeros 165 (the sort of 31 us behind them),
// the sums 67 (their gradients in the last-level cache) to 83, the join 7. 16384 tokens of
// a table of 1000 x 512 take 48 us, where the sort shows.
#include "echo_row.h"

namespace echo {
namespace {

constexpr int kSortThreads = 1024;
constexpr int kWaves = kSortThreads / 64;
constexpr int kDigitBits = 9;
constexpr int kDigits = 1 << kDigitBits;
constexpr int kSmallRounds = 16;
constexpr int64_t kSmall = kSortThreads * kSmallRounds;  // tokens that one workgroup sorts: 128 KB of LDS
constexpr int kTileRounds = 4;
constexpr int kThreads = 256;  // of the join
constexpr unsigned kClearGroups = 256;  // of kSortThreads: one to a CU

struct SortLds {
  uint32_t count[kWaves][kDigits];
  uint32_t wave_total[kWaves];
};

// The row of token t over all ranks; `rows` (behind the last) where there is none.
template <typename Args>
__device__ __forceinline__ uint32_t key_of(const Args* a, int64_t t) {
  const int64_t token = a->wide ? static_cast<const int64_t*>(a->tokens)[t] : static_cast<const int32_t*>(a->tokens)[t];
  const uint64_t v = static_cast<uint64_t>(token) - static_cast<uint64_t>(a->first), rows = static_cast<uint64_t>(a->P * a->V);
  return static_cast<uint32_t>(v < rows ? v : rows);
}

// The place of each of a thread's keys among the workgroup's, ordered by digit, then by
// position; keys lie wavefront by wavefront, round by round, lane by lane.
template <int ROUNDS>
__device__ __forceinline__ void places(const uint32_t (&key)[ROUNDS], int digit_shift, SortLds* lds, uint32_t (&place)[ROUNDS]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int d = lane; d < kDigits; d += 64) lds->count[wave][d] = 0;
  __syncthreads();
#pragma unroll
  for (int r = 0; r < ROUNDS; ++r) {
    const uint32_t d = (key[r] >> digit_shift) & (kDigits - 1);
    // the lanes with another digit, in two halves
    uint32_t low = 0, high = 0;
#pragma unroll
    for (int b = 0; b < kDigitBits; ++b) {
      const uint32_t bit = static_cast<uint32_t>(__builtin_amdgcn_sbfe(static_cast<int>(d), b, 1));  // 0 or all ones
      const uint64_t set = __ballot(bit != 0);
      low |= static_cast<uint32_t>(set) ^ bit;
      high |= static_cast<uint32_t>(set >> 32) ^ bit;
    }
    const uint64_t same = ~(static_cast<uint64_t>(high) << 32 | low);
    const uint32_t before = __builtin_amdgcn_mbcnt_hi(~high, __builtin_amdgcn_mbcnt_lo(~low, 0));
    uint32_t old = 0;
    if (before == 0) old = atomicAdd(&lds->count[wave][d], static_cast<uint32_t>(__popcll(same)));
    place[r] = __shfl(old, __ffsll(static_cast<unsigned long long>(same)) - 1) + before;
  }
  __syncthreads();
  // exclusive prefix sums of the counts, digit by digit and within a digit by wavefront:
  // eight counters to a thread
  static_assert(kWaves * kDigits == kSortThreads * 8, "counters");
  const int d = threadIdx.x >> 1, w0 = (threadIdx.x & 1) * 8;
  uint32_t c[8], sum = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    c[i] = sum;
    sum += lds->count[w0 + i][d];
  }
  uint32_t upto = sum;
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
    const uint32_t o = __shfl_up(upto, m);
    if (lane >= m) upto += o;
  }
  if (lane == 63) lds->wave_total[wave] = upto;
  __syncthreads();
  uint32_t base = upto - sum;
  for (int w = 0; w < wave; ++w) base += lds->wave_total[w];
#pragma unroll
  for (int i = 0; i < 8; ++i) lds->count[w0 + i][d] = base + c[i];
  __syncthreads();
#pragma unroll
  for (int r = 0; r < ROUNDS; ++r) place[r] += lds->count[wave][(key[r] >> digit_shift) & (kDigits - 1)];
}

// Zeros to a row's columns from `at` on, 16 bytes at most: neighbouring threads write
// neighbouring 16 bytes, where 8 columns of fp32 to each would leave half of every line to a
// second store.
template <int E>
constexpr int kZeros = 16 / sizeof(typename ElemOf<E>::T);

// STREAM: past the caches, which the sums' reads and writes would otherwise have to empty of
// zeros first (4 tables of 16384 x 4096 fp32, 16384 tokens: 252 us, 294 without; 8192 x 4096, whose
// gradients do not fit: 112 and 131); tables that the last-level cache holds, beside gradients that
// it holds, stay there (50000 x 1024 fp32, 4096 tokens: 46 us, 52 past it).
template <int E, bool STREAM>
__device__ __forceinline__ void clear_run(void* table, int64_t at, int64_t left) {
  typedef typename ElemOf<E>::T T;
  T* p = static_cast<T*>(table) + at;
  if (left >= kZeros<E>) {
    typedef uint32_t u4 __attribute__((ext_vector_type(4), aligned(2)));
    if constexpr (STREAM) __builtin_nontemporal_store(u4{0, 0, 0, 0}, reinterpret_cast<u4*>(p));
    else *reinterpret_cast<u4*>(p) = u4{0, 0, 0, 0};
  } else {
    for (int i = 0; i < left; ++i) p[i] = static_cast<T>(0.0f);
  }
}

// A table whose rows follow each other without a gap is cleared page by page of 4 KB: workgroup b
// takes every 8th only, those at addresses of one remainder of 32 KB, its wavefronts one after the
// other.  The workgroups of an XCD, which are every 8th too, then write one remainder, and 255
// of 16 wavefronts reach 6.5 TB/s of nothing but zeros, where stretches of 32 KB to a wavefront
// reach 6.1 and pages as they come 5.4.  Rows that the sums will write are written here too: with
// the tenth of them left out that 16384 tokens of 65536 rows take, the pattern breaks (4 tables of
// 16384 x 4096 fp32: 271 us in all, 252 with them).
constexpr int64_t kPage = 4096;

// Pages lo .. hi - 1 of the ranks' tables, `per` to a table of `bytes`, by the workgroups from
// `first` on, 8 at least.
template <bool STREAM, typename Args>
__device__ __forceinline__ void clear_pages_as(const Args* a, int64_t bytes, int64_t per, int64_t lo, int64_t hi, uint32_t first) {
  typedef uint32_t u4 __attribute__((ext_vector_type(4), aligned(2)));
  const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const uint32_t kind = blockIdx.x & 7, least = first + ((kind - first) & 7);
  const uint32_t groups = (gridDim.x - least + 7) >> 3, slot = (blockIdx.x - least) >> 3;
  for (int64_t r = lo / per; r < a->P && r * per < hi; ++r) {
    char* table = static_cast<char*>(a->dtable[r]);
    const int64_t from = lo - r * per, to = hi - r * per, end = to < per ? to : per;
    int64_t page = from > 0 ? from : 0;
    page += (kind - static_cast<uint32_t>(reinterpret_cast<uintptr_t>(table) >> 12) - static_cast<uint32_t>(page)) & 7;
    for (page += int64_t{slot * kWaves + wave} * 8; page < end; page += int64_t{groups} * kWaves * 8) {
      const int64_t at = page * kPage + lane * 16;
      char* p = table + at;
      if ((page + 1) * kPage <= bytes) {
#pragma unroll
        for (int i = 0; i < kPage / 1024; ++i) {
          u4* q = reinterpret_cast<u4*>(p + i * 1024);
          if constexpr (STREAM) __builtin_nontemporal_store(u4{0, 0, 0, 0}, q);
          else *q = u4{0, 0, 0, 0};
        }
      } else {
        for (int i = 0; i < kPage; i += 1024)
          for (int b = 0; b < 16 && at + i + b < bytes; b += 2) *reinterpret_cast<uint16_t*>(p + i + b) = 0;
      }
    }
  }
}

// Part `part` of `parts` of clearing tables with gaps between their rows, by workgroup `id` of `of`.
template <int E, bool STREAM, typename Args>
__device__ __forceinline__ void clear_rows_as(const Args* a, int part, int parts, uint32_t id, uint32_t of) {
  const int64_t C = a->C, V = a->V;
  constexpr int kZ = kZeros<E>;
  int shift = 0;  // 2^shift threads to a row
  while ((1 << shift) < kSortThreads && (int64_t{kZ} << shift) < C) ++shift;
  const int64_t width = int64_t{kZ} << shift, cuts = (C + width - 1) / width, per = kSortThreads >> shift;
  const int64_t blocks = (V + per - 1) / per, jobs = blocks * cuts * a->P;  // blocks of rows, cut into columns
  const int64_t lo = jobs * part / parts, hi = jobs * (part + 1) / parts;
  for (int64_t job = lo + id; job < hi; job += of) {
    const int64_t cut = job % cuts, block = job / cuts;
    const int64_t r = block / blocks, v = (block - r * blocks) * per + (threadIdx.x >> shift);
    const int64_t at = cut * width + (threadIdx.x & ((1 << shift) - 1)) * kZ;
    if (v < V) clear_run<E, STREAM>(a->dtable[r], v * a->ldt + at, C - at);
  }
}

// Part `part` of `parts` of clearing the tables, by the launch's workgroups from `first` on.  The two
// policies are apart as a whole: the compiler would make one of two stores that differ in it alone.
template <int E, typename Args>
__device__ __forceinline__ void clear_tables(const Args* a, int part, int parts, uint32_t first) {
  const uint32_t id = blockIdx.x - first, of = gridDim.x - first;
  if ((a->ldt == a->C || a->V == 1) && of >= 8) {
    const int64_t bytes = a->V * a->C * static_cast<int64_t>(sizeof(typename ElemOf<E>::T));
    const int64_t per = (bytes + kPage - 1) / kPage, pages = per * a->P, lo = pages * part / parts, hi = pages * (part + 1) / parts;
    if (a->stream) clear_pages_as<true>(a, bytes, per, lo, hi, first);
    else clear_pages_as<false>(a, bytes, per, lo, hi, first);
  } else if (a->stream) {
    clear_rows_as<E, true>(a, part, parts, id, of);
  } else {
    clear_rows_as<E, false>(a, part, parts, id, of);
  }
}

// Workgroup 0 sorts up to 1024 * ROUNDS tokens; the others clear the tables.
template <int E, int ROUNDS>
__global__ __launch_bounds__(kSortThreads) void echo_embed_sort_k(const EmbedBwdArgs given, int digits, uint32_t* keys,
                                                                  uint32_t* order) {
  __shared__ SortLds lds;
  __shared__ uint32_t sk[kSortThreads * ROUNDS];
  __shared__ uint16_t so[kSortThreads * ROUNDS];
  const auto* a = kernel_args<EmbedBwdArgs>();
  if (blockIdx.x != 0) {
    clear_tables<E>(a, 0, 1, 1);
    return;
  }
  const int T = static_cast<int>(a->T);
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  uint32_t key[ROUNDS], at[ROUNDS], place[ROUNDS];
#pragma unroll
  for (int r = 0; r < ROUNDS; ++r) {
    const int i = (wave * ROUNDS + r) * 64 + lane;
    key[r] = i < T ? key_of(a, i) : ~0u;  // behind every key in every digit
    at[r] = static_cast<uint32_t>(i);
  }
  for (int d = 0; d < digits; ++d) {
    places(key, kDigitBits * d, &lds, place);
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
      sk[place[r]] = key[r];
      so[place[r]] = static_cast<uint16_t>(at[r]);
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
      const int i = (wave * ROUNDS + r) * 64 + lane;
      key[r] = sk[i];
      at[r] = so[i];
    }
  }
#pragma unroll
  for (int r = 0; r < ROUNDS; ++r) {
    const int i = (wave * ROUNDS + r) * 64 + lane;
    if (i < T) {
      keys[i] = key[r];
      order[i] = at[r];
    }
  }
}

template <int E>
__global__ __launch_bounds__(kSortThreads) void echo_embed_clear_k(const EmbedBwdArgs given) {
  clear_tables<E>(kernel_args<EmbedBwdArgs>(), 0, 1, 0);
}

// ---- more than kSmall tokens -------------------------------------------------------------

// keys == nullptr: the keys are formed from the tokens, the order is their own.
template <typename Args>
__device__ __forceinline__ void load_tile(const Args* a, const uint32_t* keys, const uint32_t* order, uint32_t (&key)[kTileRounds],
                                          uint32_t (&at)[kTileRounds]) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
#pragma unroll
  for (int r = 0; r < kTileRounds; ++r) {
    const int64_t i = blockIdx.x * kEmbedTile + (wave * kTileRounds + r) * 64 + lane;
    key[r] = ~0u;
    at[r] = static_cast<uint32_t>(i);
    if (i < a->T) {
      key[r] = keys != nullptr ? keys[i] : key_of(a, i);
      if (order != nullptr) at[r] = order[i];
    }
  }
}

// Workgroups behind the `work` ones of a launch clear their part of the tables.
struct Share {
  uint32_t work;
  int part, parts;
};

// counts[digit * tiles + tile]
template <int E>
__global__ __launch_bounds__(kSortThreads) void echo_embed_count_k(const EmbedBwdArgs given, const Share sh, int shift,
                                                                   const uint32_t* keys, uint32_t* counts) {
  __shared__ uint32_t n[kDigits];
  const auto* a = kernel_args<EmbedBwdArgs>();
  if (blockIdx.x >= sh.work) {
    clear_tables<E>(a, sh.part, sh.parts, sh.work);
    return;
  }
  if (threadIdx.x < kDigits) n[threadIdx.x] = 0;
  __syncthreads();
  uint32_t key[kTileRounds], at[kTileRounds];
  load_tile(a, keys, nullptr, key, at);
#pragma unroll
  for (int r = 0; r < kTileRounds; ++r)
    if (static_cast<int64_t>(at[r]) < a->T) atomicAdd(&n[(key[r] >> shift) & (kDigits - 1)], 1u);
  __syncthreads();
  if (threadIdx.x < kDigits) counts[threadIdx.x * static_cast<int64_t>(sh.work) + blockIdx.x] = n[threadIdx.x];
}

// Exclusive prefix sums in place, one workgroup.
template <int E>
__global__ __launch_bounds__(kSortThreads) void echo_embed_scan_k(const EmbedBwdArgs given, const Share sh, uint32_t* counts,
                                                                  int64_t n) {
  __shared__ uint32_t total[kWaves];
  if (blockIdx.x >= sh.work) {
    clear_tables<E>(kernel_args<EmbedBwdArgs>(), sh.part, sh.parts, sh.work);
    return;
  }
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t carry = 0;
  for (int64_t lo = 0; lo < n; lo += kSortThreads * 4) {
    uint32_t c[4], sum = 0;
    const int64_t at = lo + threadIdx.x * 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      c[i] = sum;
      sum += at + i < n ? counts[at + i] : 0;
    }
    uint32_t upto = sum;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
      const uint32_t o = __shfl_up(upto, m);
      if (lane >= m) upto += o;
    }
    __syncthreads();
    if (lane == 63) total[wave] = upto;
    __syncthreads();
    uint32_t base = carry + upto - sum;
    for (int w = 0; w < kWaves; ++w) {
      if (w < wave) base += total[w];
      carry += total[w];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (at + i < n) counts[at + i] = base + c[i];
  }
}

template <int E>
__global__ __launch_bounds__(kSortThreads) void echo_embed_place_k(const EmbedBwdArgs given, const Share sh, int shift,
                                                                   const uint32_t* keys, const uint32_t* order,
                                                                   const uint32_t* counts, uint32_t* keys_to,
                                                                   uint32_t* order_to) {
  __shared__ SortLds lds;
  __shared__ uint32_t start[kDigits];  // the digit's first place in the tile
  const auto* a = kernel_args<EmbedBwdArgs>();
  if (blockIdx.x >= sh.work) {
    clear_tables<E>(a, sh.part, sh.parts, sh.work);
    return;
  }
  uint32_t key[kTileRounds], at[kTileRounds], place[kTileRounds];
  load_tile(a, keys, order, key, at);
  places(key, shift, &lds, place);
  // the first wavefront's offsets are the digits' starts
  if (threadIdx.x < kDigits) start[threadIdx.x] = lds.count[0][threadIdx.x];
  __syncthreads();
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
#pragma unroll
  for (int r = 0; r < kTileRounds; ++r) {
    const int64_t i = blockIdx.x * kEmbedTile + (wave * kTileRounds + r) * 64 + lane;
    if (i < a->T) {
      const uint32_t d = (key[r] >> shift) & (kDigits - 1);
      const uint32_t to = counts[d * static_cast<int64_t>(sh.work) + blockIdx.x] + place[r] - start[d];
      keys_to[to] = key[r];
      order_to[to] = at[r];
    }
  }
}

// ---- sums over runs ----------------------------------------------------------------------

// The columns that thread `lane` of 2^shift has in the tile; all 8 below `lo` where it
// has none.
__device__ __forceinline__ Run columns_of(uint32_t tile, uint32_t lane, int shift, int64_t C) {
  const uint32_t at = ((tile << shift) + lane) * 8;
  if (static_cast<int64_t>(at) + 8 <= C) return Run{at, 0};
  return Run{static_cast<uint32_t>(C) - 8, static_cast<int64_t>(at) < C ? static_cast<int>(at + 8 - static_cast<uint32_t>(C)) : 8};
}

template <int E, typename Args>
__device__ __forceinline__ void write_row(const Args* a, uint32_t key, Run run, const float acc[8]) {
  const uint32_t V = static_cast<uint32_t>(a->V), r = key / V, v = key - r * V;
  float o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = acc[i] * a->scale;
  store_from<E>(a->dtable[r], v * a->ldt, run, o);
}

constexpr int kBatch = 8;  // rows in flight to a thread
constexpr int kSumThreads = 512;

// A workgroup takes the tokens of kSumThreads >> shift consecutive chunks, 2^shift threads (64
// at most) to a chunk, and 8 << shift columns.  A chunk writes the rows of runs inside it and
// leaves the sums of its first and last run in LDS; a thread a column then adds those along
// the chunks.  part: two rows of C to a workgroup, for the run that crosses its start and for
// the one that crosses its end only.  WAVE: a chunk to a wavefront (shift 6), whose tokens
// come through scalar loads.  Workgroups next to each other take the tiles of the same tokens' rows,
// so that an XCD stays with a tile (4 tables of 16384 x 4096 fp32, 16384 tokens: 238 us in all, with
// the tokens first 244).
template <int O, int E, bool WAVE>
__global__ __launch_bounds__(kSumThreads) void echo_embed_sum_k(const EmbedBwdArgs given, int shift, int length,
                                                                const uint32_t* __restrict__ keys,
                                                                const uint32_t* __restrict__ order,
                                                                float* __restrict__ part) {
  __shared__ float head[kSumThreads * 8], tail[kSumThreads * 8];
  __shared__ uint32_t first[kSumThreads], last[kSumThreads];
  const auto* a = kernel_args<EmbedBwdArgs>();
  const int64_t C = a->C, T = a->T;
  const uint32_t none = static_cast<uint32_t>(a->P * a->V);
  const int subs = kSumThreads >> shift, width = 8 << shift;
  uint32_t sub = threadIdx.x >> shift;
  if constexpr (WAVE) sub = __builtin_amdgcn_readfirstlane(sub);
  const uint32_t lane = threadIdx.x & ((1u << shift) - 1);
  const Run run = columns_of(blockIdx.x, lane, shift, C);
  const int64_t block = static_cast<int64_t>(blockIdx.y) * subs * length;  // the workgroup's first token
  const int64_t lo = block + static_cast<int64_t>(sub) * length, hi = lo + length < T ? lo + length : T;
  // the tokens around the workgroup's
  const int64_t end = block + static_cast<int64_t>(subs) * length;
  const uint32_t before = block > 0 ? keys[block - 1] : ~0u, behind = end < T ? keys[end] : ~0u;
  if (lo < T) {
    float acc[8];
    uint32_t cur = keys[lo];
    const uint32_t start = cur;
    if (lane == 0) first[sub] = start;
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
    const auto leave = [&](float* to) {  // this thread's columns of the tile
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i >= run.lo) to[sub * width + lane * 8 + i - run.lo] = acc[i];
    };
    for (int64_t i = lo; i < hi; i += kBatch) {
      uint32_t k[kBatch];
      Raw<O> v[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int64_t t = i + j < hi ? i + j : hi - 1;
        k[j] = keys[t];
        load_any<O>(a->dout, order[t] * a->lddo, run, &v[j]);
      }
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        if (i + j >= hi) break;
        if (k[j] != cur) {
          if (cur == start) leave(head);
          else if (run.lo < 8) write_row<E>(a, cur, run, acc);
#pragma unroll
          for (int n = 0; n < 8; ++n) acc[n] = 0.0f;
          cur = k[j];
        }
        float w[8];
        widen<O>(v[j], w);
#pragma unroll
        for (int n = 0; n < 8; ++n) acc[n] = acc[n] + w[n];
      }
    }
    leave(cur == start ? head : tail);
    if (lane == 0) last[sub] = cur;
  }
  __syncthreads();
  const int64_t col = static_cast<int64_t>(blockIdx.x) * width + threadIdx.x;
  if (static_cast<int>(threadIdx.x) >= width || col >= C) return;
  const auto put = [&](uint32_t key, float sum, bool at_end) {
    if (key == none) return;  // tokens without a row
    if (key == before) {
      part[2 * blockIdx.y * C + col] = sum;
    } else if (at_end && key == behind) {
      part[(2 * blockIdx.y + 1) * C + col] = sum;
    } else {
      const uint32_t V = static_cast<uint32_t>(a->V), r = key / V, v = key - r * V;
      store1<E>(a->dtable[r], v * a->ldt + col, sum * a->scale);
    }
  };
  uint32_t cur = first[0];
  float sum = 0.0f;
  for (int s = 0; s < subs && block + static_cast<int64_t>(s) * length < T; ++s) {
    const uint32_t f = first[s], l = last[s];
    if (f != cur) {
      put(cur, sum, false);
      cur = f;
      sum = 0.0f;
    }
    sum = sum + head[s * width + threadIdx.x];
    if (l != f) {
      put(cur, sum, false);
      cur = l;
      sum = tail[s * width + threadIdx.x];
    }
  }
  put(cur, sum, true);
}

// The runs that cross workgroups of the sums, `length` tokens to each: the one where a run
// starts adds up its parts.  2^shift threads to its columns.
template <int E>
__global__ __launch_bounds__(kThreads) void echo_embed_join_k(const EmbedBwdArgs given, int shift, int64_t length,
                                                              const uint32_t* __restrict__ keys,
                                                              const float* __restrict__ part) {
  const auto* a = kernel_args<EmbedBwdArgs>();
  const int64_t C = a->C, T = a->T;
  const int64_t group = static_cast<int64_t>(blockIdx.x) * (kThreads >> shift) + (threadIdx.x >> shift);
  const Run run = columns_of(blockIdx.y, threadIdx.x & ((1u << shift) - 1), shift, C);
  const int64_t lo = group * length, hi = lo + length;
  if (hi >= T || run.lo == 8) return;
  const uint32_t k = keys[hi - 1];
  if (k == static_cast<uint32_t>(a->P * a->V) || keys[hi] != k) return;
  if (keys[lo] == k && lo > 0 && keys[lo - 1] == k) return;  // it starts further up
  // the run's end: the first place behind hi with another key
  int64_t b = hi, e = T;
  while (b < e) {
    const int64_t m = (b + e) >> 1;
    if (keys[m] == k) b = m + 1;
    else e = m;
  }
  const int64_t last = (b - 1) / length;
  Raw<kElemF32> v[kBatch];
  float acc[8];
  load_any<kElemF32>(part, (2 * group + 1) * C, run, &v[0]);
  widen<kElemF32>(v[0], acc);
  for (int64_t c = group + 1; c <= last; c += kBatch) {
#pragma unroll
    for (int j = 0; j < kBatch; ++j) load_any<kElemF32>(part, 2 * (c + j < last ? c + j : last) * C, run, &v[j]);
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      if (c + j > last) break;
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] = acc[i] + v[j].v[i];
    }
  }
  write_row<E>(a, k, run, acc);
}

template <bool WAVE, int O, int E>
hipError_t launch_sums(const EmbedBwdArgs& a, int shift, const uint32_t* keys, const uint32_t* order, float* part,
                       hipStream_t s) {
  const int64_t runs = (a.C + 7) / 8, length = embed_chunk(a.T), group = length * (kSumThreads >> shift);
  const int64_t groups = (a.T + group - 1) / group;
  hipLaunchKernelGGL((echo_embed_sum_k<O, E, WAVE>),
                     dim3(static_cast<unsigned>((runs + (1 << shift) - 1) >> shift), static_cast<unsigned>(groups)),
                     dim3(kSumThreads), 0, s, a, shift, static_cast<int>(length), keys, order, part);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || groups == 1) return e;
  int js = shift;
  while (js < 8 && (int64_t{1} << js) < runs) ++js;
  const int64_t per = kThreads >> js;
  hipLaunchKernelGGL((echo_embed_join_k<E>),
                     dim3(static_cast<unsigned>((groups + per - 1) / per), static_cast<unsigned>((runs + (1 << js) - 1) >> js)),
                     dim3(kThreads), 0, s, a, js, group, keys, part);
  return hipGetLastError();
}

// More than kSmall tokens.  *in: which of the two buffers they end in.
template <int E>
hipError_t launch_sort(const EmbedBwdArgs& a, int digits, uint32_t* const keys[2], uint32_t* const order[2], uint32_t* counts,
                       int* in, hipStream_t s) {
  const unsigned tiles = static_cast<unsigned>(embed_tiles(a.T));
  hipError_t e;
  Share sh{tiles, 0, 3 * digits};
  for (int d = 0; d < digits; ++d, *in ^= 1) {
    const uint32_t *k = d == 0 ? nullptr : keys[*in], *o = d == 0 ? nullptr : order[*in];
    const int shift = kDigitBits * d;
    hipLaunchKernelGGL(echo_embed_count_k<E>, dim3(tiles + kClearGroups), dim3(kSortThreads), 0, s, a, sh, shift, k, counts);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    ++sh.part;
    sh.work = 1;
    hipLaunchKernelGGL(echo_embed_scan_k<E>, dim3(1 + kClearGroups), dim3(kSortThreads), 0, s, a, sh, counts,
                       tiles * int64_t{kDigits});
    if ((e = hipGetLastError()) != hipSuccess) return e;
    ++sh.part;
    sh.work = tiles;
    hipLaunchKernelGGL(echo_embed_place_k<E>, dim3(tiles + kClearGroups), dim3(kSortThreads), 0, s, a, sh, shift, k, o, counts,
                       keys[*in ^ 1], order[*in ^ 1]);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    ++sh.part;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_embed_bwd(const EmbedBwdArgs& given, Elem dout, Elem table, hipStream_t s) {
  EmbedBwdArgs a = given;
  a.stream = a.P * a.V * a.C * elem_size(table) >= int64_t{256} << 20 || a.T * a.C * elem_size(dout) >= int64_t{256} << 20;
  const int64_t T = a.T;
  const EmbedLayout w = embed_layout(T, a.C);
  char* base = static_cast<char*>(a.workspace);
  uint32_t* const keys[2] = {reinterpret_cast<uint32_t*>(base + w.keys[0]), reinterpret_cast<uint32_t*>(base + w.keys[1])};
  uint32_t* const order[2] = {reinterpret_cast<uint32_t*>(base + w.order[0]), reinterpret_cast<uint32_t*>(base + w.order[1])};
  int digits = 1;  // of keys 0 .. P V
  while (((a.P * a.V) >> (kDigitBits * digits)) != 0) ++digits;
  int in = 0;
  const int64_t elems = a.P * a.V * a.C, want = (elems + kSortThreads * 8 - 1) / (kSortThreads * 8);
  const unsigned clear = static_cast<unsigned>(want < kClearGroups - 1 ? want : kClearGroups - 1);
  return with_types(dout, dout, table, [&](auto O, auto, auto E) -> hipError_t {
    hipError_t e = hipSuccess;
    if (T == 0)
      hipLaunchKernelGGL((echo_embed_clear_k<E()>), dim3(clear), dim3(kSortThreads), 0, s, a);
    else if (T <= kSortThreads)
      hipLaunchKernelGGL((echo_embed_sort_k<E(), 1>), dim3(1 + clear), dim3(kSortThreads), 0, s, a, digits, keys[0], order[0]);
    else if (T <= 4 * kSortThreads)
      hipLaunchKernelGGL((echo_embed_sort_k<E(), 4>), dim3(1 + clear), dim3(kSortThreads), 0, s, a, digits, keys[0], order[0]);
    else if (T <= 8 * kSortThreads)
      hipLaunchKernelGGL((echo_embed_sort_k<E(), 8>), dim3(1 + clear), dim3(kSortThreads), 0, s, a, digits, keys[0], order[0]);
    else if (T <= kSmall)
      hipLaunchKernelGGL((echo_embed_sort_k<E(), kSmallRounds>), dim3(1 + clear), dim3(kSortThreads), 0, s, a, digits, keys[0],
                         order[0]);
    else
      e = launch_sort<E()>(a, digits, keys, order, reinterpret_cast<uint32_t*>(base + w.counts), &in, s);
    if (e == hipSuccess) e = hipGetLastError();
    if (e != hipSuccess || T == 0) return e;
    const int shift = embed_shift(a.C);
    float* part = reinterpret_cast<float*>(base + w.part);
    return shift == 6 ? launch_sums<true, O(), E()>(a, shift, keys[in], order[in], part, s)
                      : launch_sums<false, O(), E()>(a, shift, keys[in], order[in], part, s);
  });
}

}  // namespace echo
