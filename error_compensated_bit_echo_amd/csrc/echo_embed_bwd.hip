// Gradient of the embedding: dtable_r[v] = scale * (sum of dout[t] over the tokens t with
// row r V + v, in rising order of t), zeros for rows without a token.
//
// The tokens are sorted by row (stable, so equal tokens stay in order), then runs of equal
// tokens are summed: no atomics, so the result is the same from call to call, and a row is
// written once.  The sort is a radix sort of 8-bit digits.  Up to kSmall tokens one
// workgroup holds them all in LDS, while the launch's other workgroups clear the tables.
// More tokens take three launches a digit: counts per tile, their prefix sums, placement.
//
// The sorted tokens are cut into chunks of equal length, whatever the runs: a chunk writes
// the rows of runs that lie inside it, and puts the sum of a run that crosses its start or
// its end into the workspace; a last launch adds those up along the chunks.  So a token
// that comes up ten thousand times costs as much as ten thousand different ones.
#include "echo_row.h"

namespace echo {
namespace {

constexpr int kSortThreads = 1024;
constexpr int kWaves = kSortThreads / 64;
constexpr int kDigits = 256;
constexpr int kSmallRounds = 16;
constexpr int64_t kSmall = kSortThreads * kSmallRounds;  // tokens that one workgroup sorts: 128 KB of LDS
constexpr int kTileRounds = 4;
constexpr int64_t kTile = kSortThreads * kTileRounds;
constexpr int kThreads = 256;

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
    uint64_t same = ~uint64_t{0};  // the lanes with this digit
#pragma unroll
    for (int b = 0; b < 8; ++b) {
      const uint64_t set = __ballot((d >> b) & 1);
      same &= (d >> b) & 1 ? set : ~set;
    }
    const int before = __popcll(same & ((uint64_t{1} << lane) - 1));
    uint32_t old = 0;
    if (before == 0) old = atomicAdd(&lds->count[wave][d], static_cast<uint32_t>(__popcll(same)));
    place[r] = __shfl(old, __ffsll(static_cast<unsigned long long>(same)) - 1) + static_cast<uint32_t>(before);
  }
  __syncthreads();
  // exclusive prefix sums of the counts, digit by digit and within a digit by wavefront:
  // four counters to a thread
  const int d = threadIdx.x >> 2, w0 = (threadIdx.x & 3) * 4;
  uint32_t c[4], sum = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
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
  for (int i = 0; i < 4; ++i) lds->count[w0 + i][d] = base + c[i];
  __syncthreads();
#pragma unroll
  for (int r = 0; r < ROUNDS; ++r) place[r] += lds->count[wave][(key[r] >> digit_shift) & (kDigits - 1)];
}

// Clears the tables, workgroup `id` of `of`.
template <int E, typename Args>
__device__ __forceinline__ void clear_tables(const Args* a, int64_t id, int64_t of) {
  const int64_t C = a->C, rows = a->P * a->V;
  const float zero[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  for (int64_t row = id; row < rows; row += of) {
    const int64_t r = row / a->V, v = row - r * a->V;
    void* table = a->dtable[r];
    for (int64_t at = static_cast<int64_t>(threadIdx.x) * 8; at < C; at += kSortThreads * 8)
      store_run<E>(table, v * a->ldt + at, run_length(at, C), zero);
  }
}

// Workgroup 0 sorts up to kSmall tokens; the others clear the tables.
template <int E>
__global__ __launch_bounds__(kSortThreads) void echo_embed_sort_k(const EmbedBwdArgs given, int digits, uint32_t* keys,
                                                                  uint32_t* order) {
  __shared__ SortLds lds;
  __shared__ uint32_t sk[kSmall], so[kSmall];
  const auto* a = kernel_args<EmbedBwdArgs>();
  if (blockIdx.x != 0) {
    clear_tables<E>(a, blockIdx.x - 1, gridDim.x - 1);
    return;
  }
  const int T = static_cast<int>(a->T);
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  uint32_t key[kSmallRounds], at[kSmallRounds], place[kSmallRounds];
#pragma unroll
  for (int r = 0; r < kSmallRounds; ++r) {
    const int i = (wave * kSmallRounds + r) * 64 + lane;
    key[r] = i < T ? key_of(a, i) : ~0u;  // behind every key in every digit
    at[r] = static_cast<uint32_t>(i);
  }
  for (int d = 0; d < digits; ++d) {
    places(key, 8 * d, &lds, place);
#pragma unroll
    for (int r = 0; r < kSmallRounds; ++r) {
      sk[place[r]] = key[r];
      so[place[r]] = at[r];
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kSmallRounds; ++r) {
      const int i = (wave * kSmallRounds + r) * 64 + lane;
      key[r] = sk[i];
      at[r] = so[i];
    }
  }
#pragma unroll
  for (int r = 0; r < kSmallRounds; ++r) {
    const int i = (wave * kSmallRounds + r) * 64 + lane;
    if (i < T) {
      keys[i] = key[r];
      order[i] = at[r];
    }
  }
}

template <int E>
__global__ __launch_bounds__(kSortThreads) void echo_embed_clear_k(const EmbedBwdArgs given) {
  clear_tables<E>(kernel_args<EmbedBwdArgs>(), blockIdx.x, gridDim.x);
}

// ---- more than kSmall tokens -------------------------------------------------------------

// keys == nullptr: the keys are formed from the tokens, the order is their own.
template <typename Args>
__device__ __forceinline__ void load_tile(const Args* a, const uint32_t* keys, const uint32_t* order, uint32_t (&key)[kTileRounds],
                                          uint32_t (&at)[kTileRounds]) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
#pragma unroll
  for (int r = 0; r < kTileRounds; ++r) {
    const int64_t i = blockIdx.x * kTile + (wave * kTileRounds + r) * 64 + lane;
    key[r] = ~0u;
    at[r] = static_cast<uint32_t>(i);
    if (i < a->T) {
      key[r] = keys != nullptr ? keys[i] : key_of(a, i);
      if (order != nullptr) at[r] = order[i];
    }
  }
}

// counts[digit * tiles + tile]
__global__ __launch_bounds__(kSortThreads) void echo_embed_count_k(const EmbedBwdArgs given, int shift, const uint32_t* keys,
                                                                   uint32_t* counts) {
  __shared__ uint32_t n[kDigits];
  const auto* a = kernel_args<EmbedBwdArgs>();
  if (threadIdx.x < kDigits) n[threadIdx.x] = 0;
  __syncthreads();
  uint32_t key[kTileRounds], at[kTileRounds];
  load_tile(a, keys, nullptr, key, at);
#pragma unroll
  for (int r = 0; r < kTileRounds; ++r)
    if (static_cast<int64_t>(at[r]) < a->T) atomicAdd(&n[(key[r] >> shift) & (kDigits - 1)], 1u);
  __syncthreads();
  if (threadIdx.x < kDigits) counts[threadIdx.x * static_cast<int64_t>(gridDim.x) + blockIdx.x] = n[threadIdx.x];
}

// Exclusive prefix sums in place, one workgroup.
__global__ __launch_bounds__(kSortThreads) void echo_embed_scan_k(uint32_t* counts, int64_t n) {
  __shared__ uint32_t total[kWaves];
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

__global__ __launch_bounds__(kSortThreads) void echo_embed_place_k(const EmbedBwdArgs given, int shift, const uint32_t* keys,
                                                                   const uint32_t* order, const uint32_t* counts,
                                                                   uint32_t* keys_to, uint32_t* order_to) {
  __shared__ SortLds lds;
  __shared__ uint32_t start[kDigits];  // the digit's first place in the tile
  const auto* a = kernel_args<EmbedBwdArgs>();
  uint32_t key[kTileRounds], at[kTileRounds], place[kTileRounds];
  load_tile(a, keys, order, key, at);
  places(key, shift, &lds, place);
  // the first wavefront's offsets are the digits' starts
  if (threadIdx.x < kDigits) start[threadIdx.x] = lds.count[0][threadIdx.x];
  __syncthreads();
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
#pragma unroll
  for (int r = 0; r < kTileRounds; ++r) {
    const int64_t i = blockIdx.x * kTile + (wave * kTileRounds + r) * 64 + lane;
    if (i < a->T) {
      const uint32_t d = (key[r] >> shift) & (kDigits - 1);
      const uint32_t to = counts[d * static_cast<int64_t>(gridDim.x) + blockIdx.x] + place[r] - start[d];
      keys_to[to] = key[r];
      order_to[to] = at[r];
    }
  }
}

// ---- sums over runs ----------------------------------------------------------------------

// Tokens to a chunk.
constexpr int64_t kRun = 32;

template <int E, typename Args>
__device__ __forceinline__ void write_row(const Args* a, uint32_t key, int64_t at, int n, const float acc[8]) {
  const int64_t r = key / a->V, v = key - r * a->V;
  float o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = acc[i] * a->scale;
  store_run<E>(a->dtable[r], v * a->ldt + at, n, o);
}

// 2^shift threads to a chunk's columns.  part: two rows of C to a chunk, for the run that
// crosses its start and for the one that crosses its end only.
template <int O, int E>
__global__ __launch_bounds__(kThreads) void echo_embed_sum_k(const EmbedBwdArgs given, int shift, const uint32_t* keys,
                                                             const uint32_t* order, float* part) {
  const auto* a = kernel_args<EmbedBwdArgs>();
  const int64_t chunk = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) >> shift, C = a->C, T = a->T;
  const int64_t at = ((static_cast<int64_t>(blockIdx.y) << shift) + (threadIdx.x & ((1 << shift) - 1))) * 8;
  const int64_t lo = chunk * kRun, hi = lo + kRun < T ? lo + kRun : T;
  if (lo >= T || at >= C) return;
  const uint32_t none = static_cast<uint32_t>(a->P * a->V);
  const int n = run_length(at, C);
  const uint32_t before = lo > 0 ? keys[lo - 1] : ~0u, behind = hi < T ? keys[hi] : ~0u, first = keys[lo];
  float acc[8];
  uint32_t cur = first;
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
  for (int64_t i = lo; i < hi; ++i) {
    const uint32_t k = keys[i];
    if (k != cur) {
      if (cur == before) store_run<kElemF32>(part, (2 * chunk) * C + at, n, acc);
      else write_row<E>(a, cur, at, n, acc);
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] = 0.0f;
      cur = k;
    }
    if (k == none) return;  // nothing but tokens without a row from here on
    float v[8];
    load_run<O>(a->dout, order[i] * a->lddo + at, n, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[j] = acc[j] + v[j];
  }
  if (cur == before) store_run<kElemF32>(part, (2 * chunk) * C + at, n, acc);
  else if (cur == behind) store_run<kElemF32>(part, (2 * chunk + 1) * C + at, n, acc);
  else write_row<E>(a, cur, at, n, acc);
}

// The runs that cross chunks: the chunk where one starts adds up its parts.
template <int E>
__global__ __launch_bounds__(kThreads) void echo_embed_join_k(const EmbedBwdArgs given, int shift, const uint32_t* keys,
                                                              const float* part) {
  const auto* a = kernel_args<EmbedBwdArgs>();
  const int64_t chunk = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) >> shift, C = a->C, T = a->T;
  const int64_t at = ((static_cast<int64_t>(blockIdx.y) << shift) + (threadIdx.x & ((1 << shift) - 1))) * 8;
  const int64_t lo = chunk * kRun, hi = lo + kRun;
  if (hi >= T || at >= C) return;
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
  const int n = run_length(at, C);
  float acc[8];
  load_run<kElemF32>(part, (2 * chunk + 1) * C + at, n, acc);
  const int64_t last = (b - 1) / kRun;
  for (int64_t c = chunk + 1; c <= last; ++c) {
    float v[8];
    load_run<kElemF32>(part, (2 * c) * C + at, n, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = acc[i] + v[i];
  }
  write_row<E>(a, k, at, n, acc);
}

size_t align256(size_t n) { return (n + 255) & ~size_t{255}; }

int64_t tiles_of(int64_t T) { return (T + kTile - 1) / kTile; }

}  // namespace

// Two pairs of keys and places, the tiles' counts, the parts of the chunks.
size_t embed_workspace(int64_t T, int64_t C) {
  if (T == 0) return 0;
  return 4 * align256(static_cast<size_t>(T) * 4) + align256(static_cast<size_t>(tiles_of(T)) * kDigits * 4) +
         static_cast<size_t>((T + kRun - 1) / kRun) * 2 * static_cast<size_t>(C) * sizeof(float);
}

hipError_t launch_embed_bwd(const EmbedBwdArgs& a, Elem dout, Elem table, hipStream_t s) {
  const int64_t T = a.T, n_rows = a.P * a.V;
  const unsigned fill = static_cast<unsigned>(n_rows < 2048 ? n_rows : 2048);
  char* w = static_cast<char*>(a.workspace);
  uint32_t *keys[2], *order[2];
  for (int i = 0; i < 2; ++i) {
    keys[i] = reinterpret_cast<uint32_t*>(w);
    w += align256(static_cast<size_t>(T) * 4);
    order[i] = reinterpret_cast<uint32_t*>(w);
    w += align256(static_cast<size_t>(T) * 4);
  }
  uint32_t* counts = reinterpret_cast<uint32_t*>(w);
  float* part = reinterpret_cast<float*>(w + align256(static_cast<size_t>(tiles_of(T)) * kDigits * 4));
  int digits = 1;  // of keys 0 .. n_rows
  while (digits < 4 && (n_rows >> (8 * digits)) != 0) ++digits;
  int in = 0;
  return with_types(dout, dout, table, [&](auto O, auto, auto E) -> hipError_t {
    hipError_t e;
    if (T == 0 || T > kSmall) {
      hipLaunchKernelGGL((echo_embed_clear_k<E()>), dim3(fill), dim3(kSortThreads), 0, s, a);
      if ((e = hipGetLastError()) != hipSuccess || T == 0) return e;
      const unsigned tiles = static_cast<unsigned>(tiles_of(T));
      for (int d = 0; d < digits; ++d, in ^= 1) {
        const uint32_t *k = d == 0 ? nullptr : keys[in], *o = d == 0 ? nullptr : order[in];
        hipLaunchKernelGGL(echo_embed_count_k, dim3(tiles), dim3(kSortThreads), 0, s, a, 8 * d, k, counts);
        if ((e = hipGetLastError()) != hipSuccess) return e;
        hipLaunchKernelGGL(echo_embed_scan_k, dim3(1), dim3(kSortThreads), 0, s, counts, tiles * int64_t{kDigits});
        if ((e = hipGetLastError()) != hipSuccess) return e;
        hipLaunchKernelGGL(echo_embed_place_k, dim3(tiles), dim3(kSortThreads), 0, s, a, 8 * d, k, o, counts, keys[in ^ 1],
                           order[in ^ 1]);
        if ((e = hipGetLastError()) != hipSuccess) return e;
      }
    } else {
      hipLaunchKernelGGL((echo_embed_sort_k<E()>), dim3(1 + fill), dim3(kSortThreads), 0, s, a, digits, keys[0], order[0]);
      if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    const int64_t runs = (a.C + 7) / 8, chunks = (T + kRun - 1) / kRun;
    int shift = 0;
    while (shift < 8 && (int64_t{1} << shift) < runs) ++shift;
    const int64_t per = kThreads >> shift;
    const dim3 grid(static_cast<unsigned>((chunks + per - 1) / per), static_cast<unsigned>((runs + (1 << shift) - 1) >> shift));
    hipLaunchKernelGGL((echo_embed_sum_k<O(), E()>), grid, dim3(kThreads), 0, s, a, shift, keys[in], order[in], part);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if (chunks > 1) {
      hipLaunchKernelGGL((echo_embed_join_k<E()>), grid, dim3(kThreads), 0, s, a, shift, keys[in], part);
      e = hipGetLastError();
    }
    return e;
  });
}

}  // namespace echo
