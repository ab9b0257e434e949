// Internal interface of the operators of a training step around the tensor-parallel
// blocks (block norm, gradient clipping, embedding): launch arguments.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "echo_layer_internal.h"

namespace echo {

constexpr int64_t kStepMaxCols = int64_t{1} << 22;  // columns of a norm's or an embedding's row

constexpr int64_t elem_size(int elem) { return elem == kElemF32 ? 4 : 2; }

// The parameters of a block's norms and gate, as both directions read them.
struct BlockParams {
  const void* gate;    // nullptr: 1
  const void* w_post;  // nullptr: 1
  const void* w_pre;   // nullptr: 1
  int64_t ldg, n_gates, rows_per_gate;  // n_gates 1 without a gate
  int64_t R, C;
  float alpha, offset, eps, inv_cols;  // inv_cols: 1 / C
  int32_t elem;  // Elem of gate, w_post and w_pre
  int32_t post;  // y is normalised
};

// Whether a call moves more than the last-level cache holds (256 MB): its 16-bit results then go
// past the caches, where they would only replace inputs that later rows, or the next call, read.
// Smaller results stay for the kernel that reads them next.
inline bool block_streams(int64_t R, int64_t C, int64_t bytes) { return R * C >= (int64_t{256} << 20) / bytes; }

struct BlockNormArgs {
  BlockParams p;
  const void* x;
  const void* y;  // nullptr: out is x and not written
  void* out;
  void* a;  // nullptr: not wanted
  int64_t ldx, ldy, ldo, lda;
};
hipError_t launch_block_norm(const BlockNormArgs& a, Elem x, Elem y, Elem out_a, hipStream_t s);

struct BlockNormBwdArgs {
  BlockParams p;
  const void* out;   // the stream as stored
  const void* y;     // nullptr: none
  const void* dout;  // nullptr: 0
  const void* da;    // nullptr: 0
  void* dx;          // nullptr: not wanted, as the other outputs
  void* dy;
  void* dgate;
  void* dw_post;
  void* dw_pre;
  int64_t ldo, ldy, lddo, ldda, lddx, lddy, lddg;
  float* part;   // workspace: column sums of the workgroups
  float4* stats;  // and the rows' statistics
};
constexpr int kMaxThreads = 1024;

// Threads for rows of C columns, 8 * `runs` of them to a thread.
inline int row_threads(int64_t C, int runs) {
  const int64_t t = (C + 8 * runs - 1) / (8 * runs);
  return static_cast<int>(t >= kMaxThreads ? kMaxThreads : (t + 63) / 64 * 64);
}

// Whether one workgroup holds a row's inputs and column sums in its registers; other rows
// take a pass for their statistics and one by columns.
inline bool block_fits(int64_t C) { return C >= 8 && C <= 8 * kMaxThreads; }

constexpr int64_t kColumnTile = 2048;  // columns of a workgroup of the pass by columns

// The split of the rows over workgroups that sum columns: `chunks` workgroups to a gate's
// rows, each taking every chunks-th of them (rows next to each other are worked on at the
// same time, so that their addresses spread over the memory channels: 16384 x 8192 bfloat16
// 344 us, with consecutive rows to a workgroup 354); or, where chunks is 0, `gates` whole
// gates of `rows` rows in all to a workgroup.
struct BlockSplit {
  int64_t groups, chunks, gates, rows;
};

inline BlockSplit block_split(int64_t R, int64_t n_gates, int64_t C) {
  BlockSplit s{};
  if (R == 0) return s;
  const int64_t per_gate = R / n_gates;
  // as many workgroups as 256 CUs hold at a time, 16 wavefronts to a CU
  const int64_t tiles = (C + kColumnTile - 1) / kColumnTile;
  int64_t most = block_fits(C) ? 256 * (kMaxThreads / row_threads(C, 1)) : tiles < 1024 ? 1024 / tiles : 1;
  // a workgroup's column sums cost two rows of fp32 each: at least 4 rows for them, where
  // that leaves a workgroup to every CU
  const int64_t few = R / 4 > 256 ? R / 4 : 256;
  if (most > few) most = few;
  if (n_gates < most) {
    const int64_t chunks = most / n_gates;
    s.chunks = per_gate < chunks ? per_gate : chunks;
    s.groups = n_gates * s.chunks;
  } else {
    s.gates = (n_gates + most - 1) / most;
    s.groups = (n_gates + s.gates - 1) / s.gates;
    s.rows = s.gates * per_gate;
  }
  return s;
}

// The workspace: every workgroup's three column sums, and, for rows that do not fit the
// registers, four statistics of each.
inline size_t block_norm_part(int64_t R, int64_t C, int64_t n_gates) {
  return static_cast<size_t>(block_split(R, n_gates, C).groups) * 3 * static_cast<size_t>(C) * sizeof(float);
}
inline size_t block_norm_workspace(int64_t R, int64_t C, int64_t n_gates) {
  return (block_norm_part(R, C, n_gates) + 15) / 16 * 16 + (block_fits(C) ? 0 : static_cast<size_t>(R) * 16);
}
hipError_t launch_block_norm_bwd(const BlockNormBwdArgs& a, Elem x, Elem y, Elem out_a, hipStream_t s);

// Gradient clipping: a launch takes its tensors in its arguments, cut into chunks of kClipChunk
// bytes (the last of each may be shorter), so a tensor is a pointer, its first chunk, and 16
// bits of its last chunk's length and its type; where the result goes elsewhere, a second
// pointer.  4 KB of arguments hold 176 tensors, or 280 where there is one pointer each.
constexpr int64_t kClipChunk = 32768;
// workgroups, and partial sums, of a launch at most: four to a CU (64 tensors of 16 Mi fp32 2215 us,
// with 2048 2277, with 256 2300; 331 mixed ones 46.2, 48.5 and 50.6)
constexpr int kClipGroups = 1024;
template <int N, bool APART>
struct ClipArgs {
  static constexpr int kTensors = N;
  const void* src[N];
  void* dst[APART ? N : 1];  // APART false: src itself
  uint32_t first[N + 1];     // the tensor's first chunk
  uint16_t tail[N];          // last chunk: bytes / 2 - 1, and Elem in the upper two bits
  int32_t tensors;
};
typedef ClipArgs<280, false> ClipInPlace;
typedef ClipArgs<176, true> ClipApart;
inline int64_t clip_chunks(int64_t bytes) { return (bytes + kClipChunk - 1) / kClipChunk; }
inline uint16_t clip_tail(int64_t bytes, int32_t elem) {
  const int64_t last = bytes - (clip_chunks(bytes) - 1) * kClipChunk;
  return static_cast<uint16_t>((last / 2 - 1) | elem << 14);
}
inline unsigned clip_grid(uint32_t chunks) {
  return chunks < static_cast<uint32_t>(kClipGroups) ? chunks : static_cast<unsigned>(kClipGroups);
}
// part: a partial sum for each of clip_grid(chunks) workgroups
hipError_t launch_clip_sum(const ClipInPlace& a, double* part, hipStream_t s);
// Results go past the caches where the tensors and they do not fit the last-level cache
// together (64 MB of fp32 in 16 tensors; 256 MB: 153 us, 123 past them).
constexpr int64_t kClipStream = int64_t{128} << 20;
// norm: written if not nullptr
hipError_t launch_clip_scale(const ClipInPlace& a, const double* part, int64_t n_part, double max_norm, float* norm,
                             bool stream, hipStream_t s);
hipError_t launch_clip_scale(const ClipApart& a, const double* part, int64_t n_part, double max_norm, float* norm,
                             bool stream, hipStream_t s);
hipError_t launch_clip_norm(const double* part, int64_t n_part, float* norm, hipStream_t s);
// part[0] = the sum of all: more partial sums than one launch leaves cost a launch of their own
// less than every workgroup of every launch adding them up (with 2048 a launch: 331 tensors, 46.8 us
// and 47.6; 1200 of 256 KB, 200 and 249; 6000, 1039 and 2484)
hipError_t launch_clip_join(double* part, int64_t n_part, hipStream_t s);

struct EmbedArgs {
  const void* table[kMaxRanks];
  void* out[kMaxRanks];
  const void* tokens;
  int64_t V, C, ldt, T, ldo, first;
  float scale;
  int32_t P, wide;  // wide: 64-bit tokens
};
hipError_t launch_embed(const EmbedArgs& a, Elem table, Elem out, hipStream_t s);

struct EmbedBwdArgs {
  void* dtable[kMaxRanks];
  const void* dout;
  const void* tokens;
  int64_t V, C, ldt, T, lddo, first;
  float scale;
  int32_t P, wide;
  int32_t stream;   // set by the launcher: zeros go past the caches
  void* workspace;  // embed_layout(...).bytes, 256-byte aligned
};

constexpr int64_t kEmbedTile = 4096;  // tokens of a tile of the sort
inline int64_t embed_tiles(int64_t T) { return (T + kEmbedTile - 1) / kEmbedTile; }

// 2^embed_shift threads, 64 at most, take the columns of a row, 8 each and as often as needed.
__host__ __device__ inline int embed_shift(int64_t C) {
  int shift = 0;
  while (shift < 6 && (int64_t{8} << shift) < C) ++shift;
  return shift;
}

// Sorted tokens to a chunk: 8 for few tokens, so that none waits for another; more for many,
// since runs over many chunks are added up chunk by chunk.
inline int64_t embed_chunk(int64_t T) {
  if (T <= 4096) return 8;
  int64_t n = 16;
  while (T > n * 8192) n *= 2;
  return n;
}

// Where the workspace's parts lie: two pairs of keys and places, the tiles' counts of 512
// digits, two rows of fp32 for every 512 threads' worth of chunks.
struct EmbedLayout {
  size_t keys[2], order[2], counts, part, bytes;
};
inline EmbedLayout embed_layout(int64_t T, int64_t C) {
  EmbedLayout w{};
  const auto take = [&w](size_t n) {
    const size_t at = w.bytes;
    w.bytes += (n + 255) & ~size_t{255};
    return at;
  };
  if (T == 0) return w;
  const int buffers = T > 4 * kEmbedTile ? 2 : 1;  // one workgroup sorts 16384 tokens in place
  for (int i = 0; i < buffers; ++i) {
    w.keys[i] = take(static_cast<size_t>(T) * 4);
    w.order[i] = take(static_cast<size_t>(T) * 4);
  }
  if (buffers == 2) w.counts = take(static_cast<size_t>(embed_tiles(T)) * 512 * 4);
  const int64_t group = embed_chunk(T) * (512 >> embed_shift(C)), groups = (T + group - 1) / group;
  w.part = take(static_cast<size_t>(groups) * 2 * static_cast<size_t>(C) * sizeof(float));
  return w;
}
hipError_t launch_embed_bwd(const EmbedBwdArgs& a, Elem dout, Elem table, hipStream_t s);

}  // namespace echo
