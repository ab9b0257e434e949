// Internal interface of the operators of a training step around the tensor-parallel
// blocks (block norm, gradient clipping, embedding): launch arguments.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "echo_layer_internal.h"

namespace echo {

constexpr int64_t kStepMaxCols = int64_t{1} << 22;  // columns of a norm's or an embedding's row

// The parameters of a block's norms and gate, as both directions read them.
struct BlockParams {
  const void* gate;    // nullptr: 1
  const void* w_post;  // nullptr: 1
  const void* w_pre;   // nullptr: 1
  int64_t ldg, n_gates, rows_per_gate;  // n_gates 1 without a gate
  int64_t R, C;
  float alpha, offset, eps;
  int32_t elem;  // Elem of gate, w_post and w_pre
  int32_t post;  // y is normalised
};

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

// Gradient clipping: a launch takes up to kClipTensors tensors in its arguments.
constexpr int kClipTensors = 120;
constexpr int kClipGroups = 2048;  // workgroups, and partial sums, of a launch at most
struct ClipArgs {
  const void* src[kClipTensors];
  void* dst[kClipTensors];
  int64_t n[kClipTensors];
  uint32_t first[kClipTensors + 1];  // the tensor's first chunk
  uint8_t elem[kClipTensors];
  int32_t tensors;
};
// chunks of a tensor of n elements
int64_t clip_chunks(int64_t n);
// part: kClipGroups doubles a launch, filled from `at` on; *used: how many it wrote
hipError_t launch_clip_sum(const ClipArgs& a, double* part, int64_t at, int64_t* used, hipStream_t s);
// norm: written (by the first of several launches) if not nullptr
hipError_t launch_clip_scale(const ClipArgs& a, const double* part, int64_t n_part, double max_norm, float* norm,
                             hipStream_t s);
hipError_t launch_clip_norm(const double* part, int64_t n_part, float* norm, hipStream_t s);

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
  void* workspace;  // embed_workspace(...) bytes, 256-byte aligned
};
size_t embed_workspace(int64_t T, int64_t C);
hipError_t launch_embed_bwd(const EmbedBwdArgs& a, Elem dout, Elem table, hipStream_t s);

}  // namespace echo
