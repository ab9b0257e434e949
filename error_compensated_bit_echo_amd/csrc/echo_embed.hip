// Rows of a table whose vocabulary is split over ranks: out_r[t] = scale * table_r[tokens[t]
// - first - r V] where that row is in [0, V), zeros elsewhere, for every rank of the call.
// A thread takes 8 columns of a row of the output; a table's row is read by its owner only.
// Bound by the memory: 16384 tokens of 131072 x 8192 bfloat16 take 91 us, 5.9 TB/s.
#include "echo_row.h"

namespace echo {
namespace {

constexpr int kThreads = 256;

// 2^shift threads to a row.
template <int E, int O>
__global__ __launch_bounds__(kThreads) void echo_embed_k(const EmbedArgs given, int shift) {
  const auto* a = kernel_args<EmbedArgs>();
  const int64_t C = a->C, rows = int64_t{gridDim.x} * (kThreads >> shift);
  const int64_t at = ((static_cast<int64_t>(blockIdx.y) << shift) + (threadIdx.x & ((1 << shift) - 1))) * 8;
  if (at >= C) return;
  const int n = run_length(at, C);
  for (int64_t row = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) >> shift; row < a->T; row += rows) {
    const int64_t token = a->wide ? static_cast<const int64_t*>(a->tokens)[row] : static_cast<const int32_t*>(a->tokens)[row];
    uint64_t v = static_cast<uint64_t>(token) - static_cast<uint64_t>(a->first);  // wraps: no row for what lies before
    for (int r = 0; r < a->P; ++r, v -= static_cast<uint64_t>(a->V)) {
      float x[8];
      if (v < static_cast<uint64_t>(a->V)) {
        load_run<E>(a->table[r], static_cast<int64_t>(v) * a->ldt + at, n, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = x[i] * a->scale;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = 0.0f;
      }
      store_run<O>(a->out[r], row * a->ldo + at, n, x);
    }
  }
}

}  // namespace

hipError_t launch_embed(const EmbedArgs& a, Elem table, Elem out, hipStream_t s) {
  const int64_t runs = (a.C + 7) / 8;
  int shift = 0;
  while (shift < 8 && (int64_t{1} << shift) < runs) ++shift;
  const int64_t rows = kThreads >> shift;
  // a launch numbers its threads along an axis in 32 bits
  const int64_t want = (a.T + rows - 1) / rows, most = ((int64_t{1} << 32) - 1) / kThreads;
  const dim3 grid(static_cast<unsigned>(want < most ? want : most), static_cast<unsigned>((runs + (1 << shift) - 1) >> shift));
  return with_types(table, table, out, [&](auto E, auto, auto O) {
    hipLaunchKernelGGL((echo_embed_k<E(), O()>), grid, dim3(kThreads), 0, s, a, shift);
    return hipGetLastError();
  });
}

}  // namespace echo
