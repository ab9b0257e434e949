// What the C-ABI host code of the layer's operators checks of its arguments: element
// types, alignment, row pitches, and which memory a strided matrix takes.
#pragma once

#include <stdint.h>

#include "echo.h"

namespace {

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

inline bool elem_bytes(int32_t dtype, int64_t* bytes) {
  if (dtype == ECHO_F32) *bytes = 4;
  else if (dtype == ECHO_BF16 || dtype == ECHO_F16) *bytes = 2;
  else return false;
  return true;
}

// Whether rows `ld` elements of `es` bytes apart do not overlap and span at most 2^48
// bytes: beyond what a device addresses, and far from where the arithmetic below wraps.
inline bool pitch_fits(int64_t rows, int64_t cols, int64_t ld, int64_t es) {
  return rows <= 1 || (ld >= cols && ld <= (int64_t{1} << 48) / (rows * es));
}

// The pitch of `rows` rows of `cols`: where there is one row, `ld` says nothing.
inline int64_t pitch_of(int64_t rows, int64_t cols, int64_t ld) { return rows > 1 ? ld : cols; }

// The memory a strided matrix takes: `count` runs of `width` bytes, `pitch` bytes
// from one run's start to the next's (pitch 0 where there is one run).
struct Area {
  uintptr_t at;
  uint64_t width, pitch, count;
  uintptr_t end() const { return at + (count - 1) * pitch + width; }
};

inline Area area(const void* p, int64_t rows, int64_t width, int64_t pitch) {
  return Area{reinterpret_cast<uintptr_t>(p), static_cast<uint64_t>(width),
              rows > 1 ? static_cast<uint64_t>(pitch) : 0, static_cast<uint64_t>(rows)};
}

// Whether two matrices share memory.  Matrices of the same pitch may lie beside
// each other in the columns of one buffer.
inline bool overlap(const Area& a, const Area& b) {
  if (a.end() <= b.at || b.end() <= a.at) return false;
  const uint64_t pitch = a.pitch != 0 ? a.pitch : b.pitch;
  if (pitch == 0 || (a.pitch != 0 && a.pitch != pitch) || (b.pitch != 0 && b.pitch != pitch)) return true;
  // where b's runs start within a's pitch
  const uint64_t d = b.at >= a.at ? (b.at - a.at) % pitch : (pitch - (a.at - b.at) % pitch) % pitch;
  return !(d >= a.width && d + b.width <= pitch);
}

// `outs` written, `ins` read: no output shares memory with anything else.
inline bool outputs_apart(const Area* outs, int n_out, const Area* ins, int n_in) {
  for (int i = 0; i < n_out; ++i) {
    for (int j = i + 1; j < n_out; ++j)
      if (overlap(outs[i], outs[j])) return false;
    for (int j = 0; j < n_in; ++j)
      if (overlap(outs[i], ins[j])) return false;
  }
  return true;
}

}  // namespace
