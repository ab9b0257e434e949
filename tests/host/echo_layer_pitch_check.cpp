// Host-logic check of pitches that say nothing, those of a single row and of a residual
// that is not there: the host code of the layer operators (csrc/echo_layer_api.hip, included
// whole) takes any value for them, does no arithmetic on it and hands the kernels a pitch that
// is safe to multiply.  Tensors are fake addresses; launches are stand-ins that record.
// Built with AddressSanitizer and UndefinedBehaviorSanitizer by
// tests/test_layer_pitches_host_cpu.py; prints "ok" and exits 0 when every check holds.
#include "echo_layer_api.hip"

#include <cstdio>

namespace {

int g_failures = 0;
echo::QuantFp8Args g_quant;
echo::GemmFp8Args g_gemm;
echo::DropoutArgs g_drop;

#define CHECK(cond)                                                                                     \
  do {                                                                                                  \
    if (!(cond) && ++g_failures <= 20) std::fprintf(stderr, "FAIL line %d (pitch %lld): %s\n", __LINE__, static_cast<long long>(ld), #cond); \
  } while (0)

void* fake(uint64_t a) { return reinterpret_cast<void*>(static_cast<uintptr_t>(a)); }

}  // namespace

namespace echo {
hipError_t launch_quantize_fp8(const QuantFp8Args& a, int, Elem, bool, hipStream_t) {
  g_quant = a;
  return hipSuccess;
}
hipError_t launch_gemm_fp8(const GemmFp8Args& a, int, bool, bool, bool, hipStream_t) {
  g_gemm = a;
  return hipSuccess;
}
hipError_t launch_dropout(const DropoutArgs& a, Elem, Elem, hipStream_t) {
  g_drop = a;
  return hipSuccess;
}
}  // namespace echo

int main() {
  void *X[1] = {fake(1u << 20)}, *q[1] = {fake(2u << 20)}, *s[1] = {fake(3u << 20)}, *w[1] = {fake(4u << 20)},
       *sw[1] = {fake(5u << 20)}, *o[1] = {fake(6u << 20)};
  const int64_t* rng = static_cast<const int64_t*>(fake(7u << 20));
  const echo_fp8 one{q, s, 256, 1, 1, ECHO_E4M3, ECHO_SCALE_F32, 1}, many{w, sw, 256, 1, 50, ECHO_E4M3, ECHO_SCALE_F32, 1};
  for (const int64_t ld : {int64_t{0}, int64_t{-1}, INT64_MIN, INT64_MAX, int64_t{1} << 41}) {
    CHECK(echo_quantize_fp8(X, 1, 1, 200, ld, ECHO_F32, &one, nullptr, nullptr) == ECHO_OK);
    CHECK(g_quant.ldx == 200);
    CHECK(echo_gemm_fp8(&one, &many, o, 1, 1, 50, 200, ld, ECHO_F32, nullptr) == ECHO_OK);
    CHECK(g_gemm.ldo == 50);
    CHECK(echo_dropout_add(X[0], q[0], o[0], 1, 200, ld, ld, ld, ECHO_F32, ECHO_F32, 0.5, rng, 0, 0, nullptr) == ECHO_OK);
    CHECK(g_drop.ldx == 200 && g_drop.ldr == 200 && g_drop.ldo == 200);
    CHECK(echo_dropout_add(X[0], nullptr, o[0], 10, 200, 200, ld, 200, ECHO_F32, ECHO_F32, 0.5, rng, 0, 0, nullptr) == ECHO_OK);
    CHECK(g_drop.residual == nullptr);
    // in place, whatever the pitches of a single row say
    CHECK(echo_dropout_add(X[0], nullptr, X[0], 1, 200, ld, 0, 7, ECHO_F32, ECHO_F32, 0.5, rng, 0, 0, nullptr) == ECHO_OK);
  }
  if (g_failures != 0) return 1;
  std::printf("ok\n");
  return 0;
}
