// Host-logic check of the layer operators' C ABI on a machine without a GPU: the host
// code (csrc/echo_layer_api.hip, included whole) runs against stand-ins of the
// launches that record their arguments.  Tensors are fake device addresses that the
// host code only does arithmetic on.  It checks that valid calls launch once with the
// arguments given, that outputs may lie beside each other in one buffer but share no
// byte with anything (against a byte-by-byte count on small layouts), and that a failed
// launch is reported.
// Built with AddressSanitizer and UndefinedBehaviorSanitizer by
// tests/test_layer_host_cpu.py; prints "ok" and exits 0 when every check holds.
#include "echo_layer_api.hip"

#include <cstdio>
#include <cstring>
#include <random>
#include <set>

namespace {

int g_checks = 0, g_failures = 0, g_launches = 0;
bool g_fail = false;
echo::QuantFp8Args g_quant;
echo::GemmFp8Args g_gemm;
echo::DropoutArgs g_drop;
int g_P;
bool g_flags[3];

#define CHECK(cond)                                                        \
  do {                                                                     \
    ++g_checks;                                                            \
    if (!(cond) && ++g_failures <= 20) std::fprintf(stderr, "FAIL line %d: %s\n", __LINE__, #cond); \
  } while (0)

void* fake(uint64_t a) { return reinterpret_cast<void*>(static_cast<uintptr_t>(a)); }

hipError_t launched() {
  ++g_launches;
  return g_fail ? hipErrorLaunchFailure : hipSuccess;
}

}  // namespace

namespace echo {
hipError_t launch_quantize_fp8(const QuantFp8Args& a, int P, Elem x, bool block128, hipStream_t) {
  g_quant = a;
  g_P = P;
  g_flags[0] = block128;
  g_flags[1] = x == kElemF32;
  return launched();
}
hipError_t launch_gemm_fp8(const GemmFp8Args& a, int P, bool a5, bool w5, bool e8, hipStream_t) {
  g_gemm = a;
  g_P = P;
  g_flags[0] = a5;
  g_flags[1] = w5;
  g_flags[2] = e8;
  return launched();
}
hipError_t launch_dropout(const DropoutArgs& a, Elem, Elem, hipStream_t) {
  g_drop = a;
  return launched();
}
}  // namespace echo

namespace {

echo_fp8 mats(void** codes, void** scales, int64_t ld, int64_t srs, int64_t sks, int fmt, int st, int block) {
  return echo_fp8{codes, scales, ld, srs, sks, fmt, st, block};
}

void check_quantizer() {
  void* X[2] = {fake(1u << 20), fake(2u << 20)};
  void *q[2] = {fake(3u << 20), fake(4u << 20)}, *s[2] = {fake(5u << 20), fake((5u << 20) + 4096)};
  void *qc[2] = {fake(6u << 20), fake(7u << 20)}, *sc[2] = {fake(8u << 20), fake((8u << 20) + 8192)};
  const echo_fp8 rows = mats(q, s, 304, 1, 100, ECHO_E5M2, ECHO_SCALE_F32, 1);
  const echo_fp8 cols = mats(qc, sc, 112, 1, 300, ECHO_E5M2, ECHO_SCALE_F32, 1);
  g_launches = 0;
  CHECK(echo_quantize_fp8(X, 2, 100, 300, 301, ECHO_F32, &rows, &cols, nullptr) == ECHO_OK);
  CHECK(g_launches == 1 && g_P == 2 && !g_flags[0] && g_flags[1]);
  CHECK(g_quant.R == 100 && g_quant.C == 300 && g_quant.ldx == 301 && g_quant.e5m2 == 1 && g_quant.e8m0 == 0);
  for (int r = 0; r < 2; ++r) {
    CHECK(g_quant.X[r] == X[r] && g_quant.rows.codes[r] == q[r] && g_quant.rows.scales[r] == s[r]);
    CHECK(g_quant.cols.codes[r] == qc[r] && g_quant.cols.scales[r] == sc[r]);
  }
  CHECK(g_quant.rows.ld == 304 && g_quant.rows.srs == 1 && g_quant.rows.sks == 100);
  CHECK(g_quant.cols.ld == 112 && g_quant.cols.srs == 1 && g_quant.cols.sks == 300);
  CHECK(echo_quantize_fp8(X, 2, 100, 300, 301, ECHO_F32, nullptr, &cols, nullptr) == ECHO_OK);
  CHECK(g_quant.rows.codes[0] == nullptr && g_quant.cols.codes[0] == qc[0]);
  g_fail = true;
  CHECK(echo_quantize_fp8(X, 2, 100, 300, 301, ECHO_F32, &rows, nullptr, nullptr) == ECHO_ERR_HIP);
  g_fail = false;
  // scales of a rank that reach into the next rank's
  void* s_close[2] = {fake(5u << 20), fake((5u << 20) + 4 * 299)};
  const echo_fp8 close = mats(q, s_close, 304, 1, 100, ECHO_E5M2, ECHO_SCALE_F32, 1);
  g_launches = 0;
  CHECK(echo_quantize_fp8(X, 2, 100, 300, 301, ECHO_F32, &close, nullptr, nullptr) == ECHO_ERR_ARG);
  CHECK(g_launches == 0);
}

void check_product() {
  void *A[1] = {fake(1u << 20)}, *sA[1] = {fake(2u << 20)}, *W[1] = {fake(3u << 20)}, *sW[1] = {fake(4u << 20)}, *o[1] = {fake(5u << 20)};
  const echo_fp8 a = mats(A, sA, 256, 1, 50, ECHO_E5M2, ECHO_SCALE_E8M0, 1);
  const echo_fp8 w = mats(W, sW, 272, 2, 1, ECHO_E4M3, ECHO_SCALE_E8M0, 128);
  g_launches = 0;
  CHECK(echo_gemm_fp8(&a, &w, o, 1, 50, 200, 250, 203, ECHO_F16, nullptr) == ECHO_OK);
  CHECK(g_launches == 1 && g_P == 1 && g_flags[0] && !g_flags[1] && g_flags[2]);
  CHECK(g_gemm.M == 50 && g_gemm.N == 200 && g_gemm.K == 250 && g_gemm.lda == 256 && g_gemm.ldw == 272 && g_gemm.ldo == 203);
  CHECK(g_gemm.sa_row == 1 && g_gemm.sa_k == 50 && g_gemm.sa_shift == 0 && g_gemm.sw_row == 2 && g_gemm.sw_k == 1 && g_gemm.sw_shift == 7);
  CHECK(g_gemm.A[0] == A[0] && g_gemm.W[0] == W[0] && g_gemm.sA[0] == sA[0] && g_gemm.sW[0] == sW[0] && g_gemm.out[0] == o[0]);
  // one scale for everything: strides of zero
  const echo_fp8 one = mats(A, sA, 256, 0, 0, ECHO_E4M3, ECHO_SCALE_E8M0, 1);
  CHECK(echo_gemm_fp8(&one, &one, o, 1, 50, 50, 250, 50, ECHO_F32, nullptr) == ECHO_OK);
  // strides beyond what the kernels' 32-bit offsets take
  const echo_fp8 far = mats(A, sA, 256, (int64_t{1} << 29) / 50 + 1, 0, ECHO_E4M3, ECHO_SCALE_E8M0, 1);
  CHECK(echo_gemm_fp8(&far, &one, o, 1, 50, 50, 250, 50, ECHO_F32, nullptr) == ECHO_ERR_SHAPE);
  // nothing along k: the operands are not looked at
  const echo_fp8 none = mats(nullptr, nullptr, 0, 0, 0, ECHO_E4M3, ECHO_SCALE_E8M0, 1);
  CHECK(echo_gemm_fp8(&none, &none, o, 1, 50, 50, 0, 50, ECHO_F32, nullptr) == ECHO_OK && g_gemm.K == 0);
}

void check_dropout() {
  g_launches = 0;
  CHECK(echo_dropout_add(fake(1 << 20), fake(2 << 20), fake(3 << 20), 10, 20, 21, 22, 23, ECHO_F32, ECHO_BF16, 0.25,
                         static_cast<const int64_t*>(fake(4 << 20)), -5, 77, nullptr) == ECHO_OK);
  CHECK(g_launches == 1 && g_drop.threshold == 16384 && g_drop.scale == 65536.0f / 49152.0f && g_drop.offset == -5 && g_drop.first == 77);
  CHECK(g_drop.R == 10 && g_drop.C == 20 && g_drop.ldx == 21 && g_drop.ldr == 22 && g_drop.ldo == 23);
  const auto p = [](double x) {
    return echo_dropout_add(fake(1 << 20), nullptr, fake(3 << 20), 1, 8, 8, 8, 8, ECHO_F32, ECHO_F32, x,
                            static_cast<const int64_t*>(fake(4 << 20)), 0, 0, nullptr);
  };
  CHECK(p(0.0) == ECHO_OK && g_drop.threshold == 0 && g_drop.scale == 1.0f);
  CHECK(p(1.0 - 1.0 / 65536) == ECHO_OK && g_drop.threshold == 65535 && g_drop.scale == 65536.0f);
  CHECK(p(1.0 / 131072) == ECHO_OK && g_drop.threshold == 0);  // a tie, to even
  CHECK(p(3.0 / 131072) == ECHO_OK && g_drop.threshold == 2);
}

// overlap() against the bytes themselves: never false where a byte is shared; exact for
// one pitch, where neither matrix wraps past its pitch.
void check_overlap() {
  std::mt19937 g(1);
  const auto pick = [&](int lo, int hi) { return std::uniform_int_distribution<int>(lo, hi)(g); };
  for (int n = 0; n < 20000; ++n) {
    const int pitch_a = pick(4, 12), pitch_b = pick(0, 2) ? pitch_a : pick(4, 12);
    const Area a = area(fake(1000 + pick(0, 60)), pick(1, 5), pick(1, pitch_a), pitch_a);
    const Area b = area(fake(1000 + pick(0, 60)), pick(1, 5), pick(1, pitch_b), pitch_b);
    std::set<uint64_t> bytes;
    for (uint64_t i = 0; i < a.count; ++i)
      for (uint64_t j = 0; j < a.width; ++j) bytes.insert(a.at + i * a.pitch + j);
    bool shared = false;
    for (uint64_t i = 0; i < b.count; ++i)
      for (uint64_t j = 0; j < b.width; ++j) shared |= bytes.count(b.at + i * b.pitch + j) != 0;
    CHECK(!shared || overlap(a, b));
    CHECK(overlap(a, b) == overlap(b, a));
  }
  // beside each other in one buffer
  CHECK(!overlap(area(fake(1000), 4, 30, 100), area(fake(1030), 4, 70, 100)));
  CHECK(!overlap(area(fake(1050), 4, 50, 100), area(fake(1000), 9, 50, 100)));
  CHECK(overlap(area(fake(1000), 4, 31, 100), area(fake(1030), 4, 70, 100)));
}

}  // namespace

int main() {
  check_quantizer();
  check_product();
  check_dropout();
  check_overlap();
  if (g_failures != 0) {
    std::fprintf(stderr, "%d of %d checks failed\n", g_failures, g_checks);
    return 1;
  }
  std::printf("ok: %d checks\n", g_checks);
  return 0;
}
