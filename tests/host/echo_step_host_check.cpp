// Host-logic check of the training step's operators' C ABI on a machine without a GPU: the
// host code (csrc/echo_step_api.hip, included whole) runs against stand-ins of the launches
// that record their arguments.  Tensors are fake device addresses that the host code only does
// arithmetic on.  It checks that valid calls launch with the arguments given, that workspaces
// hold what the launches put there, that a clipping call's launches cover every tensor once,
// byte for byte, and that a failed launch is reported.
// Built with AddressSanitizer and UndefinedBehaviorSanitizer by tests/test_step_host_cpu.py;
// prints "ok" and exits 0 when every check holds.
#include "echo_step_api.hip"

#include <cstdio>
#include <random>
#include <vector>

namespace {

int g_checks = 0, g_failures = 0, g_fail_at = -1, g_launches = 0;

#define CHECK(cond)                                                        \
  do {                                                                     \
    ++g_checks;                                                            \
    if (!(cond) && ++g_failures <= 20) std::fprintf(stderr, "FAIL line %d: %s\n", __LINE__, #cond); \
  } while (0)

void* fake(uint64_t a) { return reinterpret_cast<void*>(static_cast<uintptr_t>(a)); }

hipError_t launched() { return g_launches++ == g_fail_at ? hipErrorLaunchFailure : hipSuccess; }

echo::BlockNormArgs g_norm;
echo::BlockNormBwdArgs g_bwd;
echo::EmbedArgs g_embed;
echo::EmbedBwdArgs g_embed_bwd;
echo::Elem g_types[3];

// What the clipping launches covered: (source, bytes, type, destination) of every tensor, and
// the partial sums they wrote.
struct Seen {
  const void* src;
  void* dst;
  int64_t bytes;
  int elem;
};
std::vector<Seen> g_summed, g_scaled;
std::vector<const double*> g_parts;
int64_t g_n_part = -1, g_joined = 0;
int g_norms = 0;

template <typename Args>
void unpack(const Args& a, bool scaled) {
  CHECK(a.tensors >= 1 && a.tensors <= Args::kTensors && a.first[0] == 0);
  CHECK(sizeof(Args) <= 4096 - 64);
  for (int t = 0; t < a.tensors; ++t) {
    const int64_t chunks = static_cast<int64_t>(a.first[t + 1]) - a.first[t];
    CHECK(chunks >= 1);
    const int64_t bytes = (chunks - 1) * echo::kClipChunk + ((a.tail[t] & 0x3FFF) + 1) * 2;
    const bool apart = sizeof(a.dst) > sizeof(void*);
    (scaled ? g_scaled : g_summed)
        .push_back(Seen{a.src[t], apart ? a.dst[t] : const_cast<void*>(a.src[t]), bytes, a.tail[t] >> 14});
  }
}

}  // namespace

namespace echo {
hipError_t launch_block_norm(const BlockNormArgs& a, Elem x, Elem y, Elem o, hipStream_t) {
  g_norm = a;
  g_types[0] = x, g_types[1] = y, g_types[2] = o;
  return launched();
}
hipError_t launch_block_norm_bwd(const BlockNormBwdArgs& a, Elem x, Elem y, Elem o, hipStream_t) {
  g_bwd = a;
  g_types[0] = x, g_types[1] = y, g_types[2] = o;
  return launched();
}
hipError_t launch_clip_sum(const ClipInPlace& a, double* part, hipStream_t) {
  unpack(a, false);
  for (unsigned i = 0; i < clip_grid(a.first[a.tensors]); ++i) g_parts.push_back(part + i);
  return launched();
}
template <typename Args>
hipError_t scaled(const Args& a, int64_t n_part, float* norm) {
  unpack(a, true);
  g_n_part = n_part;
  g_norms += norm != nullptr;
  return launched();
}
hipError_t launch_clip_scale(const ClipInPlace& a, const double*, int64_t n, double, float* norm, bool, hipStream_t) {
  return scaled(a, n, norm);
}
hipError_t launch_clip_scale(const ClipApart& a, const double*, int64_t n, double, float* norm, bool, hipStream_t) {
  return scaled(a, n, norm);
}
hipError_t launch_clip_join(double* part, int64_t n, hipStream_t) {
  CHECK(!g_parts.empty() && part == g_parts[0]);
  g_joined = n;
  return launched();
}
hipError_t launch_clip_norm(const double*, int64_t n, float*, hipStream_t) {
  g_n_part = n;
  ++g_norms;
  return launched();
}
hipError_t launch_embed(const EmbedArgs& a, Elem t, Elem o, hipStream_t) {
  g_embed = a;
  g_types[0] = t, g_types[1] = o;
  return launched();
}
hipError_t launch_embed_bwd(const EmbedBwdArgs& a, Elem o, Elem t, hipStream_t) {
  g_embed_bwd = a;
  g_types[0] = t, g_types[1] = o;
  return launched();
}
}  // namespace echo

namespace {

constexpr uint64_t G = uint64_t{1} << 30;

echo_block block() {
  echo_block b{};
  b.rows = 60;
  b.cols = 300;
  b.gate = fake(5 * G);
  b.ld_gate = 303;
  b.gate_rows = 4;
  b.w_post = fake(6 * G);
  b.w_pre = fake(7 * G);
  b.residual_scale = 0.5;
  b.weight_offset = 1.0;
  b.eps = 1e-6;
  b.x_dtype = ECHO_F32;
  b.y_dtype = ECHO_BF16;
  b.a_dtype = ECHO_BF16;
  b.param_dtype = ECHO_F16;
  b.post_norm = 1;
  return b;
}

void check_block() {
  echo_block b = block();
  CHECK(echo_block_norm(&b, fake(G), 301, fake(2 * G), 302, fake(3 * G), 304, fake(4 * G), 305, nullptr) == ECHO_OK);
  CHECK(g_launches == 1 && g_norm.x == fake(G) && g_norm.y == fake(2 * G) && g_norm.out == fake(3 * G) && g_norm.a == fake(4 * G));
  CHECK(g_norm.ldx == 301 && g_norm.ldy == 302 && g_norm.ldo == 304 && g_norm.lda == 305);
  CHECK(g_norm.p.R == 60 && g_norm.p.C == 300 && g_norm.p.n_gates == 4 && g_norm.p.rows_per_gate == 15 && g_norm.p.ldg == 303);
  CHECK(g_norm.p.alpha == 0.5f && g_norm.p.offset == 1.0f && g_norm.p.eps == 1e-6f && g_norm.p.elem == ECHO_F16 && g_norm.p.post);
  CHECK(g_types[0] == echo::kElemF32 && g_types[1] == echo::kElemBf16 && g_types[2] == echo::kElemBf16);
  // one row: its pitch says nothing; types of what is not there are x's
  b.rows = 1;
  b.gate_rows = 1;
  b.w_pre = nullptr;
  CHECK(echo_block_norm(&b, fake(G), -7, fake(2 * G), 0, fake(3 * G), 1, nullptr, 9, nullptr) == ECHO_OK);
  CHECK(g_norm.ldx == 300 && g_norm.p.ldg == 300 && g_types[2] == echo::kElemF32);
  // beside each other in one buffer
  b = block();
  CHECK(echo_block_norm(&b, fake(G), 600, fake(2 * G), 300, fake(G + 1200), 600, fake(4 * G), 300, nullptr) == ECHO_OK);
  CHECK(echo_block_norm(&b, fake(G), 600, fake(2 * G), 300, fake(G + 1196), 600, fake(4 * G), 300, nullptr) == ECHO_ERR_ARG);
  g_launches = 0;
  g_fail_at = 0;
  CHECK(echo_block_norm(&b, fake(G), 301, fake(2 * G), 302, fake(3 * G), 304, fake(4 * G), 305, nullptr) == ECHO_ERR_HIP);
  g_fail_at = -1;

  const size_t need = echo_block_norm_workspace(60, 300, 4);
  CHECK(need > 0);
  CHECK(echo_block_norm_backward(&b, fake(G), 301, fake(2 * G), 302, fake(3 * G), 303, fake(4 * G), 304, fake(8 * G), 305,
                                 fake(9 * G), 306, fake(10 * G), 307, fake(11 * G), fake(12 * G), fake(13 * G), need,
                                 nullptr) == ECHO_OK);
  CHECK(g_bwd.out == fake(G) && g_bwd.y == fake(2 * G) && g_bwd.dout == fake(3 * G) && g_bwd.da == fake(4 * G));
  CHECK(g_bwd.dx == fake(8 * G) && g_bwd.dy == fake(9 * G) && g_bwd.dgate == fake(10 * G) && g_bwd.dw_post == fake(11 * G) &&
        g_bwd.dw_pre == fake(12 * G) && g_bwd.part == fake(13 * G));
  CHECK(g_bwd.ldo == 301 && g_bwd.ldy == 302 && g_bwd.lddo == 303 && g_bwd.ldda == 304 && g_bwd.lddx == 305 &&
        g_bwd.lddy == 306 && g_bwd.lddg == 307);
  CHECK(echo_block_norm_backward(&b, fake(G), 301, fake(2 * G), 302, fake(3 * G), 303, fake(4 * G), 304, fake(8 * G), 305,
                                 fake(9 * G), 306, fake(10 * G), 307, fake(11 * G), fake(12 * G), fake(13 * G), need - 1,
                                 nullptr) == ECHO_ERR_WORKSPACE);
  // the workspace holds the column sums of every workgroup and, behind them, the rows' statistics
  for (int64_t rows : {1, 2, 255, 256, 257, 1023, 4096, 100000, 1 << 22})
    for (int64_t cols : {1, 7, 8, 64, 1000, 2048, 8192, 8193, 16385, 1 << 20})
      for (int64_t gates : {int64_t{1}, int64_t{2}, int64_t{600}, rows}) {
        if (rows % gates != 0 || rows > (int64_t{1} << 40) / cols) continue;
        const echo::BlockSplit s = echo::block_split(rows, gates, cols);
        const int64_t per_gate = rows / gates;
        CHECK(s.groups >= 1 && s.groups <= (int64_t{1} << 31) - 1);
        if (s.chunks != 0) {
          CHECK(s.groups == gates * s.chunks && s.chunks <= per_gate);  // every workgroup has a row
        } else {
          CHECK(s.rows == s.gates * per_gate && s.groups * s.gates >= gates && (s.groups - 1) * s.gates < gates);
        }
        const size_t part = static_cast<size_t>(s.groups) * 3 * cols * 4, stats = echo::block_fits(cols) ? 0 : rows * 16;
        const size_t bytes = echo_block_norm_workspace(rows, cols, gates);
        CHECK(bytes >= part + stats && bytes < part + stats + 16);
      }
}

void check_clip() {
  std::mt19937 g(3);
  const auto pick = [&](int64_t lo, int64_t hi) { return std::uniform_int_distribution<int64_t>(lo, hi)(g); };
  int joins = 0;
  for (int n : {0, 1, 5, 175, 176, 177, 279, 280, 281, 353, 1000}) {
    std::vector<const void*> src;
    std::vector<void*> dst;
    std::vector<int64_t> numel;
    std::vector<int32_t> types;
    uint64_t at = G, to = 400 * G;
    int64_t whole = 0;
    for (int i = 0; i < n; ++i) {
      const int32_t t = static_cast<int32_t>(pick(0, 2));
      const int64_t es = t == ECHO_F32 ? 4 : 2;
      const int64_t edge = echo::kClipChunk / es;  // lengths around a chunk's end, short ones, none, long ones
      const int64_t m = i % 5 == 0 ? pick(0, 3) : i % 5 == 1 ? edge * pick(1, 3) + pick(-2, 2) : i == 7 ? int64_t{1} << 33 : pick(1, 100000);
      at = (at + 3) & ~uint64_t{3};
      to = (to + 3) & ~uint64_t{3};
      src.push_back(fake(at));
      dst.push_back(fake(to));
      numel.push_back(m);
      types.push_back(t);
      at += m * es;
      to += m * es;
      whole += m > 0;
    }
    const size_t bytes = echo_clip_workspace(n);
    for (int in_place = 0; in_place < 2; ++in_place) {
      g_summed.clear(), g_scaled.clear(), g_parts.clear();
      g_norms = g_launches = 0;
      g_joined = 0;
      CHECK(echo_clip_grads(src.data(), in_place ? const_cast<void* const*>(src.data()) : dst.data(), numel.data(), types.data(),
                            n, 1.0, static_cast<float*>(fake(900 * G)), fake(901 * G), bytes, nullptr) == ECHO_OK);
      CHECK(g_norms == 1 && g_summed.size() == static_cast<size_t>(whole));
      const int64_t parts = static_cast<int64_t>(g_parts.size());  // more than one launch leaves are joined first
      CHECK(g_joined == (parts > echo::kClipGroups ? parts : 0) && g_n_part == (g_joined != 0 ? 1 : parts));
      joins += g_joined != 0;
      CHECK(g_scaled.size() == g_summed.size());
      size_t k = 0;
      for (int i = 0; i < n; ++i) {
        if (numel[i] == 0) continue;
        const int64_t b = numel[i] * (types[i] == ECHO_F32 ? 4 : 2);
        for (const Seen& s : {g_summed[k], g_scaled[k]}) CHECK(s.src == src[i] && s.bytes == b && s.elem == types[i]);
        CHECK(g_scaled[k].dst == (in_place ? src[i] : dst[i]));
        ++k;
      }
      // partial sums lie one after the other, inside the workspace
      const double* base = static_cast<const double*>(fake(901 * G));
      for (size_t i = 0; i < g_parts.size(); ++i) CHECK(g_parts[i] == base + i);
      CHECK(g_parts.size() * sizeof(double) <= bytes);
    }
    g_norms = 0;
    g_parts.clear();
    CHECK(echo_grad_norm(src.data(), numel.data(), types.data(), n, static_cast<float*>(fake(900 * G)), fake(901 * G), bytes,
                         nullptr) == ECHO_OK);
    CHECK(g_norms == 1 && g_n_part == static_cast<int64_t>(g_parts.size()));
    const int launches = g_launches;
    if (n >= 280) {
      g_launches = 0;
      g_fail_at = 1;
      CHECK(echo_clip_grads(src.data(), dst.data(), numel.data(), types.data(), n, 1.0, static_cast<float*>(fake(900 * G)),
                            fake(901 * G), bytes, nullptr) == ECHO_ERR_HIP);
      CHECK(g_launches == 2 && launches > 2);  // nothing is launched behind a failed launch
      g_fail_at = -1;
    }
  }
  CHECK(joins > 0);
}

// Overlaps of clipping calls against a byte-by-byte count.
void check_clip_overlaps() {
  std::mt19937 g(4);
  const auto pick = [&](int lo, int hi) { return std::uniform_int_distribution<int>(lo, hi)(g); };
  int accepted = 0;
  for (int n = 0; n < 4000; ++n) {
    const int count = pick(1, 4);
    const void* src[4];
    void* dst[4];
    int64_t numel[4];
    int32_t types[4];
    std::vector<int> written(400, 0), read(400, 0);
    bool bad = false;
    for (int i = 0; i < count; ++i) {
      const int s = pick(0, 80) * 4, d = pick(0, 2) ? s : pick(0, 80) * 4;
      numel[i] = pick(0, 6);
      types[i] = ECHO_F32;
      src[i] = fake(4096 + s);
      dst[i] = fake(4096 + d);
      for (int b = 0; b < 4 * numel[i]; ++b) {
        ++written[d + b];
        if (s != d) ++read[s + b];
      }
    }
    for (int b = 0; b < 400; ++b) bad |= written[b] > 1 || (written[b] == 1 && read[b] > 0);
    const echo_status e = echo_clip_grads(src, dst, numel, types, count, 1.0, static_cast<float*>(fake(8192)), fake(1 << 20),
                                          echo_clip_workspace(count), nullptr);
    CHECK(e == (bad ? ECHO_ERR_ARG : ECHO_OK));
    accepted += !bad;
  }
  CHECK(accepted > 100 && accepted < 3900);
}

void check_embed_calls() {
  const void* t[2] = {fake(G), fake(2 * G)};
  void *o[2] = {fake(3 * G), fake(4 * G)}, *d[2] = {fake(5 * G), fake(6 * G)};
  CHECK(echo_embed(t, fake(7 * G), o, 2, 50, 70, 71, 9, 72, ECHO_F32, ECHO_F16, 4, 11, 0.5, nullptr) == ECHO_OK);
  CHECK(g_embed.table[1] == t[1] && g_embed.out[1] == o[1] && g_embed.tokens == fake(7 * G) && g_embed.V == 50 && g_embed.C == 70);
  CHECK(g_embed.ldt == 71 && g_embed.T == 9 && g_embed.ldo == 72 && g_embed.first == 11 && g_embed.scale == 0.5f &&
        g_embed.P == 2 && g_embed.wide == 0 && g_types[0] == echo::kElemF32 && g_types[1] == echo::kElemF16);
  const size_t need = echo_embed_workspace(9, 70);
  CHECK(echo_embed_backward(fake(8 * G), fake(7 * G), d, 2, 50, 70, 71, 9, 72, ECHO_F16, ECHO_F32, 8, 11, 0.5, fake(9 * G), need,
                            nullptr) == ECHO_OK);
  CHECK(g_embed_bwd.dout == fake(8 * G) && g_embed_bwd.dtable[1] == d[1] && g_embed_bwd.lddo == 72 && g_embed_bwd.ldt == 71 &&
        g_embed_bwd.wide == 1 && g_embed_bwd.workspace == fake(9 * G));
  // no tokens: the tables are still cleared
  g_launches = 0;
  CHECK(echo_embed_backward(nullptr, nullptr, d, 2, 50, 70, 71, 0, 72, ECHO_F16, ECHO_F32, 8, 11, 0.5, nullptr, 0, nullptr) == ECHO_OK);
  CHECK(g_launches == 1 && g_embed_bwd.T == 0);
  // an empty table: nothing is read of it
  CHECK(echo_embed(nullptr, fake(7 * G), o, 2, 0, 70, 0, 9, 72, ECHO_F32, ECHO_F16, 4, 11, 0.5, nullptr) == ECHO_OK);
  g_fail_at = g_launches;
  CHECK(echo_embed(t, fake(7 * G), o, 2, 50, 70, 71, 9, 72, ECHO_F32, ECHO_F16, 4, 11, 0.5, nullptr) == ECHO_ERR_HIP);
  g_fail_at = -1;
  // the workspace's parts lie one after the other, each as long as the launches need
  for (int64_t T : {1, 8, 4096, 4097, 16384, 16385, 1 << 17, (1 << 17) + 1, 1 << 24, 1 << 27})
    for (int64_t C : {1, 8, 9, 64, 512, 513, 4096, 1 << 22}) {
      const echo::EmbedLayout w = echo::embed_layout(T, C);
      const bool big = T > 16384;
      CHECK(w.order[0] - w.keys[0] >= static_cast<size_t>(T) * 4 && w.keys[0] == 0);
      if (big) {
        CHECK(w.keys[1] - w.order[0] >= static_cast<size_t>(T) * 4 && w.order[1] - w.keys[1] >= static_cast<size_t>(T) * 4);
        CHECK(w.counts - w.order[1] >= static_cast<size_t>(T) * 4);
        CHECK(w.part - w.counts >= static_cast<size_t>((T + 4095) / 4096) * 512 * 4);
      }
      const int64_t group = echo::embed_chunk(T) * (512 >> echo::embed_shift(C));
      CHECK(w.bytes - w.part >= static_cast<size_t>((T + group - 1) / group) * 2 * C * 4);
      CHECK(echo_embed_workspace(T, C) == w.bytes);
    }
}

}  // namespace

int main() {
  check_block();
  check_clip();
  check_clip_overlaps();
  check_embed_calls();
  if (g_failures != 0) {
    std::fprintf(stderr, "%d of %d checks failed\n", g_failures, g_checks);
    return 1;
  }
  std::printf("ok: %d checks\n", g_checks);
  return 0;
}
