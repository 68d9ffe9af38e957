// Drives csrc/moe.cpp with launchers that look at the plans they are handed: every part of
// the workspace that a launch reads or writes lies inside the size that was asked for and
// apart from the others.  Host only, built with sanitizers.
#include <algorithm>
#include <cstdio>
#include <string>
#include <utility>
#include <vector>

#include "internal.h"
#include "smlp.h"

static std::string g_detail;
static int g_bad = 0, g_launches = 0;
static char g_case[256];

static void require(bool ok, const char* what) {
  if (ok) return;
  if (g_bad++ < 20) std::printf("%s: %s\n", g_case, what);
}

static int64_t blocks128(int64_t n) { return (n + 127) / 128; }

namespace smlp {
int set_error(int status, const char* detail) {
  g_detail = detail;
  return status;
}
int launch_route(const void*, int, int64_t, int64_t, int64_t, const float*, const smlp_route&, int32_t*, float*,
                 hipStream_t) {
  return 0;
}
int launch_quant_fp8(const void*, int, int64_t, int64_t, int64_t, int64_t, int, void*, float*, int64_t, int64_t,
                     hipStream_t) {
  return 0;
}
int launch_row_fp8(const void*, const float*, const void*, const float*, void*, int64_t, int64_t, int, hipStream_t) {
  return 0;
}
int launch_narrow_fp8(const F8Plan&, const void*, const void*, const float*, void*, int64_t, int64_t, int64_t, int64_t,
                      int, float*, hipStream_t) {
  return 0;
}
// Dropped stores are aimed at byte 2^31 of a tile's results, which therefore end before it.
static bool drops(int64_t rows, int64_t ld, int64_t n) { return ((rows - 1) * ld + n) * 2 <= 0x7ffffff0; }

int launch_linear_fp8(const F8Plan& p, const void*, const float*, int64_t, int64_t, const void*, const float*, void*,
                      int64_t M, int64_t, int64_t N, int64_t ldy, int, float*, hipStream_t) {
  ++g_launches;
  if (p.kind == F8_KIND_TILE) require(!p.by_rows == !drops(M < p.bm ? M : p.bm, ldy, N), "by_rows");
  return 0;
}

int launch_experts_fp8(const ExpertsPlan& p, const ExpertsCall&, void*, hipStream_t) {
  ++g_launches;
  const int64_t HB = blocks128(p.H), IB = blocks128(p.I);
  if (!p.token && !p.y_f32)
    require(drops(p.P < p.dn.bm ? p.P : p.dn.bm, p.H, p.H), "dropped stores of y would land in it");
  std::vector<std::pair<size_t, size_t>> used;  // offset, bytes
  auto use = [&](size_t off, int64_t bytes) { used.push_back({off, (size_t)bytes}); };
  if (p.token) {
    use(p.h32_off, p.topk * p.I * 4);
  } else {
    const bool stream = p.gu.kind == F8_KIND_STREAM, short_k = p.dn.kind == F8_KIND_DOWN;
    use(p.hdr_off, (4 + 4 * p.max_tiles) * 4);
    use(p.perm_off, p.P * 4);
    use(p.place_off, p.P * 4);
    if (p.chunk) use(p.counts_off, (p.P + p.chunk - 1) / p.chunk * p.E * 4);
    use(p.x8_off, p.T * p.H);
    use(p.xs_off, p.T * HB * 4);
    if (stream) use(p.h32_off, p.P * p.I * 4);
    if (!short_k) {
      use(p.h8_off, p.P * p.I);
      use(p.hs_off, p.P * IB * 4);
    }
    use(p.y_off, p.P * p.H * (p.y_f32 ? 4 : 2));
    if (!p.y_f32) use(p.yexp_off, p.P * ((p.H + 63) / 64));
  }
  std::sort(used.begin(), used.end());
  size_t end = 0;
  for (const auto& u : used) {
    require(u.first % 256 == 0, "a region is not aligned");
    require(u.first >= end, "regions overlap");
    end = u.first + u.second;
  }
  require(end <= p.workspace_bytes, "a region ends behind the workspace");
  return 0;
}
}  // namespace smlp

static char* at(uintptr_t v) { return reinterpret_cast<char*>(v << 40); }
static float* fat(uintptr_t v) { return reinterpret_cast<float*>(at(v)); }

static void experts_regions() {
  const int64_t sizes[][2] = {{256, 512},   {512, 256},    {16, 2048},     {128, 4096},    {8208, 128},
                              {2000, 336},  {7168, 768},   {4194304, 128}, {8388608, 112}, {18000016, 16},
                              {33554432, 16}};
  for (int64_t T : {1, 2, 5, 40, 62, 127, 255, 301, 600, 5000})
    for (int64_t E : {1, 2, 3, 24, 128})
      for (int64_t topk : {1, 2, 4, 8, 12, 13, 25, 26, 39, 64})
        for (const auto& s : sizes)
          for (int partial : {0, 1}) {
            std::snprintf(g_case, sizeof g_case, "T %lld H %lld I %lld E %lld topk %lld partial %d", (long long)T,
                          (long long)s[0], (long long)s[1], (long long)E, (long long)topk, partial);
            size_t n = 0;
            if (shared_mlp_experts_fp8_workspace_bytes(T, s[0], s[1], E, topk, partial, &n)) continue;
            g_launches = 0;
            const int rc = shared_mlp_experts_fp8(at(1), reinterpret_cast<int32_t*>(at(2)), fat(3), at(4), fat(5), at(6),
                                                  fat(7), at(8), T, s[0], s[1], E, topk, 0, partial, at(9), n, nullptr);
            require(rc == SMLP_OK && g_launches == 1, g_detail.c_str());
          }
}

static void linear_rows() {
  const int64_t cases[][4] = {  // M, K, N, ldy
      {200, 128, 6000000, 6000000}, {200, 128, 5000000, 5000000}, {60, 128, 64, 35000000},  {60, 128, 64, 17000000},
      {1000, 256, 4096, 2000000},   {8192, 6144, 7168, 7168},     {300, 256, 1024, 7000000}, {63, 1024, 64, 17300000}};
  for (const auto& c : cases)
    for (int f32 : {0, 1}) {
      std::snprintf(g_case, sizeof g_case, "M %lld K %lld N %lld ldy %lld fp32 %d", (long long)c[0], (long long)c[1],
                    (long long)c[2], (long long)c[3], f32);
      g_launches = 0;
      const int rc = shared_mlp_linear_fp8(at(1), fat(2), at(3), fat(4), at(5), c[0], c[1], c[2], c[3], f32, at(6),
                                           (size_t)1 << 39, nullptr);
      require(rc == SMLP_OK && g_launches == 1, g_detail.c_str());
    }
}

// Captured launches: no counter is handed out twice.
static void captured_counters() {
  std::snprintf(g_case, sizeof g_case, "captured counters");
  smlp::CounterRun run;
  int64_t end = 0;
  for (int i = 0; i < 1000; ++i) {
    const int64_t n = 1 + i * 7 % 128, at = run.take(n, 20000);
    if (at < 0) {
      require(end + n > 20000, "refused while enough are left");
      continue;
    }
    require(at == end && at + n <= 20000, "handed out twice, or past the end");
    end = at + n;
  }
  require(run.take(20001 - end, 20000) < 0 && run.take(-1, 20000) < 0, "past the end");
}

int main() {
  experts_regions();
  linear_rows();
  captured_counters();
  std::printf(g_bad ? "%d checks failed\n" : "all checks passed\n", g_bad);
  return g_bad != 0;
}
