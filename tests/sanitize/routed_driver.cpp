// Drives the host code of csrc/moe.cpp (validation and planning of the routed half) with the
// kernel launchers replaced by stand-ins that count their calls; built with sanitizers.
#include <cstdio>
#include <cstring>
#include <string>

#include "internal.h"
#include "smlp.h"

static std::string g_detail;
static int g_launches = 0;

namespace smlp {
int set_error(int status, const char* detail) {
  g_detail = detail;
  return status;
}
int launch_route(const void*, int, int64_t, int64_t, int64_t, const float*, const smlp_route&, int32_t*, float*,
                 hipStream_t) {
  return ++g_launches, 0;
}
int launch_quant_fp8(const void*, int, int64_t, int64_t, int64_t, int64_t, int, void*, float*, int64_t, int64_t,
                     hipStream_t) {
  return ++g_launches, 0;
}
int launch_row_fp8(const void*, const float*, const void*, const float*, void*, int64_t, int64_t, int, hipStream_t) {
  return ++g_launches, 0;
}
int launch_narrow_fp8(const F8Plan&, const void*, const void*, const float*, void*, int64_t, int64_t, int64_t, int64_t,
                      int, float*, hipStream_t) {
  return ++g_launches, 0;
}
int launch_linear_fp8(const F8Plan&, const void*, const float*, int64_t, int64_t, const void*, const float*, void*,
                      int64_t, int64_t, int64_t, int64_t, int, float*, hipStream_t) {
  return ++g_launches, 0;
}
int launch_experts_fp8(const ExpertsPlan&, const ExpertsCall&, void*, hipStream_t) { return ++g_launches, 0; }
}  // namespace smlp

static int g_bad = 0;
static void expect(const char* what, int got, int want, int launched) {
  if (got != want || (g_launches > 0) != (launched != 0)) {
    std::printf("%s: status %d (want %d), launches %d: %s\n", what, got, want, g_launches, g_detail.c_str());
    ++g_bad;
  }
  g_launches = 0;
}

static char* at(uintptr_t v) { return reinterpret_cast<char*>(v); }
static float* fat(uintptr_t v) { return reinterpret_cast<float*>(v); }

int main() {
  const int64_t big = (int64_t)1 << 58;
  int32_t* ids = reinterpret_cast<int32_t*>(at(0x20000000));
  float* w = fat(0x28000000);
  smlp_route r{SMLP_SCORE_SIGMOID, 8, 4, 2, 8, 1, 2.5f};
  auto route = [&](int64_t T, int64_t E, int64_t ld) {
    return shared_mlp_route(at(0x10000000), SMLP_FP32, T, E, ld, nullptr, &r, ids, w, nullptr);
  };
  expect("route", route(100, 256, 256), SMLP_OK, 1);
  expect("route T = 0", route(0, 256, 256), SMLP_OK, 0);
  const int64_t odd[] = {-big, -1, 0, 1, 1023, 1025, (int64_t)1 << 31, big};
  for (int64_t T : odd)
    for (int64_t E : odd)
      for (int64_t ld : odd) {
        (void)route(T, E, ld);
        g_launches = 0;
      }
  for (int v = -2; v <= 70; ++v) {
    smlp_route q = r;
    for (int* f : {&q.score, &q.groups, &q.top_groups, &q.group_top, &q.topk}) {
      const int keep = *f;
      *f = v;
      (void)shared_mlp_route(at(0x10000000), SMLP_BF16, 4, 256, 256, nullptr, &q, ids, w, nullptr);
      *f = keep;
      g_launches = 0;
    }
  }
  size_t n = 0;
  for (int64_t a : odd)
    for (int64_t b : odd)
      for (int64_t c : odd) {
        (void)shared_mlp_linear_fp8_workspace_bytes(a, b, c, 0, &n);
        (void)shared_mlp_linear_fp8(at(0x1000), nullptr, at(0x100000), fat(0x200000), at(0x300000), a, b * 16, c, c, 0,
                                    at(0x40000000), 1 << 30, nullptr);
        (void)shared_mlp_quant_fp8(at(0x1000), SMLP_BF16, a, b, c, c, 1, at(0x100000), fat(0x200000), nullptr);
        (void)shared_mlp_quant_fp8(at(0x1000), SMLP_FP32, a, b, c * 16, c * 16, 128, at(0x100000), fat(0x200000), nullptr);
        for (int64_t d : odd) {
          (void)shared_mlp_experts_fp8_workspace_bytes(a, b * 16, c * 16, d, 8, 0, &n);
          (void)shared_mlp_experts_fp8_workspace_bytes(a, 256, 128, b, d, 1, &n);
        }
        g_launches = 0;
      }
  expect("linear", shared_mlp_linear_fp8(at(0x1000), nullptr, at(0x100000), fat(0x200000), at(0x300000), 5, 256, 7, 7, 0,
                                         at(0x40000000), 1 << 20, nullptr), SMLP_OK, 1);
  expect("experts bytes", shared_mlp_experts_fp8_workspace_bytes(64, 256, 128, 8, 2, 0, &n), SMLP_OK, 0);
  auto experts = [&](size_t bytes, int64_t first) {
    return shared_mlp_experts_fp8(at(0x1000000), ids, w, at(0x30000000), fat(0x38000000), at(0x39000000), fat(0x3a000000),
                                  at(0x3b000000), 64, 256, 128, 8, 2, first, 0, at(0x40000000), bytes, nullptr);
  };
  expect("experts", experts(n, 0), SMLP_OK, 1);
  expect("experts, small workspace", experts(n - 1, 0), SMLP_ERR_WORKSPACE, 0);
  expect("experts, first < 0", experts(n, -1), SMLP_ERR_ARG, 0);
  std::printf(g_bad ? "%d checks failed\n" : "all checks passed\n", g_bad);
  return g_bad != 0;
}
