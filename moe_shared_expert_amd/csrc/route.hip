// Routing of tokens to experts: scores, choice of groups, top-k, weights.
//
// Row t of the logits gives, in fp32, a score s_e (sigmoid or softmax of l_e) and a choice
// value c_e (s_e + bias_e; for softmax without a bias l_e itself, which has the same order
// without the ties that rounding s_e would make).  The experts may be cut into equal
// contiguous groups; a group counts as the sum of its one or two largest choices and only
// the best top_groups groups are eligible.  The topk largest eligible choices are taken in
// descending order, ties to the lower index, and the weights are their scores, divided by
// their sum if asked, times a factor.
//
// The score is 1 / (1 + expf(-l)) with the correctly rounded divide (not the fast forms):
// the ids are decided by comparing scores, so every rounding of the formula as it is
// written counts.
#include "device_common.h"
#include "internal.h"
#include "smlp.h"

namespace smlp {

namespace {

struct RouteArgs {
  const void* logits;
  const float* bias;
  int32_t* ids;
  float* weights;
  int T, E, ldl;
  int per;  // experts per group
  smlp_route r;
};

// Order-preserving map of a choice value to an unsigned key: 0 is kept for "not eligible",
// NaN maps to 1 (below -inf), -0 and +0 to the same key.
__device__ __forceinline__ uint32_t choice_key(float c) {
  if (c != c) return 1u;
  const uint32_t u = __float_as_uint(c + 0.0f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// Maximum / sum over the 64 lanes, in every lane.
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v = max(v, (uint32_t)__shfl_xor((int)v, d));
  return v;
}
__device__ __forceinline__ float wave_max_f32(float v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v = fmaxf(v, __shfl_xor(v, d));
  return v;
}
__device__ __forceinline__ float wave_sum_f32(float v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

constexpr int kRouteWaves = 4;

// One wave per token.  Lane p holds experts p * VPT .. p * VPT + VPT - 1, so that the
// lowest lane with the largest key holds the lowest index.
template <int VPT, bool BF>
__global__ __launch_bounds__(kRouteWaves * 64) void route_kernel(RouteArgs a) {
  __shared__ float choice_lds[kRouteWaves][VPT * 64];
  const int lane = threadIdx.x & 63;
  const int wave = threadIdx.x >> 6;
  const int t = blockIdx.x * kRouteWaves + wave;
  const bool live = t < a.T;
  const int e0 = lane * VPT;

  float score[VPT], choice[VPT];
  uint32_t key[VPT];
  float mx = -INFINITY;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    float l = -INFINITY;
    if (live && e0 + i < a.E) {
      const size_t at = (size_t)t * a.ldl + e0 + i;
      l = BF ? __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(a.logits)[at] << 16)
             : reinterpret_cast<const float*>(a.logits)[at];
    }
    score[i] = l;
    mx = fmaxf(mx, l);
  }
  if (a.r.score == SMLP_SCORE_SIGMOID) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      score[i] = 1.0f / (1.0f + expf(-score[i]));
      choice[i] = score[i];
    }
  } else {
    mx = wave_max_f32(mx);
    const float ref = mx == -INFINITY ? 0.0f : mx;  // a row of -inf: every term 0
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const float l = score[i];
      const float p = expf(l - ref);
      choice[i] = l;
      score[i] = p;
      sum += p;
    }
    sum = wave_sum_f32(sum);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      score[i] = sum == 0.0f ? 0.0f : score[i] / sum;
      if (a.bias) choice[i] = score[i];
    }
  }
  if (a.bias) {
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if (e0 + i < a.E) choice[i] += a.bias[e0 + i];
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) key[i] = e0 + i < a.E ? choice_key(choice[i]) : 0u;

  if (a.r.groups > 1) {
    // Lane g sums group g's best choices (NaN counts as -inf); then the best groups.
#pragma unroll
    for (int i = 0; i < VPT; ++i) choice_lds[wave][e0 + i] = choice[i] == choice[i] ? choice[i] : -INFINITY;
    __syncthreads();
    uint32_t gkey = 0u;
    if (lane < a.r.groups) {
      float m1 = -INFINITY, m2 = -INFINITY;
      for (int i = 0; i < a.per; ++i) {
        const float c = choice_lds[wave][lane * a.per + i];
        m2 = fmaxf(m2, fminf(m1, c));
        m1 = fmaxf(m1, c);
      }
      gkey = choice_key(a.r.group_top == 2 ? m1 + m2 : m1);
    }
    uint64_t stay = 0;
    for (int j = 0; j < a.r.top_groups; ++j) {
      const uint32_t best = wave_max_u32(gkey);
      const int g = __ffsll((unsigned long long)__ballot(gkey == best)) - 1;
      stay |= 1ull << g;
      if (lane == g) gkey = 0u;
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if (e0 + i >= a.E || !((stay >> ((e0 + i) / a.per)) & 1)) key[i] = 0u;
  }

  int my_id = 0;
  float my_score = 0.0f;
  for (int j = 0; j < a.r.topk; ++j) {
    uint32_t best = key[0];
    int at = 0;
    float s = score[0];
#pragma unroll
    for (int i = 1; i < VPT; ++i)
      if (key[i] > best) {
        best = key[i];
        at = i;
        s = score[i];
      }
    const uint32_t top = wave_max_u32(best);
    const int src = __ffsll((unsigned long long)__ballot(best == top)) - 1;
    const int id = __shfl(e0 + at, src);
    const float sc = __shfl(s, src);
    if (lane == src) {
#pragma unroll
      for (int i = 0; i < VPT; ++i)
        if (i == at) key[i] = 0u;
    }
    if (lane == j) {
      my_id = id;
      my_score = sc;
    }
  }
  const float sum = wave_sum_f32(my_score);  // lanes past topk hold 0
  if (!live || lane >= a.r.topk) return;
  float w = my_score;
  if (a.r.renormalize) w = sum == 0.0f ? 0.0f : w / sum;
  const size_t at = (size_t)t * a.r.topk + lane;
  a.ids[at] = my_id;
  a.weights[at] = w * a.r.scale;
}

}  // namespace

int launch_route(const void* logits, int bf16, int64_t T, int64_t E, int64_t ldl, const float* bias,
                 const smlp_route& r, int32_t* ids, float* weights, hipStream_t s) {
  RouteArgs a{};
  a.logits = logits;
  a.bias = bias;
  a.ids = ids;
  a.weights = weights;
  a.T = (int)T;
  a.E = (int)E;
  a.ldl = (int)ldl;
  a.per = (int)E / r.groups;
  a.r = r;
  const dim3 grid((unsigned)((T + kRouteWaves - 1) / kRouteWaves)), block(kRouteWaves * 64);
#define SMLP_R(V)                                                                   \
  if (E <= 64 * V) {                                                                \
    if (bf16) hipLaunchKernelGGL((route_kernel<V, true>), grid, block, 0, s, a);    \
    else hipLaunchKernelGGL((route_kernel<V, false>), grid, block, 0, s, a);        \
    return (int)hipGetLastError();                                                  \
  }
  SMLP_R(1) SMLP_R(2) SMLP_R(4) SMLP_R(8) SMLP_R(16)
#undef SMLP_R
  return (int)hipErrorInvalidConfiguration;
}

}  // namespace smlp
