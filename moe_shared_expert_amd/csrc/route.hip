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
  int per;    // experts per group
  int whole;  // E a multiple of the experts per lane, rows and bias aligned to 32 bytes
  smlp_route r;
};

// Order-preserving map of a choice value to an unsigned key: 0 is kept for "not eligible",
// NaN maps to 1 (below -inf), -0 and +0 to the same key.
__device__ __forceinline__ uint32_t choice_key(float c) {
  if (c != c) return 1u;
  const uint32_t u = __float_as_uint(c + 0.0f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// Data-parallel moves inside the wave (no LDS traffic): the lane `CTRL` names, or `old` where
// there is none.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v, uint32_t old) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)old, (int)v, CTRL, 0xf, 0xf, false);
}
enum { SHR1 = 0x111, SHR2 = 0x112, SHR4 = 0x114, SHR8 = 0x118, BCAST15 = 0x142, BCAST31 = 0x143 };
enum { XOR1 = 0xB1, XOR2 = 0x4E, HALF_MIRROR = 0x141, MIRROR = 0x140 };

// Reductions over the 64 lanes: the last lane collects, the result is wave-uniform.
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
  v = max(v, dpp<SHR1>(v, 0));
  v = max(v, dpp<SHR2>(v, 0));
  v = max(v, dpp<SHR4>(v, 0));
  v = max(v, dpp<SHR8>(v, 0));
  v = max(v, dpp<BCAST15>(v, 0));
  v = max(v, dpp<BCAST31>(v, 0));
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
template <int CTRL>
__device__ __forceinline__ float dpp_f(float v, float old) {
  return __uint_as_float(dpp<CTRL>(__float_as_uint(v), __float_as_uint(old)));
}
__device__ __forceinline__ float wave_max_f32(float v) {
  v = fmaxf(v, dpp_f<SHR1>(v, -INFINITY));
  v = fmaxf(v, dpp_f<SHR2>(v, -INFINITY));
  v = fmaxf(v, dpp_f<SHR4>(v, -INFINITY));
  v = fmaxf(v, dpp_f<SHR8>(v, -INFINITY));
  v = fmaxf(v, dpp_f<BCAST15>(v, -INFINITY));
  v = fmaxf(v, dpp_f<BCAST31>(v, -INFINITY));
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), 63));
}
__device__ __forceinline__ float wave_sum_f32(float v) {
  v += dpp_f<SHR1>(v, 0.f);
  v += dpp_f<SHR2>(v, 0.f);
  v += dpp_f<SHR4>(v, 0.f);
  v += dpp_f<SHR8>(v, 0.f);
  // The broadcasts add row 0 to row 1 and row 2 to row 3, then rows 0-1 to rows 2-3; only
  // the last lane's sum is read, and it takes each row once.
  v += dpp_f<BCAST15>(v, 0.f);
  v += dpp_f<BCAST31>(v, 0.f);
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), 63));
}

// The two largest of (a1 >= a2) and (b1 >= b2).
__device__ __forceinline__ void merge2(float& a1, float& a2, float b1, float b2) {
  a2 = fmaxf(fminf(a1, b1), fmaxf(a2, b2));
  a1 = fmaxf(a1, b1);
}

__device__ __forceinline__ void wave_fence() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_wave_barrier();
}

constexpr int kRouteWaves = 4;

// One wave per token.  Lane p holds experts p * VPT .. p * VPT + VPT - 1, so that the
// lowest lane with the largest key holds the lowest index.  One token takes 3.6 us, nearly all
// of it latency; 8192 x 256 (top 8 of 4 of 8 groups) 10.8 us against 2 us for its 8.9 MB: about
// 800 instructions per token are issued, half of them in the eight rounds of the choice.  Two
// tokens per wave share the reductions but scan twice the experts per lane, and took the same.
template <int VPT, bool BF>
__global__ __launch_bounds__(kRouteWaves * 64) void route_kernel(RouteArgs a) {
  __shared__ float lds[kRouteWaves][VPT * 64];  // this wave's choices, then its scores
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int t = blockIdx.x * kRouteWaves + wave;
  if (t >= a.T) return;  // waves are independent: no workgroup barrier below
  const int e0 = lane * VPT;
  float* mine = lds[wave];

  float score[VPT], choice[VPT], bias[VPT];
  const size_t row = (size_t)t * a.ldl + e0;
  if (a.whole) {
    // Every lane's experts exist and sit at aligned addresses: one wide load each.
    typedef float fvec __attribute__((ext_vector_type(VPT)));
    typedef uint16_t hvec __attribute__((ext_vector_type(VPT)));
    if (e0 < a.E) {
      if constexpr (BF) {
        const hvec v = *reinterpret_cast<const hvec*>(reinterpret_cast<const uint16_t*>(a.logits) + row);
#pragma unroll
        for (int i = 0; i < VPT; ++i) score[i] = __uint_as_float((uint32_t)v[i] << 16);
      } else {
        const fvec v = *reinterpret_cast<const fvec*>(reinterpret_cast<const float*>(a.logits) + row);
#pragma unroll
        for (int i = 0; i < VPT; ++i) score[i] = v[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < VPT; ++i) score[i] = -INFINITY;
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) bias[i] = 0.0f;
    if (a.bias && e0 < a.E) {
      const fvec v = *reinterpret_cast<const fvec*>(a.bias + e0);
#pragma unroll
      for (int i = 0; i < VPT; ++i) bias[i] = v[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPT; ++i) bias[i] = a.bias && e0 + i < a.E ? a.bias[e0 + i] : 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      float l = -INFINITY;
      if (e0 + i < a.E)
        l = BF ? __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(a.logits)[row + i] << 16)
               : reinterpret_cast<const float*>(a.logits)[row + i];
      score[i] = l;
    }
  }
  if (a.r.score == SMLP_SCORE_SIGMOID) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      score[i] = 1.0f / (1.0f + expf(-score[i]));
      choice[i] = a.bias ? score[i] + bias[i] : score[i];
    }
  } else {
    float mx = score[0];
#pragma unroll
    for (int i = 1; i < VPT; ++i) mx = fmaxf(mx, score[i]);
    mx = wave_max_f32(mx);
    const float ref = mx == -INFINITY ? 0.0f : mx;  // a row of -inf: every term 0
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      choice[i] = score[i];
      score[i] = expf(score[i] - ref);
      sum += score[i];
    }
    sum = wave_sum_f32(sum);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      score[i] = sum == 0.0f ? 0.0f : score[i] / sum;
      if (a.bias) choice[i] = score[i] + bias[i];
    }
  }
  uint32_t key[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) key[i] = e0 + i < a.E ? choice_key(choice[i]) : 0u;

  if (a.r.groups > 1) {
    // 2^s lanes per group scan its choices (NaN counts as -inf) and merge their two largest;
    // then the best groups are taken one by one.
#pragma unroll
    for (int i = 0; i < VPT; ++i) mine[e0 + i] = choice[i] == choice[i] ? choice[i] : -INFINITY;
    wave_fence();
    const int sh = __builtin_clz(a.r.groups - 1) - 26;  // 64 >> sh lanes hold all groups: 2^sh lanes each
    const int grp = lane >> sh;
    float m1 = -INFINITY, m2 = -INFINITY;
    if (grp < a.r.groups)
      for (int i = lane & ((1 << sh) - 1); i < a.per; i += 1 << sh) {
        const float c = mine[grp * a.per + i];
        m2 = fmaxf(m2, fminf(m1, c));
        m1 = fmaxf(m1, c);
      }
    // Within 2^k equal lanes, the mirrored lane of the next larger run stands for the other half.
    if (sh > 0) merge2(m1, m2, dpp_f<XOR1>(m1, 0.f), dpp_f<XOR1>(m2, 0.f));
    if (sh > 1) merge2(m1, m2, dpp_f<XOR2>(m1, 0.f), dpp_f<XOR2>(m2, 0.f));
    if (sh > 2) merge2(m1, m2, dpp_f<HALF_MIRROR>(m1, 0.f), dpp_f<HALF_MIRROR>(m2, 0.f));
    if (sh > 3) merge2(m1, m2, dpp_f<MIRROR>(m1, 0.f), dpp_f<MIRROR>(m2, 0.f));
    if (sh > 4) merge2(m1, m2, __shfl_xor(m1, 16), __shfl_xor(m2, 16));
    uint32_t gkey = grp < a.r.groups ? choice_key(a.r.group_top == 2 ? m1 + m2 : m1) : 0u;
    uint64_t stay = 0;
    for (int j = 0; j < a.r.top_groups; ++j) {
      const uint32_t best = wave_max_u32(gkey);
      const int g = (__ffsll((unsigned long long)__ballot(gkey == best)) - 1) >> sh;
      stay |= 1ull << g;
      if (grp == g) gkey = 0u;
    }
    int of = e0 / a.per, left = a.per - (e0 - of * a.per);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      if (!((stay >> (of & 63)) & 1)) key[i] = 0u;
      if (--left == 0) {
        ++of;
        left = a.per;
      }
    }
  }
  wave_fence();
#pragma unroll
  for (int i = 0; i < VPT; ++i) mine[e0 + i] = score[i];

  int my_id = 0;
  for (int j = 0; j < a.r.topk; ++j) {
    uint32_t best = key[0];
    int at = 0;
#pragma unroll
    for (int i = 1; i < VPT; ++i)
      if (key[i] > best) {
        best = key[i];
        at = i;
      }
    const uint32_t top = wave_max_u32(best);
    const int src = __ffsll((unsigned long long)__ballot(best == top)) - 1;
    const int id = __builtin_amdgcn_readlane(e0 + at, src);
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if (e0 + i == id) key[i] = 0u;
    if (lane == j) my_id = id;
  }
  wave_fence();
  const float my_score = lane < a.r.topk ? mine[my_id] : 0.0f;
  const float sum = wave_sum_f32(my_score);
  if (lane >= a.r.topk) return;
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
  const int64_t eb = bf16 ? 2 : 4;
  const bool aligned = ldl * eb % 32 == 0 && (uintptr_t)logits % 32 == 0 && (uintptr_t)bias % 32 == 0;
#define SMLP_R(V)                                                                   \
  if (E <= 64 * V) {                                                                \
    a.whole = V <= 8 && E % V == 0 && aligned;                                      \
    if (bf16) hipLaunchKernelGGL((route_kernel<V, true>), grid, block, 0, s, a);    \
    else hipLaunchKernelGGL((route_kernel<V, false>), grid, block, 0, s, a);        \
    return (int)hipGetLastError();                                                  \
  }
  SMLP_R(1) SMLP_R(2) SMLP_R(4) SMLP_R(8) SMLP_R(16)
#undef SMLP_R
  return (int)hipErrorInvalidConfiguration;
}

}  // namespace smlp
