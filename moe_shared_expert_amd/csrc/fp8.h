// Device helpers of the 8-bit (e4m3) block-scaled kernels.
#pragma once
#include "device_common.h"

namespace smlp {

typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr float kE4M3Max = 448.0f;
// Groups whose largest magnitude is below this are scaled as if it were this, so that the
// scale and its reciprocal stay normal fp32 numbers.
constexpr float kAmaxMin = 1e-30f;

// Four floats -> four packed e4m3 values (element 0 in bits 0..7), round to nearest even.
__device__ __forceinline__ uint32_t pack_fp8x4(float a, float b, float c, float d) {
  int r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  r = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
  return (uint32_t)r;
}

// SiLU(g) * u in fp32, SiLU first: it is at most |g|, so only a result past the range of fp32
// overflows (g * u formed first would, and be a NaN where e^-g does too).
__device__ __forceinline__ float silu_then_mul(float g, float u) { return g / (1.0f + __expf(-g)) * u; }

// A 16x16x128 product of e4m3 operands, from zero.  Lane l holds 32 K elements of A row
// l % 16 and of B column l % 16; any assignment of K elements to (l / 16, position) serves
// as long as A and B use the same one.  Lane l, element j of the result: row
// 4 * (l / 16) + j of A, column l % 16 of B.
__device__ __forceinline__ f32x4 mfma_fp8(i32x8 a, i32x8 b) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}

// The same product through bf16: an e4m3 value is a bf16 value, and the bf16 instructions add
// the exact products in fp32.  The 8-bit instructions drop low bits as they add (those of 32 and
// of 128 elements alike): measured on N(0, 1) data they are 1.5e-5 (2-norm) off the exact sum,
// without a bias (so the same for 1 and for 512 blocks), the bf16 form 1e-8.
struct frag_bf16 {
  u32x4 q[4];  // 32 K elements
};
__device__ __forceinline__ frag_bf16 widen(i32x8 v) {
  frag_bf16 f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const auto lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((unsigned)v[i], 1.0f, false);
    const auto hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((unsigned)v[i], 1.0f, true);
    f.q[i >> 1][2 * (i & 1)] = __builtin_bit_cast(uint32_t, lo);
    f.q[i >> 1][2 * (i & 1) + 1] = __builtin_bit_cast(uint32_t, hi);
  }
  return f;
}
__device__ __forceinline__ f32x4 mfma_widened(const frag_bf16& a, const frag_bf16& b) {
  f32x4 c{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; ++i) c = mfma16x16x32(a.q[i], b.q[i], c);
  return c;
}

// Operand fragment of one 16-row x 128-byte tile in LDS (rows of 128 bytes, 16-byte chunk c
// of row r stored at slot c ^ ((r / 2) % 8)): lane l reads chunks l / 16 and 4 + l / 16 of
// row l % 16.  The sixteen lanes of a quarter wave touch sixteen different 16-byte columns
// of the 256-byte bank row pair.
__device__ __forceinline__ i32x8 lds_frag(const char* tile, int lane) {
  const int r = lane & 15, g = lane >> 4, sw = (r >> 1) & 7;
  const u32x4 lo = *reinterpret_cast<const u32x4*>(tile + r * 128 + ((g ^ sw) * 16));
  const u32x4 hi = *reinterpret_cast<const u32x4*>(tile + r * 128 + (((g + 4) ^ sw) * 16));
  i32x8 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = (int)lo[i];
    v[4 + i] = (int)hi[i];
  }
  return v;
}

// One half (16 K elements per lane) of such a fragment into v[4 half .. 4 half + 3].
__device__ __forceinline__ void lds_half(const char* tile, int lane, int half, i32x8& v) {
  const int r = lane & 15, g = lane >> 4, sw = (r >> 1) & 7;
  const u32x4 q = *reinterpret_cast<const u32x4*>(tile + r * 128 + (((g + 4 * half) ^ sw) * 16));
#pragma unroll
  for (int i = 0; i < 4; ++i) v[4 * half + i] = (int)q[i];
}

// 4 bytes per lane from each lane's own address into 256 consecutive bytes of LDS.
typedef const __attribute__((address_space(1))) void glb_void;
__device__ __forceinline__ void glb_ld_lds4(const void* p, char* dst) {
  __builtin_amdgcn_global_load_lds((glb_void*)p, (lds_void*)dst, 4, 0, 0);
}

}  // namespace smlp
