// Host-side interface between the C ABI (api.cpp) and the kernel launchers.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "smlp.h"

namespace smlp {

// Record a status and its detail (shared_mlp_last_error) and return the status (api.cpp);
// SMLP_OK clears the detail.
int set_error(int status, const char* msg);

// One weight-streaming (small-M) stage: out-features in blocks of 16, K split into
// `ksplit` slices over workgroups and into `waves` slices inside a workgroup.
struct SkinnyPlan {
  int kind;      // SKINNY_STREAM16 or SKINNY_DIRECT16
  int mt;        // 16-token tiles (M <= 16 * mt)
  int nb;        // output tiles per workgroup (SKINNY_STREAM16: 16-row MFMA tiles holding
                 // 8 gate_up features or 16 down rows; SKINNY_DIRECT16: 16-feature blocks)
  int waves;     // waves per workgroup (they split K)
  int u;         // SKINNY_STREAM16: LDS ring stages; SKINNY_DIRECT16: 64-element K steps
                 // per wave per pipeline stage
  int ksplit;    // workgroups along K (1 = no cross-workgroup reduction)
  int kslice;    // K elements per workgroup slice (multiple of 64)
  int blocks;    // total workgroups
  int fpw;       // SKINNY_STREAM16: features (gate_up) or rows (down) per workgroup
  int ttiles;    // SKINNY_STREAM16 token split: workgroups along M, 16 * mt tokens each
                 // (0 or 1 = none; blocks counts every workgroup)
  int red_ok;    // a K split may be reduced in the same launch (off for a pinned shape)
};

enum { SKINNY_DIRECT16 = 2, SKINNY_STREAM16 = 3 };

// One stage of the LDS-tiled GEMM path (gemm.hip).
struct GemmPlan {
  int bm, bn;    // tile: tokens x weight rows (gate_up: bn/2 features)
  int wm, wn;    // wave grid
  int ns;        // LDS stages
  int tiles_m;   // tiles along M (tiles = tiles_m * tiles along N)
  int tiles;
  int ksplit;    // workgroups along K
  int kslice;    // K elements per slice (multiple of 64)
  int ntb;       // weight loads non-temporal (a tile of SMLP_GEMM_NT_CONFIGS)
};

struct Plan {
  int path;                 // SMLP_PATH_*
  int64_t M, H, I;
  int dtype;
  int partial_fp32;
  int h_dtype;              // SMLP_FP32, SMLP_BF16, SMLP_BF16_HILO or SMLP_FP16
  size_t h_offset, h_bytes;
  size_t part_offset, part_bytes;   // split-K partial sums
  size_t wd16_offset, wd16_bytes;   // fp16 copy of w_down [H, I] (dense) when the down stage
                                    // multiplies fp16 h by pre-converted weights
  size_t workspace_bytes;
  SkinnyPlan gu, dn;
  GemmPlan ggu, gdn;
  // Large-M stages split by output columns: ggu / gdn cover features / rows [0, split)
  // in whole rounds of workgroups and the tail plan the rest (split = 0: no split).
  GemmPlan ggu_tail, gdn_tail;
  int64_t gu_split, dn_split;
  // Large-M path with the gate_up stage run by the weight-streaming kernel split over
  // tokens (plan gu) instead of the tiled GEMM (ggu).
  int gu_tsplit;
  int kernels;
  // Weight views (a rank's slice read in place from full weights): rows between a gate
  // row and its up row in w_gate_up (I for whole weights), and the row stride of w_down
  // in elements (I for whole weights).
  int64_t up_off, ldwd;
};

// Weight-streaming stages (skinny.hip).  Return a hipError_t.
int launch_skinny_gate_up(const Plan& p, const void* x, const void* w_gate_up, void* ws,
                          hipStream_t s);
int launch_skinny_down(const Plan& p, const void* w_down, void* out, void* ws, hipStream_t s);
// One-launch decode layer (both stages in one grid; skinny.hip): whether plan p has the
// stage configurations it is built for, and the launch with counter slot `slot` and a
// consumer wait of at most `limit` polls.  Returns a hipError_t.
constexpr int kLayerSyncSlots = 16;
// Counter slot of `stream` on the current device (api.cpp; -1 when all are taken), and
// whether one-launch forms and in-launch reductions are enabled (shared_mlp_tune_layer_fusion).
int stream_slot(hipStream_t stream);
bool fusion_enabled();
// Per-column counters for an in-launch K-split reduction over `columns` columns on
// `stream`, or null (then a finalize launch reduces) (skinny.hip).
constexpr int kRedColumns = 256;  // most columns
uint32_t* reduce_counters(hipStream_t stream, int columns);
// The same for a product whose launch may be captured: a captured launch keeps its counters
// wherever and whenever its graph is replayed, so it gets `columns` of its own (null once they
// are used up), any other launch its stream's (skinny.hip).
uint32_t* product_counters(hipStream_t stream, int columns);
// Counters given out once each: the first of n, or -1 when fewer are left of `all`.
struct CounterRun {
  int64_t used = 0;
  int64_t take(int64_t n, int64_t all) {
    if (n < 0 || n > all - used) return -1;
    used += n;
    return used - n;
  }
};
bool decode_layer_eligible(const Plan& p);
int launch_decode_layer(const Plan& p, const void* x, const void* w_gate_up, const void* w_down, void* out,
                        void* ws, int slot, int limit, hipStream_t s);

// Sum K-split partials [ksplit][M][P*N] in slice order and apply the stage epilogue
// (gate_up: SiLU-and-mul into h, h_fmt 1 = one bf16 plane, 2 = bf16 hi + lo, 3 = fp16;
// down: bf16 or fp32 out).
int launch_finalize(bool gate_up, const float* part, int ksplit, int M, int N, void* out,
                    int ldo, int out_f32, int h_fmt, hipStream_t s);

// Plain projection y = x . w^T (bf16 operands; y bf16 or fp32 with row stride ldy):
// the streaming kernel (plan kind SKINNY_STREAM16, M <= 32) or the LDS-tiled kernel,
// with `part` holding ksplit x M x N fp32 partials when the plan splits K.
int launch_skinny_linear(const SkinnyPlan& sp, const void* x, const void* w, void* y, int M, int K,
                         int N, int ldy, int out_f32, float* part, hipStream_t s, int ldw = 0);
int launch_gemm_linear(const GemmPlan& gp, const void* x, const void* w, void* y, int M, int K,
                       int N, int ldy, int out_f32, float* part, hipStream_t s);
// Rank-major -> logical column order of a gathered merged-column output (latent.hip);
// arguments validated by the caller.
int launch_restore_logical(const void* src, void* dst, int64_t M, int64_t N, const int64_t* sizes,
                           int nr, int tp, int elem_bytes, hipStream_t s);

// LDS-tiled GEMM stages (gemm.hip).
int launch_gemm_gate_up(const Plan& p, const void* x, const void* w_gate_up, void* ws, hipStream_t s);
int launch_gemm_down(const Plan& p, const void* w_down, void* out, void* ws, hipStream_t s);

// Device address of this device's static scratch array (noalloc.hip), looked up with
// hipGetSymbolAddress on the first call per device and cached.  Returns a hipError_t.
int noalloc_scratch(void** ptr);

// fp32 stages and helpers (aux.hip).
int launch_fp32_gate_up(const Plan& p, const float* x, const float* w_gate_up, void* ws,
                        hipStream_t s);
int launch_fp32_down(const Plan& p, const float* w_down, float* out, void* ws, hipStream_t s);
// Both fp32 stages in one single-workgroup launch, h in LDS, where M * I <= kFp32SmallH and
// M * H * I <= 2^20 (fp32_small_layer); the same bits as the two launches above.
constexpr int kFp32SmallH = 4096;
inline bool fp32_small_layer(int64_t M, int64_t H, int64_t I) {
  return M * I <= kFp32SmallH && M * H * I <= ((int64_t)1 << 20);
}
int launch_fp32_layer(const Plan& p, const float* x, const float* w_gate_up, const float* w_down, float* out,
                      hipStream_t s);
int launch_slice_rank(const void* wgu, const void* wd, void* wgu_r, void* wd_r, int64_t H,
                      int64_t I, int tp, int rank, int elem_bytes, hipStream_t s);
int launch_rms_rescale(const float* in, uint16_t* out, int64_t M, int64_t H, hipStream_t s);
// bf16 -> fp16 copy of a rows x cols weight matrix (source row stride ld_src) into a dense
// destination (aux.hip).
int launch_bf16_to_f16(const void* src, int64_t ld_src, int64_t rows, int64_t cols, void* dst, hipStream_t s);

// Routing to experts (route.hip); arguments validated by the caller.
int launch_route(const void* logits, int bf16, int64_t T, int64_t E, int64_t ldl, const float* bias,
                 const smlp_route& r, int32_t* ids, float* weights, hipStream_t s);

constexpr int kCUs = 256;  // compute units the grids are sized for
// Limits of the short-K down kernel (16-row weight tiles per workgroup) and of the kernels
// for one token (blocks of 128 in H; blocks of 128 in I over all pairs).
constexpr int kDownRun = 496, kTokenBlocks = 64, kTokenPairBlocks = 64;
// Most pairs that one workgroup sorts, and most chunks otherwise.
constexpr int kOneSort = 4096, kSortChunks = 64;
// Most K slices of a projection.
constexpr int kSlices = 8;

// Whether `rows` rows of n 2-byte elements, ld apart, fit a buffer resource whose stores can be
// dropped: an offset of 2^31 has to be past its end, so it spans at most 2^31 - 16 bytes.
constexpr bool rows_fit_buffer(int64_t rows, int64_t ld, int64_t n) {
  return ((rows - 1) * ld + n) * 2 <= ((int64_t)1 << 31) - 16;
}

// One 8-bit block-scaled product (fp8.hip).
enum { F8_KIND_STREAM = 0, F8_KIND_TILE = 1, F8_KIND_DOWN = 2, F8_KIND_ROW = 3, F8_KIND_NARROW = 4 };
struct F8Plan {
  int kind;
  int bm;                     // activation rows per tile
  int nt;                     // streaming: 16-row weight tiles per workgroup
  int run;                    // short-K down: 16-row weight tiles per workgroup
  int bn;                     // tiled: weight rows per workgroup
  int exact;                  // tiled: products through bf16 (fp32 results)
  int by_rows;                // tiled projection: a tile's rows of y fit one buffer (rows_fit_buffer)
  int ksplit, kslice;         // tiled projection: K slices over workgroups, 128-element blocks per slice
};

// Rows (parts x rows, row stride ldx elements) to e4m3 with one scale per row (block_rows 1;
// scale of row r, group b at scales[r * s_row + b * s_kb]) or per block of 128 rows of a part
// (dense [parts, row blocks, column blocks]) and 128 columns.
int launch_quant_fp8(const void* x, int bf16, int64_t parts, int64_t rows, int64_t cols, int64_t ldx,
                     int block_rows, void* q, float* scales, int64_t s_row, int64_t s_kb, hipStream_t s);
// The product for one row (K <= 128 * kTokenBlocks): x bf16 (xs null) or e4m3 with scales.
int launch_row_fp8(const void* x, const float* xs, const void* w, const float* ws, void* y, int64_t K, int64_t N,
                   int out_f32, hipStream_t s);
// The product for up to 16 bf16 rows (M * K < 2^30) in one launch; with a K split `part` holds
// ksplit x columns of workgroups x nt x 256 fp32 partials.
int launch_narrow_fp8(const F8Plan& p, const void* x, const void* w, const float* ws, void* y, int64_t M, int64_t K,
                      int64_t N, int64_t ldy, int out_f32, float* part, hipStream_t s);
int launch_linear_fp8(const F8Plan& p, const void* a8, const float* as, int64_t as_row, int64_t as_kb,
                      const void* w, const float* ws, void* y, int64_t M, int64_t K, int64_t N, int64_t ldy,
                      int out_f32, float* part, hipStream_t s);

// The routed experts: sort, gate_up, (requantisation of h,) down, weighted sum (fp8.hip).
struct ExpertsPlan {
  int64_t T, H, I, E, topk;
  int64_t P;            // pairs = T * topk
  int64_t max_tiles;    // row tiles that any routing can need
  F8Plan gu, dn;
  int chunk;            // pairs per workgroup of the sort in two launches (0: one workgroup)
  int token;            // one token: two launches without a sort
  int y_f32;            // rows of y held in fp32 (1) or fp16 with exponents (0)
  size_t hdr_off, perm_off, place_off, counts_off, yexp_off, x8_off, xs_off, h8_off, hs_off, h32_off, y_off, workspace_bytes;
};
struct ExpertsCall {
  const void* x;
  const int32_t* ids;
  const float* weights;
  const void* w_gate_up;
  const float* s_gate_up;
  const void* w_down;
  const float* s_down;
  void* out;
  int64_t first;
  int out_f32;
};
int launch_experts_fp8(const ExpertsPlan& p, const ExpertsCall& c, void* workspace, hipStream_t s);

}  // namespace smlp
