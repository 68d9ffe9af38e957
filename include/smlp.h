/*
 * smlp.h -- C ABI of the MI355X (gfx950) shared-expert SwiGLU MLP library (libsmlp.so).
 *
 * The operation (vLLM PR 50656, "[Kimi-K3] Add option to shard the shared expert
 * instead of replicating", sections "Problem" and "Change"; the equivalence test in
 * the prhub.com.cn digest of that PR, section 关键源码片段):
 *
 *     G   = x . Wg^T            Wg = w_gate_up rows [0, I)       (gate_up_proj)
 *     U   = x . Wu^T            Wu = w_gate_up rows [I, 2I)
 *     h   = SiLU(G) * U         SiLU(g) = g / (1 + e^-g)          (SiluAndMul)
 *     out = h . Wd^T            Wd = w_down, stored [H, I]        (down_proj)
 *
 * Replicated layout: the caller passes the full weights (I = 6144 for Kimi-K3) and
 * gets the layer output.  TP-sharded layout: the caller passes one rank's shard
 * ([gate_r; up_r] and the matching column block of Wd, I = I_full / tp) and asks for
 * an fp32 output, which is that rank's partial over its intermediate slice -- the
 * tensor the sharded block hands to its reduce-scatter (down_proj with the
 * reduction turned off, digest section 实现拆解 step 3).
 *
 * Conventions for every entry point
 *  - Layouts are row-major [out, in]: x [M, H], w_gate_up [2I, H], w_down [H, I],
 *    out [M, H].  Element type is given by `dtype` (SMLP_BF16 or SMLP_FP32).
 *  - Device pointers only (memory from hipMalloc or any allocator of the same
 *    device).  The caller owns every buffer; the library keeps no pointer after a
 *    call returns and allocates no device memory.
 *  - Work is enqueued on `stream` (0 = the legacy default stream) and the call
 *    returns without synchronising.  The library never synchronises a stream.
 *    The GPU of the stream and the buffers must be the current one (hipSetDevice).
 *  - Return value: SMLP_OK (0) or an error status.  On any error nothing was
 *    launched; shared_mlp_last_error() gives a detail string (thread-local).
 *    Argument validation happens on the host before any HIP call, so every
 *    validation error is reported without touching a GPU.
 *  - There is no silent fallback: an unsupported shape or layout is an error, never
 *    a different computation.
 *  - M == 0 is a valid no-op (nothing is launched).  H and I must be >= 1.
 *  - Size limits: M*H, M*I and 2*I*H must each be < 2^31 elements.
 *  - SMLP_BF16: H % 8 == 0, I % 8 == 0 and every pointer 16-byte aligned.
 *    Accumulation is fp32; the bf16 output is rounded once, to nearest even.
 *  - SMLP_FP32: any sizes; pointers 4-byte aligned; out is fp32.
 *  - Output buffers must not overlap any input buffer or the workspace.
 *  - Calls that share a workspace must not run concurrently.
 */
#ifndef SMLP_H
#define SMLP_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Element types.  SMLP_BF16_HILO and SMLP_FP16 only describe the intermediate h in a
 * workspace: two bf16 planes [M, I] (hi first, then lo) whose sum is the fp32 value, or
 * one fp16 plane [M, I] (rounded once to nearest even; |h| must stay below 65504). */
enum { SMLP_BF16 = 0, SMLP_FP32 = 1, SMLP_BF16_HILO = 2, SMLP_FP16 = 3 };

/* Status codes. */
enum {
  SMLP_OK = 0,
  SMLP_ERR_NULL = 1,      /* a required pointer is NULL                                  */
  SMLP_ERR_SHAPE = 2,     /* a size is out of range or breaks a divisibility rule        */
  SMLP_ERR_ALIGN = 3,     /* a pointer is not aligned as the dtype requires              */
  SMLP_ERR_ALIAS = 4,     /* an output overlaps an input or the workspace                */
  SMLP_ERR_WORKSPACE = 5, /* workspace_bytes is smaller than shared_mlp_workspace_bytes  */
  SMLP_ERR_DTYPE = 6,     /* unknown dtype, or a flag the dtype does not support         */
  SMLP_ERR_HIP = 7,       /* a HIP runtime call or kernel launch failed                  */
  SMLP_ERR_ARG = 8        /* another argument is out of range (tp, rank, threshold)     */
};

/* Kernel path chosen by the M-dispatch. */
enum {
  SMLP_PATH_NONE = 0,     /* M == 0                                                       */
  SMLP_PATH_FP32 = 1,     /* fp32 inputs: plain fp32 kernels, any shape                   */
  SMLP_PATH_SMALL_M = 2,  /* bf16, M < large-M threshold: weight-streaming kernels        */
  SMLP_PATH_LARGE_M = 3   /* bf16, M >= threshold: LDS-tiled bf16 MFMA GEMM kernels       */
};

/* Static name of a status code. */
const char* shared_mlp_status_string(int status);

/* Detail of the last non-OK status returned on this thread ("" if none). */
const char* shared_mlp_last_error(void);

/* Dispatch plan of one forward call.  Filled by shared_mlp_plan (host-only). */
typedef struct {
  int path;               /* SMLP_PATH_*                                                  */
  int h_dtype;            /* storage type of the intermediate h in the workspace          */
  size_t h_offset;        /* byte offset of h [M, I] (row-major) inside the workspace     */
  size_t workspace_bytes; /* bytes of workspace the call needs                            */
  int gate_up_ksplit;     /* K-split factor of the gate_up stage (1 = none)              */
  int down_ksplit;        /* K-split factor of the down stage                             */
  int gate_up_blocks;     /* workgroups of the gate_up stage's main kernel                */
  int down_blocks;        /* workgroups of the down stage's main kernel                   */
  int kernels;            /* kernel launches per forward call (1 for the one-launch      */
                          /* decode layer, 2 there on a stream past the 16th per device;  */
                          /* 1 for a small fp32 layer, M*I <= 4096 and M*H*I <= 2^20)      */
} smlp_plan;

/* Plan of shared_mlp_forward for these sizes.  Host-only; no HIP call. */
int shared_mlp_plan(int64_t M, int64_t H, int64_t I, int dtype, int partial_fp32,
                    smlp_plan* plan);

/* Bytes of workspace shared_mlp_forward needs for these sizes (host-only). */
int shared_mlp_workspace_bytes(int64_t M, int64_t H, int64_t I, int dtype, size_t* bytes);

/*
 * Forward pass of the SwiGLU MLP (formula above).
 *   x            [M, H]   dtype
 *   w_gate_up    [2I, H]  dtype, rows [0, I) gate, rows [I, 2I) up
 *   w_down       [H, I]   dtype
 *   out          [M, H]   fp32 if dtype == SMLP_FP32 or partial_fp32 != 0, else bf16
 *   partial_fp32 nonzero: write fp32 (a TP rank's partial sum); zero: bf16 output
 *   workspace    device scratch of >= shared_mlp_workspace_bytes(...) bytes, 256-byte
 *                aligned; contents on entry are ignored, on exit unspecified
 * One to five kernels are enqueued on `stream` (see smlp_plan.kernels).  At M <= 32
 * with bf16 weights the two stages run as one launch whose down workgroups wait
 * (bounded) for the gate_up workgroups of the same launch; it keeps a few counters per
 * stream in a static device array (16 streams per GPU; further streams get the
 * two-launch form).  Calls on one stream, and on different streams, may run as usual.  A
 * captured launch keeps the counters of the stream it was captured on, wherever its graph
 * is replayed: what was captured on one stream must not run at the same time as anything
 * else captured on that stream or launched on it (a second replay of the same graph,
 * another graph, an eager call).  The same holds for shared_mlp_linear (smlp_latent.h).  If a down workgroup ever gives up waiting, its output
 * rows are NaN.  A small fp32 layer (M * I <= 4096, M * H * I <= 2^20) runs both stages
 * in one single-workgroup launch with h in LDS; the workspace is still required.
 * SiLU(g) * u is formed as (g * u) / (1 + e^-g): a g * u past fp32's range gives an
 * infinity or a NaN, also where SiLU(g) * u itself would be in it.
 */
int shared_mlp_forward(const void* x, const void* w_gate_up, const void* w_down, void* out,
                       int64_t M, int64_t H, int64_t I, int dtype, int partial_fp32,
                       void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * shared_mlp_forward without a workspace argument and without any allocation, for
 * callers that cannot allocate device memory: code under HIP graph capture, tight
 * serving loops, harnesses that forbid allocation.  The intermediate h and any K-split
 * partial sums live in a static device array of SMLP_NOALLOC_SCRATCH_BYTES bytes
 * (32 MiB), one per GPU, held from library load until the process ends.  A call whose
 * plan needs more (shared_mlp_plan's workspace_bytes; e.g. the M = 8192 prefill) returns
 * SMLP_ERR_WORKSPACE before any HIP call.  Every call on one GPU uses that GPU's array:
 * calls that overlap on one GPU (concurrent streams or threads) race and must be
 * serialised by the caller.  The array keeps the last call's contents; nothing in it
 * needs to start at zero.  Arguments and results are those of shared_mlp_forward.
 */
#define SMLP_NOALLOC_SCRATCH_BYTES (32u << 20)
int shared_mlp_forward_noalloc(const void* x, const void* w_gate_up, const void* w_down, void* out,
                               int64_t M, int64_t H, int64_t I, int dtype, int partial_fp32,
                               hipStream_t stream);

/*
 * The two halves of shared_mlp_forward, for callers that time or test them apart.
 * shared_mlp_gate_up_act computes h = SiLU(x Wg^T) * (x Wu^T) into the workspace
 * (at smlp_plan.h_offset, as smlp_plan.h_dtype); shared_mlp_down then computes out
 * from that h.  Both calls must get the same M, H, I, dtype, partial_fp32 and
 * workspace; together they equal one shared_mlp_forward.
 */
int shared_mlp_gate_up_act(const void* x, const void* w_gate_up, int64_t M, int64_t H,
                           int64_t I, int dtype, int partial_fp32, void* workspace,
                           size_t workspace_bytes, hipStream_t stream);
int shared_mlp_down(const void* w_down, void* out, int64_t M, int64_t H, int64_t I, int dtype,
                    int partial_fp32, void* workspace, size_t workspace_bytes,
                    hipStream_t stream);

/*
 * M-dispatch threshold: bf16 calls with M >= threshold take the LDS-tiled MFMA path,
 * smaller M the weight-streaming path (which serves at most 128 tokens, so M > 128
 * always takes the tiled path).  The initial value is 33, or the value of the
 * environment variable SMLP_LARGE_M_MIN (an integer in [1, 129]) read at library
 * load.  Returns the previous threshold, or -1 (SMLP_ERR_ARG detail) if threshold is
 * outside [1, 129].  Process-wide; not synchronised with calls in flight on other
 * threads.
 */
int64_t shared_mlp_set_large_m_threshold(int64_t threshold);

/*
 * Shard-gating predicate (prhub digest of PR 50656, section 实现拆解 step 2): returns
 * 1 when the MLP should be TP-sharded -- the opt-in flag is on, sequence
 * parallelism is on, the call site is eligible, tp > 1, and H and I both divide
 * by tp -- and 0 when it stays replicated.  Pure host function; it is the only
 * place where "replicate instead" is an answer, and it is an explicit query.
 */
int shared_mlp_shard_eligible(int flag_on, int use_sequence_parallel, int caller_eligible,
                              int tp, int64_t H, int64_t I);

/*
 * Copy rank `rank`'s shard out of full weights (digest section 关键源码片段): with
 * s = I / tp, w_gate_up_r [2s, H] = [gate rows r*s..(r+1)*s ; up rows I+r*s..I+(r+1)*s]
 * and w_down_r [H, s] = columns r*s..(r+1)*s of w_down [H, I].  Requires I % tp == 0
 * and 0 <= rank < tp (else SMLP_ERR_ARG); bit-exact copy; destination buffers must
 * not overlap the sources.  Same pointer and alignment rules as the forward call.
 */
int shared_mlp_slice_rank(const void* w_gate_up, const void* w_down, void* w_gate_up_r,
                          void* w_down_r, int64_t H, int64_t I, int tp, int rank, int dtype,
                          hipStream_t stream);

/*
 * Rank `rank`'s fp32 partial of the TP-sharded layer, computed straight from the full
 * weights without copying a shard (the slice of shared_mlp_slice_rank, read in place):
 * with s = I / tp, gate rows [r*s, (r+1)*s) and up rows I + [r*s, (r+1)*s) of w_gate_up
 * [2I, H], and columns [r*s, (r+1)*s) of w_down [H, I] (row stride I).  Lets a caller
 * that keeps the replicated weights resident run the sharded layout on any step.
 *   x [M, H], out [M, H] fp32 (always the partial); workspace as for
 *   shared_mlp_workspace_bytes(M, H, I / tp, dtype).  Requires I % tp == 0 and
 *   0 <= rank < tp (else SMLP_ERR_ARG), and for bf16 s % 8 == 0 (SMLP_ERR_SHAPE).
 * Equal, up to fp32 summation order, to shared_mlp_forward(partial_fp32 = 1) on the
 * copied shard.
 */
int shared_mlp_forward_rank(const void* x, const void* w_gate_up, const void* w_down, void* out,
                            int64_t M, int64_t H, int64_t I, int tp, int rank, int dtype,
                            void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * Per-token rescale to unit RMS, the glue between the layers of a stacked-layer
 * chain: out[m, :] = bf16_rne(in[m, :] / sqrt(mean_k in[m, k]^2)), computed in fp32.
 *   in   [M, H] fp32 (e.g. a partial output), out [M, H] bf16; no epsilon: a row
 *   whose RMS is zero yields NaN.  Pointers 16-byte aligned, H % 4 == 0, out must
 *   not overlap in.
 */
int shared_mlp_rms_rescale(const float* in, void* out, int64_t M, int64_t H,
                           hipStream_t stream);

/* ---------------------------------------------------------------------------------------
 * The routed half of the layer: routing to experts, the 8-bit block-scaled product, the
 * routed experts' SwiGLU.
 * ------------------------------------------------------------------------------------- */

#define SMLP_MAX_EXPERTS 1024
#define SMLP_MAX_TOPK 64
#define SMLP_MAX_GROUPS 64

enum { SMLP_SCORE_SIGMOID = 0, SMLP_SCORE_SOFTMAX = 1 };

/* How shared_mlp_route chooses. */
typedef struct {
  int score;       /* SMLP_SCORE_*                                                        */
  int groups;      /* equal contiguous groups of experts (1 = none)                       */
  int top_groups;  /* groups that stay eligible, 1 .. groups                              */
  int group_top;   /* a group counts as the sum of this many largest choices (1 or 2)     */
  int topk;        /* experts per token                                                   */
  int renormalize; /* nonzero: weights divided by their sum                               */
  float scale;     /* factor on the weights                                               */
} smlp_route;

/*
 * Routing of tokens to experts.  For row t, with l = fp32(logits[t, :]):
 *   score   sigmoid: s_e = 1 / (1 + e^-l_e); softmax: s_e = e^(l_e - max l) / sum (a row of
 *           -inf only: all 0)
 *   choice  c_e = s_e + bias_e (bias NULL: 0); softmax without a bias: c_e = l_e, the same
 *           order.  A NaN choice counts below -inf.
 *   groups  the top_groups groups with the largest sums of their group_top best choices
 *   ids     the topk eligible experts of largest choice, in descending order
 *   weights their scores; renormalize: over their sum (0 where it is 0); times scale
 * Ties go to the lower index everywhere.  Scores, choices and sums are fp32.
 *   logits  T rows of E elements, row t at logits + t * ldl; dtype SMLP_BF16 or SMLP_FP32
 *   bias    [E] fp32 or NULL
 *   ids     [T, topk] int32, weights [T, topk] fp32
 * E in [1, SMLP_MAX_EXPERTS] and a multiple of groups; topk in [1, SMLP_MAX_TOPK] and at
 * most top_groups * E / groups; group_top <= E / groups; softmax with group_top 2 needs a
 * bias (SMLP_ERR_ARG otherwise); ldl >= E; T * max(ldl, topk) < 2^31.  T == 0 is a no-op.
 */
int shared_mlp_route(const void* logits, int dtype, int64_t T, int64_t E, int64_t ldl, const float* bias,
                     const smlp_route* route, int32_t* ids, float* weights, hipStream_t stream);

/*
 * The 8-bit form of a tensor: e4m3 values (OCP, largest finite value 448) with one fp32
 * scale per group, the value being q * scale.  With a = max(max|x| over the group, 1e-30):
 *   scale = a / 448,   q = e4m3_rne(x * (448 * (1 / a)))  (each operation rounded to fp32)
 * A NaN stays a NaN; an infinity makes every product with its group a NaN.
 *   x       parts * rows rows of cols elements, row stride ldx; dtype SMLP_BF16 or
 *           SMLP_FP32; 16-byte aligned, ldx * element size a multiple of 16
 *   block_rows  1 (activations): groups of 1 row x 128 columns, scales [parts * rows,
 *           ceil(cols / 128)]; 128 (weights): blocks of 128 rows x 128 columns that start
 *           anew with each part, scales [parts, ceil(rows / 128), ceil(cols / 128)]
 *   q       dense [parts * rows, cols], 16-byte aligned
 * cols a positive multiple of 16; rows >= 1; parts * rows * max(ldx, cols) < 2^40 and at
 * most 2^31 - 1 blocks.  parts == 0 is a no-op.  (Merged gate_up weights of E experts are
 * 2 E parts of I rows, down weights E parts of H rows.)
 */
int shared_mlp_quant_fp8(const void* x, int dtype, int64_t parts, int64_t rows, int64_t cols, int64_t ldx,
                         int block_rows, void* q, float* scales, hipStream_t stream);

/* Bytes of workspace shared_mlp_linear_fp8 needs (host-only; x_fp8: x is given as e4m3). */
int shared_mlp_linear_fp8_workspace_bytes(int64_t M, int64_t K, int64_t N, int x_fp8, size_t* bytes);

/*
 * y[m, n] = sum_b xs[m, b] ws[n / 128, b] sum_{k in block b} xq[m, k] wq[n, k], blocks b of
 * 128 K elements; fp32 accumulation.
 *   x         x_scales given: e4m3 [M, K] with x_scales [M, ceil(K / 128)]; x_scales NULL:
 *             bf16 [M, K], brought to that form first (as shared_mlp_quant_fp8 does)
 *   w         e4m3 [N, K], w_scales [ceil(N / 128), ceil(K / 128)]
 *   y         M rows of N elements, row m at y + m * ldy; bf16 (out_fp32 == 0, rounded once)
 *             or fp32 (out_fp32 == 1)
 * K a positive multiple of 16; N >= 1; ldy >= N; M * K, N * K and M * ldy < 2^31; x and w
 * 16-byte aligned, y aligned to its element; workspace 256-byte aligned (may be NULL when
 * 0 bytes are needed).  y must not overlap an input or the workspace.  M == 0 is a no-op.
 * Products are exact and summed in fp32, except where M > 32, K > 512 and y is bf16: there
 * the 8-bit matrix instructions are used at twice the rate, whose sums are about 1.5e-5 off
 * (2-norm; one bf16 value in about 500 rounds the other way for it).  out_fp32 == 1 always
 * takes the exact products.
 * A product whose K is split over workgroups (few outputs) counts arrivals in a static device
 * array: on its stream's counters (16 streams per GPU; further ones run without the split),
 * or, captured, on counters of its own (2^18 tiles per GPU over the life of the process;
 * captures beyond that run without the split).  So graphs may be replayed beside one another
 * and beside eager calls, as long as their buffers are apart; one graph not twice at a time.
 */
int shared_mlp_linear_fp8(const void* x, const float* x_scales, const void* w, const float* w_scales, void* y,
                          int64_t M, int64_t K, int64_t N, int64_t ldy, int out_fp32, void* workspace,
                          size_t workspace_bytes, hipStream_t stream);

/* Bytes of workspace shared_mlp_experts_fp8 needs for these sizes (host-only). */
int shared_mlp_experts_fp8_workspace_bytes(int64_t T, int64_t H, int64_t I, int64_t E, int64_t topk,
                                           int partial_fp32, size_t* bytes);

/*
 * The routed experts' SwiGLU on 8-bit weights, over ids and weights of shared_mlp_route:
 *   xq = 8-bit form of x (rows in groups of 128);  for each pair (t, j) with
 *   e = ids[t, j] - first_expert in [0, E):
 *     g = xq[t] Wg_e^T,  u = xq[t] Wu_e^T,  h = SiLU(g) * u (fp32), hq = 8-bit form of h
 *     y = hq Wd_e^T
 *   out[t] = sum_j weights[t, j] * y      (pairs of other experts add nothing; 0 if none)
 * first_expert and E select the experts this rank holds (expert parallelism); with an
 * intermediate slice of every expert it is the tensor-parallel partial.
 *   x           [T, H] bf16
 *   ids         [T, topk] int32 (any values), weights [T, topk] fp32
 *   w_gate_up   e4m3 [E, 2 I, H] (gate rows, then up rows), s_gate_up [E, 2 ceil(I / 128),
 *               ceil(H / 128)]: the row blocks of the gate rows, then those of the up rows
 *   w_down      e4m3 [E, H, I], s_down [E, ceil(H / 128), ceil(I / 128)]
 *   out         [T, H] bf16 (rounded once; with many tokens each expert's y passes through
 *               fp16 with a common exponent per 64 columns) or fp32 (partial_fp32 != 0)
 * With at most 12 pairs per expert on average, and with partial_fp32 != 0, products are exact
 * and summed in fp32.  Otherwise the 8-bit matrix instructions are used: g and u are about
 * 1.5e-5 off (2-norm), so one value of h in some thousands is stored as the neighbouring e4m3
 * value, and out is 2.0e-3 to 2.3e-3 off the definition instead of the 1.7e-3 that rounding
 * to bf16 alone makes.  partial_fp32 != 0 is how a caller has the exact products (8192 tokens,
 * 8 of 64 experts of 768: 2.98 ms instead of 1.52).
 *   workspace   >= shared_mlp_experts_fp8_workspace_bytes(...), 256-byte aligned
 * H and I positive multiples of 16; E in [1, SMLP_MAX_EXPERTS]; topk in [1, SMLP_MAX_TOPK];
 * T * H, T * topk, T * topk * I and 2 * I * H < 2^31; x, w_gate_up, w_down and out 16-byte
 * aligned.  out must not overlap an input or the workspace.  T == 0 is a no-op.
 */
int shared_mlp_experts_fp8(const void* x, const int32_t* ids, const float* weights, const void* w_gate_up,
                           const float* s_gate_up, const void* w_down, const float* s_down, void* out, int64_t T,
                           int64_t H, int64_t I, int64_t E, int64_t topk, int64_t first_expert, int partial_fp32,
                           void* workspace, size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* SMLP_H */
