// C ABI of the routed half: routing, the 8-bit block-scaled product, the routed experts.
// Host-side validation and planning; every check runs before the first HIP call.
#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdio>

#include "internal.h"
#include "smlp.h"

namespace {

constexpr int64_t kLimit = (int64_t)1 << 31;

int fail(int status, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  return smlp::set_error(status, buf);
}

int ok() { return smlp::set_error(SMLP_OK, ""); }

int hip_status(int rc, const char* what) {
  if (rc == (int)hipSuccess) return SMLP_OK;
  return fail(SMLP_ERR_HIP, "%s: %s", what, hipGetErrorString((hipError_t)rc));
}

int check_ptr(const void* p, const char* name, size_t align) {
  if (!p) return fail(SMLP_ERR_NULL, "%s is NULL", name);
  if ((uintptr_t)p % align) return fail(SMLP_ERR_ALIGN, "%s is not %zu-byte aligned", name, align);
  return SMLP_OK;
}

struct Range {
  const void* p;
  size_t n;
};
bool overlap(Range a, Range b) {
  if (!a.p || !b.p || !a.n || !b.n) return false;
  const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
  return x < y + b.n && y < x + a.n;
}

int64_t blocks128(int64_t n) { return (n + 127) / 128; }
size_t round_up(size_t v) { return (v + 255) / 256 * 256; }

// a * b < 2^31 for non-negative a and b, without overflow.
bool fits(int64_t a, int64_t b) { return a < kLimit && b < kLimit && a * b < kLimit; }

// Streaming tiles of 8, 16 or 32 activation rows.
smlp::F8Plan stream_plan(int64_t rows, int64_t KB) {
  smlp::F8Plan p{};
  p.kind = smlp::F8_KIND_STREAM;
  p.nt = 2;
  p.bm = rows > 16 ? 32 : rows > 8 ? 16 : 8;
  p.ksplit = 1;
  p.kslice = (int)KB;
  return p;
}

smlp::F8Plan tile_plan(int bm, int bn, int64_t KB, int exact) {
  smlp::F8Plan p{};
  p.kind = smlp::F8_KIND_TILE;
  p.bm = bm;
  p.bn = bn;
  p.exact = exact;
  p.ksplit = 1;
  p.kslice = (int)KB;
  return p;
}

struct LinearF8Plan {
  smlp::F8Plan f;
  size_t x8_off, xs_off, part_off, workspace_bytes;
};

// Outputs of the one-launch projection of few rows, and tiles of a projection with a K split.
constexpr int64_t kNarrowN = 1536, kSplitTiles = smlp::kCUs / 2;
static_assert(kNarrowN / 16 <= smlp::kRedColumns && kSplitTiles <= smlp::kRedColumns, "a counter for each");

int make_linear_plan(int64_t M, int64_t K, int64_t N, int x_fp8, int out_fp32, LinearF8Plan* out) {
  if (M < 0) return fail(SMLP_ERR_SHAPE, "M = %lld < 0", (long long)M);
  if (K < 16 || K % 16) return fail(SMLP_ERR_SHAPE, "K = %lld is not a positive multiple of 16", (long long)K);
  if (N < 1) return fail(SMLP_ERR_SHAPE, "N = %lld < 1", (long long)N);
  if (!fits(M, K) || !fits(N, K) || !fits(M, N))
    return fail(SMLP_ERR_SHAPE, "M*K, N*K and M*N must be below 2^31");
  LinearF8Plan p{};
  const int64_t KB = blocks128(K);
  size_t part = 0;
  if (M == 1 && KB <= smlp::kTokenBlocks) {
    p.f = stream_plan(M, KB);
    p.f.kind = smlp::F8_KIND_ROW;  // x is brought to its 8-bit form in each workgroup
    x_fp8 = 1;
  } else if (M <= 16 && N <= kNarrowN && !x_fp8 && M * K < kLimit / 2) {
    // Few rows of w: x is brought to its 8-bit form by the workgroups that use it (16 x 512 x
    // 7168: 6.8 us against 14 us with a launch of its own; at N = 2112 they took the same, 11.7 us
    // with the launch, of which it is 2.5).
    p.f = stream_plan(M, KB);
    p.f.kind = smlp::F8_KIND_NARROW;
    p.f.nt = 1;
    x_fp8 = 1;
    // Up to two workgroups per compute unit, at least one block per wave.
    const int64_t cols = (N + 15) / 16;
    int64_t slices = 2 * smlp::kCUs / cols;
    if (slices > (KB + 7) / 8) slices = (KB + 7) / 8;
    if (slices > smlp::kSlices) slices = smlp::kSlices;
    if (slices > 1) {
      p.f.kslice = (int)((KB + slices - 1) / slices);
      p.f.ksplit = (int)((KB + p.f.kslice - 1) / p.f.kslice);
      part = (size_t)p.f.ksplit * (size_t)cols * 256 * 4;
    }
  } else if (M <= 32) {
    p.f = stream_plan(M, KB);
  } else {
    const int64_t t256 = ((M + 255) / 256) * ((N + 255) / 256), t128 = blocks128(M) * blocks128(N);
    // fp32 results go through the bf16 instructions, since the 8-bit ones are 1.5e-5 off (8192 x
    // 7168 x 6144 706 us against 325 us for a bf16 result), and so do short K, where the time is
    // in the stores.
    const int exact = out_fp32 || KB <= 4;
    const int b = t256 >= 256 ? 256 : t128 >= 256 ? 128 : 64;
    p.f = tile_plan(b, b, KB, exact);
    const int64_t tiles = ((M + b - 1) / b) * ((N + b - 1) / b);
    if (b == 64 && tiles <= kSplitTiles) {
      // Not even one tile for every second compute unit: K over workgroups too, at least
      // eight blocks each.  A K step takes 0.33 us and the join of the slices' sums 2.2 us, so
      // short slices gain little (e4m3 x, bf16 y; without and with the split: 333 x 1000 x 2000
      // 9.9 and 9.4 us, 64 x 7168 x 7168 22.9 and 16.1 us, 64 x 2112 x 7168 22.7 and 12.2 us).
      int64_t slices = 2 * smlp::kCUs / tiles;
      if (slices > KB / 8) slices = KB / 8;
      if (slices > smlp::kSlices) slices = smlp::kSlices;
      if (slices > 1) {
        p.f.kslice = (int)((KB + slices - 1) / slices);
        p.f.ksplit = (int)((KB + p.f.kslice - 1) / p.f.kslice);
        part = (size_t)p.f.ksplit * (size_t)tiles * 64 * 64 * 4;
      }
    }
  }
  size_t off = 0;
  p.x8_off = off;
  if (!x_fp8) off += round_up((size_t)(M * K));
  p.xs_off = off;
  if (!x_fp8) off += round_up((size_t)(M * KB) * 4);
  p.part_off = off;
  off += round_up(part);
  p.workspace_bytes = off;
  *out = p;
  return SMLP_OK;
}

int make_experts_plan(int64_t T, int64_t H, int64_t I, int64_t E, int64_t topk, int partial_fp32,
                      smlp::ExpertsPlan* out) {
  if (T < 0) return fail(SMLP_ERR_SHAPE, "T = %lld < 0", (long long)T);
  if (H < 16 || H % 16 || I < 16 || I % 16)
    return fail(SMLP_ERR_SHAPE, "H = %lld and I = %lld must be positive multiples of 16", (long long)H, (long long)I);
  if (E < 1 || E > SMLP_MAX_EXPERTS)
    return fail(SMLP_ERR_ARG, "E = %lld outside [1, %d]", (long long)E, SMLP_MAX_EXPERTS);
  if (topk < 1 || topk > SMLP_MAX_TOPK)
    return fail(SMLP_ERR_ARG, "topk = %lld outside [1, %d]", (long long)topk, SMLP_MAX_TOPK);
  if (!fits(T, H) || !fits(T, topk) || !fits(T * topk, I) || !fits(2 * I, H))
    return fail(SMLP_ERR_SHAPE, "T*H, T*topk, T*topk*I and 2*I*H must be below 2^31");
  smlp::ExpertsPlan p{};
  p.T = T;
  p.H = H;
  p.I = I;
  p.E = E;
  p.topk = topk;
  p.P = T * topk;
  const int64_t HB = blocks128(H), IB = blocks128(I);
  // Rows per expert as if every pair were of an expert held here: a rank of an expert-parallel
  // group plans for more rows than it has.
  const int64_t active = p.P < E ? p.P : E;
  const int64_t rows = active ? p.P / active : 0;
  // Streaming against tiles of 64 rows, the same experts: 8 rows per expert 198 and 235 us, 16
  // rows 265 and 241 us.
  if (rows <= 12) {
    p.gu = stream_plan(rows * 2, HB);
    p.dn = stream_plan(rows * 2, IB);
    if (IB * p.dn.bm <= 256 && IB <= 16) {
      // The whole K of a tile's activations fits LDS: about four workgroups per compute unit
      // over the (tile, run of weight tiles) pairs, at least four weight tiles each.
      p.dn.kind = smlp::F8_KIND_DOWN;
      const int64_t ht = (H + 15) / 16, tiles = active ? p.P / p.dn.bm + active : 1;
      const int64_t runs = (4 * smlp::kCUs + tiles - 1) / tiles, run = (ht + runs - 1) / runs;
      p.dn.run = (int)(run < 4 ? 4 : run > smlp::kDownRun ? smlp::kDownRun : (run + 3) / 4 * 4);
    }
  } else {
    // 8 of 64 experts of 768, H = 7168: 96 rows per expert take 369 us on tiles of 256 rows and
    // 376 us on tiles of 64, 128 rows 390 and 416 us, 64 rows 343 and 303 us.
    const int bm = rows >= 112 ? 256 : 64;
    p.gu = tile_plan(bm, 256, HB, partial_fp32 != 0);
    p.dn = tile_plan(bm, 256, IB, partial_fp32 != 0);
  }
  p.token = T == 1 && HB <= smlp::kTokenBlocks && topk * IB <= smlp::kTokenPairBlocks;
  const bool stream = p.gu.kind == smlp::F8_KIND_STREAM;
  // fp32 rows of y as long as they stay in the caches (301 tokens of 4 pairs of 2000: weighted
  // sum 4.0 us against 5.7 us from fp16 rows).
  p.y_f32 = stream || partial_fp32 || p.P * H <= (4 << 20);
  // fp16 rows are stored through a buffer per tile; rows too long for that stay fp32.
  if (!p.y_f32 && !smlp::rows_fit_buffer(p.P < p.dn.bm ? p.P : p.dn.bm, H, H)) p.y_f32 = 1;
  // An expert with c rows needs ceil(c / bm) tiles.
  p.max_tiles = p.P / p.gu.bm + active;
  size_t off = 0;
  auto take = [&](size_t n) {
    const size_t at = off;
    off += round_up(n);
    return at;
  };
  p.hdr_off = take((size_t)(4 + 4 * p.max_tiles) * 4);
  p.perm_off = take((size_t)p.P * 4);
  if (p.P > smlp::kOneSort) {
    const int64_t least = (p.P + smlp::kSortChunks - 1) / smlp::kSortChunks;
    p.chunk = (int)(least < 2048 ? 2048 : (least + 1023) / 1024 * 1024);
  }
  p.counts_off = take(p.chunk ? (size_t)smlp::kSortChunks * (size_t)E * 4 : 0);
  p.place_off = take((size_t)p.P * 4);
  p.yexp_off = take(p.y_f32 ? 0 : (size_t)p.P * (size_t)((H + 63) / 64));
  p.x8_off = take((size_t)(T * H));
  p.xs_off = take((size_t)(T * HB) * 4);
  p.h8_off = take((size_t)(p.P * I));
  p.hs_off = take((size_t)(p.P * IB) * 4);
  // fp32 h: the streaming gate_up, and the two launches of one token whatever p.gu says (many
  // choices among few experts make p.gu tiled).
  p.h32_off = take(stream || p.token ? (size_t)(p.P * I) * 4 : 0);
  p.y_off = take((size_t)p.P * (size_t)H * (p.y_f32 ? 4 : 2));
  p.workspace_bytes = off;
  *out = p;
  return SMLP_OK;
}

}  // namespace

extern "C" {

int shared_mlp_route(const void* logits, int dtype, int64_t T, int64_t E, int64_t ldl, const float* bias,
                     const smlp_route* route, int32_t* ids, float* weights, hipStream_t stream) {
  if (dtype != SMLP_BF16 && dtype != SMLP_FP32) return fail(SMLP_ERR_DTYPE, "logits dtype %d", dtype);
  if (!route) return fail(SMLP_ERR_NULL, "route is NULL");
  const smlp_route r = *route;
  if (r.score != SMLP_SCORE_SIGMOID && r.score != SMLP_SCORE_SOFTMAX)
    return fail(SMLP_ERR_ARG, "score = %d", r.score);
  if (T < 0) return fail(SMLP_ERR_SHAPE, "T = %lld < 0", (long long)T);
  if (E < 1 || E > SMLP_MAX_EXPERTS)
    return fail(SMLP_ERR_ARG, "E = %lld outside [1, %d]", (long long)E, SMLP_MAX_EXPERTS);
  if (r.groups < 1 || r.groups > SMLP_MAX_GROUPS || E % r.groups)
    return fail(SMLP_ERR_ARG, "groups = %d outside [1, %d] or no divisor of E = %lld", r.groups, SMLP_MAX_GROUPS,
                (long long)E);
  const int64_t per = E / r.groups;
  if (r.top_groups < 1 || r.top_groups > r.groups)
    return fail(SMLP_ERR_ARG, "top_groups = %d outside [1, %d]", r.top_groups, r.groups);
  if ((r.group_top != 1 && r.group_top != 2) || (r.groups > 1 && r.group_top > per))
    return fail(SMLP_ERR_ARG, "group_top = %d with %lld experts per group", r.group_top, (long long)per);
  if (r.groups > 1 && r.group_top == 2 && r.score == SMLP_SCORE_SOFTMAX && !bias)
    return fail(SMLP_ERR_ARG, "softmax without a bias is chosen by logits: a group's score is its largest one");
  if (r.topk < 1 || r.topk > SMLP_MAX_TOPK || r.topk > r.top_groups * per)
    return fail(SMLP_ERR_ARG, "topk = %d outside [1, %d] or above the %lld eligible experts", r.topk, SMLP_MAX_TOPK,
                (long long)(r.top_groups * per));
  if (ldl < E) return fail(SMLP_ERR_SHAPE, "ldl = %lld < E", (long long)ldl);
  if (!fits(T, ldl) || !fits(T, r.topk)) return fail(SMLP_ERR_SHAPE, "T * max(ldl, topk) must be below 2^31");
  if (T == 0) return ok();
  const size_t eb = dtype == SMLP_BF16 ? 2 : 4;
  int rc;
  if ((rc = check_ptr(logits, "logits", eb)) || (rc = check_ptr(ids, "ids", 4)) ||
      (rc = check_ptr(weights, "weights", 4)))
    return rc;
  if ((uintptr_t)bias % 4) return fail(SMLP_ERR_ALIGN, "bias is not 4-byte aligned");
  const size_t n = (size_t)(T * r.topk) * 4;
  const Range in[2] = {{logits, ((size_t)(T - 1) * ldl + E) * eb}, {bias, (size_t)E * 4}};
  if (overlap({ids, n}, {weights, n})) return fail(SMLP_ERR_ALIAS, "ids and weights overlap");
  for (const Range& q : in)
    if (overlap({ids, n}, q) || overlap({weights, n}, q))
      return fail(SMLP_ERR_ALIAS, "ids or weights overlap an input");
  (void)hipGetLastError();
  if ((rc = hip_status(smlp::launch_route(logits, dtype == SMLP_BF16, T, E, ldl, bias, r, ids, weights, stream),
                       "routing launch")))
    return rc;
  return ok();
}

int shared_mlp_quant_fp8(const void* x, int dtype, int64_t parts, int64_t rows, int64_t cols, int64_t ldx,
                         int block_rows, void* q, float* scales, hipStream_t stream) {
  if (dtype != SMLP_BF16 && dtype != SMLP_FP32) return fail(SMLP_ERR_DTYPE, "x dtype %d", dtype);
  const int64_t eb = dtype == SMLP_BF16 ? 2 : 4;
  if (block_rows != 1 && block_rows != 128) return fail(SMLP_ERR_ARG, "block_rows = %d is neither 1 nor 128", block_rows);
  if (parts < 0 || rows < 1 || parts >= kLimit || rows >= kLimit)
    return fail(SMLP_ERR_SHAPE, "parts = %lld, rows = %lld", (long long)parts, (long long)rows);
  if (cols < 16 || cols % 16 || cols >= kLimit)
    return fail(SMLP_ERR_SHAPE, "cols = %lld is not a positive multiple of 16", (long long)cols);
  if (ldx < cols || ldx >= kLimit || ldx * eb % 16)
    return fail(SMLP_ERR_SHAPE, "ldx = %lld is below cols or no multiple of 16 bytes", (long long)ldx);
  if (parts == 0) return ok();
  const int64_t most = (int64_t)1 << 40;
  if (parts > most / rows || parts * rows > most / ldx)
    return fail(SMLP_ERR_SHAPE, "parts * rows * ldx must be at most 2^40");
  const int64_t nblk = (block_rows == 1 ? parts * rows : parts * blocks128(rows)) * blocks128(cols);
  if (block_rows != 1 && nblk >= kLimit) return fail(SMLP_ERR_SHAPE, "2^31 or more blocks");
  int rc;
  if ((rc = check_ptr(x, "x", 16)) || (rc = check_ptr(q, "q", 16)) || (rc = check_ptr(scales, "scales", 4))) return rc;
  const Range xr{x, (size_t)((parts * rows - 1) * ldx + cols) * eb}, qr{q, (size_t)(parts * rows) * cols},
      sr{scales, (size_t)nblk * 4};
  if (overlap(qr, xr) || overlap(sr, xr) || overlap(qr, sr)) return fail(SMLP_ERR_ALIAS, "q, scales and x overlap");
  (void)hipGetLastError();
  if ((rc = hip_status(smlp::launch_quant_fp8(x, dtype == SMLP_BF16, parts, rows, cols, ldx, block_rows, q, scales,
                                              blocks128(cols), 1, stream),
                       "quantisation launch")))
    return rc;
  return ok();
}

int shared_mlp_linear_fp8_workspace_bytes(int64_t M, int64_t K, int64_t N, int x_fp8, size_t* bytes) {
  if (!bytes) return fail(SMLP_ERR_NULL, "bytes is NULL");
  LinearF8Plan p;
  const int rc = make_linear_plan(M, K, N, x_fp8 != 0, 0, &p);
  if (rc) return rc;
  *bytes = p.workspace_bytes;
  return ok();
}

int shared_mlp_linear_fp8(const void* x, const float* x_scales, const void* w, const float* w_scales, void* y,
                          int64_t M, int64_t K, int64_t N, int64_t ldy, int out_fp32, void* workspace,
                          size_t workspace_bytes, hipStream_t stream) {
  if (out_fp32 != 0 && out_fp32 != 1) return fail(SMLP_ERR_DTYPE, "out_fp32 = %d is neither 0 nor 1", out_fp32);
  LinearF8Plan p;
  int rc = make_linear_plan(M, K, N, x_scales != nullptr, out_fp32, &p);
  if (rc) return rc;
  if (ldy < N || !fits(M, ldy)) return fail(SMLP_ERR_SHAPE, "ldy = %lld is below N or M * ldy not below 2^31", (long long)ldy);
  if (M == 0) return ok();
  p.f.by_rows = smlp::rows_fit_buffer(M < p.f.bm ? M : p.f.bm, ldy, N);
  const size_t oe = out_fp32 ? 4 : 2;
  if ((rc = check_ptr(x, "x", 16)) || (rc = check_ptr(w, "w", 16)) || (rc = check_ptr(w_scales, "w_scales", 4)) ||
      (rc = check_ptr(y, "y", oe)))
    return rc;
  if ((uintptr_t)x_scales % 4) return fail(SMLP_ERR_ALIGN, "x_scales is not 4-byte aligned");
  if (p.workspace_bytes) {
    if ((rc = check_ptr(workspace, "workspace", 256))) return rc;
    if (workspace_bytes < p.workspace_bytes)
      return fail(SMLP_ERR_WORKSPACE, "workspace_bytes = %zu < %zu needed", workspace_bytes, p.workspace_bytes);
  }
  const int64_t KB = blocks128(K);
  const Range yr{y, ((size_t)(M - 1) * ldy + N) * oe}, wsr{workspace, p.workspace_bytes};
  const Range in[4] = {{x, (size_t)(M * K) * (x_scales ? 1 : 2)},
                       {x_scales, (size_t)(M * KB) * 4},
                       {w, (size_t)(N * K)},
                       {w_scales, (size_t)(blocks128(N) * KB) * 4}};
  for (const Range& q : in)
    if (overlap(yr, q) || overlap(wsr, q)) return fail(SMLP_ERR_ALIAS, "y or the workspace overlaps an input");
  if (overlap(yr, wsr)) return fail(SMLP_ERR_ALIAS, "y overlaps the workspace");
  (void)hipGetLastError();
  if (p.f.kind == smlp::F8_KIND_ROW) {
    rc = smlp::launch_row_fp8(x, x_scales, w, w_scales, y, K, N, out_fp32, stream);
    if ((rc = hip_status(rc, "8-bit product launch"))) return rc;
    return ok();
  }
  if (p.f.kind == smlp::F8_KIND_NARROW) {
    rc = smlp::launch_narrow_fp8(p.f, x, w, w_scales, y, M, K, N, ldy, out_fp32,
                                 reinterpret_cast<float*>(static_cast<char*>(workspace) + p.part_off), stream);
    if ((rc = hip_status(rc, "8-bit product launch"))) return rc;
    return ok();
  }
  char* base = static_cast<char*>(workspace);
  const void* x8 = x;
  const float* xs = x_scales;
  int64_t s_row = KB, s_kb = 1;
  if (!x_scales) {
    x8 = base + p.x8_off;
    xs = reinterpret_cast<const float*>(base + p.xs_off);
    s_row = 1;
    s_kb = M;
    rc = smlp::launch_quant_fp8(x, 1, 1, M, K, K, 1, base + p.x8_off, reinterpret_cast<float*>(base + p.xs_off), s_row,
                                s_kb, stream);
    if ((rc = hip_status(rc, "quantisation launch"))) return rc;
  }
  rc = smlp::launch_linear_fp8(p.f, x8, xs, s_row, s_kb, w, w_scales, y, M, K, N, ldy, out_fp32,
                               reinterpret_cast<float*>(base + p.part_off), stream);
  if ((rc = hip_status(rc, "8-bit product launch"))) return rc;
  return ok();
}

int shared_mlp_experts_fp8_workspace_bytes(int64_t T, int64_t H, int64_t I, int64_t E, int64_t topk,
                                           int partial_fp32, size_t* bytes) {
  if (!bytes) return fail(SMLP_ERR_NULL, "bytes is NULL");
  smlp::ExpertsPlan p;
  const int rc = make_experts_plan(T, H, I, E, topk, partial_fp32 != 0, &p);
  if (rc) return rc;
  *bytes = p.workspace_bytes;
  return ok();
}

int shared_mlp_experts_fp8(const void* x, const int32_t* ids, const float* weights, const void* w_gate_up,
                           const float* s_gate_up, const void* w_down, const float* s_down, void* out, int64_t T,
                           int64_t H, int64_t I, int64_t E, int64_t topk, int64_t first_expert, int partial_fp32,
                           void* workspace, size_t workspace_bytes, hipStream_t stream) {
  smlp::ExpertsPlan p;
  int rc = make_experts_plan(T, H, I, E, topk, partial_fp32 != 0, &p);
  if (rc) return rc;
  if (first_expert < 0 || first_expert >= kLimit)
    return fail(SMLP_ERR_ARG, "first_expert = %lld", (long long)first_expert);
  if (T == 0) return ok();
  if ((rc = check_ptr(x, "x", 16)) || (rc = check_ptr(ids, "ids", 4)) || (rc = check_ptr(weights, "weights", 4)) ||
      (rc = check_ptr(w_gate_up, "w_gate_up", 16)) || (rc = check_ptr(s_gate_up, "s_gate_up", 4)) ||
      (rc = check_ptr(w_down, "w_down", 16)) || (rc = check_ptr(s_down, "s_down", 4)) ||
      (rc = check_ptr(out, "out", 16)) || (rc = check_ptr(workspace, "workspace", 256)))
    return rc;
  if (workspace_bytes < p.workspace_bytes)
    return fail(SMLP_ERR_WORKSPACE, "workspace_bytes = %zu < %zu needed", workspace_bytes, p.workspace_bytes);
  const int64_t HB = blocks128(H), IB = blocks128(I);
  const Range o{out, (size_t)(T * H) * (partial_fp32 ? 4 : 2)}, wsr{workspace, p.workspace_bytes};
  const Range in[7] = {{x, (size_t)(T * H) * 2},
                       {ids, (size_t)p.P * 4},
                       {weights, (size_t)p.P * 4},
                       {w_gate_up, (size_t)E * (size_t)(2 * I * H)},
                       {s_gate_up, (size_t)(E * 2 * IB * HB) * 4},
                       {w_down, (size_t)E * (size_t)(H * I)},
                       {s_down, (size_t)(E * HB * IB) * 4}};
  for (const Range& q : in)
    if (overlap(o, q) || overlap(wsr, q)) return fail(SMLP_ERR_ALIAS, "out or the workspace overlaps an input");
  if (overlap(o, wsr)) return fail(SMLP_ERR_ALIAS, "out overlaps the workspace");
  (void)hipGetLastError();
  const smlp::ExpertsCall c{x,      ids,    weights, w_gate_up, s_gate_up,
                            w_down, s_down, out,     first_expert, partial_fp32 != 0};
  if ((rc = hip_status(smlp::launch_experts_fp8(p, c, workspace, stream), "experts launch"))) return rc;
  return ok();
}

}  // extern "C"
