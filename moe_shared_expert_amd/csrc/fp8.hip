// 8-bit (e4m3) block-scaled products: the plain projection and the two products of the
// routed experts, and the kernels around them (quantisation, the sort of token-expert
// pairs, the weighted sum of a token's experts).
//
// y[m, n] = sum_b as[m, b] ws[n / 128, b] sum_{k in block b} a[m, k] w[n, k]
//
// b runs over blocks of 128 K elements.  One 16x16x128 matrix instruction multiplies
// exactly one block of a 16 x 16 output tile, starting from zero; its four results per lane
// are then added into fp32 accumulators with one multiply-add each, scaled by as * ws.  The
// weights are the instruction's A operand, so a lane holds one token's results (one
// activation scale per lane and tile) for four consecutive output features (one 8- or
// 16-byte store), and the weight scale is the same for the whole wave.
//
// Operands reach LDS by direct loads in 1 KB blocks of 8 rows x 128 bytes, the 16-byte
// chunks of a row permuted so that the fragment reads are free of bank conflicts.  The
// scales of a K block travel the same way, as one 4-byte-per-lane load beside the data.
//
// The streaming kernel, every product that is returned in fp32 and projections of at most four
// blocks go through the bf16 instructions (exact products, fp32 sums); the tiled kernel with
// bf16 results uses the 8-bit instruction at twice the rate, whose sums are about 1.5e-5 off.
// In a projection that is far below the rounding of the result.  In gate_up it moves about one
// value of h in 5000 to the neighbouring e4m3 value: the experts' output is then 2.0e-3 to
// 2.3e-3 off the definition (2-norm), of which its rounding to bf16 is 1.7e-3.  The exact form
// costs what it is worth to few: 8192 tokens of 8 pairs 2.98 ms (fp32 result) against 1.52 ms,
// 301 tokens of an expert-parallel rank 43 against 35 us.
#include "fp8.h"
#include "internal.h"
#include "smlp.h"

namespace smlp {

namespace {

enum { F8_LINEAR = 0, F8_GATE_UP = 1, F8_DOWN = 2 };
constexpr int kGuarded = 2;  // F8Args::out_f32

struct F8Args {
  const uint8_t* a;    // activations [rows, K]
  uint32_t a_bytes;
  const float* as;     // scale of activation row r, block b: as[r * as_row + b * as_kb]
  int as_row, as_kb;
  const uint8_t* w;    // weights of expert e at w + e * w_stride, rows of K bytes
  size_t w_stride;
  uint32_t w_bytes;    // bytes of one expert's weights
  const float* ws;     // block scales of expert e at ws + e * ws_stride, rows of KB
  size_t ws_stride;
  int K, KB;           // K elements and blocks of 128
  int N;               // features (gate_up: of h)
  int nblk;            // 128-row blocks of N
  int M;               // projection: rows of a
  int tiles_m, tiles_n;
  const int* hdr;      // experts: tile list (SortHeader layout below)
  const int* perm;     // experts: pair at each sorted position
  int topk;
  void* out;           // projection: y; gate_up: h; down: y (rows: sorted positions)
  int ldo;
  int out_f32;         // fp32 (1) or bf16 (0) output; gate_up: fp32 h (1) or e4m3 h (0); down:
                       // fp32 y (1) or fp16 y with exponents (0); tiled projection: kGuarded for
                       // bf16 rows that do not fit a buffer
  float* hs;           // gate_up with e4m3 h: scales, block b of position p at hs[b * hs_ld + p]
  int hs_ld;
  uint8_t* yexp;       // down with fp16 y: exponent of position p and columns 64 c .. + 63 at
                       // yexp[c * hs_ld + p]
  float* part;         // projection with a K split: fp32 partials, and one arrival counter per
  uint32_t* arrived;   // tile, 16 words apart, zero between launches
  int kslice;          // K blocks per slice
};

// Index of expert `id` among the E held from `first` on, or -1.
__device__ __forceinline__ int local_expert(int id, int first, int E) {
  return id >= first && id - first < E ? id - first : -1;
}

// Tile list of the experts' products: hdr[0] = tiles, then (expert, first sorted position,
// rows) of each.
__device__ __forceinline__ bool f8_tile(const F8Args& g, int mode, int bm, int tile, int& expert, int& start,
                                        int& count) {
  if (mode == F8_LINEAR) {
    expert = 0;
    start = tile * bm;
    count = min(bm, g.M - start);
    return true;
  }
  if (tile >= g.hdr[0]) return false;
  expert = g.hdr[4 + tile * 4];
  start = g.hdr[5 + tile * 4];
  count = g.hdr[6 + tile * 4];
  return true;
}

// Activation row of row r of a tile.
__device__ __forceinline__ int f8_arow(const F8Args& g, int mode, int start, int r) {
  if (mode == F8_GATE_UP) return g.perm[start + r] / g.topk;
  return start + r;
}

// Byte offsets that make a buffer load return zeros: kNoRow in place of a row's offset,
// kNoChunk added to one.  Operands hold at most 2^31 - 16 bytes, so a real offset plus
// kNoChunk, and kNoRow plus any, is out of range, and nothing wraps.  kNoRow also drops a
// store: results that are stored through a buffer are held to the same size (the planner's
// rows_fit_buffer; h of a tile is less than 2^31 bytes because h of all pairs is).
constexpr uint32_t kNoRow = 0x80000000u, kNoChunk = 0x7ffffff0u;

__device__ __forceinline__ void f8_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
}

// Store four consecutive features n .. n+3 of one output row.
__device__ __forceinline__ void f8_store4(const F8Args& g, size_t row, int n, f32x4 v) {
  const size_t at = row * (size_t)g.ldo + n;
  if (g.out_f32 & 1) {
    float* p = reinterpret_cast<float*>(g.out) + at;
    if (n + 3 < g.N && ((uintptr_t)p & 15) == 0) {
      *reinterpret_cast<f32x4*>(p) = v;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (n + j < g.N) p[j] = v[j];
    }
  } else {
    uint16_t* p = reinterpret_cast<uint16_t*>(g.out) + at;
    if (n + 3 < g.N && ((uintptr_t)p & 7) == 0) {
      *reinterpret_cast<u32x2*>(p) = u32x2{pack_bf2(v[0], v[1]), pack_bf2(v[2], v[3])};
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (n + j < g.N) p[j] = (uint16_t)f2bf(v[j]);
    }
  }
}

// Eight elements at p (16-byte aligned).
__device__ __forceinline__ void load8(const void* x, size_t at, int bf16, float (&v)[8]) {
  if (bf16) {
    const u32x4 u = ld16(reinterpret_cast<const uint16_t*>(x) + at);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf_lo(u[i]);
      v[2 * i + 1] = bf_hi(u[i]);
    }
  } else {
    const float* p = reinterpret_cast<const float*>(x) + at;
    const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = a[i];
      v[4 + i] = b[i];
    }
  }
}

// Activation tiles of the streaming kernels come in AH blocks of 8 rows.  One block serves
// up to 8 rows (lanes 8-15 of a fragment read it again): a product's column depends on its
// own activation row only, so columns without a row may hold anything and are not stored.
__device__ __forceinline__ i32x8 act_frag(const char* tile, int row, int lg) {
  const int sw = (row >> 1) & 7;
  const u32x4 lo = *reinterpret_cast<const u32x4*>(tile + row * 128 + ((lg ^ sw) * 16));
  const u32x4 hi = *reinterpret_cast<const u32x4*>(tile + row * 128 + (((lg + 4) ^ sw) * 16));
  i32x8 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = (int)lo[i];
    v[4 + i] = (int)hi[i];
  }
  return v;
}

// Weight streaming (few rows per tile), bound by HBM: the gate_up of 32 tokens of 8 pairs over
// 128 experts (H = 7168, I = 768) reads its 105 active experts' 1.16 GB in 164 us, 7.0 TB/s.
// Tiles of 8 rows instead of 16 and three ring stages instead of four let a second workgroup
// live on a compute unit (180 -> 164 us).  A workgroup owns NT tiles of 16 weight rows
// (gate_up: NT / 2 tiles of gate rows and the matching up rows) and one tile of 8 * AH
// activation rows; its waves take the K blocks in turn, each through a ring of its own, and
// their sums are added in wave order.
template <int NT, int AH, int WAVES, int STAGES, int MODE>
__global__ __launch_bounds__(WAVES * 64) void f8_stream_kernel(F8Args g) {
  constexpr bool GU = MODE == F8_GATE_UP;
  constexpr int FT = GU ? NT / 2 : NT;  // feature tiles
  constexpr int AR = 8 * AH, MT = (AH + 1) / 2;
  constexpr int SLOT = NT * 2048 + AH * 1024 + 256;
  constexpr int LPS = 2 * NT + AH + 1;
  constexpr int RING = WAVES * STAGES * SLOT;
  constexpr int RED = WAVES * NT * MT * 64 * 16;
  static_assert(LPS * (STAGES - 1) < 64 && AR <= 32, "loads in flight");
  __shared__ __attribute__((aligned(1024))) char lds[RING > RED ? RING : RED];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ln = lane & 15, lg = lane >> 4, lr = lane >> 3;
  int expert, start, count;
  if (!f8_tile(g, MODE, AR, blockIdx.y, expert, start, count)) return;
  const int f0 = blockIdx.x * (16 * FT);
  const int K = g.K;
  const uint8_t* w = g.w + (size_t)expert * g.w_stride;
  const float* ws = g.ws + (size_t)expert * g.ws_stride;
  const __amdgpu_buffer_rsrc_t wr = make_rsrc(w, g.w_bytes);
  const __amdgpu_buffer_rsrc_t ar = make_rsrc(g.a, g.a_bytes);

  int ch[2];
  uint32_t wo[NT][2], ao[AH];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    ch[h] = (lane & 7) ^ (((8 * h + lr) >> 1) & 7);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int f = f0 + 16 * (t % FT) + 8 * h + lr;
      const int row = t < FT ? f : g.N + f;
      wo[t][h] = f < g.N ? (uint32_t)row * (uint32_t)K + ch[h] * 16 : kNoRow;
    }
  }
#pragma unroll
  for (int h = 0; h < AH; ++h) {
    const int r = 8 * h + lr;
    ao[h] = r < count ? (uint32_t)f8_arow(g, MODE, start, r) * (uint32_t)K + ch[h & 1] * 16 : kNoRow;
  }
  // Scale source of this lane: lanes 0 .. AR - 1 the activation rows, lanes 32 and up the
  // weight blocks (even lanes the gate or only one, odd lanes the up block).
  const float* sp;
  int sstep;
  if (lane < 32) {
    sp = g.as + (size_t)f8_arow(g, MODE, start, min(lane & (AR - 1), count - 1)) * g.as_row;
    sstep = g.as_kb;
  } else {
    const int blk = min(f0 / 128, g.nblk - 1) + (GU && (lane & 1) ? g.nblk : 0);
    sp = ws + (size_t)blk * g.KB;
    sstep = 1;
  }

  char* my = lds + wave * (STAGES * SLOT);
  const int nst = (g.KB + WAVES - 1) / WAVES;
  auto issue = [&](int slot, int i) {
    const int kb = i * WAVES + wave;
    const int k = kb * 128;
    char* sl = my + slot * SLOT;
    const uint32_t ko[2] = {k + ch[0] * 16 < K ? (uint32_t)k : kNoChunk, k + ch[1] * 16 < K ? (uint32_t)k : kNoChunk};
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int h = 0; h < 2; ++h) buf_ld_lds_nt(wr, sl + t * 2048 + h * 1024, wo[t][h] + ko[h]);
#pragma unroll
    for (int h = 0; h < AH; ++h) buf_ld_lds(ar, sl + NT * 2048 + h * 1024, ao[h] + ko[h & 1]);
    glb_ld_lds4(sp + (size_t)min(kb, g.KB - 1) * sstep, sl + NT * 2048 + AH * 1024);
  };

  f32x4 acc[NT][MT];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[t][m] = f32x4{0.f, 0.f, 0.f, 0.f};

#pragma unroll
  for (int st = 0; st < STAGES - 1; ++st) issue(st, st);
  for (int i = 0; i < nst; ++i) {
    // The fragments of the slot about to be refilled were all read (and waited for) in the
    // previous step.  Steps past K arrive as zeros without memory traffic.
    issue((i + STAGES - 1) % STAGES, i + STAGES - 1);
    wait_vmcnt<(STAGES - 1) * LPS>();
    asm volatile("" ::: "memory");
    const char* sl = my + (i % STAGES) * SLOT;
    const float* sc = reinterpret_cast<const float*>(sl + NT * 2048 + AH * 1024);
    frag_bf16 af[MT];
    float sg[MT], su[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int row = (16 * m + ln) & (AR - 1);
      af[m] = widen(act_frag(sl + NT * 2048, row, lg));
      const float s = sc[row];
      sg[m] = s * sc[32];
      su[m] = GU ? s * sc[33] : sg[m];
    }
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const frag_bf16 wf = widen(lds_frag(sl + t * 2048, lane));
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const f32x4 p = mfma_widened(wf, af[m]);
        const float s = t < FT ? sg[m] : su[m];
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[t][m][j] = fmaf(p[j], s, acc[t][m][j]);
      }
    }
    __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): this slot's reads are done
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
  }
  wait_vmcnt<0>();

  // Add the waves' sums in wave order; wave 0 finishes.
  if constexpr (WAVES > 1) {
    f32x4* red = reinterpret_cast<f32x4*>(lds);
    __syncthreads();
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int m = 0; m < MT; ++m) red[(wave * NT * MT + t * MT + m) * 64 + lane] = acc[t][m];
    __syncthreads();
    if (wave != 0) return;
    for (int v = 1; v < WAVES; ++v)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[t][m] += red[(v * NT * MT + t * MT + m) * 64 + lane];
  }
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int r = 16 * m + ln;
    if (r >= count) continue;
#pragma unroll
    for (int t = 0; t < FT; ++t) {
      const int n = f0 + 16 * t + 4 * lg;
      if (n >= g.N) continue;
      f32x4 v = acc[t][m];
      if constexpr (GU) {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = silu_then_mul(v[j], acc[t + FT][m][j]);
      }
      f8_store4(g, (size_t)(start + r), n, v);
    }
  }
}

// Most 128-row blocks that a run of the short-K down kernel touches.
constexpr int kDownBlocks = kDownRun / 8 + 2;

// Down product of few rows per expert and a short K (KB <= KBMAX blocks), bound by HBM: the
// same experts' 0.58 GB in 97 us, 6.0 TB/s; with K split over the waves as above, six blocks
// left each wave one or two steps and the time was in starting and ending workgroups (221 us).
// A workgroup holds
// its tile's activations (h in fp32, brought to the 8-bit form here) in LDS and streams a run
// of `run` 16-row weight tiles; its waves take the tiles in turn, each wave with the whole K
// and a ring of D blocks of 16 rows x 128 bytes that runs on from tile to tile.
template <int AH, int KBMAX, int D>
__global__ __launch_bounds__(256) void f8_down_kernel(F8Args g, const float* h, int run) {
  constexpr int WAVES = 4, AR = 8 * AH, MT = (AH + 1) / 2;
  constexpr int RING = WAVES * D * 2048, ACT = KBMAX * AR * 128;
  __shared__ __attribute__((aligned(1024))) char lds[RING + ACT + KBMAX * (AR + kDownBlocks) * 4];
  char* act = lds + RING;
  float* sx = reinterpret_cast<float*>(lds + RING + ACT);
  float* sw = sx + KBMAX * AR;  // this run's weight scales, from the block of its first row on

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ln = lane & 15, lg = lane >> 4, lr = lane >> 3;
  int expert, start, count;
  if (!f8_tile(g, F8_DOWN, AR, blockIdx.y, expert, start, count)) return;
  const int K = g.K, KB = g.KB;
  const int tiles = min(run, (g.N + 15) / 16 - (int)blockIdx.x * run);
  const int n0 = blockIdx.x * run * 16;
  const __amdgpu_buffer_rsrc_t wr = make_rsrc(g.w + (size_t)expert * g.w_stride, g.w_bytes);
  const float* ws = g.ws + (size_t)expert * g.ws_stride;

  const int mine = tiles > wave ? (tiles - wave + WAVES - 1) / WAVES : 0;
  char* my = lds + wave * (D * 2048);
  int ch[2];
  uint32_t wo[2];  // this lane's two row offsets in the tile being issued
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    ch[q] = (lane & 7) ^ (((8 * q + lr) >> 1) & 7);
    wo[q] = (uint32_t)(n0 + wave * 16 + 8 * q + lr) * (uint32_t)K + ch[q] * 16;
  }
  int ikb = 0, itile = 0;  // next block to issue
  auto issue = [&](int slot) __attribute__((always_inline)) {
    const int k = ikb * 128;
#pragma unroll
    for (int q = 0; q < 2; ++q)
      buf_ld_lds_nt(wr, my + slot * 2048 + q * 1024,
                    itile < mine && k + ch[q] * 16 < K ? wo[q] + (uint32_t)k : kNoRow);
    if (++ikb == KB) {
      ikb = 0;
      ++itile;
      wo[0] += (uint32_t)(WAVES * 16) * (uint32_t)K;
      wo[1] += (uint32_t)(WAVES * 16) * (uint32_t)K;
    }
  };
  // h rows -> e4m3 in LDS, 16 lanes per row and group of 128.  Loads complete in order, so
  // the first HP rounds of h and the weight scales are loaded ahead of the ring's weights; more rounds only come with more than HP * 16 / KB rows.
  constexpr int HP = 3;
  const int l = threadIdx.x & 15;
  float hv[HP][8];
  auto load_h = [&](int q, float (&v)[8]) __attribute__((always_inline)) {
    const int r = q / KB, c = (q - r * KB) * 128 + l * 8;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 0.f;
    if (q < count * KB && c < K) load8(h, (size_t)(start + r) * K + c, 0, v);
  };
#pragma unroll
  for (int i = 0; i < HP; ++i) load_h(i * 16 + (threadIdx.x >> 4), hv[i]);
  const int blk0 = n0 / 128, nb = (min(n0 + tiles * 16, g.N) + 127) / 128 - blk0;
  float swv = 0.f;
  if ((int)threadIdx.x < nb * KB) swv = ws[(size_t)blk0 * KB + threadIdx.x];
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int d = 0; d < D - 1; ++d) issue(d);
  __builtin_amdgcn_sched_barrier(0);
  auto put_h = [&](int q, const float (&v)[8]) __attribute__((always_inline)) {
    const int r = q / KB, b = q - r * KB;
    float mx = kAmaxMin;
#pragma unroll
    for (int i = 0; i < 8; ++i) mx = fmaxf(mx, fabsf(v[i]));
#pragma unroll
    for (int d = 8; d >= 1; d >>= 1) mx = fmaxf(mx, __shfl_xor(mx, d));
    if (q >= count * KB) return;
    const float inv = kE4M3Max * (1.0f / mx);
    *reinterpret_cast<u32x2*>(act + b * (AR * 128) + r * 128 + (((l >> 1) ^ ((r >> 1) & 7)) * 16) + (l & 1) * 8) =
        u32x2{pack_fp8x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
              pack_fp8x4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv)};
    if (l == 0) sx[b * AR + r] = mx / kE4M3Max;
  };
#pragma unroll
  for (int i = 0; i < HP; ++i) put_h(i * 16 + (threadIdx.x >> 4), hv[i]);
  for (int q0 = HP * 16; q0 < count * KB; q0 += 16) {
    float v[8];
    load_h(q0 + (threadIdx.x >> 4), v);
    put_h(q0 + (threadIdx.x >> 4), v);
  }
  if ((int)threadIdx.x < nb * KB) sw[threadIdx.x] = swv;
  for (int q = 256 + threadIdx.x; q < nb * KB; q += 256) sw[q] = ws[(size_t)blk0 * KB + q];
  // LDS writes of every wave done; the ring's loads stay in flight.
  __builtin_amdgcn_s_waitcnt(0xc07f);
  f8_barrier();

  f32x4 acc[MT];
  int slot = 0;
  for (int t = 0; t < mine; ++t) {
    const int n = n0 + (wave + t * WAVES) * 16;
    const float* swr = sw + (n / 128 - blk0) * KB;
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[m] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int kb = 0; kb < KB; ++kb) {
      issue(slot == 0 ? D - 1 : slot - 1);
      wait_vmcnt<2 * (D - 1)>();
      asm volatile("" ::: "memory");
      const frag_bf16 wf = widen(lds_frag(my + slot * 2048, lane));
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int r = (16 * m + ln) & (AR - 1);
        const f32x4 p = mfma_widened(wf, widen(act_frag(act + kb * (AR * 128), r, lg)));
        const float s = sx[kb * AR + r] * swr[kb];
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[m][j] = fmaf(p[j], s, acc[m][j]);
      }
      __builtin_amdgcn_s_waitcnt(0xc07f);  // this slot's reads are done
      __builtin_amdgcn_sched_barrier(0);
      asm volatile("" ::: "memory");
      slot = slot == D - 1 ? 0 : slot + 1;
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
      if (16 * m + ln < count) f8_store4(g, (size_t)(start + 16 * m + ln), n + 4 * lg, acc[m]);
  }
  wait_vmcnt<0>();
}

// Projection of up to 16 bf16 rows in one launch: a lane loads the 32 elements of x that it
// holds of a fragment, finds the group's largest magnitude with the three other lanes of its
// row, and has both its fragment and its scale (of the column it holds results for) in
// registers.  A workgroup owns NT tiles of 16 weight rows; its 8 waves take the K blocks in
// turn, D blocks of loads in flight, and their sums are added in wave order.  The work on x
// (about 200 instructions a block, for every workgroup anew) bounds a workgroup, so with few
// weight rows K is split over workgroups too (gridDim.y); the last one to arrive at a counter
// adds the slices in order (16 x 132 x 7168: 13.4 us on nine workgroups, 6.2 us on 63).
struct NarrowArgs {
  const void* x;   // [M, K] bf16
  const uint8_t* w;
  const float* ws;
  F8Args g;        // M, K, KB, N, nblk, out, ldo, out_f32, w_bytes; kslice, part: K split
  uint32_t* arrived;  // one counter per blockIdx.x, 16 words apart, zero between launches
};

template <int NT, int D>
__global__ __launch_bounds__(512, 2) void f8_narrow_kernel(NarrowArgs a) {
  constexpr int WAVES = 8;
  __shared__ f32x4 red[WAVES][NT][64];
  __shared__ int last;
  const F8Args& g = a.g;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ln = lane & 15, lg = lane >> 4;
  const int K = g.K, n0 = blockIdx.x * (16 * NT);
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(a.x, (uint32_t)g.M * (uint32_t)K * 2u), wr = make_rsrc(a.w, g.w_bytes);
  const uint32_t xo = ln < g.M ? ((uint32_t)ln * (uint32_t)K + lg * 16) * 2u : kNoRow;
  uint32_t wo[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int n = n0 + 16 * t + ln;
    wo[t] = n < g.N ? (uint32_t)n * (uint32_t)K + lg * 16 : kNoRow;
  }
  struct Block {
    u32x4 x[4], w[NT][2];
    float s;
  };
  Block q[D];
  const float* ws = a.ws + (size_t)min(n0 / 128, g.nblk - 1) * g.KB;
  const int kb0 = blockIdx.y * g.kslice, kb1 = min(g.KB, kb0 + g.kslice);
  auto load = [&](Block& b, int i) __attribute__((always_inline)) {
    const int kb = kb0 + i * WAVES + wave, k = kb * 128;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bool in = kb < kb1 && k + 64 * h + lg * 16 < K;
      const uint32_t ko = in ? (uint32_t)(k + 64 * h) : kNoChunk;
      const uint32_t kx = in ? 2u * (uint32_t)(k + 64 * h) : kNoChunk;
      b.x[2 * h] = buf_ld(xr, xo + kx);
      b.x[2 * h + 1] = buf_ld(xr, xo + kx + (in ? 16u : 0u));
#pragma unroll
      for (int t = 0; t < NT; ++t) b.w[t][h] = buf_ld_nt(wr, wo[t] + ko);
    }
    b.s = ws[min(kb, g.KB - 1)];
  };
  f32x4 acc[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto use = [&](const Block& b) __attribute__((always_inline)) {
    float v[32], mx = kAmaxMin;
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[8 * c + 2 * i] = bf_lo(b.x[c][i]);
        v[8 * c + 2 * i + 1] = bf_hi(b.x[c][i]);
      }
#pragma unroll
    for (int i = 0; i < 32; ++i) mx = fmaxf(mx, fabsf(v[i]));
    mx = fmaxf(mx, __shfl_xor(mx, 16));
    mx = fmaxf(mx, __shfl_xor(mx, 32));
    const float inv = kE4M3Max * (1.0f / mx);
    i32x8 af;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      af[i] = (int)pack_fp8x4(v[4 * i] * inv, v[4 * i + 1] * inv, v[4 * i + 2] * inv, v[4 * i + 3] * inv);
    const frag_bf16 fa = widen(af);
    const float s = (mx / kE4M3Max) * b.s;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      i32x8 wf;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        wf[i] = (int)b.w[t][0][i];
        wf[4 + i] = (int)b.w[t][1][i];
      }
      const f32x4 p = mfma_widened(widen(wf), fa);
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[t][j] = fmaf(p[j], s, acc[t][j]);
    }
  };
  const int nst = (kb1 - kb0 + WAVES - 1) / WAVES;  // blocks past the slice are zeros
#pragma unroll
  for (int d = 0; d < D; ++d) load(q[d], d);
  int i0 = 0;
  for (; i0 + D < nst; i0 += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      use(q[d]);
      load(q[d], i0 + D + d);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
#pragma unroll
  for (int d = 0; d < D; ++d)
    if (i0 + d < nst) use(q[d]);
#pragma unroll
  for (int t = 0; t < NT; ++t) red[wave][t][lane] = acc[t];
  __syncthreads();
  f32x4 sum{0.f, 0.f, 0.f, 0.f};
  if (wave < NT) {
    sum = red[0][wave][lane];
#pragma unroll
    for (int v = 1; v < WAVES; ++v) sum += red[v][wave][lane];
  }
  const int slices = gridDim.y;
  if (slices > 1) {
    // Partial sums, agent-coherent: [slice][column of workgroups][tile][lane][4].
    const size_t col = ((size_t)blockIdx.x * NT + wave) * 256 + lane * 4, step = (size_t)gridDim.x * NT * 256;
    if (wave < NT) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        __hip_atomic_store(g.part + blockIdx.y * step + col + j, sum[j], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    wait_vmcnt<0>();
    __syncthreads();
    if (threadIdx.x == 0) {
      uint32_t* c = a.arrived + 16 * blockIdx.x;
      const bool l = __hip_atomic_fetch_add(c, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == (uint32_t)slices - 1;
      if (l) __hip_atomic_store(c, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      last = l;
    }
    __syncthreads();
    if (!last || wave >= NT) return;
    const __amdgpu_buffer_rsrc_t pr = make_rsrc(g.part, (uint32_t)(slices * step * 4));
    f32x4 v[kSlices];
#pragma unroll
    for (int q = 0; q < kSlices; ++q)
      v[q] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(
                 pr, (int)(q < slices ? (uint32_t)((q * step + col) * 4) : kNoRow), 0, 16));
    sum = v[0];
#pragma unroll
    for (int q = 1; q < kSlices; ++q) sum += v[q];  // slices past the last are zeros
  }
  if (wave >= NT) return;
  const int n = n0 + 16 * wave + 4 * lg;
  if (ln < g.M && n < g.N) f8_store4(g, (size_t)ln, n, sum);
}

// ---- one activation row ----
// A single row leaves the matrix instructions with one column in sixteen, so these kernels
// multiply in the vector unit, straight from registers (one token of 8 experts, H = 7168, I =
// 768: gate_up 88 MB in 16.7 us, 5.3 TB/s; down 44 MB in 12.2 us; a projection of 2112 x 7168
// 7.0 us, mostly latency): a 16-byte load per lane covers 8
// weight rows x 128 bytes (8 whole lines), lane l holding 16 K elements of row l / 8, and
// each lane keeps NB such loads in flight: 14 for rows of K (a wave's quarter of K = 7168, the
// hidden size this serves, in one round), 12 for down (two pairs of six blocks).  Other sizes
// take more rounds, the last of them partly of zeros.  The row of x sits in LDS in its 8-bit form.

// Eight values -> e4m3 with the scale of the 16 lanes that share a group.
__device__ __forceinline__ u32x2 quant8(const float (&v)[8], float& scale) {
  float mx = kAmaxMin;
#pragma unroll
  for (int i = 0; i < 8; ++i) mx = fmaxf(mx, fabsf(v[i]));
#pragma unroll
  for (int d = 8; d >= 1; d >>= 1) mx = fmaxf(mx, __shfl_xor(mx, d));
  const float inv = kE4M3Max * (1.0f / mx);
  scale = mx / kE4M3Max;
  return u32x2{pack_fp8x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
               pack_fp8x4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv)};
}

// One row of K bf16 values to e4m3 and scales in LDS, by a workgroup of 256 threads, in two
// halves: the loads, and, once the weights' loads are out too, the rest (loads complete in
// order, so a load issued behind the weights would wait for them).  The tail of the last
// block is filled with zeros.
struct RowLoad {
  u32x4 v[kTokenBlocks / 16];
};
__device__ __forceinline__ void row_load(RowLoad& r, const void* x, int K) {
#pragma unroll
  for (int i = 0; i < kTokenBlocks / 16; ++i) {
    const int c = i * 2048 + (int)threadIdx.x * 8;
    r.v[i] = c < K ? ld16(reinterpret_cast<const uint16_t*>(x) + c) : u32x4{0, 0, 0, 0};
  }
}
__device__ __forceinline__ void row_to_lds(const RowLoad& r, int KB, char* x8, float* sx) {
#pragma unroll
  for (int i = 0; i < kTokenBlocks / 16; ++i) {
    const int b = i * 16 + (threadIdx.x >> 4);
    if (b >= KB) break;
    float v[8], sc;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      v[2 * q] = bf_lo(r.v[i][q]);
      v[2 * q + 1] = bf_hi(r.v[i][q]);
    }
    *reinterpret_cast<u32x2*>(x8 + i * 2048 + threadIdx.x * 8) = quant8(v, sc);
    if ((threadIdx.x & 15) == 0) sx[b] = sc;
  }
}

// Sum of 16 products of e4m3 values (exact in fp32) in fp32.
__device__ __forceinline__ float dot16(u32x4 w, u32x4 x) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  float a = 0.f, b = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const f32x2 w0 = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], false), w1 = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i], true);
    const f32x2 x0 = __builtin_amdgcn_cvt_pk_f32_fp8((int)x[i], false), x1 = __builtin_amdgcn_cvt_pk_f32_fp8((int)x[i], true);
    a = fmaf(w0[0], x0[0], a);
    b = fmaf(w0[1], x0[1], b);
    a = fmaf(w1[0], x1[0], a);
    b = fmaf(w1[1], x1[1], b);
  }
  return a + b;
}

// Sum over the 8 lanes that share a weight row.
__device__ __forceinline__ float row_sum(float v) {
  v += __shfl_xor(v, 1);
  v += __shfl_xor(v, 2);
  return v + __shfl_xor(v, 4);
}

struct TokenArgs {
  const void* x;         // bf16 [H] (projection: bf16, or e4m3 with xs)
  const float* xs;
  const int32_t* ids;    // [topk]
  const float* weights;  // [topk]
  const uint8_t* w;      // gate_up, or down, of expert e at w + e * w_stride
  size_t w_stride;
  uint32_t w_bytes;
  const float* ws;
  size_t ws_stride;
  int H, I, HB, IB, E, first, topk;
  float* h;              // [topk, I] fp32
  void* out;
  int out_f32;
};

// GU: workgroup (b, j) makes features 8 b .. 8 b + 7 of pair j's h from 8 gate rows and 8 up
// rows of H elements.  Otherwise output rows 8 b .. 8 b + 7 of a projection of x [H] (I: the
// number of outputs).  The four waves take the K blocks in turn; their sums are added in
// wave order.
template <bool GU, int NB>
__global__ __launch_bounds__(256, 4) void f8_row_kernel(TokenArgs a) {
  constexpr int WAVES = 4, P = GU ? 2 : 1;
  __shared__ __attribute__((aligned(16))) char x8[kTokenBlocks * 128];
  __shared__ float sx[kTokenBlocks], sw[P][kTokenBlocks], red[WAVES][P][8];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int f0 = blockIdx.x * 8, K = a.H, KB = a.HB;
  int expert = 0;
  if (GU) {
    expert = local_expert(a.ids[blockIdx.y], a.first, a.E);
    if (expert < 0) return;
  }
  const __amdgpu_buffer_rsrc_t wr = make_rsrc(a.w + (size_t)expert * a.w_stride, a.w_bytes);
  const int ch = (lane & 7) * 16;
  const uint32_t wo = (uint32_t)(f0 + (lane >> 3)) * (uint32_t)K + ch;
  const uint32_t up = GU ? (uint32_t)a.I * (uint32_t)K : 0u;
  // Unit u of this wave: block (u / P) * WAVES + wave of the gate (or only) or the up rows.
  const int units = P * ((KB - wave + WAVES - 1) / WAVES);
  u32x4 v[NB];
  auto load = [&](int u) {
    const int k = ((u / P) * WAVES + wave) * 128;
    return buf_ld_nt(wr, k + ch < K ? wo + (uint32_t)(u % P) * up + (uint32_t)k : kNoRow);
  };
  static_assert(NB % P == 0, "a buffer slot stays with the gate or the up rows");
  // x and the scales first, then the weights, then x's 8-bit form.
  const bool given = !GU && a.xs;
  RowLoad x;
  u32x4 xq[kTokenBlocks / 32];
  float xsv = 0.f, wsv[P];
  const int b0 = min((int)threadIdx.x, KB - 1);
  if (given) {
#pragma unroll
    for (int i = 0; i < kTokenBlocks / 32; ++i) {
      const int c = i * 4096 + (int)threadIdx.x * 16;
      xq[i] = c < K ? ld16(static_cast<const char*>(a.x) + c) : u32x4{0, 0, 0, 0};
    }
    xsv = a.xs[b0];
  } else {
    row_load(x, a.x, K);
  }
  const float* ws = a.ws + (size_t)expert * a.ws_stride + (size_t)(f0 / 128) * KB;
#pragma unroll
  for (int q = 0; q < P; ++q) wsv[q] = ws[(size_t)q * a.IB * KB + b0];
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int i = 0; i < NB; ++i) v[i] = load(i);
  __builtin_amdgcn_sched_barrier(0);
  if (given) {
#pragma unroll
    for (int i = 0; i < kTokenBlocks / 32; ++i) *reinterpret_cast<u32x4*>(x8 + i * 4096 + threadIdx.x * 16) = xq[i];
    if ((int)threadIdx.x < KB) sx[threadIdx.x] = xsv;
  } else {
    row_to_lds(x, KB, x8, sx);
  }
#pragma unroll
  for (int q = 0; q < P; ++q)
    if ((int)threadIdx.x < KB) sw[q][threadIdx.x] = wsv[q];
  __syncthreads();

  float acc[P];
#pragma unroll
  for (int q = 0; q < P; ++q) acc[q] = 0.f;
  // Units past the last are zeros.
  auto use = [&](int u, int i) __attribute__((always_inline)) {
    const int kb = min((u / P) * WAVES + wave, KB - 1);
    const float p = dot16(v[i], *reinterpret_cast<const u32x4*>(x8 + kb * 128 + ch));
    acc[i % P] = fmaf(p, sx[kb] * sw[i % P][kb], acc[i % P]);
  };
  int u0 = 0;
  for (; u0 + NB < units; u0 += NB) {
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      use(u0 + i, i);
      v[i] = load(u0 + NB + i);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
#pragma unroll
  for (int i = 0; i < NB; ++i) use(u0 + i, i);
#pragma unroll
  for (int q = 0; q < P; ++q) {
    const float s = row_sum(acc[q]);
    if ((lane & 7) == 0) red[wave][q][lane >> 3] = s;
  }
  __syncthreads();
  if (threadIdx.x >= 8 || f0 + (int)threadIdx.x >= a.I) return;
  float s[P];
#pragma unroll
  for (int q = 0; q < P; ++q) {
    s[q] = red[0][q][threadIdx.x];
#pragma unroll
    for (int v2 = 1; v2 < WAVES; ++v2) s[q] += red[v2][q][threadIdx.x];
  }
  const int n = f0 + threadIdx.x;
  if (GU) a.h[(size_t)blockIdx.y * a.I + n] = silu_then_mul(s[0], s[P - 1]);
  else if (a.out_f32) reinterpret_cast<float*>(a.out)[n] = s[0];
  else reinterpret_cast<uint16_t*>(a.out)[n] = (uint16_t)f2bf(s[0]);
}

// Down product of one token and the sum over its pairs.  Workgroup b: output rows 8 b .. + 7;
// wave w takes pairs w, w + 4, ... with the whole K; the waves' sums are added in wave order.
template <int NB>
__global__ __launch_bounds__(256, 4) void f8_token_down_kernel(TokenArgs a) {
  constexpr int WAVES = 4;
  __shared__ __attribute__((aligned(16))) char h8[kTokenPairBlocks * 128];
  __shared__ float sc[kTokenPairBlocks], sw[kTokenPairBlocks], red[WAVES][8];
  __shared__ int expert_of[SMLP_MAX_TOPK];
  __shared__ float wt[SMLP_MAX_TOPK];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = blockIdx.x * 8, K = a.I, KB = a.IB;
  // h first (its loads do not wait for the weights'), then ids, scales and weights.
  constexpr int HP = kTokenPairBlocks / 16;
  float hv[HP][8];
#pragma unroll
  for (int i = 0; i < HP; ++i) {
    const int q = i * 16 + (threadIdx.x >> 4), j = q / KB, c = (q - j * KB) * 128 + (threadIdx.x & 15) * 8;
#pragma unroll
    for (int e = 0; e < 8; ++e) hv[i][e] = 0.f;
    if (q < a.topk * KB && c < K) load8(a.h, (size_t)j * K + c, 0, hv[i]);
  }
  if ((int)threadIdx.x < a.topk) {
    expert_of[threadIdx.x] = local_expert(a.ids[threadIdx.x], a.first, a.E);
    wt[threadIdx.x] = a.weights[threadIdx.x];
  }
  __syncthreads();
  float wsv = 0.f;
  if ((int)threadIdx.x < a.topk * KB) {
    const int j = threadIdx.x / KB, e = expert_of[j];
    if (e >= 0) wsv = a.ws[(size_t)e * a.ws_stride + (size_t)(n0 / 128) * KB + threadIdx.x - j * KB];
  }
  const int ch = (lane & 7) * 16;
  const uint32_t wo = (uint32_t)(n0 + (lane >> 3)) * (uint32_t)K + ch;
  // Unit u of this wave: block u % KB of pair wave + WAVES * (u / KB); a pair of another rank
  // reads nothing.
  const int units = a.topk > wave ? KB * ((a.topk - wave + WAVES - 1) / WAVES) : 0;
  int lj = wave, lkb = 0;
  u32x4 v[NB];
  auto load = [&]() {
    const int e = lj < a.topk ? __builtin_amdgcn_readfirstlane(expert_of[lj]) : -1;
    const __amdgpu_buffer_rsrc_t wr = make_rsrc(a.w + (size_t)max(e, 0) * a.w_stride, e < 0 ? 0u : a.w_bytes);
    const int k = lkb * 128;
    const u32x4 r = buf_ld_nt(wr, k + ch < K ? wo + (uint32_t)k : kNoRow);
    if (++lkb == KB) {
      lkb = 0;
      lj += WAVES;
    }
    return r;
  };
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int i = 0; i < NB; ++i) v[i] = load();
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int i = 0; i < HP; ++i) {
    const int q = i * 16 + (threadIdx.x >> 4);
    float s;
    const u32x2 v8 = quant8(hv[i], s);  // rows of other ranks' pairs hold anything and are not summed
    if (q < a.topk * KB) {
      *reinterpret_cast<u32x2*>(h8 + q * 128 + (threadIdx.x & 15) * 8) = v8;
      if ((threadIdx.x & 15) == 0) sc[q] = s;
    }
  }
  if ((int)threadIdx.x < a.topk * KB) sw[threadIdx.x] = wsv;
  __syncthreads();

  float sum = 0.f, acc = 0.f;
  int j = wave, kb = 0;
  // Blocks past the last are zeros; a finished pair's sum is weighted and restarted.
  auto use = [&](int i) __attribute__((always_inline)) {
    const int q = min(j * KB + kb, a.topk * KB - 1);
    acc = fmaf(dot16(v[i], *reinterpret_cast<const u32x4*>(h8 + q * 128 + ch)), sc[q] * sw[q], acc);
    if (++kb == KB) {
      if (j < a.topk && __builtin_amdgcn_readfirstlane(expert_of[j]) >= 0) sum = fmaf(wt[j], acc, sum);
      acc = 0.f;
      kb = 0;
      j += WAVES;
    }
  };
  int u0 = 0;
  for (; u0 + NB < units; u0 += NB) {
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      use(i);
      v[i] = load();
      __builtin_amdgcn_sched_barrier(0);
    }
  }
#pragma unroll
  for (int i = 0; i < NB; ++i) use(i);
  sum = row_sum(sum);
  if ((lane & 7) == 0) red[wave][lane >> 3] = sum;
  __syncthreads();
  if (threadIdx.x >= 8) return;
  float s = red[0][threadIdx.x];
#pragma unroll
  for (int v2 = 1; v2 < WAVES; ++v2) s += red[v2][threadIdx.x];
  const int n = n0 + threadIdx.x;
  if (a.out_f32) reinterpret_cast<float*>(a.out)[n] = s;
  else reinterpret_cast<uint16_t*>(a.out)[n] = (uint16_t)f2bf(s);
}

// Position `lin` of the launch order -> (tile_m, tile_n): each XCD (workgroups are handed out
// round-robin over the 8) takes a contiguous run of the tiles, walked in groups of GROUP_M
// row tiles, so that the workgroups resident on one XCD share weight and activation tiles in
// its L2.
template <int GROUP_M>
__device__ __forceinline__ bool f8_coords(int tiles_m, int tiles_n, int lin, int& tm, int& tn) {
  constexpr int XCDS = 8;
  const int total = tiles_m * tiles_n;
  if (lin >= total) return false;
  const int per = total / XCDS, rem = total % XCDS;
  const int xcd = lin % XCDS, idx = lin / XCDS;
  const int f = xcd * per + min(xcd, rem) + idx;
  const int group = GROUP_M * tiles_n;
  const int gi = f / group, first = gi * GROUP_M;
  const int gsize = min(tiles_m - first, GROUP_M);
  const int in = f - gi * group;
  tm = first + in % gsize;
  tn = in / gsize;
  return true;
}

// 16-byte, 4-byte and 1-byte stores through a buffer resource: one past its end is dropped.
__device__ __forceinline__ void buf_st16(__amdgpu_buffer_rsrc_t r, uint32_t off, u32x4 v) {
  __builtin_amdgcn_raw_buffer_store_b128(v, r, (int)off, 0, 2);
}
__device__ __forceinline__ void buf_st4(__amdgpu_buffer_rsrc_t r, uint32_t off, uint32_t v) {
  __builtin_amdgcn_raw_buffer_store_b32(v, r, (int)off, 0, 0);
}
__device__ __forceinline__ void buf_st1(__amdgpu_buffer_rsrc_t r, uint32_t off, uint32_t v) {
  __builtin_amdgcn_raw_buffer_store_b8((unsigned char)v, r, (int)off, 0, 0);
}

// LDS-tiled kernel: BM activation rows x BN weight rows (gate_up: BN / 2 features and
// both their rows) per tile, WM x WN waves; a workgroup takes tiles lin, lin + gridDim.x, ...
// EXACT: products through bf16.
//
// 8192 x 7168 x 6144 in 322 us, 2.24 PFLOP/s (torch's library product with one scale for a
// whole tensor 299 us): the matrix cores are busy 53% of the time at 2.0 GHz; of the rest, half
// a round of tiles (896 over 256 compute units) is 12%, and without the loads or without the
// scaling's multiply-adds, which share the issue slots, the kernel would take 292 or 297 us.
// gate_up of 65536 pairs (I = 768) 700 us, 2.1 PFLOP/s with an eighth of the rows empty; down
// 530 us, 1.36 PFLOP/s: six blocks of K per tile against 128 KB of results, whose stores the
// next tile's second step has to wait for.
template <int BM, int BN, int WM, int WN, int NS, int MODE, bool EXACT>
__global__ __launch_bounds__(WM * WN * 64) void f8_tile_kernel(F8Args g) {
  constexpr bool GU = MODE == F8_GATE_UP;
  constexpr int W = WM * WN;
  constexpr int TM = BM / WM / 16, TN = BN / WN / 16;
  constexpr int FT = GU ? TN / 2 : TN;
  constexpr int FN = GU ? BN / 2 : BN;  // features per tile
  constexpr int AL = BM / 8 / W, BL = BN / 8 / W;
  constexpr int RPW = BM / W;  // activation rows whose scales a wave fetches
  static_assert(AL * W * 8 == BM && BL * W * 8 == BN && RPW <= 32, "tile / wave mismatch");
  static_assert(!GU || (TN % 2 == 0 && FN == 128), "a gate_up tile covers one scale group of h");
  static_assert(MODE != F8_DOWN || 16 * TN == 64, "64 columns share an exponent");
  static_assert(BN / WN <= 128 && 128 % (16 * FT) == 0, "one weight scale per wave");
  constexpr int A_BYTES = BM * 128, B_BYTES = BN * 128;
  constexpr int STAGE = A_BYTES + B_BYTES + W * 256;
  constexpr int LPS = AL + BL + 1;
  static_assert(NS >= 2 && LPS * (NS - 1) < 40, "loads in flight");
  // Results pass through a staging area of their own, so that the next tile's first loads
  // can fill the ring meanwhile.
  constexpr int PITCH = 32 * TN + 16;
  constexpr int STAGING = W * 16 * PITCH;
  static_assert(STAGING >= WN * BM * 4, "the row maxima of gate_up fit too");
  constexpr int PERM = GU ? (BM < 64 * W ? BM : 64 * W) * 4 : 0;  // the next tile's pairs
  __shared__ __attribute__((aligned(1024))) char lds[NS * STAGE + STAGING + PERM];
  static_assert(NS * STAGE + STAGING + PERM <= 160 * 1024, "LDS");
  static_assert(!GU || BM % 64 == 0, "64 pairs per load");

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;  // the waves that share a SIMD have different rows
  const int ln = lane & 15, lg = lane >> 4, lr = lane >> 3;
  const int tiles_m = MODE == F8_LINEAR ? g.tiles_m : g.hdr[0];
  const int K = g.K;
  const int kb0 = blockIdx.y * g.kslice;
  const int nk = min(g.KB - kb0, g.kslice);
  const __amdgpu_buffer_rsrc_t ar = make_rsrc(g.a, g.a_bytes);

  // Block i of this wave: tile rows (i * W + wave) * 8 .. + 7; this lane's row and chunk.
  static_assert(W % 2 == 0, "one chunk permutation for all blocks of a wave");
  const int chk = (lane & 7) ^ ((4 * wave + (lr >> 1)) & 7);

  // A tile's place.
  struct Place {
    int expert, start, count, f0;
  };
  auto place = [&](int lin, Place& t) __attribute__((always_inline)) {
    int tm, tn;
    // A projection's rows share all weights; row tiles of the experts mostly belong to different
    // ones (8192 tokens: groups of 2 / 4 / 8 1506 / 1526 / 1545 us; projection 336 / 330 / 334 us).
    if (!f8_coords<MODE == F8_LINEAR ? 4 : 2>(tiles_m, g.tiles_n, lin, tm, tn)) return false;
    f8_tile(g, MODE, BM, tm, t.expert, t.start, t.count);
    t.f0 = tn * FN;
    return true;
  };
  // gate_up: the pairs of a tile's rows on their way to LDS (every wave one load).
  int* const pairs = reinterpret_cast<int*>(lds + NS * STAGE + STAGING);
  auto fetch_pairs = [&](const Place& t) __attribute__((always_inline)) {
    if constexpr (GU) {
      const int r0 = wave * 64 % BM;
      glb_ld_lds4(g.perm + t.start + min(r0 + lane, t.count - 1), reinterpret_cast<char*>(pairs + r0));
    }
  };
  // Activation row of tile row r.
  auto arow = [&](const Place& t, int r) __attribute__((always_inline)) {
    if constexpr (GU) return pairs[r] / g.topk;
    else return t.start + min(r, t.count - 1);
  };

  uint32_t aoff[AL], boff[BL];
  __amdgpu_buffer_rsrc_t wr;
  const float* sp;
  int sstep;
  // Lane number that the compiler takes for new in each tile: what is derived from it is
  // computed again instead of being kept in registers through the product.
  auto fresh = [&]() __attribute__((always_inline)) {
    int l = threadIdx.x & 63;
    asm volatile("" : "+v"(l));
    return l;
  };
  auto aim = [&](const Place& t) __attribute__((always_inline)) {
    const int lane = fresh(), lr = lane >> 3;
    wr = make_rsrc(g.w + (size_t)t.expert * g.w_stride, g.w_bytes);
#pragma unroll
    for (int i = 0; i < AL; ++i)
      aoff[i] = (i * W + wave) * 8 + lr < t.count ? (uint32_t)arow(t, (i * W + wave) * 8 + lr) * (uint32_t)K + chk * 16
                                                  : kNoRow;
#pragma unroll
    for (int i = 0; i < BL; ++i) {
      const int r = (i * W + wave) * 8 + lr;
      int f = t.f0 + r, row = f;
      if (GU) {
        // Each wave column's 16 * TN rows: its gate rows, then the matching up rows.
        const int wc = r / (16 * TN), rr = r % (16 * TN);
        f = t.f0 + wc * 16 * FT + rr % (16 * FT);
        row = rr < 16 * FT ? f : g.N + f;
      }
      boff[i] = f < g.N ? (uint32_t)row * (uint32_t)K + chk * 16 : kNoRow;
    }
    // Scale source of this lane: lanes 0 .. RPW - 1 activation rows wave * RPW + lane, lanes
    // 32 and up the block of this wave's weight rows (odd lanes: of its up rows).
    if (lane < 32) {
      sp = g.as + (size_t)arow(t, wave * RPW + lane % RPW) * g.as_row;
      sstep = g.as_kb;
    } else {
      const int blk = min((t.f0 + wn * 16 * FT) / 128, g.nblk - 1) + (GU && (lane & 1) ? g.nblk : 0);
      sp = g.ws + (size_t)t.expert * g.ws_stride + (size_t)blk * g.KB;
      sstep = 1;
    }
    sp += (size_t)kb0 * sstep;
  };

  // Load l of the LPS per wave and step: activation blocks, weight blocks, scales.  Data past
  // the end of K arrives as zeros.  Steps are issued in order, so the scale pointer advances
  // by one block each time, up to the last one.
  auto issue_one = [&](int buf, int kb, int l) __attribute__((always_inline)) {
    char* st = lds + buf * STAGE;
    const uint32_t k = kb * 128 + chk * 16 < K ? (uint32_t)kb * 128u : kNoChunk;
    if (l < AL) {
      buf_ld_lds(ar, st + (l * W + wave) * 1024, aoff[l] + k);
    } else if (l < AL + BL) {
      buf_ld_lds(wr, st + A_BYTES + ((l - AL) * W + wave) * 1024, boff[l - AL] + k);
    } else {
      glb_ld_lds4(sp, st + A_BYTES + B_BYTES + wave * 256);
      sp += kb + 1 < g.KB ? sstep : 0;
    }
  };
  auto issue = [&](int buf, int kb) __attribute__((always_inline)) {
#pragma unroll
    for (int l = 0; l < LPS; ++l) issue_one(buf, kb, l);
  };
  constexpr int SLOTS = TM * TN;
  constexpr int Q = (LPS + SLOTS - 1) / SLOTS;       // loads per slot of the pinned schedule
  constexpr int HALF = Q * TN < LPS ? Q * TN : LPS;  // loads issued in the last row tile
  // Every step of the ring is issued, those past the slice too (they are not used, and past K
  // they read nothing), so the loop has no branches and its waits are constants.
  auto first_loads = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int st = 0; st < NS - 1; ++st) issue(st, kb0 + st);
    if constexpr (!EXACT) {
#pragma unroll
      for (int l = 0; l < HALF; ++l) issue_one(NS - 1, kb0 + NS - 1, l);
    }
  };
  constexpr int AHEAD = (NS - 2) * LPS + (EXACT ? 0 : HALF);  // loads behind step 0's

  f32x4 acc[TM][TN];
  // Scale of row tile i in a stage: the fetching wave's region and place.
  auto row_scale = [&](const char* sc, int i) __attribute__((always_inline)) {
    const int r = (wm * TM + i) * 16 + ln;
    return *reinterpret_cast<const float*>(sc + (r / RPW) * 256 + (r % RPW) * 4);
  };

  int lin = blockIdx.x;
  Place cur;
  if (!place(lin, cur)) return;
  if constexpr (GU) {
    fetch_pairs(cur);
    wait_vmcnt<0>();
    f8_barrier();
  }
  aim(cur);
  if constexpr (GU) {
    __builtin_amdgcn_s_waitcnt(0xc07f);
    f8_barrier();  // the pairs are read before the next tile's arrive
  }
  first_loads();
  wait_vmcnt<AHEAD>();
  for (;;) {
    f8_barrier();  // step 0 has landed in every wave's view
    // The next tile's place and pairs are looked up while this one is multiplied.
    Place nxt_place;
    const bool more = place(lin + (int)gridDim.x, nxt_place);
    if (more) fetch_pairs(nxt_place);
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    if constexpr (!EXACT) {
      // Pinned schedule.  A step is TM x TN slots, row tile by row tile.  Slot m issues one
      // matrix instruction and, while it runs, the four multiply-adds of slot m - 2, whose
      // result has arrived by then; the fragments and scale of the next row tile are read
      // during the present one.  The barrier that hands a stage back sits before the last row
      // tile, whose operands every wave then holds in registers: that tile's matrix
      // instructions cover the barrier, the reads of the next step's weights (each fragment
      // right after its last use) and the first loads into the released stage; the remaining
      // loads go out one per slot at the top of the next step.
      static_assert(TM >= 2 && TM % 2 == 0 && SLOTS % 4 == 0, "fragment and result buffers alternate");
      i32x8 wf[TN], af[2];
      f32x4 p[4];
      float sg[2] = {0.f, 0.f}, su[2] = {0.f, 0.f}, swg, swu;
      p[2] = p[3] = f32x4{0.f, 0.f, 0.f, 0.f};  // the first step's slots 0 and 1 add nothing
      auto madd = [&](int m) __attribute__((always_inline)) {
        const int i = m / TN, j = m % TN;
        const float sc = GU && j >= FT ? su[i & 1] : sg[i & 1];
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = fmaf(p[m & 3][e], sc, acc[i][j][e]);
      };
      auto read_af = [&](const char* st, int i, int half) __attribute__((always_inline)) {
        lds_half(st + (wm * TM + i) * 2048, lane, half, af[i & 1]);
      };
      auto read_wf = [&](const char* st, int j) __attribute__((always_inline)) {
        lds_half(st + A_BYTES + (wn * TN + j) * 2048, lane, 0, wf[j]);
        lds_half(st + A_BYTES + (wn * TN + j) * 2048, lane, 1, wf[j]);
      };
      auto scales_of = [&](float s, int slot) __attribute__((always_inline)) {
        sg[slot] = s * swg;
        if constexpr (GU) su[slot] = s * swu;
      };
      // Slots of row tile i of a step (stage st); nst: the next step's stage (read in the last
      // tile); loads l0 .. l1 - 1 of step lkb into stage lbuf go out Q per slot from the top.
      auto row_tile = [&](int i, const char* st, const char* nst, int lbuf, int lkb, int l0, int l1)
          __attribute__((always_inline)) {
        const bool last = i == TM - 1;
        const char* rst = last ? nst : st;
        const int ri = last ? 0 : i + 1;
        float s_next = 0.f, g_next = 0.f, u_next = 0.f;
#pragma unroll
        for (int j = 0; j < TN; ++j) {
          const int m = i * TN + j;
          // The matrix instruction goes first whenever both waves of a SIMD have something to issue.
          __builtin_amdgcn_s_setprio(1);
          p[m & 3] = mfma_fp8(wf[j], af[i & 1]);
          __builtin_amdgcn_s_setprio(0);
          madd((m + SLOTS - 2) % SLOTS);
          if (last) read_wf(nst, j);
          if (j == 0) {
            s_next = row_scale(rst + A_BYTES + B_BYTES, ri);
            read_af(rst, ri, 0);
          }
          if (j == 1) read_af(rst, ri, 1);
          if (last && j == TN - 1) {
            const float* w2 = reinterpret_cast<const float*>(nst + A_BYTES + B_BYTES + wave * 256 + 128);
            g_next = w2[0];
            if constexpr (GU) u_next = w2[1];
          }
#pragma unroll
          for (int q = 0; q < Q; ++q)
            if (l0 + j * Q + q < l1) issue_one(lbuf, lkb, l0 + j * Q + q);
          __builtin_amdgcn_sched_barrier(0);
        }
        if (last) {
          swg = g_next;
          swu = u_next;
        }
        scales_of(s_next, ri & 1);
      };
      // A wave none of whose rows exist only moves data (an expert's last tile): the other wave
      // of its SIMD has the matrix core to itself.
      const bool idle = WM > 1 && wm * TM * 16 >= cur.count;
      if (idle) {
        for (int kt = 0; kt < nk; ++kt) {
#pragma unroll
          for (int l = HALF; l < LPS; ++l) issue_one((kt + NS - 1) % NS, kb0 + kt + NS - 1, l);
          wait_vmcnt<(NS - 2) * LPS>();
          f8_barrier();
#pragma unroll
          for (int l = 0; l < HALF; ++l) issue_one(kt % NS, kb0 + kt + NS, l);
        }
      } else {
        const char* st = lds;
        const float* w2 = reinterpret_cast<const float*>(st + A_BYTES + B_BYTES + wave * 256 + 128);
        swg = w2[0];
        swu = GU ? w2[1] : 0.f;
#pragma unroll
        for (int j = 0; j < TN; ++j) read_wf(st, j);
        read_af(st, 0, 0);
        read_af(st, 0, 1);
        scales_of(row_scale(st + A_BYTES + B_BYTES, 0), 0);
        __builtin_amdgcn_sched_barrier(0);
      }
      for (int kt = 0; kt < (idle ? 0 : nk); ++kt) {
        const int now = kt % NS, nxt = (kt + 1) % NS;
        const char* st = lds + now * STAGE;
        const char* nst = lds + nxt * STAGE;
        // The rest of step kt + NS - 1's loads (its first HALF went out in the last row tile of
        // the step before).
#pragma unroll
        for (int i = 0; i < TM - 1; ++i)
          row_tile(i, st, nst, (kt + NS - 1) % NS, kb0 + kt + NS - 1, HALF + i * TN * Q, LPS);
        static_assert(HALF + (TM - 1) * TN * Q >= LPS, "a step's slots hold its loads");
        // Every wave holds the last row tile's operands (lgkmcnt 0) and step kt + 1 has landed.
        // (After the last step the reads below fetch fragments that are never used.)
        __builtin_amdgcn_s_waitcnt(0xc07f);
        wait_vmcnt<(NS - 2) * LPS>();
        f8_barrier();
        row_tile(TM - 1, st, nst, now, kb0 + kt + NS, 0, HALF);
      }
      // The last two slots' multiply-adds; sg / su of the last row tile are still in place.
      if (!idle) {
        madd(SLOTS - 2);
        madd(SLOTS - 1);
      }
      __builtin_amdgcn_s_waitcnt(0xc07f);
    } else {
      for (int kt = 0; kt < nk; ++kt) {
        if (kt) {
          wait_vmcnt<(NS - 2) * LPS>();
          f8_barrier();
        }
        issue((kt + NS - 1) % NS, kb0 + kt + NS - 1);
        const char* st = lds + (kt % NS) * STAGE;
        const char* sc = st + A_BYTES + B_BYTES;
        const float swg = *reinterpret_cast<const float*>(sc + wave * 256 + 128);
        const float swu = GU ? *reinterpret_cast<const float*>(sc + wave * 256 + 132) : swg;
        frag_bf16 wf[TN];
#pragma unroll
        for (int j = 0; j < TN; ++j) wf[j] = widen(lds_frag(st + A_BYTES + (wn * TN + j) * 2048, lane));
#pragma unroll
        for (int i = 0; i < TM; ++i) {
          const frag_bf16 af = widen(lds_frag(st + (wm * TM + i) * 2048, lane));
          const float s = row_scale(sc, i);
          const float sg = s * swg, su = s * swu;
#pragma unroll
          for (int j = 0; j < TN; ++j) {
            const f32x4 p = mfma_widened(wf[j], af);
            const float sj = j < FT ? sg : su;
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][j][e] = fmaf(p[e], sj, acc[i][j][e]);
          }
        }
        __builtin_amdgcn_s_waitcnt(0xc07f);
      }
    }
    // The ring is free once every wave's loads have landed and its reads are done: the next
    // tile's first loads go out ahead of this tile's stores.  Loads and stores complete in
    // order, so the wait at the end counts the stores behind them, a fixed number (rows past
    // the tile's are dropped by the buffer bounds, not skipped).
    wait_vmcnt<0>();
    f8_barrier();
    if (more) {
      aim(nxt_place);
      first_loads();
    }
    __builtin_amdgcn_sched_barrier(0);  // the stores below stay behind these loads
    int stores = 0;  // known when inlined; -1: not fixed
    const int lane = fresh(), ln = lane & 15, lg = lane >> 4;
    if constexpr (MODE == F8_LINEAR) {
      if (gridDim.y > 1) {
        // K split over workgroups (one tile each, at most kCUs / 2): this slice's sums go
        // out agent-coherent as [slice][tile][row tile, column tile][lane][4]; the last slice
        // of a tile to arrive adds all of them in slice order and goes on with the sum.
        const uint32_t tile = blockIdx.x, per = BM * BN * 4, step = gridDim.x * per;
        const __amdgpu_buffer_rsrc_t pr = make_rsrc(g.part, gridDim.y * step);
        const uint32_t base = tile * per + (uint32_t)(wave * TM * TN * 64 + lane) * 16u;
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int j = 0; j < TN; ++j)
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, acc[i][j]), pr,
                                                   (int)(blockIdx.y * step + base + (i * TN + j) * 1024), 0, 16);
        wait_vmcnt<0>();
        f8_barrier();
        int* last = reinterpret_cast<int*>(lds + NS * STAGE);
        if (threadIdx.x == 0) {
          uint32_t* c = g.arrived + 16 * tile;
          const bool l = __hip_atomic_fetch_add(c, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == gridDim.y - 1;
          if (l) __hip_atomic_store(c, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
          *reinterpret_cast<volatile int*>(last) = l;
        }
        __syncthreads();
        if (!*reinterpret_cast<volatile int*>(last)) return;
        __syncthreads();  // the flag is read before the staging area is used
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
          for (int j = 0; j < TN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
        for (uint32_t q = 0; q < gridDim.y; ++q)
#pragma unroll
          for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j)
              acc[i][j] += __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(
                               pr, (int)(q * step + base + (i * TN + j) * 1024), 0, 16));
      }
    }
    char* const stg = lds + NS * STAGE + wave * (16 * PITCH);
    if constexpr (GU) {
      // h = SiLU(gate) * up, then e4m3 with one scale per row and 128 features: the rows'
      // largest magnitudes over this wave's features, then over the waves of a row.
      float* red = reinterpret_cast<float*>(lds + NS * STAGE);
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        float mx = 0.f;
#pragma unroll
        for (int j = 0; j < FT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float v = silu_then_mul(acc[i][j][e], acc[i][j + FT][e]);
            acc[i][j][e] = v;
            mx = fmaxf(mx, fabsf(v));
          }
        mx = fmaxf(mx, __shfl_xor(mx, 16));
        mx = fmaxf(mx, __shfl_xor(mx, 32));
        if (lg == 0) red[wn * BM + (wm * TM + i) * 16 + ln] = mx;
      }
      __builtin_amdgcn_s_waitcnt(0xc07f);
      f8_barrier();
      float top[TM];
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        top[i] = kAmaxMin;
#pragma unroll
        for (int v = 0; v < WN; ++v) top[i] = fmaxf(top[i], red[v * BM + (wm * TM + i) * 16 + ln]);
      }
      __builtin_amdgcn_s_waitcnt(0xc07f);
      f8_barrier();  // the staging area changes hands
      const __amdgpu_buffer_rsrc_t hr =
          make_rsrc(static_cast<uint8_t*>(g.out) + (size_t)cur.start * g.N, (uint32_t)cur.count * (uint32_t)g.N);
      const __amdgpu_buffer_rsrc_t sr =
          make_rsrc(g.hs + (size_t)(cur.f0 / 128) * g.hs_ld + cur.start, (uint32_t)cur.count * 4u);
#pragma unroll
      for (int i = 0; i < TM; i += 4) {
        // Lane group q stores the scales of row tile i + q (the first wave column's lanes).
        float t4 = top[i];
#pragma unroll
        for (int q = 1; q < 4; ++q)
          if (i + q < TM && lg == q) t4 = top[i + q];
        const uint32_t r = (uint32_t)((wm * TM + i + lg) * 16 + ln);
        buf_st4(sr, wn == 0 && i + lg < TM ? r * 4u : kNoRow, __float_as_uint(t4 / kE4M3Max));
      }
      constexpr int HB = 16 * FT;  // bytes of a row: two 16-byte chunks (FT == 2)
      static_assert(FT == 2 && TM % 2 == 0, "two row tiles per store");
#pragma unroll
      for (int i = 0; i < TM; i += 2) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const float inv = kE4M3Max * (1.0f / top[i + q]);
#pragma unroll
          for (int j = 0; j < FT; ++j)
            *reinterpret_cast<uint32_t*>(stg + (q * 16 + ln) * (HB + 4) + j * 16 + lg * 4) =
                pack_fp8x4(acc[i + q][j][0] * inv, acc[i + q][j][1] * inv, acc[i + q][j][2] * inv,
                           acc[i + q][j][3] * inv);
        }
        __builtin_amdgcn_wave_barrier();
        const int rr = lane >> 1, c = lane & 1;
        const uint32_t* from = reinterpret_cast<const uint32_t*>(stg + rr * (HB + 4) + c * 16);
        const u32x4 v{from[0], from[1], from[2], from[3]};
        const uint32_t r = (uint32_t)((wm * TM + i) * 16 + rr);
        const int n = cur.f0 + wn * HB + c * 16;  // N is a multiple of 16
        // Rows past the tile's are dropped here: with a wide N their offsets would wrap.
        buf_st16(hr, n < g.N && (int)r < cur.count ? r * (uint32_t)g.N + (uint32_t)n : kNoRow, v);
        __builtin_amdgcn_wave_barrier();
      }
      stores = (TM + 3) / 4 + TM / 2;
    } else {
      constexpr int CPR = 2 * TN, RPI = 64 / CPR;  // 16-byte chunks per staged row, rows per store
      const bool whole = MODE == F8_DOWN
                             ? !g.out_f32
                             : !g.out_f32 && cur.f0 + FN <= g.N && g.ldo % 8 == 0 && ((uintptr_t)g.out & 15) == 0;
      if (whole) {
        // Rows through LDS: a lane's four features are 8 bytes of 16 different rows, the
        // stores below whole runs of 32 TN bytes per row.  Projection: bf16.  Experts: fp16
        // with a power of two per row and 64 columns (11 significant bits at the range of
        // fp32; bf16 here would show beside the rounding of the sum).
        const uint32_t rowb = (uint32_t)g.ldo * 2u;
        const __amdgpu_buffer_rsrc_t yr =
            make_rsrc(static_cast<char*>(g.out) + (size_t)cur.start * rowb, (uint32_t)(cur.count - 1) * rowb + (uint32_t)g.N * 2u);
        uint32_t ex[TM];
#pragma unroll
        for (int i = 0; i < TM; ++i) {
          float up = 1.f;
          if constexpr (MODE == F8_DOWN) {
            float mx = 0.f;
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
              for (int e = 0; e < 4; ++e) mx = fmaxf(mx, fabsf(acc[i][j][e]));
            mx = fmaxf(mx, __shfl_xor(mx, 16));
            mx = fmaxf(mx, __shfl_xor(mx, 32));
            // A result past the range stays an infinity; the exponent is the finite ones'.
            if (__ballot(mx == INFINITY)) {
              mx = 0.f;
#pragma unroll
              for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const float v = fabsf(acc[i][j][e]);
                  mx = fmaxf(mx, v < INFINITY ? v : 0.f);
                }
              mx = fmaxf(mx, __shfl_xor(mx, 16));
              mx = fmaxf(mx, __shfl_xor(mx, 32));
            }
            ex[i] = max(__float_as_uint(mx) >> 23, 15u);        // exponent field of the largest
            up = __uint_as_float((268u - ex[i]) << 23);         // brings it to [2^14, 2^15)
          }
#pragma unroll
          for (int j = 0; j < TN; ++j) {
            u32x2 v;
            if constexpr (MODE == F8_DOWN)
              v = u32x2{f2h(acc[i][j][0] * up) | f2h(acc[i][j][1] * up) << 16,
                        f2h(acc[i][j][2] * up) | f2h(acc[i][j][3] * up) << 16};
            else
              v = u32x2{pack_bf2(acc[i][j][0], acc[i][j][1]), pack_bf2(acc[i][j][2], acc[i][j][3])};
            *reinterpret_cast<u32x2*>(stg + ln * PITCH + j * 32 + lg * 8) = v;
          }
          __builtin_amdgcn_wave_barrier();
#pragma unroll
          for (int q = 0; q < 16 / RPI; ++q) {
            const int rr = q * RPI + lane / CPR;
            const u32x4 v = *reinterpret_cast<const u32x4*>(stg + rr * PITCH + (lane % CPR) * 16);
            const uint32_t r = (uint32_t)((wm * TM + i) * 16 + rr);
            const int n = cur.f0 + wn * 16 * TN + (lane % CPR) * 8;
            buf_st16(yr, n < g.N && (int)r < cur.count ? r * rowb + (uint32_t)n * 2u : kNoRow, v);
          }
          __builtin_amdgcn_wave_barrier();
        }
        if constexpr (MODE == F8_DOWN) {
          const __amdgpu_buffer_rsrc_t er = make_rsrc(
              g.yexp + (size_t)(cur.f0 / 64 + wn) * g.hs_ld + cur.start, cur.f0 + wn * 64 < g.N ? (uint32_t)cur.count : 0u);
#pragma unroll
          for (int i = 0; i < TM; i += 4) {
            uint32_t e4 = ex[i];
#pragma unroll
            for (int q = 1; q < 4; ++q)
              if (i + q < TM && lg == q) e4 = ex[i + q];
            buf_st1(er, i + lg < TM ? (uint32_t)((wm * TM + i + lg) * 16 + ln) : kNoRow, e4);
          }
        }
        stores = TM * (16 / RPI) + (MODE == F8_DOWN ? (TM + 3) / 4 : 0);
      } else {
        stores = -1;
#pragma unroll
        for (int i = 0; i < TM; ++i) {
          const int r = (wm * TM + i) * 16 + ln;
          if (r >= cur.count) continue;
          const size_t row = (size_t)(cur.start + r);
#pragma unroll
          for (int j = 0; j < TN; ++j) {
            const int n = cur.f0 + (wn * TN + j) * 16 + 4 * lg;
            if (n >= g.N) continue;
            f8_store4(g, row, n, acc[i][j]);
          }
        }
      }
    }
    if (!more) break;
    constexpr int CPRW = 2 * TN;
    constexpr int FIXED = GU ? (TM + 3) / 4 + TM / 2 : TM * (16 * CPRW / 64) + (MODE == F8_DOWN ? (TM + 3) / 4 : 0);
    static_assert(AHEAD + FIXED < 64, "vmcnt range");
    if (stores == FIXED) wait_vmcnt<AHEAD + FIXED>();
    else wait_vmcnt<0>();
    lin += (int)gridDim.x;
    cur = nxt_place;
  }
}

// Quantisation of rows in groups of 128 columns: 16 lanes per group, 8 elements each.
// scale of row r, group b: s[r * s_row + b * s_kb].  Bound by HBM: 8192 x 6144 bf16 in 33 us,
// 4.6 TB/s read and written.
struct QuantArgs {
  const void* x;
  int64_t rows;
  int cols;      // multiple of 16
  int64_t ldx;
  int bf16;
  uint8_t* q;    // dense [rows, cols]
  float* s;
  int64_t s_row, s_kb;
};

__device__ __forceinline__ void quant_group(const QuantArgs& a, int64_t group, int KB) {
  const int l = threadIdx.x & 15;
  const int64_t row = group / KB;
  const int b = (int)(group - row * KB);
  const int c = b * 128 + l * 8;
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  const bool in = row < a.rows && c < a.cols;
  if (in) load8(a.x, (size_t)row * a.ldx + c, a.bf16, v);
  float mx = kAmaxMin;
#pragma unroll
  for (int i = 0; i < 8; ++i) mx = fmaxf(mx, fabsf(v[i]));
#pragma unroll
  for (int d = 8; d >= 1; d >>= 1) mx = fmaxf(mx, __shfl_xor(mx, d));
  if (!in) return;
  const float inv = kE4M3Max * (1.0f / mx);
  *reinterpret_cast<u32x2*>(a.q + (size_t)row * a.cols + c) =
      u32x2{pack_fp8x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
            pack_fp8x4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv)};
  if (l == 0) a.s[row * a.s_row + b * a.s_kb] = mx / kE4M3Max;
}

__global__ __launch_bounds__(256) void quant_rows_kernel(QuantArgs a) {
  const int KB = (a.cols + 127) / 128;
  const int64_t groups = a.rows * KB;
  const int64_t step = (int64_t)gridDim.x * 16;
  // Whole workgroups iterate together: the last round's idle groups read nothing.
  for (int64_t g = (int64_t)blockIdx.x * 16; g < groups; g += step) quant_group(a, g + (threadIdx.x >> 4), KB);
}

// Quantisation in 128 x 128 blocks of parts x rows x cols: one workgroup per block.
__global__ __launch_bounds__(256) void quant_blocks_kernel(QuantArgs a, int rows_per_part) {
  __shared__ float red[4];
  const int KB = (a.cols + 127) / 128, RB = (rows_per_part + 127) / 128;
  const int64_t id = blockIdx.x;
  const int b = (int)(id % KB);
  const int64_t rb = id / KB;
  const int64_t part = rb / RB;
  const int r0 = (int)(rb % RB) * 128;
  const int nr = min(128, rows_per_part - r0);
  const int64_t row0 = part * rows_per_part + r0;
  const int l = threadIdx.x & 15, rr = threadIdx.x >> 4;
  const int c = b * 128 + l * 8;
  float mx = kAmaxMin;
  for (int r = rr; r < nr; r += 16) {
    if (c >= a.cols) break;
    float v[8];
    load8(a.x, (size_t)(row0 + r) * a.ldx + c, a.bf16, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) mx = fmaxf(mx, fabsf(v[i]));
  }
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) mx = fmaxf(mx, __shfl_xor(mx, d));
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = mx;
  __syncthreads();
  mx = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  const float inv = kE4M3Max * (1.0f / mx);
  for (int r = rr; r < nr; r += 16) {
    if (c >= a.cols) break;
    float v[8];
    load8(a.x, (size_t)(row0 + r) * a.ldx + c, a.bf16, v);
    *reinterpret_cast<u32x2*>(a.q + (size_t)(row0 + r) * a.cols + c) =
        u32x2{pack_fp8x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
              pack_fp8x4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv)};
  }
  if (threadIdx.x == 0) a.s[(rb * KB) + b] = mx / kE4M3Max;
}

// First launches of the experts: sort the pairs (token, choice) by expert, write the tile
// list, and quantise x beside that.  Pairs whose expert is outside [first, first + E) are
// dropped.  Up to kOneSort pairs one workgroup sorts; above, workgroup b counts its chunk of
// pairs, and a second launch places them from the counts (65536 pairs: one workgroup took
// 90 us, most of it waiting for its own loads).
struct PrepArgs {
  const int32_t* ids;
  int pairs, E, first, bm;
  int* hdr;     // [0] tiles, then 4 words per tile
  int* perm;    // pair at each sorted position
  int* place;   // sorted position of each pair, -1 for other ranks' pairs
  int* counts;  // [chunks][E]
  int chunk, chunks;
  QuantArgs q;
};

constexpr int kPrepThreads = 1024;

__device__ __forceinline__ void prep_quant(const PrepArgs& a, int block, int blocks) {
  const int KB = (a.q.cols + 127) / 128;
  const int64_t groups = a.q.rows * KB;
  constexpr int PER = kPrepThreads / 16;
  for (int64_t g = (int64_t)block * PER; g < groups; g += (int64_t)blocks * PER) quant_group(a.q, g + (threadIdx.x >> 4), KB);
}

// Rows of each local expert among pairs p0 .. p1 - 1, into count (LDS, kPrepThreads words).
__device__ __forceinline__ void prep_count(const PrepArgs& a, int p0, int p1, int* count) {
  static_assert(SMLP_MAX_EXPERTS <= kPrepThreads, "one thread per expert");
  count[threadIdx.x] = 0;
  __syncthreads();
  for (int p = p0 + (int)threadIdx.x; p < p1; p += kPrepThreads) {
    const int e = local_expert(a.ids[p], a.first, a.E);
    if (e >= 0) atomicAdd(&count[e], 1);
  }
  __syncthreads();
}

// Thread e holds expert e's rows c: its first sorted position, and (write) its tiles.
__device__ __forceinline__ int prep_scan(const PrepArgs& a, int c, bool write, int (*wsum)[kPrepThreads / 64]) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int nt = (c + a.bm - 1) / a.bm;
  int o = c, t = nt;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int uo = __shfl_up(o, d), ut = __shfl_up(t, d);
    if (lane >= d) {
      o += uo;
      t += ut;
    }
  }
  if (lane == 63) {
    wsum[0][wave] = o;
    wsum[1][wave] = t;
  }
  __syncthreads();
  for (int v = 0; v < wave; ++v) {
    o += wsum[0][v];
    t += wsum[1][v];
  }
  if (write) {
    if (tid == kPrepThreads - 1) a.hdr[0] = t;
    for (int i = 0, q = t - nt; i < c; i += a.bm, ++q) {
      a.hdr[4 + 4 * q] = tid;
      a.hdr[5 + 4 * q] = o - c + i;
      a.hdr[6 + 4 * q] = min(a.bm, c - i);
    }
  }
  return o - c;
}

// Place pairs p0 .. p1 - 1 from the next free positions in off (LDS).  The order within an
// expert does not change any result (a row's sums do not depend on its place in a tile);
// rounds of the workgroup keep it near token order.
__device__ __forceinline__ void prep_place(const PrepArgs& a, int p0, int p1, int* off) {
  for (int q = p0; q < p1; q += kPrepThreads) {
    const int p = q + (int)threadIdx.x;
    if (p < p1) {
      const int e = local_expert(a.ids[p], a.first, a.E);
      const int at = e >= 0 ? atomicAdd(&off[e], 1) : -1;
      a.place[p] = at;
      if (e >= 0) a.perm[at] = p;
    }
    __syncthreads();
  }
}

__global__ __launch_bounds__(kPrepThreads) void experts_prep_kernel(PrepArgs a) {
  if (blockIdx.x > 0) {
    prep_quant(a, blockIdx.x - 1, gridDim.x - 1);
    return;
  }
  __shared__ int count[kPrepThreads], off[kPrepThreads], wsum[2][kPrepThreads / 64];
  prep_count(a, 0, a.pairs, count);
  off[threadIdx.x] = prep_scan(a, count[threadIdx.x], true, wsum);
  __syncthreads();
  prep_place(a, 0, a.pairs, off);
}

__global__ __launch_bounds__(kPrepThreads) void experts_count_kernel(PrepArgs a) {
  const int b = blockIdx.x;
  if (b >= a.chunks) {
    prep_quant(a, b - a.chunks, gridDim.x - a.chunks);
    return;
  }
  __shared__ int count[kPrepThreads];
  prep_count(a, b * a.chunk, min(a.pairs, (b + 1) * a.chunk), count);
  if ((int)threadIdx.x < a.E) a.counts[b * a.E + threadIdx.x] = count[threadIdx.x];
}

__global__ __launch_bounds__(kPrepThreads) void experts_place_kernel(PrepArgs a) {
  __shared__ int off[kPrepThreads], wsum[2][kPrepThreads / 64];
  const int b = blockIdx.x, e = threadIdx.x;
  int all = 0, before = 0;
  if (e < a.E)
    for (int v = 0; v < a.chunks; ++v) {
      const int c = a.counts[v * a.E + e];
      all += c;
      if (v < b) before += c;
    }
  off[e] = before + prep_scan(a, all, b == 0, wsum);
  __syncthreads();
  prep_place(a, b * a.chunk, min(a.pairs, (b + 1) * a.chunk), off);
}

// out[t] = sum_j weights[t, j] y[place of (t, j)] over the local experts, in fp32.
struct CombineArgs {
  const void* y;         // fp32, or fp16 with exponents
  const uint8_t* yexp;
  int P;
  const int* place;
  const float* weights;
  void* out;
  int T, H, topk, out_f32;
};

// F32: few pairs, whose latency counts: a token's places and rows are loaded together (32
// tokens of 8 pairs: 6.5 -> 4.5 us).  Otherwise the rows come from HBM, one after the other
// (8192 tokens of 8 pairs of 7168: 215 us for 1.06 GB; two at a time behind branches 370 us).
template <bool F32>
__global__ __launch_bounds__(256) void experts_combine_kernel(CombineArgs a) {
  const int per = a.H / 8;
  const int64_t total = (int64_t)a.T * per;
  constexpr int B = F32 ? 8 : 1;  // pairs whose loads are in flight together
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int t = (int)(i / per), c = (int)(i - (int64_t)t * per) * 8;
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int j0 = 0; j0 < a.topk; j0 += B) {
      int at[B];
      float w[B];
#pragma unroll
      for (int j = 0; j < B; ++j) {
        const bool in = j0 + j < a.topk;
        at[j] = in ? a.place[(size_t)t * a.topk + j0 + j] : -1;
        w[j] = in ? a.weights[(size_t)t * a.topk + j0 + j] : 0.f;
      }
      if constexpr (F32) {
        f32x4 y[B][2];
#pragma unroll
        for (int j = 0; j < B; ++j)
          if (at[j] >= 0) {
            const float* p = reinterpret_cast<const float*>(a.y) + (size_t)at[j] * a.H + c;
            y[j][0] = *reinterpret_cast<const f32x4*>(p);
            y[j][1] = *reinterpret_cast<const f32x4*>(p + 4);
          }
#pragma unroll
        for (int j = 0; j < B; ++j)
          if (at[j] >= 0) {
#pragma unroll
            for (int q = 0; q < 8; ++q) acc[q] = fmaf(w[j], y[j][q >> 2][q & 3], acc[q]);
          }
      } else {
        if (at[0] < 0) continue;
        const u32x4 u = __builtin_nontemporal_load(
            reinterpret_cast<const u32x4*>(reinterpret_cast<const uint16_t*>(a.y) + (size_t)at[0] * a.H + c));
        const float down = __uint_as_float((uint32_t)(a.yexp[(size_t)(c / 64) * a.P + at[0]] - 14) << 23);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float lo = (float)__builtin_bit_cast(_Float16, (uint16_t)(u[q] & 0xffffu));
          const float hi = (float)__builtin_bit_cast(_Float16, (uint16_t)(u[q] >> 16));
          acc[2 * q] = fmaf(w[0], lo * down, acc[2 * q]);
          acc[2 * q + 1] = fmaf(w[0], hi * down, acc[2 * q + 1]);
        }
      }
    }
    const size_t at = (size_t)t * a.H + c;
    if (a.out_f32) {
      f32x4* o = reinterpret_cast<f32x4*>(reinterpret_cast<float*>(a.out) + at);
      o[0] = f32x4{acc[0], acc[1], acc[2], acc[3]};
      o[1] = f32x4{acc[4], acc[5], acc[6], acc[7]};
    } else {
      *reinterpret_cast<u32x4*>(reinterpret_cast<uint16_t*>(a.out) + at) =
          u32x4{pack_bf2(acc[0], acc[1]), pack_bf2(acc[2], acc[3]), pack_bf2(acc[4], acc[5]),
                pack_bf2(acc[6], acc[7])};
    }
  }
}

unsigned quant_grid(int64_t groups, int per) {
  const int64_t n = (groups + per - 1) / per;
  return (unsigned)(n < 1 ? 1 : n > 2048 ? 2048 : n);
}

template <int MODE>
int launch_f8(const F8Plan& p, const F8Args& a, int max_tiles, hipStream_t s) {
  if (p.kind == F8_KIND_STREAM) {
    const int per = (MODE == F8_GATE_UP ? 8 : 16) * p.nt;
    const dim3 grid((unsigned)((a.N + per - 1) / per), (unsigned)max_tiles);
#define SMLP_F8(NT_, AH_, W_, S_)                                                                      \
  if (p.nt == NT_ && p.bm == 8 * AH_) {                                                                \
    hipLaunchKernelGGL((f8_stream_kernel<NT_, AH_, W_, S_, MODE>), grid, dim3(W_ * 64), 0, s, a);      \
    return (int)hipGetLastError();                                                                     \
  }
    SMLP_F8(2, 1, 4, 3) SMLP_F8(2, 2, 4, 3) SMLP_F8(2, 4, 4, 4)
#undef SMLP_F8
    return (int)hipErrorInvalidConfiguration;
  }
  const int fn = MODE == F8_GATE_UP ? p.bn / 2 : p.bn;
  F8Args g = a;
  g.tiles_n = (a.N + fn - 1) / fn;
  g.tiles_m = max_tiles;
  // One workgroup per compute unit (two of the small tiles), each taking every so-manieth tile.
  const int resident = (p.bm * p.bn <= 128 * 128 ? 2 : 1) * kCUs, tiles = g.tiles_n * max_tiles;
  const dim3 grid((unsigned)(tiles < resident ? tiles : resident), (unsigned)p.ksplit);
#define SMLP_F8(BM_, BN_, WM_, WN_, NS_)                                                               \
  if (p.bm == BM_ && p.bn == BN_) {                                                                    \
    if (p.exact)                                                                                       \
      hipLaunchKernelGGL((f8_tile_kernel<BM_, BN_, WM_, WN_, NS_, MODE, true>), grid,                  \
                         dim3(WM_ * WN_ * 64), 0, s, g);                                               \
    else                                                                                               \
      hipLaunchKernelGGL((f8_tile_kernel<BM_, BN_, WM_, WN_, NS_, MODE, false>), grid,                 \
                         dim3(WM_ * WN_ * 64), 0, s, g);                                               \
    return (int)hipGetLastError();                                                                     \
  }
  SMLP_F8(256, 256, 2, 4, 2)
  if constexpr (MODE != F8_LINEAR) { SMLP_F8(64, 256, 2, 4, 3) }
  if constexpr (MODE == F8_LINEAR) { SMLP_F8(64, 64, 2, 2, 4) SMLP_F8(128, 128, 2, 2, 2) }
#undef SMLP_F8
  return (int)hipErrorInvalidConfiguration;
}

}  // namespace

int launch_quant_fp8(const void* x, int bf16, int64_t parts, int64_t rows, int64_t cols, int64_t ldx,
                     int block_rows, void* q, float* scales, int64_t s_row, int64_t s_kb, hipStream_t s) {
  QuantArgs a{};
  a.x = x;
  a.rows = parts * rows;
  a.cols = (int)cols;
  a.ldx = ldx;
  a.bf16 = bf16;
  a.q = static_cast<uint8_t*>(q);
  a.s = scales;
  a.s_row = s_row;
  a.s_kb = s_kb;
  const int64_t KB = (cols + 127) / 128;
  if (block_rows == 1) {
    hipLaunchKernelGGL(quant_rows_kernel, dim3(quant_grid(a.rows * KB, 16)), dim3(256), 0, s, a);
  } else {
    const int64_t blocks = parts * ((rows + 127) / 128) * KB;
    hipLaunchKernelGGL(quant_blocks_kernel, dim3((unsigned)blocks), dim3(256), 0, s, a, (int)rows);
  }
  return (int)hipGetLastError();
}

int launch_row_fp8(const void* x, const float* xs, const void* w, const float* ws, void* y, int64_t K, int64_t N,
                   int out_f32, hipStream_t s) {
  TokenArgs t{};
  t.x = x;
  t.xs = xs;
  t.w = static_cast<const uint8_t*>(w);
  t.w_bytes = (uint32_t)(N * K);
  t.ws = ws;
  t.H = (int)K;
  t.I = (int)N;
  t.HB = (int)((K + 127) / 128);
  t.IB = (int)((N + 127) / 128);
  t.out = y;
  t.out_f32 = out_f32;
  hipLaunchKernelGGL((f8_row_kernel<false, 14>), dim3((unsigned)((N + 7) / 8)), dim3(256), 0, s, t);
  return (int)hipGetLastError();
}

int launch_narrow_fp8(const F8Plan& p, const void* x, const void* w, const float* ws, void* y, int64_t M, int64_t K,
                      int64_t N, int64_t ldy, int out_f32, float* part, hipStream_t s) {
  NarrowArgs a{};
  a.x = x;
  a.w = static_cast<const uint8_t*>(w);
  a.ws = ws;
  a.g.w_bytes = (uint32_t)(N * K);
  a.g.K = (int)K;
  a.g.KB = (int)((K + 127) / 128);
  a.g.N = (int)N;
  a.g.nblk = (int)((N + 127) / 128);
  a.g.M = (int)M;
  a.g.out = y;
  a.g.ldo = (int)ldy;
  a.g.out_f32 = out_f32;
  const int cols = (int)((N + 16 * p.nt - 1) / (16 * p.nt));
  a.arrived = p.ksplit > 1 ? product_counters(s, cols) : nullptr;
  const int slices = a.arrived ? p.ksplit : 1;  // no counters left: no split
  a.g.kslice = slices > 1 ? p.kslice : a.g.KB;
  a.g.part = part;
  const dim3 grid((unsigned)cols, (unsigned)slices);
  hipLaunchKernelGGL((f8_narrow_kernel<1, 4>), grid, dim3(512), 0, s, a);
  return (int)hipGetLastError();
}

int launch_linear_fp8(const F8Plan& p, const void* a8, const float* as, int64_t as_row, int64_t as_kb,
                      const void* w, const float* ws, void* y, int64_t M, int64_t K, int64_t N, int64_t ldy,
                      int out_f32, float* part, hipStream_t s) {
  F8Args g{};
  g.a = static_cast<const uint8_t*>(a8);
  g.a_bytes = (uint32_t)(M * K);
  g.as = as;
  g.as_row = (int)as_row;
  g.as_kb = (int)as_kb;
  g.w = static_cast<const uint8_t*>(w);
  g.w_bytes = (uint32_t)(N * K);
  g.ws = ws;
  g.K = (int)K;
  g.KB = (int)((K + 127) / 128);
  g.N = (int)N;
  g.nblk = (int)((N + 127) / 128);
  g.M = (int)M;
  g.out = y;
  g.ldo = (int)ldy;
  g.out_f32 = out_f32;
  if (p.kind == F8_KIND_TILE && !out_f32 && !p.by_rows) g.out_f32 = kGuarded;
  g.part = part;
  const int tiles = (int)((M + p.bm - 1) / p.bm);
  F8Plan q = p;
  if (p.ksplit > 1) {
    g.arrived = product_counters(s, (int)(tiles * ((N + p.bn - 1) / p.bn)));
    if (!g.arrived) {  // no counters left: no split
      q.ksplit = 1;
      q.kslice = g.KB;
    }
  }
  g.kslice = q.kslice;
  return launch_f8<F8_LINEAR>(q, g, tiles, s);
}

namespace {

int launch_f8_down(const F8Plan& p, const F8Args& a, const float* h, int max_tiles, hipStream_t s) {
  const dim3 grid((unsigned)(((a.N + 15) / 16 + p.run - 1) / p.run), (unsigned)max_tiles);
#define SMLP_F8(AH_, KB_, D_)                                                                             \
  if (p.bm == 8 * AH_ && a.KB <= KB_) {                                                                   \
    hipLaunchKernelGGL((f8_down_kernel<AH_, KB_, D_>), grid, dim3(256), 0, s, a, h, p.run);               \
    return (int)hipGetLastError();                                                                        \
  }
  SMLP_F8(1, 8, 6) SMLP_F8(2, 8, 6) SMLP_F8(4, 8, 6) SMLP_F8(1, 16, 6) SMLP_F8(2, 16, 5)
#undef SMLP_F8
  return (int)hipErrorInvalidConfiguration;
}

}  // namespace

int launch_experts_fp8(const ExpertsPlan& p, const ExpertsCall& c, void* workspace, hipStream_t s) {
  char* base = static_cast<char*>(workspace);
  const int64_t HB = (p.H + 127) / 128, IB = (p.I + 127) / 128;
  int* hdr = reinterpret_cast<int*>(base + p.hdr_off);
  int* perm = reinterpret_cast<int*>(base + p.perm_off);
  uint8_t* x8 = reinterpret_cast<uint8_t*>(base + p.x8_off);
  float* xs = reinterpret_cast<float*>(base + p.xs_off);
  uint8_t* h8 = reinterpret_cast<uint8_t*>(base + p.h8_off);
  float* hs = reinterpret_cast<float*>(base + p.hs_off);
  float* h32 = reinterpret_cast<float*>(base + p.h32_off);
  void* y = base + p.y_off;

  if (p.token) {
    TokenArgs t{};
    t.x = c.x;
    t.ids = c.ids;
    t.weights = c.weights;
    t.w = static_cast<const uint8_t*>(c.w_gate_up);
    t.w_stride = (size_t)(2 * p.I * p.H);
    t.w_bytes = (uint32_t)(2 * p.I * p.H);
    t.ws = c.s_gate_up;
    t.ws_stride = (size_t)(2 * IB * HB);
    t.H = (int)p.H;
    t.I = (int)p.I;
    t.HB = (int)HB;
    t.IB = (int)IB;
    t.E = (int)p.E;
    t.first = (int)c.first;
    t.topk = (int)p.topk;
    t.h = h32;
    t.out = c.out;
    t.out_f32 = c.out_f32;
    hipLaunchKernelGGL((f8_row_kernel<true, 14>), dim3((unsigned)(p.I / 8), (unsigned)p.topk), dim3(256), 0, s, t);
    int rc = (int)hipGetLastError();
    if (rc) return rc;
    t.w = static_cast<const uint8_t*>(c.w_down);
    t.w_stride = (size_t)(p.H * p.I);
    t.w_bytes = (uint32_t)(p.H * p.I);
    t.ws = c.s_down;
    t.ws_stride = (size_t)(HB * IB);
    hipLaunchKernelGGL((f8_token_down_kernel<12>), dim3((unsigned)(p.H / 8)), dim3(256), 0, s, t);
    return (int)hipGetLastError();
  }
  PrepArgs pa{};
  pa.ids = c.ids;
  pa.pairs = (int)p.P;
  pa.E = (int)p.E;
  pa.first = (int)c.first;
  pa.bm = p.gu.bm;
  pa.hdr = hdr;
  pa.perm = perm;
  pa.place = reinterpret_cast<int*>(base + p.place_off);
  pa.q.x = c.x;
  pa.q.rows = p.T;
  pa.q.cols = (int)p.H;
  pa.q.ldx = p.H;
  pa.q.bf16 = 1;
  pa.q.q = x8;
  pa.q.s = xs;
  pa.q.s_row = 1;
  pa.q.s_kb = p.T;
  pa.counts = reinterpret_cast<int*>(base + p.counts_off);
  pa.chunk = p.chunk;
  pa.chunks = p.chunk ? (pa.pairs + p.chunk - 1) / p.chunk : 1;
  const unsigned qgrid = quant_grid(p.T * HB, kPrepThreads / 16);
  if (!p.chunk) {
    hipLaunchKernelGGL(experts_prep_kernel, dim3(1 + qgrid), dim3(kPrepThreads), 0, s, pa);
  } else {
    hipLaunchKernelGGL(experts_count_kernel, dim3((unsigned)pa.chunks + qgrid), dim3(kPrepThreads), 0, s, pa);
    if (int e = (int)hipGetLastError()) return e;
    hipLaunchKernelGGL(experts_place_kernel, dim3((unsigned)pa.chunks), dim3(kPrepThreads), 0, s, pa);
  }
  int rc = (int)hipGetLastError();
  if (rc) return rc;

  F8Args g{};
  g.a = x8;
  g.a_bytes = (uint32_t)(p.T * p.H);
  g.as = xs;
  g.as_row = 1;
  g.as_kb = (int)p.T;
  g.w = static_cast<const uint8_t*>(c.w_gate_up);
  g.w_stride = (size_t)(2 * p.I * p.H);
  g.w_bytes = (uint32_t)(2 * p.I * p.H);
  g.ws = c.s_gate_up;
  g.ws_stride = (size_t)(2 * IB * HB);
  g.K = (int)p.H;
  g.KB = (int)HB;
  g.N = (int)p.I;
  g.nblk = (int)IB;
  g.hdr = hdr;
  g.perm = perm;
  g.topk = (int)p.topk;
  g.ldo = (int)p.I;
  g.kslice = (int)HB;
  const bool stream = p.gu.kind == F8_KIND_STREAM;
  g.out = stream ? static_cast<void*>(h32) : h8;
  g.out_f32 = stream;
  g.hs = hs;
  g.hs_ld = (int)p.P;
  if ((rc = launch_f8<F8_GATE_UP>(p.gu, g, (int)p.max_tiles, s))) return rc;
  const bool short_k = p.dn.kind == F8_KIND_DOWN;
  if (stream && !short_k && (rc = launch_quant_fp8(h32, 0, 1, p.P, p.I, p.I, 1, h8, hs, 1, p.P, s))) return rc;

  F8Args d{};
  d.a = h8;
  d.a_bytes = (uint32_t)(p.P * p.I);
  d.as = hs;
  d.as_row = 1;
  d.as_kb = (int)p.P;
  d.w = static_cast<const uint8_t*>(c.w_down);
  d.w_stride = (size_t)(p.H * p.I);
  d.w_bytes = (uint32_t)(p.H * p.I);
  d.ws = c.s_down;
  d.ws_stride = (size_t)(HB * IB);
  d.K = (int)p.I;
  d.KB = (int)IB;
  d.N = (int)p.H;
  d.nblk = (int)HB;
  d.hdr = hdr;
  d.perm = perm;
  d.topk = (int)p.topk;
  d.out = y;
  d.ldo = (int)p.H;
  d.out_f32 = p.y_f32;
  d.hs_ld = (int)p.P;
  d.yexp = reinterpret_cast<uint8_t*>(base + p.yexp_off);
  d.kslice = (int)IB;
  rc = short_k ? launch_f8_down(p.dn, d, h32, (int)p.max_tiles, s) : launch_f8<F8_DOWN>(p.dn, d, (int)p.max_tiles, s);
  if (rc) return rc;

  CombineArgs ca{};
  ca.y = y;
  ca.yexp = reinterpret_cast<const uint8_t*>(base + p.yexp_off);
  ca.P = (int)p.P;
  ca.place = reinterpret_cast<const int*>(base + p.place_off);
  ca.weights = c.weights;
  ca.out = c.out;
  ca.T = (int)p.T;
  ca.H = (int)p.H;
  ca.topk = (int)p.topk;
  ca.out_f32 = c.out_f32;
  const int64_t n = (p.T * (p.H / 8) + 255) / 256;
  const dim3 cgrid((unsigned)(n > 16384 ? 16384 : n));
  if (p.y_f32) hipLaunchKernelGGL(experts_combine_kernel<true>, cgrid, dim3(256), 0, s, ca);
  else hipLaunchKernelGGL(experts_combine_kernel<false>, cgrid, dim3(256), 0, s, ca);
  return (int)hipGetLastError();
}

}  // namespace smlp
