// prefill_q8.cu -- attention of a chunk of new tokens over an 8-bit paged cache.
//
// What it computes: the chunked prefill of prefill_sm100.cu ("Phase 08" page,
// Concepts: chunked prefill, paged attention; Lab 03 step 4) over the 8-bit
// cache of decode_q8.cu: the element is scale * code, one float32 scale per
// (page, K/V head) of K and of V, and chunk query t of a sequence, at position
// ctx + t, sees keys 0 .. ctx + t (less those behind a window).
//
// How it maps to sm_100a.  The two products run on tcgen05 (kind::f16, f16
// operands, f32 accumulators in TMEM), which takes its B operand from shared
// memory in 16 bits, so the codes are widened on the way there.  Doing that in
// the kernel keeps the cache's traffic at one byte per element; widening the
// cache in a pass of its own would write and read twice that.
//  * Rows: the query heads that share a K/V head are rows of one tile.  A CTA
//    has two tiles of 128 rows, each floor(128 / G) tokens by G heads (G = Hq /
//    Hkv, or a divisor of it up to 128), so a widened tile serves the whole
//    group, and a chunk of a few tokens fills a tile instead of G of them.
//  * 16 warps in four warpgroups:
//      warp 0       allocates TMEM and issues every tcgen05.mma;
//      warps 4-7    widen: each takes two pages of every 128-key tile, copies
//                   their codes to shared memory three tiles ahead, converts them
//                   and stores them into a ring of NST slots in the
//                   128-byte-swizzled layout that the MMAs read;
//      warps 8-11   softmax, correction and epilogue of tile 0, warps 12-15 of
//                   tile 1; before that they bring the tiles' queries to f16.
//  * What bounds it, and what it measured (B200, d = 128, 32 query and 8 K/V heads;
//    cycles by timestamps in the kernel).  16 chunks of 512 tokens after up to 7680,
//    E4M3: 567 us, 938 TFLOP/s or 58 % of the measured bf16 rate, with the SMs at
//    1.81 GHz; 606 us at 1.70 GHz, in a run long enough for the power limit.  An SM
//    has seven CTAs one after another and 219 key tiles.  A key tile takes 3870
//    cycles, in which the tensor cores work 2048, the widening warps all but the 490
//    that they wait for free slots, and a row tile's softmax all but the 820 that it
//    waits for scores: 85 % of the time.  A CTA's start and end take 22600 (4500 for
//    its pages, 11100 for the queries and the first scores, 7000 for the last product
//    and the rows): 15 %.
//    Four sequences of five tokens (20 rows a K/V head) over 8 K to 32 K keys, INT8:
//    72 us, 2.5 TB/s of codes or 38 % of the measured copy rate, at 1.82 GHz.  The
//    longest CTA has 39 key tiles of 2320 cycles, 1160 each for K and V, of which the
//    widening warps wait 130 for a slot: widening is what bounds them.  50 us, and
//    11 us for the CTA's plan, start and end; the rest is launches and the joining.
//  * Exactness.  Codes are exact in f16.  Queries are scaled by a power of two
//    per row before rounding to f16, exact for elements within 2^28 of the
//    row's largest.  The K scale multiplies the f32 scores, per page.  The V
//    scale multiplies P in f32 before it is rounded to f16 (2^-11 of each, against
//    bf16's 2^-8 of the output), relative to the largest of the row's own
//    contributions so far, P times V scale over the keys that it sees: what it does
//    not see, and what it barely attends, moves nothing.  (Terms under 2^-18 of
//    that largest one lose bits, 2^-29 of it at most.  Relative to the largest V
//    scale of the CTA's pages, one later large value took the bits of every row
//    before it; that took 561 us for the 16 chunks above, 945 with ALiBi and 481
//    with d = 64, this 566, 949 and 487.  Scaling the codes on their way
//    costs two roundings, and as much time.)
//  * Few rows and long keys.  A chunk that fits one row tile gives both tiles the
//    same rows and half of the CTA's keys each ("twin"), which overlaps what one
//    tile alone does in turn: 146 us -> 89 us for the 20 rows above, with the
//    even split below.  With at most 32 rows every quarter of a tile's lanes
//    holds all of them and its warp works on a quarter of the columns.  When the
//    row tiles alone leave SMs idle, each tile's keys are split over several
//    CTAs, by each sequence's length, which write normalised partials and their
//    log2-sum-exps to the workspace; a second kernel, scheduled behind the first,
//    joins them.
//  * NaN behind the mask: a masked score is replaced, whatever it was.  In the
//    P V product a zero weight would not cancel a NaN value, so in tiles that
//    some row sees only in part such values enter as zeros and are noted by
//    key; a row that does see a noted key gets NaN in the elements it has one in,
//    as the product gives in the other tiles.  A V scale that is no number makes
//    every element NaN in the rows that see its page.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>

#include <mutex>

#include "common.cuh"
#include "internal.h"

namespace exattn {
namespace {

constexpr int BM = 128;  // rows of a tile
constexpr int BN = 128;  // keys of a tile
constexpr int kPage = 16;
constexpr int kPagesPerTile = BN / kPage;
constexpr int NUM_THREADS = 512;
// Registers a thread by role; the widening of twin tiles holds a whole raw tile.
template <bool kTwin>
struct Regs {
  static constexpr int kMma = kTwin ? 64 : 88, kWiden = kTwin ? 104 : 88, kSoft = 168;
  static_assert(128 * (kMma + kWiden + 2 * kSoft) <= NUM_THREADS * 128,
                "setmaxnreg split must fit the block's launch registers");
};
constexpr int kRankMax = NUM_THREADS;   // sequences ranked by length
constexpr int CHUNK_BYTES = 128 * 128;  // one 128-row x 128-byte swizzle column block
constexpr int kSMs = 148;
constexpr int kScaleRing = 8;  // tiles whose page scales are kept in shared memory
constexpr int kEdge = 4;       // tiles that a row may see in part, at either end of the walk
constexpr float kTop = 4.f;    // log2 of what a row's reference contribution is in f16

template <int D, bool kTwin>
struct Cfg {
  static constexpr int TILE_BYTES = BM * D * 2;  // a Q, K or V tile in f16
  static constexpr int NQ = kTwin ? 1 : 2;       // Q tiles (twin tiles have one)
  static constexpr int NST = (D == 64 ? 8 : 5) - NQ;  // ring slots: what is left
  static constexpr int RAW_BYTES = BN * D;       // a K or V tile in codes
  static constexpr int NRAW = 4;                 // raw slots
  static constexpr int RING_OFF = NQ * TILE_BYTES;
  static constexpr int RAW_OFF = RING_OFF + NST * TILE_BYTES;
  static constexpr int BAR_OFF = RAW_OFF + NRAW * RAW_BYTES;
  static constexpr int SMEM_BYTES = BAR_OFF + 1024 + 1024;  // + 1 KB align slack
  static constexpr uint32_t IDESC_QK =  // as idesc_bf16_f32, with both operand formats 0 (f16)
      idesc_bf16_f32(BM, BN, false, false) & ~((7u << 7) | (7u << 10));
  static constexpr uint32_t IDESC_PV =
      idesc_bf16_f32(BM, D, false, true) & ~((7u << 7) | (7u << 10));
  static_assert(SMEM_BYTES <= 232448 && NST >= 3 && NST <= 8, "fits an SM");
};

struct Shared {
  uint64_t full[8];
  uint64_t empty[8];
  uint64_t q_full[2];
  uint64_t s_full[2];
  uint64_t p_half[2];
  uint64_t p_full[2];
  uint64_t o_half[2];
  uint64_t o_full[2];
  uint64_t mrg_full;  // twin: what tile 1 knows of its rows is published
  uint64_t mma_done;
  alignas(16) float k_scale[kScaleRing][kPagesPerTile];
  alignas(16) float v_scale[kScaleRing][kPagesPerTile];
  unsigned v_bad[2 * kEdge][BN / 32];  // keys of edge tiles with codes that are no numbers
  int any_bad;
  int seq, hkv, edge_hi, edge_0, jlo, jhi;  // of the CTA, for the epilogue's rare reader
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(sizeof(Shared) <= 1024, "fits behind the ring");

struct Params {
  const __nv_bfloat16 *q;
  const uint8_t *k_pages, *v_pages;
  const float *k_scales, *v_scales;
  const int *block_table, *seq_lens, *cu_q;
  __nv_bfloat16 *o;
  float *lse;
  // Split over keys (split): each sequence's first CTA and its parts per work
  // item, [2][S]; and every CTA's rows, normalised, with their log2-sum-exps,
  // [CTA][rows_cap][D] and [CTA][rows_cap].
  int *plan;
  float *o_part, *l2_part;
  const float *slopes;
  unsigned *status;
  int S, Hq, Hkv, T, max_q, max_blocks, num_pages;
  int heads;      // query heads per CTA (rows of a token)
  int tokens;     // tokens per tile: floor(128 / heads)
  int span;       // tokens of a CTA: those of two tiles, or of one (twin)
  int pairs;      // CTAs for max_q tokens
  int split, rows_cap;
  float scale_log2;
  int window;
};

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
  return d;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ __half2 as_h2(uint32_t w) { return *reinterpret_cast<__half2 *>(&w); }
__device__ __forceinline__ uint32_t as_u32(__half2 h) { return *reinterpret_cast<uint32_t *>(&h); }
// 16 bytes from global to shared memory behind this thread's back, or zeros where
// `size` is 0; a group of them is closed, and waited for but for the N newest.
__device__ __forceinline__ void copy_async16(uint32_t dst, const void *src, int size) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(size) : "memory");
}
__device__ __forceinline__ void copy_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// A barrier of the softmax warps alone.
__device__ __forceinline__ void soft_barrier() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred one;\n\t"
      "elect.sync _|one, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, one;\n\t}"
      : "=r"(p));
  return p != 0;
}
// Shared-memory stores of this thread become visible to the tensor core's reads.
__device__ __forceinline__ void fence_async_shared() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Four codes of a word -> two f16x2, exactly (element 0 in the low half of a).
template <int FMT>
__device__ __forceinline__ void widen4(uint32_t w, uint32_t &a, uint32_t &b) {
  if constexpr (FMT == ATTN_KV_E4M3) {
    asm("{ .reg .b16 l, h; mov.b32 {l, h}, %2; cvt.rn.f16x2.e4m3x2 %0, l; cvt.rn.f16x2.e4m3x2 %1, h; }"
        : "=r"(a), "=r"(b)
        : "r"(w));
  } else {
    // The byte, sign flipped, in the mantissa of 1024 is code + 1152.
    const uint32_t u = w ^ 0x80808080u;
    const __half2 bias = as_h2(0x64806480u);
    a = as_u32(__hsub2(as_h2(prmt(u, 0x64646464u, 0x4140u)), bias));
    b = as_u32(__hsub2(as_h2(prmt(u, 0x64646464u, 0x4342u)), bias));
  }
}

// N columns of a score row -> N / 2 f16 pairs of P = 2^(s*c - m), c
// the multiplier of the columns' page, times their page's weight v; returns the
// part of the row sum, which has no weights.
template <int N>
__device__ __forceinline__ float exp_cols(const uint32_t (&sv)[N], const float *c, const float *v,
                                          float m, uint32_t (&pk)[N / 2]) {
  const float2 nm2 = make_float2(-m, -m);
  float2 sum_a = make_float2(0.f, 0.f), sum_b = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const float2 c2 = make_float2(c[i / kPage], c[i / kPage]);
    const float2 x0 = fma2(make_float2(__uint_as_float(sv[i]), __uint_as_float(sv[i + 1])), c2, nm2);
    const float2 x1 = fma2(make_float2(__uint_as_float(sv[i + 2]), __uint_as_float(sv[i + 3])), c2, nm2);
    float2 p0 = make_float2(ex2(x0.x), ex2(x0.y));
    float2 p1 = make_float2(ex2(x1.x), ex2(x1.y));
    sum_a = add2(sum_a, p0);
    sum_b = add2(sum_b, p1);
    const float2 v2 = make_float2(v[i / kPage], v[i / kPage]), z2 = make_float2(0.f, 0.f);
    p0 = fma2(p0, v2, z2);
    p1 = fma2(p1, v2, z2);
    pk[i >> 1] = pack_f16x2(p0.x, p0.y);
    pk[(i >> 1) + 1] = pack_f16x2(p1.x, p1.y);
  }
  return (sum_a.x + sum_a.y) + (sum_b.x + sum_b.y);
}
__device__ __forceinline__ void store_half(uint32_t addr, const uint32_t (&pk)[32]) {
  tmem_st32(addr, pk);
}
// Four columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_st4(uint32_t addr, float a, float b, float c, float d) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr),
               "r"(__float_as_uint(a)), "r"(__float_as_uint(b)), "r"(__float_as_uint(c)), "r"(__float_as_uint(d))
               : "memory");
}
__device__ __forceinline__ float4 tmem_ld4(uint32_t addr) {
  uint32_t r[4];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3])::"memory");
  return make_float4(__uint_as_float(r[0]), __uint_as_float(r[1]), __uint_as_float(r[2]), __uint_as_float(r[3]));
}

// A row's references, log2: m of its scaled scores, for the sum of P, and mv of its
// contributions, scores plus log2 |V scale| of the keys it sees, for P V.  The
// weight of a page's P in f16 is V scale * 2^(m - mv + kTop), taken as two factors
// h: far scales can put the whole outside float32.
__device__ __forceinline__ float half_weight(float m, float mv) {
  return m == -INFINITY ? 0.f : ex2(0.5f * (m - mv + kTop));
}
__device__ __forceinline__ bool finite(float x) { return fabsf(x) <= 3.4028235e38f; }
// log2 |V scale| for the references, at least that of the smallest normal number (a
// page of zeros contributes nothing, but its rows need a finite reference); that
// too for a scale that is no number, whose page counts as zeros.
__device__ __forceinline__ float scale_log2(float v) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(fabsf(v)));
  return finite(v) ? fmaxf(y, -126.f) : -126.f;
}
// Weights of N pages against a row's references, from their V scales v; visible
// columns [lo, hi).  Where a scale is no number its page weighs nothing and a row
// that sees it is poisoned.  A weight may be as large as P is small (their product is
// 2^12 at most, or the reference would have moved): both are taken from the middle of
// float32's range, weights 2^-kLift times and P 2^kLift times as large.  One that is
// still beyond float32 becomes its largest: its P is below 2^-176 of the row's
// largest.  (Without a branch: one around the rare part cost 2 % of the time of 16
// chunks of 512.)
constexpr float kLift = 60.f;
template <int N>
__device__ __forceinline__ void weigh(float (&v)[N], float h, int lo, int hi, bool &poison) {
  const float2 h2 = make_float2(h, h), z2 = make_float2(0.f, 0.f);
  const float2 low2 = make_float2(h * 0x1p-60f, h * 0x1p-60f);  // first: v h may overflow
#pragma unroll
  for (int g = 0; g < N; g += 2) {
    const float2 x = fma2(fma2(make_float2(v[g], v[g + 1]), low2, z2), h2, z2);
    const float w[2] = {x.x, x.y};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const bool number = finite(v[g + k]);
      poison |= !number && lo < kPage * (g + k + 1) && hi > kPage * (g + k);
      v[g + k] = number ? fminf(fmaxf(w[k], -3.4028235e38f), 3.4028235e38f) : 0.f;
    }
  }
}

// A sequence's chunk: rows q0 .. q0 + nq - 1, its last token the n-th.  False
// where the lengths do not fit.
struct Chunk {
  int q0, nq, n, ctx;
};
__device__ __forceinline__ bool chunk_of(const Params &p, int s, Chunk &c) {
  c.q0 = p.cu_q[s];
  const int q1 = p.cu_q[s + 1];
  c.n = p.seq_lens[s];
  const long long nq = static_cast<long long>(q1) - c.q0;  // (a corrupt pair could wrap)
  c.nq = static_cast<int>(nq);
  c.ctx = c.n - c.nq;
  return c.q0 >= 0 && nq >= 0 && nq <= p.max_q && q1 <= p.T && c.n >= nq &&
         c.n <= static_cast<long long>(p.max_blocks) * kPage;
}

// The work item of a CTA of a split call: at most kSMs CTAs share the work items'
// key tiles, an item of `tiles` tiles in ceil(tiles / c) parts with the smallest c
// (found from below) that needs no more CTAs.  Every warp works it out alike.
struct Item {
  int seq, pair, group, part, parts, first;  // first: the sequence's first CTA
};
__device__ __forceinline__ bool plan_of(const Params &p, int cta, int lane, Item &it) {
  constexpr int kMost = (kSMs + 31) / 32;  // a split call has fewer sequences than SMs
  constexpr int kFewest = 4;               // tiles worth a part of its own
  const int groups = p.Hq / p.heads;
  int items[kMost], tiles[kMost];
  int total = 0;
#pragma unroll
  for (int k = 0; k < kMost; ++k) {
    const int s = k * 32 + lane;
    items[k] = 0;
    tiles[k] = 1;
    if (s < p.S) {
      Chunk c;
      if (!chunk_of(p, s, c)) {
        items[k] = 1;  // (to say so)
      } else if (c.nq > 0) {
        items[k] = (c.nq + p.span - 1) / p.span * groups;
        tiles[k] = (c.n + BN - 1) / BN;
        if (p.window > 0) tiles[k] = min(tiles[k], (min(p.window, c.n) + p.span) / BN + 2);
      }
    }
    total += items[k] * tiles[k];
  }
  total = __reduce_add_sync(0xffffffffu, total);
  int c = max(kFewest, (total + kSMs - 1) / kSMs);
  while (true) {
    int n = 0;
#pragma unroll
    for (int k = 0; k < kMost; ++k) n += items[k] * ((tiles[k] + c - 1) / c);
    if (__reduce_add_sync(0xffffffffu, n) <= kSMs) break;
    c += max(1, c >> 4);  // (ends: one part an item is no more than kSMs CTAs)
  }
  int before = 0;
#pragma unroll
  for (int k = 0; k < kMost; ++k) {
    const int parts = (tiles[k] + c - 1) / c, mine = items[k] * parts;
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    const unsigned here = __ballot_sync(0xffffffffu, cta < before + upto);
    if (here) {
      const int src = __ffs(here) - 1;
      it.seq = k * 32 + src;
      it.parts = __shfl_sync(0xffffffffu, parts, src);
      it.first = before + __shfl_sync(0xffffffffu, upto - mine, src);
      const int at = cta - it.first, item = at / it.parts;
      it.part = at - item * it.parts;
      it.pair = item / groups;
      it.group = item - it.pair * groups;
      return true;
    }
    before += __shfl_sync(0xffffffffu, upto, 31);
  }
  return false;
}

// Entry i of the order in which a CTA's `total` K and V tiles (of total / 2 key
// tiles from jlo on) go through the rings: its tensor, key tile and the slot of its
// page scales.  Two row tiles share every key tile: K(s) V(s) in turn.  Twin tiles,
// which hold the same rows, each walk half of the key tiles (n0, and n1 = n0 or
// n0 - 1): K0(0) K1(0), then V0(s) K0(s+1) V1(s) K1(s+1) without those past the ends.
template <bool kTwin>
__device__ __forceinline__ void entry(int i, int jlo, int total, bool &v, int &j, int &slot) {
  int t = 0, s = i >> 1;
  v = i & 1;
  if (kTwin) {
    const int n = total >> 1, n0 = (n + 1) >> 1;
    if (i == total - 1) {  // the last V: of tile 1 where the halves are equal
      t = (n & 1) ^ 1;
      s = n0 - 1;
      v = true;
    } else if (i < 2) {
      t = i;
      s = 0;
      v = false;
    } else {
      t = ((i - 2) >> 1) & 1;
      v = (i & 1) == 0;
      s = ((i - 2) >> 2) + (v ? 0 : 1);
    }
    j = jlo + (t ? n0 : 0) + s;
    slot = (2 * s + t) % kScaleRing;
  } else {
    j = jlo + s;
    slot = s % kScaleRing;
  }
}

template <int D, int FMT, bool kAlibi, bool kTwin>
__global__ void __launch_bounds__(NUM_THREADS, 1) prefill_q8_kernel(const Params p) {
  using C = Cfg<D, kTwin>;
  grid_dependents_launch();  // the joining kernel may be scheduled behind this grid
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t *sRing = smem + C::RING_OFF;
  Shared *sh = reinterpret_cast<Shared *>(smem + C::BAR_OFF);
  volatile int *abort_flag = &sh->abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // ---- work item.  A split call's by its plan; else the longest sequence first,
  // its last (heaviest) pair first, so that the last wave holds the short ones.
  // Past kRankMax sequences the order stays as given.
  const int groups = p.Hq / p.heads;  // head groups of a token
  const int lin = static_cast<int>(blockIdx.x);
  int seq, pair, group, part = 0, parts = 1;
  if (p.split) {
    Item it;
    if (!plan_of(p, lin, lane, it)) return;
    seq = it.seq;
    pair = it.pair;
    group = it.group;
    part = it.part;
    parts = it.parts;
    if (lin == it.first && threadIdx.x == 0) {
      p.plan[seq] = it.first;
      p.plan[p.S + seq] = it.parts;
    }
  } else {
    const int per_seq = p.pairs * groups;
    const int rank_of = lin / per_seq, rem = lin - rank_of * per_seq;
    pair = p.pairs - 1 - rem / groups;
    group = rem % groups;
    seq = rank_of;
    if (p.S > 1 && p.S <= kRankMax) {
      int *s_len = reinterpret_cast<int *>(smem);  // (where the queries come later)
      int &s_seq = s_len[kRankMax];
      const int t = static_cast<int>(threadIdx.x);
      if (t < p.S) s_len[t] = p.seq_lens[t];
      __syncthreads();
      if (t < p.S) {
        const int nt = s_len[t];
        int rank = 0;
        for (int u = 0; u < p.S; ++u) rank += (s_len[u] > nt) || (s_len[u] == nt && u < t);
        if (rank == rank_of) s_seq = t;
      }
      __syncthreads();
      seq = s_seq;
      __syncthreads();
    }
  }
  Chunk ck;
  if (!chunk_of(p, seq, ck)) {
    if (threadIdx.x == 0 && pair == 0 && group == 0 && part == 0) atomicOr(p.status, ATTN_DEV_BAD_PAGE);
    return;
  }
  const int tok0 = pair * p.span;  // first token of tile 0 (and, twin, of tile 1)
  if (tok0 >= ck.nq) return;
  const int h0 = group * p.heads;                            // first query head
  const int hkv = h0 / (p.Hq / p.Hkv);
  const bool rows1 = !kTwin && tok0 + p.tokens < ck.nq;      // tile 1 has rows of its own
  // Key tiles [js_t, je_t) of each row tile.
  int je0 = (ck.ctx + min(tok0 + p.tokens, ck.nq) - 1) / BN + 1;
  int je1 = rows1 ? (ck.ctx + min(tok0 + 2 * p.tokens, ck.nq) - 1) / BN + 1 : 0;
  int js0 = p.window > 0 ? max(0, ck.ctx + tok0 - p.window + 1) / BN : 0;
  int js1 = p.window > 0 && rows1 ? max(0, ck.ctx + tok0 + p.tokens - p.window + 1) / BN : 0;
  // Tiles from edge_hi on, and (with a window) the first few from edge_0, hold
  // keys that some row of this CTA does not see.  At most kEdge of each: the rows
  // span at most 256 positions.
  const int edge_hi = (ck.ctx + tok0 + 1) / BN;
  const int edge_0 = js0;
  int jlo = js0, jhi = max(je0, je1);
  if (parts > 1) {  // this CTA's part of them
    const int n = jhi - jlo, first = jlo;
    jlo = first + static_cast<int>(static_cast<long long>(n) * part / parts);
    jhi = first + static_cast<int>(static_cast<long long>(n) * (part + 1) / parts);
    js0 = max(js0, jlo);
    js1 = max(js1, jlo);
    je0 = min(je0, jhi);
    je1 = min(je1, jhi);
  }
  if (kTwin) {
    js0 = jlo;
    je0 = js1 = jlo + (jhi - jlo + 1) / 2;
    je1 = jhi;
  }
  const int total = 2 * (jhi - jlo);  // K and V tiles of the walk
  // The first page that a row sees: those before it may have been given back.
  const int pg_first = p.window > 0 ? max(0, ck.ctx + tok0 - p.window + 1) / kPage : 0;
  // Twin tiles with at most a warp of rows: every quarter of a tile's lanes holds
  // all of them, and takes a quarter of its columns.
  const int rows_here = min(p.span, ck.nq - tok0) * p.heads;
  const bool few = kTwin && rows_here <= 32;

  // ---- every page of those tiles that a row sees must be in the pool.
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NST; ++i) {
      mbar_init(&sh->full[i], 128);
      mbar_init(&sh->empty[i], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&sh->q_full[t], BM);
      mbar_init(&sh->s_full[t], 1);
      mbar_init(&sh->p_half[t], BM);
      mbar_init(&sh->p_full[t], BM);
      mbar_init(&sh->o_half[t], 1);
      mbar_init(&sh->o_full[t], 1);
    }
    mbar_init(&sh->mrg_full, BM);
    mbar_init(&sh->mma_done, 1);
    sh->abort_flag = 0;
    sh->any_bad = 0;
    sh->seq = seq;
    sh->hkv = hkv;
    sh->edge_hi = edge_hi;
    sh->edge_0 = edge_0;
    sh->jlo = jlo;
    sh->jhi = jhi;
    fence_mbar_init();
  }
  if (threadIdx.x < 2 * kEdge * (BN / 32)) (&sh->v_bad[0][0])[threadIdx.x] = 0;
  __syncthreads();
  {
    const int pg_end = min(jhi * kPagesPerTile, (ck.n + kPage - 1) / kPage);
    bool bad = false;
    for (int i = max(jlo * kPagesPerTile, pg_first) + static_cast<int>(threadIdx.x); i < pg_end; i += NUM_THREADS) {
      const int pid = p.block_table[static_cast<size_t>(seq) * p.max_blocks + i];
      bad |= pid < 0 || pid >= p.num_pages;
    }
    if (__syncthreads_or(bad) || jlo >= jhi) {
      // NaN rows for a bad page; nothing (weight zero) for a part without keys.
      const bool none = jlo >= jhi;
      if (!none && threadIdx.x == 0) atomicOr(p.status, ATTN_DEV_BAD_PAGE);
      const float fill = none ? 0.f : NAN;
      const int ntok = min(p.span, ck.nq - tok0);
      for (int i = threadIdx.x; i < ntok * p.heads * D; i += NUM_THREADS) {
        const int c = i % D, r = i / D;
        if (!p.split) {
          const size_t row = static_cast<size_t>(ck.q0 + tok0 + r / p.heads) * p.Hq + h0 + r % p.heads;
          p.o[row * D + c] = __float2bfloat16_rn(fill);
          if (c == 0) p.lse[row] = fill;
        } else {
          const size_t row = static_cast<size_t>(lin) * p.rows_cap + r;
          p.o_part[row * D + c] = fill;
          if (c == 0) p.l2_part[row] = none ? -INFINITY : fill;
        }
      }
      return;
    }
  }
  if (warp == 0) {
    tmem_alloc(&sh->tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh->tmem_base;

  if (warp < 4) {
    // ================================================================== MMA
    regs_dec<Regs<kTwin>::kMma>();
    if (warp == 0) {
      // The whole warp walks the schedule and one elected lane issues: with the
      // control flow uniform, the descriptors stay in uniform registers.  (One
      // lane alone took 110-160 cycles an MMA, more than the 64 it runs for: 680
      // us for the 16 chunks of 512, against 586 this way.)
      const bool one = elect_one();
      const uint32_t ring_base = smem_u32(sRing);
      auto slot_of = [](int i) { return i % C::NST; };
      auto wait_full = [&](int i) {
        return mbar_wait(&sh->full[i % C::NST], (i / C::NST) & 1, abort_flag, p.status);
      };
      const uint64_t qdesc0 = sdesc_sw128(smem_u32(smem), 16, 1024);
      const uint64_t kdesc0 = sdesc_sw128(ring_base, 16, 1024);
      const uint64_t vdesc0 = sdesc_sw128(ring_base, CHUNK_BYTES, 1024);
      auto issue_s = [&](int t, int kidx) {  // S_t = Q_t K^T
        const uint64_t qd = qdesc0 + (((kTwin ? 0 : t) * C::TILE_BYTES) >> 4);
        const uint64_t kd = kdesc0 + ((slot_of(kidx) * C::TILE_BYTES) >> 4);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t off = ((ks >> 2) * CHUNK_BYTES + (ks & 3) * 32) >> 4;
          if (one) mma_ss(tmem + t * 128, qd + off, kd + off, C::IDESC_QK, ks > 0);
        }
        if (one) tc_commit(&sh->s_full[t]);
      };
      // O_t (+)= P_t V, in halves of 64 keys as their P comes; st: step of the tile.
      auto issue_pv = [&](int t, int vidx, int st) {
        const uint64_t vd = vdesc0 + ((slot_of(vidx) * C::TILE_BYTES) >> 4);
        if (!mbar_wait(&sh->p_half[t], st & 1, abort_flag, p.status)) return false;
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < BN / 32; ++ks)
          if (one)
            mma_ts(tmem + 256 + t * 128, tmem + t * 128 + ks * 8, vd + ((ks * 16 * 128) >> 4),
                   C::IDESC_PV, (st > 0 || ks > 0) ? 1u : 0u);
        if (one) tc_commit(&sh->o_half[t]);
        if (!mbar_wait(&sh->p_full[t], st & 1, abort_flag, p.status)) return false;
        tc_fence_after();
#pragma unroll
        for (int ks = BN / 32; ks < BN / 16; ++ks)
          if (one)
            mma_ts(tmem + 256 + t * 128, tmem + t * 128 + ks * 8, vd + ((ks * 16 * 128) >> 4),
                   C::IDESC_PV, 1u);
        if (one) tc_commit(&sh->o_full[t]);
        return true;
      };
      bool ok = wait_full(0);
      if (ok && js0 < je0) ok = mbar_wait(&sh->q_full[0], 0, abort_flag, p.status);
      if (!kTwin && ok && js1 < je1) ok = mbar_wait(&sh->q_full[1], 0, abort_flag, p.status);
      if constexpr (kTwin) {
        // Each entry feeds one product and is released right behind it.
        const int n0 = je0 - js0, n1 = je1 - js1;
        int e = 0;
        auto release = [&]() {
          if (one) tc_commit(&sh->empty[slot_of(e)]);
          ++e;
        };
        if (ok) {
          tc_fence_after();
          issue_s(0, e);
          release();
          if (n1 > 0 && (ok = wait_full(e))) {
            tc_fence_after();
            issue_s(1, e);
            release();
          }
        }
        for (int st = 0; ok && st < n0; ++st) {
          if (!(ok = wait_full(e) && issue_pv(0, e, st))) break;
          release();
          if (st + 1 < n0) {
            if (!(ok = wait_full(e))) break;
            tc_fence_after();
            issue_s(0, e);  // behind PV0(st), which read the P that lies over S0
            release();
          }
          if (st < n1) {
            if (!(ok = wait_full(e) && issue_pv(1, e, st))) break;
            release();
          }
          if (st + 1 < n1) {
            if (!(ok = wait_full(e))) break;
            tc_fence_after();
            issue_s(1, e);
            release();
          }
        }
      } else {
        // Tile j sits at ring index 2 * (j - jlo) (K) and one behind (V).
        auto has = [&](int t, int j) {
          return t == 0 ? (j >= js0 && j < je0) : (j >= js1 && j < je1);
        };
        if (ok) {
          tc_fence_after();
          if (has(0, jlo)) issue_s(0, 0);
          if (has(1, jlo)) issue_s(1, 0);
          if (one) tc_commit(&sh->empty[slot_of(0)]);
        }
        for (int rj = 0; ok && rj < jhi - jlo; ++rj) {
          const int j = jlo + rj;
          const bool more = j + 1 < jhi;
          if (!(ok = wait_full(2 * rj + 1))) break;
          if (more && !(ok = wait_full(2 * rj + 2))) break;
          if (has(0, j) && !(ok = issue_pv(0, 2 * rj + 1, j - js0))) break;
          // P_t(j) lies over S_t: the MMAs of one thread run in order, so S_t(j+1)
          // is written only after P_t(j) has been read.
          if (more && has(0, j + 1)) issue_s(0, 2 * rj + 2);
          if (has(1, j) && !(ok = issue_pv(1, 2 * rj + 1, j - js1))) break;
          if (one) tc_commit(&sh->empty[slot_of(2 * rj + 1)]);
          if (more && has(1, j + 1)) issue_s(1, 2 * rj + 2);
          if (more && one) tc_commit(&sh->empty[slot_of(2 * rj + 2)]);
        }
      }
      // Every MMA issued above must finish before TMEM is released.
      if (one) tc_commit(&sh->mma_done);
      mbar_wait_drain(&sh->mma_done, 0, p.status);
    }
  } else if (warp < 8) {
    // =============================================================== widening
    regs_dec<Regs<kTwin>::kWiden>();
    const int w = warp - 4;
    constexpr int LPR = D / 16;         // lanes per row
    constexpr int RPP = 32 / LPR;       // rows per 512-byte pass
    constexpr int PASSES = kPage / RPP; // passes per page
    // A lane takes 16 columns: two 16-byte pieces of a 128-byte row of f16.  The
    // second column block (d = 128) lies a multiple of all banks behind the
    // first, so its lanes take the other row of each pair: the swizzle then
    // sends the eight lanes of a store to eight different bank groups.
    const int piece = lane % LPR;
    const int blk = piece >> 2, k0 = (piece & 3) * 2;
    const int row = (lane / LPR) ^ blk;
    const int from = w * (2 * kPage * D) + row * D + piece * 16;  // in a raw tile
    // One lane's 16 codes as two 16-byte pieces, to row r of the tile at dst.
    auto put = [&](uint8_t *dst, int r, const uint4 &a, const uint4 &b) {
      uint8_t *line = dst + blk * CHUNK_BYTES + r * 128;
      const int x = r & 7;
      *reinterpret_cast<uint4 *>(line + ((k0 ^ x) << 4)) = a;
      *reinterpret_cast<uint4 *>(line + (((k0 + 1) ^ x) << 4)) = b;
    };
    // A lane's share of a raw tile, unscaled.  The compiler keeps loads and stores
    // of shared memory in order, so that one load at a time waits for the store
    // before it; twin tiles, where this is what bounds the kernel, load all of it
    // first (200 of 900 cycles a tile less when it was brought in; beside two busy
    // softmaxes that gained nothing: 560 us against 549 for 16 chunks of 512).
    auto widen = [&](const uint8_t *src, uint8_t *dst) {
      constexpr int A = kTwin ? 2 * PASSES : 1;
#pragma unroll
      for (int u0 = 0; u0 < 2 * PASSES; u0 += A) {
        uint4 c[A];
#pragma unroll
        for (int u = 0; u < A; ++u) c[u] = *reinterpret_cast<const uint4 *>(src + (u0 + u) * 512);
#pragma unroll
        for (int u = 0; u < A; ++u) {
          uint4 a, b;
          widen4<FMT>(c[u].x, a.x, a.y);
          widen4<FMT>(c[u].y, a.z, a.w);
          widen4<FMT>(c[u].z, b.x, b.y);
          widen4<FMT>(c[u].w, b.z, b.w);
          put(dst, 2 * w * kPage + (u0 + u) * RPP + row, a, b);
        }
      }
    };
    // This warp's two pages of a tile: lane 2e + u holds the number of page u of
    // entry e of a round of 16, and its scales (with K: the softmax applies both).
    // Numbers are read two rounds ahead and scales one, so that neither's latency
    // is waited for.
    const int *table = p.block_table + static_cast<size_t>(seq) * p.max_blocks;
    auto page_of = [&](int i0) {
      const int i = i0 + (lane >> 1);
      if (i >= total) return -1;
      bool v;
      int j, slot;
      entry<kTwin>(i, jlo, total, v, j, slot);
      const int pg = j * kPagesPerTile + 2 * w + (lane & 1);
      return pg >= pg_first && pg * kPage < ck.n ? table[pg] : -1;
    };
    auto scales_of = [&](int i0, int pid) {
      bool v;
      int j, slot;
      float2 x = make_float2(0.f, 0.f);
      if (pid < 0) return x;
      entry<kTwin>(i0 + (lane >> 1), jlo, total, v, j, slot);
      if (v) return x;
      const size_t slice = static_cast<size_t>(pid) * p.Hkv + hkv;
      x.x = p.k_scales[slice];
      x.y = p.v_scales[slice];
      return x;
    };
    int pid = page_of(0), pid1 = page_of(16);  // of entry i's round, and the next
    float2 scale = scales_of(0, pid), scale1 = make_float2(0.f, 0.f);
    int pid2 = -1;
    // Copies this lane's bytes of entry i of the round that `pids` is of into its
    // raw slot: only this lane reads them, so its own wait is all they need.
    // Slots of pages before or behind the keys get zeros.  (Bulk copies of the 2 KB
    // slices, by two warps of their own, went at 12.6 bytes a cycle and SM, and
    // bounded calls of few rows: 73 us against 70 for 20 rows over 8 K to 32 K keys.)
    auto copy = [&](int i, int pids) {
      if (i < total) {
        bool v;
        int j, slot;
        entry<kTwin>(i, jlo, total, v, j, slot);
        const uint8_t *pool = v ? p.v_pages : p.k_pages;
        const uint32_t dst = smem_u32(smem + C::RAW_OFF + (i % C::NRAW) * C::RAW_BYTES + from);
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const int pg = __shfl_sync(0xffffffffu, pids, 2 * (i & 15) + g);
          const uint8_t *src = pool + (static_cast<size_t>(max(pg, 0)) * p.Hkv + hkv) * (kPage * D) +
                               row * D + piece * 16;
#pragma unroll
          for (int u = 0; u < PASSES; ++u)
            copy_async16(dst + (g * PASSES + u) * 512, src + u * 512, pg < 0 ? 0 : 16);
        }
      }
      copy_async_commit();
    };
    auto done = [&](int i) {
      fence_async_shared();
      mbar_arrive(&sh->full[i % C::NST]);
    };
    for (int i = 0; i < C::NRAW - 1; ++i) copy(i, pid);
    for (int i = 0; i < total; ++i) {
      if ((i & 15) == 0) {
        if (i > 0) {
          pid = pid1;
          pid1 = pid2;
          scale = scale1;
        }
        scale1 = scales_of(i + 16, pid1);
        pid2 = page_of(i + 32);
      }
      copy(i + C::NRAW - 1, ((i + C::NRAW - 1) >> 4) == (i >> 4) ? pid : pid1);
      bool v;
      int j, scale_slot;
      entry<kTwin>(i, jlo, total, v, j, scale_slot);
#ifdef EXATTN_TEST_WITHHOLD
      // Test build only: stop before ring index EXATTN_TEST_WITHHOLD, so that the
      // consumers' waits run out.
      if (i == EXATTN_TEST_WITHHOLD) break;
#endif
      // The ring's slot is free, and (of this lane) entry i has come.
      const bool ok = i < C::NST || mbar_wait(&sh->empty[i % C::NST], (i / C::NST - 1) & 1, abort_flag, p.status);
      if (!__all_sync(0xffffffffu, ok)) break;
      copy_async_wait<C::NRAW - 1>();
      // (A scale slot comes round after eight tiles; the ring holds at most four
      // between here and the softmax.)
      if (!v && (lane >> 1) == (i & 15)) {
        sh->k_scale[scale_slot][2 * w + (lane & 1)] = scale.x;
        sh->v_scale[scale_slot][2 * w + (lane & 1)] = scale.y;
      }
      uint8_t *dst = sRing + (i % C::NST) * C::TILE_BYTES;
      widen(smem + C::RAW_OFF + (i % C::NRAW) * C::RAW_BYTES + from, dst);
      // V tiles that some row sees only in part: their slot in v_bad, or -1.  (An
      // INT8 code is always a number.)
      const int edge = FMT != ATTN_KV_E4M3 || !v ? -1
                       : j >= edge_hi            ? min(j - edge_hi, kEdge - 1)
                       : p.window > 0 && j - edge_0 < kEdge ? kEdge + j - edge_0 : -1;
      if (edge >= 0) {
        // What this lane stored, again: codes that are no numbers leave.
#pragma unroll 1
        for (int u = 0; u < 2 * PASSES; ++u) {
          const int r = 2 * w * kPage + u * RPP + row;
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            uint32_t *at = reinterpret_cast<uint32_t *>(dst + blk * CHUNK_BYTES + r * 128 + (((k0 + h) ^ (r & 7)) << 4));
            bool bad = false;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint32_t f = at[e];
              if ((f & 0x7c00u) == 0x7c00u) { f &= 0xffff0000u; bad = true; }
              if ((f & 0x7c000000u) == 0x7c000000u) { f &= 0xffffu; bad = true; }
              if (bad) at[e] = f;
            }
            if (bad) {
              atomicOr(&sh->v_bad[edge][r >> 5], 1u << (r & 31));
              sh->any_bad = 1;
            }
          }
        }
      }
      done(i);
    }
    copy_async_wait<0>();  // no copy may still be on its way when the CTA exits
  } else {
    // ====================================================== softmax / epilogue
    regs_inc<Regs<kTwin>::kSoft>();
    const int t = (warp - 8) >> 2;   // row tile of this warpgroup
    const int quarter = warp & 3;    // TMEM lane quarter this warp may access
    const int r = quarter * 32 + lane;
    const int rr = few ? lane : r;   // row of this thread
    const int tl = rr / p.heads;     // token of the tile; rows behind tokens * heads are idle
    const int tok = tok0 + (kTwin ? 0 : t * p.tokens) + tl;
    const int hq = h0 + rr - tl * p.heads;
    const bool valid = tl < p.tokens && tok < ck.nq;
    const int jst = t == 0 ? js0 : js1, jen = t == 0 ? je0 : je1;
    const int nt = jen - jst;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t s_addr = tmem + lane_off + t * 128;
    const uint32_t o_addr = tmem + lane_off + 256 + t * 128;
    const size_t out_row = static_cast<size_t>(ck.q0 + (valid ? tok : 0)) * p.Hq + hq;
    float c_row = p.scale_log2;  // from a raw score to log2 units, but for the page's K scale
    if (nt > 0) {
      // This row of Q to f16, its largest element in [2^14, 2^15).  (Twin tiles
      // have one Q tile, which tile 0's threads fill.)
      uint4 u[D / 8];
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        u[i] = valid ? __ldg(reinterpret_cast<const uint4 *>(p.q + out_row * D) + i) : make_uint4(0, 0, 0, 0);
        top = __vmaxu2(top, __vmaxu2(__vmaxu2(u[i].x & 0x7fff7fffu, u[i].y & 0x7fff7fffu),
                                     __vmaxu2(u[i].z & 0x7fff7fffu, u[i].w & 0x7fff7fffu)));
      }
      top = max(top & 0xffffu, top >> 16);
      int ex = 0;
      if (top > 0 && top < 0x7f80u) ex = min(100, max(-113, 14 - (static_cast<int>(top >> 7) - 127)));
      const float up = __uint_as_float(static_cast<uint32_t>(127 + ex) << 23);
      c_row *= __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
      uint8_t *line = smem + t * C::TILE_BYTES + r * 128;
      if (!kTwin || t == 0) {
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          const uint32_t in[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
          uint32_t f[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            f[e] = pack_f16x2(__uint_as_float(in[e] << 16) * up, __uint_as_float(in[e] & 0xffff0000u) * up);
          *reinterpret_cast<uint4 *>(line + (i >> 3) * CHUNK_BYTES + (((i & 7) ^ (r & 7)) << 4)) =
              make_uint4(f[0], f[1], f[2], f[3]);
        }
        fence_async_shared();
        mbar_arrive(&sh->q_full[t]);
      }
    }
    const float slope2 = kAlibi && valid ? p.slopes[hq] * 1.4426950408889634f : 0.f;
    // A warp without a row of its own (a chunk of a few tokens) only hands on.
    const bool idle = !__any_sync(0xffffffffu, valid);
    float m = -INFINITY, mv = -INFINITY;  // references (see half_weight)
    float h = 0.f;                        // half_weight(m, mv)
    float l = 0.f;
    bool poison = false;  // the row sees a page whose V scale is no number
    bool ok = true;
    if (few) {
      // The softmax of this thread's row over columns 32 * quarter .. of every
      // tile, with a reference and a sum of its own; P is zero in the others.
      // Else as below.
      const int c0 = 32 * quarter;
      for (int jj = 0; jj < nt; ++jj) {
        const int j = jst + jj;
        const int hi = min(min(BN, ck.n - j * BN), ck.ctx + tok - j * BN + 1) - c0;
        const int lo = (p.window > 0 ? ck.ctx + min(tok, ck.nq - 1) - p.window + 1 - j * BN : 0) - c0;
        const bool masked = !__all_sync(0xffffffffu, lo <= 0 && hi >= 32);
        ok = mbar_wait(&sh->s_full[t], jj & 1, abort_flag, p.status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        uint32_t sv[32], pk[16];
        tmem_ld32(s_addr + c0, sv);
        const int slot = (2 * jj + t) % kScaleRing;
        const float2 ks = *reinterpret_cast<const float2 *>(&sh->k_scale[slot][2 * quarter]);
        const float2 vs = *reinterpret_cast<const float2 *>(&sh->v_scale[slot][2 * quarter]);
        const float cp[2] = {ks.x * c_row, ks.y * c_row};
        tmem_ld_wait(sv);
        const float rb = kAlibi ? slope2 * static_cast<float>(j * BN + c0 - (ck.ctx + tok)) : 0.f;
        float m0 = -INFINITY, m1 = -INFINITY;  // of either page
#pragma unroll
        for (int i = 0; i < kPage; ++i) {
#pragma unroll
          for (int k = i; k < 2 * kPage; k += kPage) {
            float x = __uint_as_float(sv[k]) * cp[k / kPage];
            if (kAlibi) x += fmaf(slope2, static_cast<float>(k), rb);
            if (masked && (k < lo || k >= hi)) x = -INFINITY;
            sv[k] = __float_as_uint(x);
          }
          m0 = fmaxf(m0, __uint_as_float(sv[i]));
          m1 = fmaxf(m1, __uint_as_float(sv[i + kPage]));
        }
        const float m_new = fmaxf(m, fmaxf(m0, m1));
        const float mv_new = fmaxf(mv, fmaxf(m0 + scale_log2(vs.x), m1 + scale_log2(vs.y)));
        if (m_new > m + 8.0f) {
          l *= ex2(m - m_new);
          m = m_new;
        }
        const bool resc = mv_new > mv + 8.0f;
        const float alpha = resc ? ex2(mv - mv_new) : 1.0f;
        if (resc) mv = mv_new;
        if (jj > 0 && __any_sync(0xffffffffu, resc)) {
#pragma unroll 1
          for (int cc = 0; cc < D / 32; ++cc) {
            uint32_t ov[32];
            tmem_ld32(o_addr + cc * 32, ov);
            tmem_ld_wait(ov);
#pragma unroll
            for (int i = 0; i < 32; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
            tmem_st32(o_addr + cc * 32, ov);
          }
        }
        float vp[2] = {vs.x, vs.y};
        weigh(vp, half_weight(m, mv), lo, hi, poison);
        const float ones[2] = {1.f, 1.f};
        l = fmaf(exp_cols(sv, ones, vp, (m == -INFINITY ? 0.f : m) - kLift, pk), 0x1p-60f, l);
        const uint32_t zero[16] = {};
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          if (g == quarter) tmem_st16(s_addr + 16 * g, pk);
          else tmem_st16(s_addr + 16 * g, zero);
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&sh->p_half[t]);
        mbar_arrive(&sh->p_full[t]);
      }
    }
    for (int jj = few ? nt : 0; jj < nt; ++jj) {
      const int j = jst + jj;
      // Visible columns [lo, hi) of this row.  (A row without a token takes one
      // that forces no masking on a warp whose real rows need none.)
      const int hi = min(min(BN, ck.n - j * BN), ck.ctx + tok - j * BN + 1);
      const int lo = p.window > 0 ? ck.ctx + min(tok, ck.nq - 1) - p.window + 1 - j * BN : 0;
      const bool masked = !__all_sync(0xffffffffu, lo <= 0 && hi >= BN);
      const bool attempt = !kAlibi && !masked && jj > 0 && __all_sync(0xffffffffu, m != -INFINITY);
      ok = mbar_wait(&sh->s_full[t], jj & 1, abort_flag, p.status);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      if (idle) {
        mbar_arrive(&sh->p_half[t]);
        mbar_arrive(&sh->p_full[t]);
        continue;
      }
      tc_fence_after();
      const int slot = (kTwin ? 2 * jj + t : j - jlo) % kScaleRing;
      // The multipliers of each page's columns.
      float cp[kPagesPerTile];
      {
        const float4 *ks = reinterpret_cast<const float4 *>(sh->k_scale[slot]);
        const float4 a = ks[0], b = ks[1];
        cp[0] = a.x * c_row; cp[1] = a.y * c_row; cp[2] = a.z * c_row; cp[3] = a.w * c_row;
        cp[4] = b.x * c_row; cp[5] = b.y * c_row; cp[6] = b.z * c_row; cp[7] = b.w * c_row;
      }
      auto four = [](const float *at, float *to) {
        const float4 a = *reinterpret_cast<const float4 *>(at);
        to[0] = a.x; to[1] = a.y; to[2] = a.z; to[3] = a.w;
      };
      // The row goes in halves of 64 columns, and the first half's P is handed
      // on while the second is worked on.  P of columns 0-63 lies over S columns
      // 0-31, that of 64-127 over 32-63.
      uint32_t sv[64], pk[32];
      bool first_done = false;  // the first half's P is out, against m as it was
      if (attempt) {
        // An unmasked tile first takes P against the running references as they
        // stand, without looking for its own.  Where a half's sum is at most 255
        // in every row, each of its terms is below 2^8 and the max-first step
        // below would have kept m too; and where that times the weights' sum is at
        // most 2^15 (and so no NaN), no product passes f16's largest.
        tmem_ld64(s_addr, sv);
        // The V scales, which P takes here, as weights against the references.
        float vp[kPagesPerTile];
        four(&sh->v_scale[slot][0], vp);
        four(&sh->v_scale[slot][4], vp + 4);
#pragma unroll
        for (int g = 0; g < kPagesPerTile; g += 2) {
          const float2 h2 = make_float2(h, h), z2 = make_float2(0.f, 0.f);
          const float2 x = fma2(fma2(make_float2(vp[g], vp[g + 1]), h2, z2), h2, z2);
          vp[g] = x.x;
          vp[g + 1] = x.y;
        }
        const float all = ((fabsf(vp[0]) + fabsf(vp[1])) + (fabsf(vp[2]) + fabsf(vp[3]))) +
                          ((fabsf(vp[4]) + fabsf(vp[5])) + (fabsf(vp[6]) + fabsf(vp[7])));
        auto fits = [&](float sum) { return sum <= 255.0f && sum * all <= 32768.0f; };
        tmem_ld_wait64(sv);
        const float l0 = exp_cols(sv, cp, vp, m, pk);
        if (__all_sync(0xffffffffu, fits(l0))) {
          first_done = true;
          tmem_ld64(s_addr + 64, sv);
          store_half(s_addr, pk);
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(&sh->p_half[t]);
          l += l0;
          tmem_ld_wait64(sv);
          const float l1 = exp_cols(sv, cp + 4, vp + 4, m, pk);
          if (__all_sync(0xffffffffu, fits(l1))) {
            l += l1;
            store_half(s_addr + 32, pk);
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(&sh->p_full[t]);
            continue;
          }
        }
      }
      // Max first, over what is not out yet.
      // To scaled scores (log2 units) with the bias; masked ones to -inf,
      // whatever they were.
      const float rb = kAlibi ? slope2 * static_cast<float>(j * BN - (ck.ctx + tok)) : 0.f;
      auto scaled_half = [&](int hf) {
        tmem_ld64(s_addr + 64 * hf, sv);
        tmem_ld_wait64(sv);
#pragma unroll
        for (int i = 0; i < 64; ++i) {
          float x = __uint_as_float(sv[i]) * (hf ? cp[4 + i / kPage] : cp[i / kPage]);
          if (kAlibi) x += fmaf(slope2, static_cast<float>(64 * hf + i), rb);
          sv[i] = __float_as_uint(x);
        }
        if (masked) {
          const int lo_h = lo - 64 * hf, hi_h = hi - 64 * hf;
#pragma unroll
          for (int i = 0; i < 64; ++i)
            if (i < lo_h || i >= hi_h) sv[i] = 0xff800000u;
        }
      };
      float m_new = m, mv_new = mv;
#pragma unroll 1
      for (int hf = first_done; hf < 2; ++hf) {
        scaled_half(hf);
        float vp[4];
        four(&sh->v_scale[slot][4 * hf], vp);
#pragma unroll
        for (int g = 0; g < 4; ++g) {  // a page's columns
          float top = fmaxf(__uint_as_float(sv[16 * g]), __uint_as_float(sv[16 * g + 1]));
#pragma unroll
          for (int i = 16 * g + 2; i < 16 * g + 16; i += 2)
            top = fmax3(top, __uint_as_float(sv[i]), __uint_as_float(sv[i + 1]));
          m_new = fmaxf(m_new, top);
          mv_new = fmaxf(mv_new, top + scale_log2(vp[g]));
        }
      }
      // The references move where they must (by 2^8 or more), and after a miss.
      if (m_new > m + 8.0f || (attempt && m_new > m)) {
        l *= ex2(m - m_new);
        m = m_new;
      }
      const bool resc = mv_new > mv + 8.0f || (attempt && mv_new > mv);
      const float alpha = resc ? ex2(mv - mv_new) : 1.0f;
      if (resc) mv = mv_new;
      h = half_weight(m, mv);
      if (jj > 0 && __any_sync(0xffffffffu, resc)) {
        // Lazy rescale of O.  S(j) being there implies that PV(j-1) is done; of
        // PV(j), the first half may be under way if its P is out.
        if (first_done) {
          ok = mbar_wait(&sh->o_half[t], jj & 1, abort_flag, p.status);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after();
        }
#pragma unroll 1
        for (int cc = 0; cc < D / 32; ++cc) {
          uint32_t ov[32];
          tmem_ld32(o_addr + cc * 32, ov);
          tmem_ld_wait(ov);
#pragma unroll
          for (int i = 0; i < 32; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
          tmem_st32(o_addr + cc * 32, ov);
        }
      }
      // A row that has seen no visible key yet keeps m = -inf; its masked scores
      // must still give P = 0, not -inf - (-inf).
      const float m_use = (m == -INFINITY) ? 0.f : m;
      const float ones[4] = {1.f, 1.f, 1.f, 1.f};
#pragma unroll 1
      for (int hf = first_done; hf < 2; ++hf) {
        scaled_half(hf);
        float vp[4];
        four(&sh->v_scale[slot][4 * hf], vp);
        weigh(vp, h, lo - 64 * hf, hi - 64 * hf, poison);
        l = fmaf(exp_cols(sv, ones, vp, m_use - kLift, pk), 0x1p-60f, l);
        store_half(s_addr + 32 * hf, pk);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(hf ? &sh->p_full[t] : &sh->p_half[t]);
      }
    }
    if (ok && nt > 0) {
      ok = mbar_wait(&sh->o_full[t], (nt - 1) & 1, abort_flag, p.status);
      ok = __all_sync(0xffffffffu, ok);
    }
    // Codes that are no numbers were left out of the edge tiles: the elements that
    // they make NaN in the row of token tk, stored as row `at`, are written over, by
    // reading the row's keys that have one again.  (In the other tiles, which every
    // row sees whole, the product does it.  What this needs of the CTA waits in
    // shared memory: held in registers through the softmax it took every call 2 %.)
    auto spoil = [&](int tk, size_t at) {
      const volatile Shared *cta = sh;
      const int pos = ck.ctx + tk;
#pragma unroll 1
      for (int e = 0; e < 2 * kEdge; ++e) {
        const int j = e < kEdge ? cta->edge_hi + e : cta->edge_0 + e - kEdge;
        if (j < cta->jlo || j >= cta->jhi || (e >= kEdge && j >= cta->edge_hi)) continue;
        const int hi = min(BN, pos - j * BN + 1);
        const int lo = p.window > 0 ? max(0, pos - p.window + 1 - j * BN) : 0;
#pragma unroll 1
        for (int i = lo; i < hi; ++i) {
          if (!(cta->v_bad[e][i >> 5] >> (i & 31) & 1u)) continue;
          const int key = j * BN + i;
          const int pid = p.block_table[static_cast<size_t>(cta->seq) * p.max_blocks + key / kPage];
          const uint8_t *code = p.v_pages + ((static_cast<size_t>(pid) * p.Hkv + cta->hkv) * kPage + key % kPage) * D;
#pragma unroll 1
          for (int c = 0; c < D; ++c) {
            if ((code[c] & 0x7fu) != 0x7fu) continue;
            if (p.split) p.o_part[at * D + c] = NAN;
            else p.o[at * D + c] = __float2bfloat16_rn(NAN);
          }
        }
      }
    };
    if (few) {
      // Eight partial results of every row, over disjoint keys: joined through
      // the ring, which is free once both tiles' products are done.
      soft_barrier();
      float4 *all = reinterpret_cast<float4 *>(sRing);
      const int me = warp - 8;
      all[me * 32 + lane] = make_float4(m, l, poison ? 1.f : 0.f, 0.f);
      soft_barrier();
      float mm = -INFINITY, sum = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 x = all[i * 32 + lane];
        mm = fmaxf(mm, x.x);
        poison |= x.z != 0.f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float4 x = all[i * 32 + lane];
        if (x.y != 0.f) sum += x.y * ex2(x.x - mm);
      }
      const bool use = ok && nt > 0 && l != 0.f;
      // O is relative to 2^(mv - kTop); in two factors, as that may be far from 1.
      const float part = ex2(0.5f * (mv - mm - kTop)), last = part * (poison ? NAN : 1.0f / sum);
      // (A row that sees keys, and none with a score above -inf, is 0 / 0.)
      const float unseen = !p.split && sum == 0.f ? NAN : 0.f;
      constexpr int kRow = D + 4;  // floats; keeps a store's eight lanes in different banks
      float *joint = reinterpret_cast<float *>(sRing + 8 * 32 * sizeof(float4));
      tc_fence_after();
#pragma unroll 1
      for (int cc = 0; cc < D / 32; ++cc) {
        uint32_t ov[32];
        tmem_ld32(o_addr + cc * 32, ov);
        tmem_ld_wait(ov);
        float4 *dst = reinterpret_cast<float4 *>(joint + (me * 32 + lane) * kRow + cc * 32);
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
          float x[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) x[k] = use ? __uint_as_float(ov[i + k]) * part * last : unseen;
          dst[i >> 2] = make_float4(x[0], x[1], x[2], x[3]);
        }
      }
      soft_barrier();
      for (int i = static_cast<int>(threadIdx.x) - 256; i < rows_here * (D / 4); i += 256) {
        const int row = i / (D / 4), c = (i % (D / 4)) * 4;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float4 y = *reinterpret_cast<const float4 *>(joint + (k * 32 + row) * kRow + c);
          x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
        }
        if (!p.split) {
          const int tk = row / p.heads;
          const size_t at = static_cast<size_t>(ck.q0 + tok0 + tk) * p.Hq + h0 + row - tk * p.heads;
          *reinterpret_cast<uint2 *>(p.o + at * D + c) = make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
        } else {
          *reinterpret_cast<float4 *>(p.o_part + (static_cast<size_t>(lin) * p.rows_cap + row) * D + c) = x;
        }
      }
      if (me == 0 && valid) {
        const float l2 = sum != 0.f ? mm + log2f(sum) : -INFINITY;
        if (!p.split) p.lse[out_row] = l2 * 0.6931471805599453f;
        else p.l2_part[static_cast<size_t>(lin) * p.rows_cap + lane] = l2;
      }
      if (FMT == ATTN_KV_E4M3) {
        // The rows are stored.  (Every warp takes the barrier: after a wait that ran
        // out the flag may still change, and they may read it differently.)
        soft_barrier();
        if (me == 0 && valid && *reinterpret_cast<volatile int *>(&sh->any_bad))
          spoil(tok, p.split ? static_cast<size_t>(lin) * p.rows_cap + lane : out_row);
      }
      ok = false;  // nothing more for these warps
    }
    // (l != 0 for a NaN too; 0 for a row that saw no key here: part of them only.)
    bool use0 = nt > 0 && l != 0.f, use1 = false;  // the O tiles that count
    float mv1 = 0.f;
    if (kTwin && !few) {
      // The tiles hold partial results of the same rows over disjoint keys: tile
      // 1's threads publish what they know of their rows in the first columns of
      // its S, which nothing needs any more, and tile 0's, whose lanes are the
      // same, join them.
      if (t == 1) {
        if (ok) {
          tmem_st4(s_addr, m, l, mv, poison ? 1.f : 0.f);
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(&sh->mrg_full);
        }
        ok = false;  // nothing more for this warpgroup
      } else if (ok) {
        ok = __all_sync(0xffffffffu, mbar_wait(&sh->mrg_full, 0, abort_flag, p.status));
        if (ok) {
          tc_fence_after();
          const float4 x = tmem_ld4(s_addr + 128);
          const float mm = fmaxf(m, x.x);
          use1 = x.y != 0.f;
          l = (use0 ? ex2(m - mm) * l : 0.f) + (use1 ? ex2(x.x - mm) * x.y : 0.f);
          m = mm;
          mv1 = x.z;
          poison |= x.w != 0.f;
        }
      }
    }
    if (ok && (nt > 0 || p.split)) {
      tc_fence_after();
      const bool seen = l != 0.f;
      const float inv = poison ? NAN : (seen ? 1.0f / l : 0.f);
      // (A row that sees keys, and none with a score above -inf, is 0 / 0.)
      const float unseen = !p.split && !seen ? NAN : 0.f;
      const float l2 = seen ? m + log2f(l) : -INFINITY;
      // O is relative to 2^(mv - kTop); in two factors, as that may be far from 1.
      const float a0 = ex2(0.5f * (mv - m - kTop)), a1 = ex2(0.5f * (mv1 - m - kTop));
      const float b0 = a0 * inv, b1 = a1 * inv;
      const size_t prow = static_cast<size_t>(lin) * p.rows_cap + (kTwin ? 0 : t * p.tokens * p.heads) + r;
#pragma unroll
      for (int cc = 0; cc < D / 32; ++cc) {
        uint32_t ov[32], ov1[kTwin ? 32 : 1];
        tmem_ld32(o_addr + cc * 32, ov);
        if constexpr (kTwin) tmem_ld32(o_addr + 128 + cc * 32, ov1);
        tmem_ld_wait(ov);
        if constexpr (kTwin) tmem_ld_wait(ov1);
        // (A tile that has seen nothing may hold anything.)
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          float x = use0 ? __uint_as_float(ov[i]) * a0 * b0 : unseen;
          if constexpr (kTwin) x += use1 ? __uint_as_float(ov1[i]) * a1 * b1 : 0.f;
          ov[i] = __float_as_uint(x);
        }
        if (valid && !p.split) {
          uint4 *dst = reinterpret_cast<uint4 *>(p.o + out_row * D + cc * 32);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t pk[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              pk[i] = pack_bf16x2(__uint_as_float(ov[8 * q + 2 * i]), __uint_as_float(ov[8 * q + 2 * i + 1]));
            dst[q] = make_uint4(pk[0], pk[1], pk[2], pk[3]);
          }
        } else if (valid) {
          uint4 *dst = reinterpret_cast<uint4 *>(p.o_part + prow * D + cc * 32);
#pragma unroll
          for (int q = 0; q < 8; ++q) dst[q] = make_uint4(ov[4 * q], ov[4 * q + 1], ov[4 * q + 2], ov[4 * q + 3]);
        }
      }
      if (valid) {
        if (!p.split) p.lse[out_row] = l2 * 0.6931471805599453f;
        else p.l2_part[prow] = l2;
        if (FMT == ATTN_KV_E4M3 && *reinterpret_cast<volatile int *>(&sh->any_bad)) spoil(tok, p.split ? prow : out_row);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of a split call: one warp per (token, query head), weights
// 2^(L_part - L).  Block: token of a sequence's chunk (x), eight heads (y).
constexpr int kJoinWarps = 8;
template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32) prefill_q8_join_kernel(const Params p) {
  grid_dependency_wait();
  const int s = blockIdx.x / p.max_q, tok = blockIdx.x % p.max_q;
  const int h = blockIdx.y * kJoinWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  Chunk ck;
  if (h >= p.Hq || !chunk_of(p, s, ck) || tok >= ck.nq) return;
  const size_t row = static_cast<size_t>(ck.q0 + tok) * p.Hq + h;
  // The CTAs that hold this row, and its place among theirs.
  const int pair = tok / p.span, group = h / p.heads;
  const int parts = p.plan[p.S + s];
  const int cta = p.plan[s] + (pair * (p.Hq / p.heads) + group) * parts;
  const int at = (tok - pair * p.span) * p.heads + h - group * p.heads;
  const size_t slot = static_cast<size_t>(cta) * p.rows_cap + at;
  float top = -INFINITY;
  bool failed = false;
  for (int i = lane; i < parts; i += 32) {
    const float x = p.l2_part[slot + static_cast<size_t>(i) * p.rows_cap];
    failed |= isnan(x);
    top = fmaxf(top, x);
  }
  failed = __any_sync(0xffffffffu, failed);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  constexpr int E = D / 32;  // consecutive elements of this lane
  float acc[E], sum = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  for (int i = 0; i < parts; ++i) {
    const size_t from = slot + static_cast<size_t>(i) * p.rows_cap;
    const float w = ex2(p.l2_part[from] - top);  // NaN where a part failed
    sum += w;
    const float *o = p.o_part + from * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      const float2 v = *reinterpret_cast<const float2 *>(o + e);
      acc[e] += w * v.x;
      acc[e + 1] += w * v.y;
    }
  }
  const float inv = 1.f / sum;
#pragma unroll
  for (int e = 0; e < E; e += 2)
    *reinterpret_cast<uint32_t *>(p.o + row * D + lane * E + e) = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
  // (Scores that are all -inf: O is 0 / 0, and their log-sum-exp -inf.)
  if (lane == 0) p.lse[row] = top == -INFINITY && !failed ? top : (top + log2f(sum)) * 0.6931471805599453f;
}

// How a call is cut: query heads per CTA, tokens per tile and CTA, CTAs.
struct Cut {
  int heads, tokens, span, pairs, rows_cap;
  bool twin, split;
  long long ctas;
};
Cut cut(int S, int Hq, int Hkv, int max_q, int max_blocks) {
  Cut c;
  const int G = Hq / Hkv;
  c.heads = G < BM ? G : BM;  // the fewest equal head groups of at most 128
  while (G % c.heads) --c.heads;
  const int n = G / c.heads;
  c.tokens = BM / c.heads;
  const bool many = max_blocks > kPagesPerTile;  // more than one key tile
  // Chunks that fit one row tile: both tiles take the same rows and half the
  // keys each (both sides measured: see the top of the file).
  c.twin = many && max_q <= c.tokens;
  c.span = c.twin ? c.tokens : 2 * c.tokens;
  c.pairs = (max_q - 1) / c.span + 1;
  c.rows_cap = (max_q < c.span ? max_q : c.span) * c.heads;
  c.ctas = static_cast<long long>(S) * Hkv * n * c.pairs;
  // Fewer work items than SMs: their keys are split over as many CTAs.
  c.split = many && c.ctas < kSMs;
  if (c.split) c.ctas = kSMs;
  return c;
}
size_t plan_bytes(int S) { return (2 * S * sizeof(int) + 255) / 256 * 256; }

template <int D, int FMT, bool kAlibi, bool kTwin>
attn_status_t launch(const Params &p, long long ctas, cudaStream_t stream) {
  using C = Cfg<D, kTwin>;
  // The attribute belongs to the kernel on one device: set once on each.
  constexpr int kMaxDevices = 64;
  static std::mutex mutex;
  static bool set[kMaxDevices] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return ATTN_ERR_CUDA;
  {
    std::lock_guard<std::mutex> lock(mutex);
    if (!set[dev]) {
      if (cudaFuncSetAttribute(prefill_q8_kernel<D, FMT, kAlibi, kTwin>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM_BYTES) != cudaSuccess)
        return ATTN_ERR_CUDA;
      set[dev] = true;
    }
  }
  prefill_q8_kernel<D, FMT, kAlibi, kTwin><<<static_cast<unsigned>(ctas), NUM_THREADS, C::SMEM_BYTES, stream>>>(p);
  if (cudaGetLastError() != cudaSuccess) return ATTN_ERR_CUDA;
  if (!p.split) return ATTN_OK;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.S) * p.max_q, (p.Hq + kJoinWarps - 1) / kJoinWarps);
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, prefill_q8_join_kernel<D>, p) != cudaSuccess) return ATTN_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

template <int D, int FMT>
attn_status_t launch_variant(const Params &p, const Cut &c, cudaStream_t stream) {
  if (p.slopes)
    return c.twin ? launch<D, FMT, true, true>(p, c.ctas, stream) : launch<D, FMT, true, false>(p, c.ctas, stream);
  return c.twin ? launch<D, FMT, false, true>(p, c.ctas, stream) : launch<D, FMT, false, false>(p, c.ctas, stream);
}

}  // namespace

size_t prefill_q8_workspace_bytes(int S, int Hq, int Hkv, int T, int max_q, int d, int max_blocks) {
  const Cut c = cut(S, Hq, Hkv, max_q, max_blocks);
  if (!c.split || T == 0) return 0;
  return plan_bytes(S) + static_cast<size_t>(kSMs) * c.rows_cap * (d + 1) * sizeof(float);
}

attn_status_t launch_prefill_paged_q8(const void *q, const void *k_pages, const void *v_pages,
                                      const float *k_scales, const float *v_scales, int kv_format,
                                      const int *block_table, const int *seq_lens, const int *cu_q,
                                      void *o, float *lse, int S, int Hq, int Hkv, int T, int max_q,
                                      int d, int max_blocks, int num_pages, float scale, int window,
                                      const float *slopes, void *workspace, cudaStream_t stream,
                                      unsigned *status) {
  const Cut c = cut(S, Hq, Hkv, max_q, max_blocks);
  if (c.ctas > 0x7fffffffLL || (Hq + kJoinWarps - 1) / kJoinWarps > 65535 ||
      static_cast<long long>(c.pairs) * (Hq / c.heads) > 0x7fffffffLL ||
      (c.split && static_cast<long long>(S) * max_q > 0x7fffffffLL))
    return ATTN_ERR_INVALID_ARG;
  Params p{};
  p.q = static_cast<const __nv_bfloat16 *>(q);
  p.k_pages = static_cast<const uint8_t *>(k_pages);
  p.v_pages = static_cast<const uint8_t *>(v_pages);
  p.k_scales = k_scales;
  p.v_scales = v_scales;
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.cu_q = cu_q;
  p.o = static_cast<__nv_bfloat16 *>(o);
  p.lse = lse;
  if (c.split) {
    p.plan = static_cast<int *>(workspace);
    p.o_part = reinterpret_cast<float *>(static_cast<char *>(workspace) + plan_bytes(S));
    p.l2_part = p.o_part + static_cast<size_t>(kSMs) * c.rows_cap * d;
  }
  p.slopes = slopes;
  p.status = status;
  p.S = S;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.T = T;
  p.max_q = max_q;
  p.max_blocks = max_blocks;
  p.num_pages = num_pages;
  p.heads = c.heads;
  p.tokens = c.tokens;
  p.span = c.span;
  p.pairs = c.pairs;
  p.split = c.split;
  p.rows_cap = c.rows_cap;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.window = window < max_blocks * kPage ? window : 0;  // (one past every length hides nothing)
  const bool e4m3 = kv_format == ATTN_KV_E4M3;
  if (d == 128)
    return e4m3 ? launch_variant<128, ATTN_KV_E4M3>(p, c, stream) : launch_variant<128, ATTN_KV_INT8>(p, c, stream);
  return e4m3 ? launch_variant<64, ATTN_KV_E4M3>(p, c, stream) : launch_variant<64, ATTN_KV_INT8>(p, c, stream);
}

}  // namespace exattn
