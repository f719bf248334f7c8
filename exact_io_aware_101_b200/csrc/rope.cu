// rope.cu -- rotary positions of queries and keys, with or without an RMS norm
// of each head before them, and the gradients of that.
//
// What it computes.  For a head's row x of d elements at position t, the first
// `rot` elements form rot/2 pairs (x_i, x_{i+rot/2}), or (x_2i, x_{2i+1})
// interleaved, and pair i turns by the angle t * f_i:
//   y_i = F (x_i cos - x'_i sin),   y'_i = F (x_i sin + x'_i cos)
// with F the attention factor; the elements from rot on pass as they are.  The
// map is linear, so its gradient is its transpose: the same turn by -t * f_i,
// again times F.  With a norm, xhat = x * r, r = (mean(x^2) + eps)^(-1/2), and
// the turn acts on w * xhat.  Its gradient, from u = (transposed turn of dy):
//   dw = sum over rows of u * xhat,   dx = r (w u - xhat * mean(w u * xhat)).
//
// What bounds it: HBM.  Every row is read once (in the gradient x and dy) and
// written once, and the arithmetic of a row is about 100 operations per 16
// elements.  Measured (B200): norm and rotation of 4 x 4096 tokens of 40 bf16
// heads, d = 128, 56 us (6.0 TB/s, 92 % of the measured copy rate), its gradient
// 89 us (5.7 TB/s, 87 %), a partial fp32 rotation of 2 x 2047 tokens of 32
// heads, d = 64, 11.0 us (6.2 TB/s), one decode step of 64 tokens 3.3 us, the bare
// bf16 turn of the 4 x 4096 tokens 59 us (5.6 TB/s; interleaved 60).  Half layouts
// that go element by element (below) take twice that: 121 us for 90 of 128 turned,
// 124 with a norm, 207 for its gradient.  So:
//  * One thread holds the same 16 elements (8 pairs) of its rows and walks the
//    heads of one token, q's and then k's: the cosines and sines of its 8 pairs
//    stay in registers, worked out once for all those heads.  LPR = d/16 lanes
//    hold a row, and a norm's two sums are log2(LPR) shuffles.
//  * Each lane moves 16-byte words, and the next rows (one to three) are on their
//    way, packed as they lie in memory, while a row is worked on.  (Four rows loaded
//    and unpacked together took 128 registers: 95 us for 4 x 4096 tokens of 40
//    bf16 heads with norms, and 197 us for the gradient.)  Half layouts whose rot
//    is not a multiple of two such words would put the partner elements at odd
//    addresses: they go element by element.
//  * Angles: t * f_i / 2 pi is taken in 64 bits and reduced to the nearest
//    whole turn there (a far position's angle has no fraction left in 32
//    bits); the remainder, at most half a turn, goes to sincospi in 32 bits.
//    One 64-bit product serves all heads of the token.
//  * Sums, norms and products are float32, rounded once when a row is stored.
//  * The weights' gradients: each thread adds its 16 elements' products over a
//    token's heads in registers and over its tokens in shared memory, the block
//    adds its lanes' sums and writes one row of partial sums, and a second
//    kernel, scheduled behind the first, adds those rows in a fixed order.  No
//    atomics: the result does not depend on the order in which blocks run.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "internal.h"

namespace exattn {
namespace {

constexpr int kThreads = 128;
constexpr int kSMs = 148;
constexpr double kInvTwoPi = 0.15915494309189533577;

enum Mode { kHalf, kPairs, kScalar };   // where a thread's pairs lie (see Slots)
enum Op { kTurn, kNormTurn, kNormTurnBwd };

// One of the two tensors of a call: q or k.
struct Side {
  const void *x, *dy;  // dy: gradient only
  void *y;             // output, or dx
  const void *w;       // norm weights [d]
  long long xb, xh, xn, yb, yh, yn, gb, gh, gn;  // element strides: batch, head, token
  int H;
};

struct RopeParams {
  Side side[2];
  const int *positions;
  long long pos_stride;  // of a batch entry; 0: shared
  const double *inv_freq;
  float *partial;  // gradient: [2][blocks][d], block (x, y) at row y * gridDim.x + x
  long long tokens;
  int N, rot;
  int per_group;  // heads (q's and k's together) of a block
  float factor, sign, eps;
};

// One 16-byte word of elements as floats, and back.
template <typename T>
struct Word {
  static constexpr int L = 16 / sizeof(T);  // elements
  static __device__ __forceinline__ void get(const uint4 &u, float *v) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 2) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      } else {
        v[i] = __uint_as_float(w[i]);
      }
    }
  }
  static __device__ __forceinline__ uint4 put(const float *v) {
    if constexpr (sizeof(T) == 2)
      return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                        pack_bf16x2(v[6], v[7]));
    else
      return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                        __float_as_uint(v[3]));
  }
};
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f32(float *p, float v) { *p = v; }
__device__ __forceinline__ void from_f32(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

// The 16 elements of a row that belong to lane `lane` of its LPR lanes, as 8
// slots (a[j], b[j]).  Slots of a row are numbered 0 .. d/2-1; slot s < rot/2 is
// pair s, and slot s >= rot/2 the two unturned elements 2s and 2s+1.
//  kHalf, kPairs: groups of G slots in a row, group g of all lanes side by side
//  before group g + 1 of any, so that the lanes' 16-byte words lie side by side
//  too.  In the half layout a group that turns is two words rot/2 elements
//  apart (rot/2 a multiple of G, so it turns as a whole), in the interleaved
//  layout every group is one word.  kScalar: slots lane + LPR * j, any rot.
template <typename T, int D, int MODE>
struct Slots {
  static constexpr int LPR = D / 16;
  static constexpr int L = Word<T>::L;
  static constexpr int G = MODE == kPairs ? L / 2 : L;
  static constexpr int W = MODE == kScalar ? 1 : 16 / L;  // words of a row's share
  // A row's share as it was loaded.
  struct Words {
    uint4 w[W];
  };
  struct Single {
    T a[8], b[8];
  };
  using Held = typename std::conditional<MODE == kScalar, Single, Words>::type;
  int lane, half;
  int at[W];  // elements where the words begin
  __device__ __forceinline__ Slots(int lane_, int rot) : lane(lane_), half(rot >> 1) {
#pragma unroll
    for (int w = 0; w < W; ++w) {
      if (MODE == kPairs) at[w] = 2 * slot(w * G);
      else at[w] = w & 1 ? second((w >> 1) * G) : first((w >> 1) * G);
    }
  }
  __device__ __forceinline__ int slot(int j) const {
    return MODE == kScalar ? lane + LPR * j : (j / G) * (G * LPR) + G * lane + j % G;
  }
  __device__ __forceinline__ bool turns(int j) const {
    return (MODE == kHalf ? slot(j - j % G) : slot(j)) < half;
  }
  __device__ __forceinline__ int first(int j) const {  // element of a[j] (half layouts)
    const int s = slot(j);
    if (MODE == kScalar) return s < half ? s : 2 * s;
    return turns(j) ? s : 2 * slot(j - j % G) + j % G;
  }
  __device__ __forceinline__ int second(int j) const {
    const int s = slot(j);
    if (MODE == kScalar) return s < half ? s + half : 2 * s + 1;
    return turns(j) ? s + half : 2 * slot(j - j % G) + G + j % G;
  }
  // The element that slot j's a (which = 0) or b holds.
  __device__ __forceinline__ int element(int j, int which) const {
    if (MODE == kPairs) return 2 * slot(j) + which;
    return which ? second(j) : first(j);
  }
  __device__ __forceinline__ void load(const T *row, Held &r) const {
    if constexpr (MODE == kScalar) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        r.a[j] = row[first(j)];
        r.b[j] = row[second(j)];
      }
    } else {
#pragma unroll
      for (int w = 0; w < W; ++w) r.w[w] = *reinterpret_cast<const uint4 *>(row + at[w]);
    }
  }
  __device__ __forceinline__ void get(const Held &r, float (&a)[8], float (&b)[8]) const {
    if constexpr (MODE == kScalar) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        a[j] = to_f32(r.a[j]);
        b[j] = to_f32(r.b[j]);
      }
    } else if constexpr (MODE == kHalf) {
#pragma unroll
      for (int g = 0; g < 8 / G; ++g) {
        Word<T>::get(r.w[2 * g], a + g * G);
        Word<T>::get(r.w[2 * g + 1], b + g * G);
      }
    } else {
#pragma unroll
      for (int g = 0; g < 8 / G; ++g) {
        float v[L];
        Word<T>::get(r.w[g], v);
#pragma unroll
        for (int i = 0; i < G; ++i) {
          a[g * G + i] = v[2 * i];
          b[g * G + i] = v[2 * i + 1];
        }
      }
    }
  }
  __device__ __forceinline__ void store(T *row, const float (&a)[8], const float (&b)[8]) const {
    if constexpr (MODE == kScalar) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        from_f32(row + first(j), a[j]);
        from_f32(row + second(j), b[j]);
      }
    } else if constexpr (MODE == kHalf) {
#pragma unroll
      for (int g = 0; g < 8 / G; ++g) {
        *reinterpret_cast<uint4 *>(row + at[2 * g]) = Word<T>::put(a + g * G);
        *reinterpret_cast<uint4 *>(row + at[2 * g + 1]) = Word<T>::put(b + g * G);
      }
    } else {
#pragma unroll
      for (int g = 0; g < 8 / G; ++g) {
        float v[L];
#pragma unroll
        for (int i = 0; i < G; ++i) {
          v[2 * i] = a[g * G + i];
          v[2 * i + 1] = b[g * G + i];
        }
        *reinterpret_cast<uint4 *>(row + at[g]) = Word<T>::put(v);
      }
    }
  }
};

// 16 bytes from global to shared memory behind this thread's back; a group of
// them is closed, and waited for but for the N newest.
__device__ __forceinline__ void copy_async16(void *dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Sum over the LPR lanes of a row.
template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Blocks that an SM holds at a time (the registers' limit is set to that), and rows
// on their way while one is worked on.  One block more takes 63 us instead of 56 for
// the norm and 111 instead of 89 for its gradient.  At these limits the bf16 kernels
// spill a little in some layouts: the bare turn 20 bytes (halves) and 40
// (interleaved), single elements 56 with a norm and 76 in its gradient.  The norms'
// rows wait in shared memory, where words lie as they do in global memory; bare turns
// and layouts of single elements hold theirs in registers.
// (In registers: 60 us for the norm and 100 for its gradient instead of 56 and 89,
// 4 x 4096 tokens of 40 bf16 heads.  Staged: 11.4 us for the fp32 turn of 2 x 2047
// tokens instead of 11.0.)
constexpr int blocks_per_sm(int op, int size) {
  return op == kTurn ? 7 : (op == kNormTurn ? (size == 4 ? 5 : 6) : (size == 4 ? 3 : 4));
}
constexpr bool rows_staged(int mode, int op) { return op != kTurn && mode != kScalar; }
constexpr int rows_ahead(int mode, int op, int size) {
  return rows_staged(mode, op) ? (op == kNormTurn ? (size == 4 ? 2 : 3) : (size == 4 ? 1 : 2))
                               : (op == kTurn && mode != kScalar && size == 2 ? 2 : 1);
}

// Block (x, y): group y of the heads, token tiles x, x + gridDim.x, ...
template <typename T, int D, int MODE, int OP>
__global__ void __launch_bounds__(kThreads, blocks_per_sm(OP, sizeof(T))) rope_kernel(const RopeParams p) {
  constexpr int LPR = D / 16, TT = kThreads / LPR;
  constexpr int A = rows_ahead(MODE, OP, sizeof(T));
  constexpr bool kBwd = OP == kNormTurnBwd;
  constexpr bool kStaged = rows_staged(MODE, OP);
  if constexpr (kBwd) grid_dependents_launch();
  using S = Slots<T, D, MODE>;
  const int lane = threadIdx.x % LPR, slot_row = threadIdx.x / LPR;
  const S sl(lane, p.rot);
  const int hb = blockIdx.y * p.per_group, he = hb + p.per_group;
  // Rows on their way: this thread's words of A rows, and of the one at hand.
  constexpr int kTensors = kBwd ? 2 : 1;
  __shared__ uint4 stage[kStaged ? A + 1 : 1][kStaged ? kTensors * S::W : 1][kThreads];
  // Gradient: this thread's sums of its 16 elements' dw, for q and for k.
  __shared__ float sums[kBwd ? 2 : 1][kBwd ? 16 : 1][kThreads];
  if constexpr (kBwd) {
#pragma unroll
    for (int j = 0; j < 16; ++j) sums[0][j][threadIdx.x] = sums[1][j][threadIdx.x] = 0.f;
  }

  for (long long tile = blockIdx.x; tile * TT < p.tokens; tile += gridDim.x) {
    const long long m = tile * TT + slot_row;
    // Lanes without a token take part in the shuffles with the last one's rows.
    const bool live = m < p.tokens;
    const long long mm = live ? m : p.tokens - 1;
    const long long bi = mm / p.N, n = mm - bi * p.N;
    float cs[8], sn[8];
    {
      const double t = static_cast<double>(p.positions[bi * p.pos_stride + n]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        cs[j] = 1.f;
        sn[j] = 0.f;
        if (sl.turns(j)) {
          const double turns = t * (p.inv_freq[sl.slot(j)] * kInvTwoPi);
          float s, c;
          sincospif(2.f * static_cast<float>(turns - rint(turns)), &s, &c);
          cs[j] = c * p.factor;
          sn[j] = s * (p.factor * p.sign);
        }
      }
    }
    // Turns the 8 slots of a row.  (What does not turn is left alone, not turned
    // by cosine 1 and sine 0: an infinity would make its neighbour NaN.)
    auto turn = [&](float (&a)[8], float (&b)[8]) {
#pragma unroll
      for (int g = 0; g < 8; g += S::G) {
        if (MODE == kHalf && !sl.turns(g)) continue;  // here a group turns as a whole
#pragma unroll
        for (int j = g; j < g + S::G; ++j) {
          const float y = a[j] * cs[j] - b[j] * sn[j], z = a[j] * sn[j] + b[j] * cs[j];
          const bool t = MODE == kHalf || sl.turns(j);
          a[j] = t ? y : a[j];
          b[j] = t ? z : b[j];
        }
      }
    };
#pragma unroll 1
    for (int side = 0; side < 2; ++side) {
      const Side &sd = p.side[side];
      const int off = side ? p.side[0].H : 0;
      const int h0 = max(hb - off, 0), h1 = min(he - off, sd.H);
      if (h0 >= h1) continue;
      float wa[8], wb[8];  // norm weights of this lane's elements
      if constexpr (OP != kTurn) {
        typename S::Held w;
        sl.load(static_cast<const T *>(sd.w), w);
        sl.get(w, wa, wb);
      }
      float ga[8], gb[8];  // their gradients, over this token's heads
      if constexpr (kBwd) {
#pragma unroll
        for (int j = 0; j < 8; ++j) ga[j] = gb[j] = 0.f;
      }
      const T *x = static_cast<const T *>(sd.x) + bi * sd.xb + n * sd.xn;
      T *y = static_cast<T *>(sd.y) + bi * sd.yb + n * sd.yn;
      const T *dy = kBwd ? static_cast<const T *>(sd.dy) + bi * sd.gb + n * sd.gn : nullptr;
      // Row h's words to their stage, closed as a group (an empty one past the last).
      auto ahead = [&](int h) {
        if constexpr (kStaged) {
          if (h < h1) {
            uint4(*at)[kThreads] = stage[(h - h0) % (A + 1)];
#pragma unroll
            for (int w = 0; w < S::W; ++w) {
              copy_async16(&at[w][threadIdx.x], x + h * sd.xh + sl.at[w]);
              if constexpr (kBwd) copy_async16(&at[S::W + w][threadIdx.x], dy + h * sd.gh + sl.at[w]);
            }
          }
          copy_async_commit();
        }
      };
      // One row, loaded as r0 (and its gradient g0).  In place, its lanes store after
      // all of them have read it; the rows on their way are other rows.
      auto work = [&](int h, const typename S::Held &r0, const typename S::Held &g0) {
        float a[8], b[8], c[kBwd ? 8 : 1], e[kBwd ? 8 : 1];
        sl.get(r0, a, b);
        if constexpr (kBwd) sl.get(g0, c, e);
        if constexpr (OP == kTurn) {
          turn(a, b);
        } else {
          float ss = 0.f;
#pragma unroll
          for (int j = 0; j < 8; ++j) ss += a[j] * a[j] + b[j] * b[j];
          const float r = __frsqrt_rn(row_sum<LPR>(ss) * (1.f / D) + p.eps);
          if constexpr (OP == kNormTurn) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              a[j] = a[j] * r * wa[j];
              b[j] = b[j] * r * wb[j];
            }
            turn(a, b);
          } else {
            float dot = 0.f;
            turn(c, e);  // u: sign is -1 here
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              a[j] *= r;  // xhat
              b[j] *= r;
              ga[j] += c[j] * a[j];
              gb[j] += e[j] * b[j];
              c[j] *= wa[j];
              e[j] *= wb[j];
              dot += c[j] * a[j] + e[j] * b[j];
            }
            dot = row_sum<LPR>(dot) * (1.f / D);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              a[j] = r * (c[j] - a[j] * dot);
              b[j] = r * (e[j] - b[j] * dot);
            }
          }
        }
        if (live) sl.store(y + h * sd.yh, a, b);
      };
      if constexpr (kStaged) {
#pragma unroll
        for (int i = 0; i < A; ++i) ahead(h0 + i);
        for (int h = h0; h < h1; ++h) {
          // (The stage that row h + A goes to held row h - 1, which has been used.)
          ahead(h + A);
          copy_async_wait<A>();
          const uint4(*at)[kThreads] = stage[(h - h0) % (A + 1)];
          typename S::Held r0, g0;
#pragma unroll
          for (int w = 0; w < S::W; ++w) {
            r0.w[w] = at[w][threadIdx.x];
            if constexpr (kBwd) g0.w[w] = at[S::W + w][threadIdx.x];
          }
          work(h, r0, g0);
        }
      } else {
        typename S::Held xr[A], gr[A];
#pragma unroll
        for (int i = 0; i < A; ++i)
          if (h0 + i < h1) {
            sl.load(x + (h0 + i) * sd.xh, xr[i]);
            if constexpr (kBwd) sl.load(dy + (h0 + i) * sd.gh, gr[i]);
          }
        for (int hh = h0; hh < h1; hh += A) {
#pragma unroll
          for (int i = 0; i < A; ++i) {
            const int h = hh + i;
            if (h >= h1) break;  // (the same for every lane)
            const typename S::Held r0 = xr[i], g0 = gr[i];
            if (h + A < h1) {
              sl.load(x + (h + A) * sd.xh, xr[i]);
              if constexpr (kBwd) sl.load(dy + (h + A) * sd.gh, gr[i]);
            }
            work(h, r0, g0);
          }
        }
      }
      if constexpr (kBwd) {
        if (live) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            sums[side][j][threadIdx.x] += ga[j];
            sums[side][8 + j][threadIdx.x] += gb[j];
          }
        }
      }
    }
  }

  if constexpr (kBwd) {
    // The block's row of sums: lanes of a warp that hold the same elements
    // first, then the warps, in a fixed order.
    static_assert(!kStaged || sizeof(stage) >= kThreads / 32 * D * sizeof(float), "by_warp lies over the stages");
    __shared__ float own[kStaged ? 1 : kThreads / 32][kStaged ? 1 : D];
    float(*by_warp)[D] = kStaged ? reinterpret_cast<float(*)[D]>(&stage[0][0][0]) : reinterpret_cast<float(*)[D]>(&own[0][0]);
    __syncthreads();  // every thread is through with its stages
    const int warp = threadIdx.x >> 5;
    const long long block = static_cast<long long>(blockIdx.y) * gridDim.x + blockIdx.x;
    const long long blocks = static_cast<long long>(gridDim.y) * gridDim.x;
#pragma unroll 1
    for (int side = 0; side < 2; ++side) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float a = sums[side][j][threadIdx.x], b = sums[side][8 + j][threadIdx.x];
#pragma unroll
        for (int o = LPR; o < 32; o <<= 1) {
          a += __shfl_xor_sync(0xffffffffu, a, o);
          b += __shfl_xor_sync(0xffffffffu, b, o);
        }
        if ((threadIdx.x & 31) < LPR) {
          by_warp[warp][sl.element(j, 0)] = a;
          by_warp[warp][sl.element(j, 1)] = b;
        }
      }
      __syncthreads();
      if (threadIdx.x < D) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) s += by_warp[w][threadIdx.x];
        p.partial[(side * blocks + block) * D + threadIdx.x] = s;
      }
      __syncthreads();
    }
  }
}

// dw[side][e] = sum of the side's rows of partial sums.  Block (e / 8, side):
// 8 elements, 32 threads each over every 32nd row; then a tree over those.
constexpr int kSumThreads = 256;
template <int D>
__global__ void __launch_bounds__(kSumThreads)
    rope_dw_kernel(const float *partial, float *dw0, float *dw1, int rows) {
  grid_dependency_wait();
  const int side = blockIdx.y;
  float *dw = side ? dw1 : dw0;
  if (!dw) return;
  const float *src = partial + static_cast<long long>(side) * rows * D;
  const int e = blockIdx.x * 8 + (threadIdx.x & 7), part = threadIdx.x >> 3;
  float s = 0.f;
  for (int r = part; r < rows; r += kSumThreads / 8) s += src[static_cast<long long>(r) * D + e];
  __shared__ float sh[kSumThreads];
  sh[threadIdx.x] = s;
  __syncthreads();
  for (int o = kSumThreads / 2; o >= 8; o >>= 1) {
    if (threadIdx.x < o) sh[threadIdx.x] += sh[threadIdx.x + o];
    __syncthreads();
  }
  if (threadIdx.x < 8) dw[e] = sh[threadIdx.x];
}

// How a call is cut into blocks: token tiles by groups of heads.
struct Cut {
  int per, groups, grid_x;
};

Cut cut(long long tokens, int heads, int d, int op, int size) {
  const int tt = kThreads / (d / 16);
  const long long tiles = (tokens + tt - 1) / tt;
  const long long slots = kSMs * blocks_per_sm(op, size);  // blocks that run at a time
  // A block's time is about its heads plus the angles, which take as long as
  // kAngles heads; all blocks take as many turns as they fill the slots.
  // More groups balance the turns better and work the angles out more often.
  constexpr int kAngles = 3;
  Cut c{1, heads, 0};
  long long best = -1, turns = 1;
  // (A head a block where all of those run at once.)
  for (int g = 1; tiles * heads > slots && g <= heads && g <= 64; ++g) {
    const int per = (heads + g - 1) / g;
    const long long t = (tiles * g + slots - 1) / slots, cost = t * (per + kAngles);
    if (best < 0 || cost < best) {
      best = cost;
      turns = t;
      c.per = per;
      c.groups = (heads + per - 1) / per;
    }
  }
  // The gradient has a row of partial sums per block: there a block takes its
  // turns itself, tile after tile.
  const long long gx = op == kNormTurnBwd ? (tiles + turns - 1) / turns : tiles;
  c.grid_x = gx > 0x7fffffffLL ? -1 : static_cast<int>(gx);
  return c;
}

template <typename T, int D, int OP>
attn_status_t launch_mode(const RopeParams &p, const Cut &c, bool interleaved, cudaStream_t stream) {
  const dim3 grid(c.grid_x, c.groups);
  if (interleaved)
    rope_kernel<T, D, kPairs, OP><<<grid, kThreads, 0, stream>>>(p);
  else if (p.rot % (2 * Word<T>::L) == 0)
    rope_kernel<T, D, kHalf, OP><<<grid, kThreads, 0, stream>>>(p);
  else
    rope_kernel<T, D, kScalar, OP><<<grid, kThreads, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

template <int OP>
attn_status_t launch_op(const RopeParams &p, const Cut &c, int dtype, int d, bool interleaved,
                        cudaStream_t stream) {
  if (dtype == ATTN_DTYPE_BF16)
    return d == 128 ? launch_mode<__nv_bfloat16, 128, OP>(p, c, interleaved, stream)
                    : launch_mode<__nv_bfloat16, 64, OP>(p, c, interleaved, stream);
  return d == 128 ? launch_mode<float, 128, OP>(p, c, interleaved, stream)
                  : launch_mode<float, 64, OP>(p, c, interleaved, stream);
}

}  // namespace

size_t norm_rope_bwd_workspace_bytes(long long tokens, int Hq, int Hkv, int d) {
  // (Whichever type the call has.)
  const Cut a = cut(tokens, Hq + Hkv, d, kNormTurnBwd, 2), b = cut(tokens, Hq + Hkv, d, kNormTurnBwd, 4);
  const long long rows = std::max(static_cast<long long>(a.grid_x) * a.groups,
                                   static_cast<long long>(b.grid_x) * b.groups);
  return static_cast<size_t>(2) * rows * d * sizeof(float);
}

attn_status_t launch_rope(const RopeSide &q, const RopeSide &k, const int *positions,
                          long long pos_stride, const double *inv_freq, int dtype, int op, int B,
                          int N, int d, int rot, int interleaved, float factor, int transpose,
                          float eps, void *workspace, cudaStream_t stream) {
  const bool bwd = op == kNormTurnBwd;
  RopeParams p{};
  p.tokens = static_cast<long long>(B) * N;
  const Cut c = cut(p.tokens, q.H + k.H, d, op, dtype == ATTN_DTYPE_BF16 ? 2 : 4);
  if (c.grid_x < 0 || c.groups > 65535) return ATTN_ERR_INVALID_ARG;
  const RopeSide *in[2] = {&q, &k};
  for (int i = 0; i < 2; ++i) {
    const RopeSide &s = *in[i];
    Side &o = p.side[i];
    o = Side{s.x, s.dy, s.y, s.w, s.x_st.batch, s.x_st.head, s.x_st.token, s.y_st.batch, s.y_st.head,
             s.y_st.token, s.dy_st.batch, s.dy_st.head, s.dy_st.token, s.H};
  }
  p.positions = positions;
  p.pos_stride = pos_stride;
  p.inv_freq = inv_freq;
  p.partial = static_cast<float *>(workspace);
  p.N = N;
  p.per_group = c.per;
  p.rot = rot;
  p.factor = factor;
  p.sign = (transpose || bwd) ? -1.f : 1.f;
  p.eps = eps;
  if (op == kTurn) return launch_op<kTurn>(p, c, dtype, d, interleaved, stream);
  if (op == kNormTurn) return launch_op<kNormTurn>(p, c, dtype, d, interleaved, stream);
  attn_status_t st = launch_op<kNormTurnBwd>(p, c, dtype, d, interleaved, stream);
  if (st != ATTN_OK) return st;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(d / 8, 2);
  cfg.blockDim = dim3(kSumThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const float *partial = p.partial;
  const int rows = c.grid_x * c.groups;
  const cudaError_t err =
      d == 128 ? cudaLaunchKernelEx(&cfg, rope_dw_kernel<128>, partial, q.dw, k.dw, rows)
               : cudaLaunchKernelEx(&cfg, rope_dw_kernel<64>, partial, q.dw, k.dw, rows);
  if (err != cudaSuccess) return ATTN_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace exattn
