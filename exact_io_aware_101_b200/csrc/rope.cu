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
// elements.  So:
//  * One thread holds the same 16 elements (8 pairs) of its rows and walks the
//    heads of one token: the cosines and sines of its 8 pairs and its weights
//    stay in registers, worked out once for all those heads.  LPR = d/16 lanes
//    hold a row, and a norm's two sums are log2(LPR) shuffles.
//  * Each lane moves 16-byte words, and kUnroll rows are loaded before the
//    first is used.  Half layouts whose rot is not a multiple of 16 would put
//    the partner elements at odd addresses: they go element by element.
//  * q and k go in one launch; each block works on heads of one of the two.
//  * Angles: t * f_i / 2 pi is taken in 64 bits and reduced to the nearest
//    whole turn there (a far position's angle has no fraction left in 32
//    bits); the remainder, at most half a turn, goes to sincospi in 32 bits.
//    One 64-bit product serves all heads of the token.
//  * Sums, norms and products are float32, rounded once when a row is stored.
//  * The weights' gradients: each thread adds its 16 elements' products over
//    all its rows, the block adds its lanes' sums in shared memory and writes
//    one row of partial sums per block, and a second kernel, scheduled behind
//    the first, adds those rows in a fixed order.  No atomics: the result does
//    not depend on the order in which blocks run.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "common.cuh"
#include "internal.h"

namespace exattn {
namespace {

constexpr int kThreads = 128;
constexpr int kUnroll = 4;       // rows in flight per thread
constexpr int kSMs = 148;
constexpr double kInvTwoPi = 0.15915494309189533577;

enum Mode { kHalf, kPairs, kScalar };   // where a thread's pairs lie (see load_row)
enum Op { kTurn, kNormTurn, kNormTurnBwd };

// One of the two tensors of a call: q or k.
struct Side {
  const void *x, *dy;  // dy: gradient only
  void *y;             // output, or dx
  const void *w;       // norm weights [d]
  long long xb, xh, xn, yb, yh, yn, gb, gh, gn;  // element strides: batch, head, token
  float *dw;           // float32 [d] (gradient)
  int H, groups, per_group;
};

struct RopeParams {
  Side side[2];
  const int *positions;
  long long pos_stride;  // of a batch entry; 0: shared
  const double *inv_freq;
  float *partial;  // gradient: [blocks][d], block (x, y) at row y * gridDim.x + x
  long long tokens;
  int N, rot;
  float factor, sign, eps;
};

template <typename T>
__device__ __forceinline__ void load8(const T *p, float (&v)[8]);
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16 *p, float (&v)[8]) {
  const uint4 u = *reinterpret_cast<const uint4 *>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
template <>
__device__ __forceinline__ void load8<float>(const float *p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&v)[8]) {
  *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                             pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ void store8(float *p, const float (&v)[8]) {
  reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f32(float *p, float v) { *p = v; }
__device__ __forceinline__ void from_f32(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

// The 16 elements of a row that belong to lane `i` of its LPR lanes, as 8
// slots (a[j], b[j]).  Slots are numbered 0 .. d/2-1; slot s < rot/2 is pair s,
// and slot s >= rot/2 the two unturned elements 2s and 2s+1.  kHalf and kPairs:
// lane i holds slots 8i .. 8i+7; in the half layout with rot % 16 == 0 they are
// either 8 pairs, two runs of 8 elements rot/2 apart, or 16 unturned ones; in
// the interleaved layout always 16 elements in a row.  kScalar: slots i + LPR*j.
template <int D, int MODE>
struct Slots {
  static constexpr int LPR = D / 16;
  int o0, o1;    // kHalf, kPairs: first elements of the two runs of 8
  int nturn;     // kHalf, kPairs: slots j < nturn turn
  int lane, half;
  __device__ __forceinline__ Slots(int lane_, int rot) : lane(lane_), half(rot >> 1) {
    const bool pair_runs = MODE == kHalf && 8 * lane < half;
    o0 = pair_runs ? 8 * lane : 16 * lane;
    o1 = pair_runs ? half + 8 * lane : 16 * lane + 8;
    nturn = min(8, max(0, half - 8 * lane));
  }
  __device__ __forceinline__ int slot(int j) const { return MODE == kScalar ? lane + LPR * j : 8 * lane + j; }
  __device__ __forceinline__ bool turns(int j) const { return MODE == kScalar ? slot(j) < half : j < nturn; }
  __device__ __forceinline__ int first(int j) const {  // kScalar: element of a[j]
    const int s = slot(j);
    return s < half ? s : 2 * s;
  }
  __device__ __forceinline__ int second(int j) const {
    const int s = slot(j);
    return s < half ? s + half : 2 * s + 1;
  }
  // Element of the weights' gradient that slot j's a (which = 0) or b holds.
  __device__ __forceinline__ int element(int j, int which) const {
    if (MODE == kScalar) return which ? second(j) : first(j);
    if (MODE == kPairs) return 16 * lane + 2 * j + which;
    return (which ? o1 : o0) + j;
  }
  template <typename T>
  __device__ __forceinline__ void load(const T *row, float (&a)[8], float (&b)[8]) const {
    if constexpr (MODE == kScalar) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        a[j] = to_f32(row[first(j)]);
        b[j] = to_f32(row[second(j)]);
      }
    } else {
      float u[8], v[8];
      load8(row + o0, u);
      load8(row + o1, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if constexpr (MODE == kHalf) {
          a[j] = u[j];
          b[j] = v[j];
        } else {
          a[j] = j < 4 ? u[(2 * j) & 7] : v[(2 * j) & 7];
          b[j] = j < 4 ? u[(2 * j + 1) & 7] : v[(2 * j + 1) & 7];
        }
      }
    }
  }
  template <typename T>
  __device__ __forceinline__ void store(T *row, const float (&a)[8], const float (&b)[8]) const {
    if constexpr (MODE == kScalar) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        from_f32(row + first(j), a[j]);
        from_f32(row + second(j), b[j]);
      }
    } else {
      float u[8], v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if constexpr (MODE == kHalf) {
          u[j] = a[j];
          v[j] = b[j];
        } else if (j < 4) {
          u[(2 * j) & 7] = a[j];
          u[(2 * j + 1) & 7] = b[j];
        } else {
          v[(2 * j) & 7] = a[j];
          v[(2 * j + 1) & 7] = b[j];
        }
      }
      store8(row + o0, u);
      store8(row + o1, v);
    }
  }
};

// Sum over the LPR lanes of a row.
template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Block (x, y): group y of heads of one tensor, token tiles x, x + gridDim.x, ...
template <typename T, int D, int MODE, int OP>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeParams p) {
  constexpr int LPR = D / 16, TT = kThreads / LPR;
  if constexpr (OP == kNormTurnBwd) grid_dependents_launch();
  const int lane = threadIdx.x % LPR, slot_row = threadIdx.x / LPR;
  const int which = blockIdx.y < p.side[0].groups ? 0 : 1;
  const Side &sd = p.side[which];
  const int group = blockIdx.y - (which ? p.side[0].groups : 0);
  const int h0 = group * sd.per_group, h1 = min(sd.H, h0 + sd.per_group);
  const Slots<D, MODE> sl(lane, p.rot);

  float wa[8], wb[8];  // norm weights of this lane's elements
  if constexpr (OP != kTurn) sl.load(static_cast<const T *>(sd.w), wa, wb);
  float ga[8], gb[8];  // their gradients, over this thread's rows
  if constexpr (OP == kNormTurnBwd) {
#pragma unroll
    for (int j = 0; j < 8; ++j) ga[j] = gb[j] = 0.f;
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
    auto turn = [&](float &a, float &b, int j) {
      const float y = a * cs[j] - b * sn[j], z = a * sn[j] + b * cs[j];
      // (Not by cos 1, sin 0 for the rest: an infinity beside it would turn to NaN.)
      a = sl.turns(j) ? y : a;
      b = sl.turns(j) ? z : b;
    };
    const T *x = static_cast<const T *>(sd.x) + bi * sd.xb + n * sd.xn;
    T *y = static_cast<T *>(sd.y) + bi * sd.yb + n * sd.yn;
    const T *dy = OP == kNormTurnBwd ? static_cast<const T *>(sd.dy) + bi * sd.gb + n * sd.gn : nullptr;
    constexpr int U = OP == kNormTurnBwd ? 2 : kUnroll;
    for (int h = h0; h < h1; h += U) {
      float a[U][8], b[U][8], c[OP == kNormTurnBwd ? U : 1][8], e[OP == kNormTurnBwd ? U : 1][8];
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (h + i < h1) {
          sl.load(x + (h + i) * sd.xh, a[i], b[i]);
          if constexpr (OP == kNormTurnBwd) sl.load(dy + (h + i) * sd.gh, c[i], e[i]);
        }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        if (h + i >= h1) break;  // (the same for every lane)
        if constexpr (OP == kTurn) {
#pragma unroll
          for (int j = 0; j < 8; ++j) turn(a[i][j], b[i][j], j);
        } else {
          float ss = 0.f;
#pragma unroll
          for (int j = 0; j < 8; ++j) ss += a[i][j] * a[i][j] + b[i][j] * b[i][j];
          const float r = __frsqrt_rn(row_sum<LPR>(ss) * (1.f / D) + p.eps);
          if constexpr (OP == kNormTurn) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              a[i][j] = a[i][j] * r * wa[j];
              b[i][j] = b[i][j] * r * wb[j];
              turn(a[i][j], b[i][j], j);
            }
          } else {
            float dot = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              turn(c[i][j], e[i][j], j);  // u: sign is -1 here
              a[i][j] *= r;               // xhat
              b[i][j] *= r;
              if (live) {
                ga[j] += c[i][j] * a[i][j];
                gb[j] += e[i][j] * b[i][j];
              }
              c[i][j] *= wa[j];
              e[i][j] *= wb[j];
              dot += c[i][j] * a[i][j] + e[i][j] * b[i][j];
            }
            dot = row_sum<LPR>(dot) * (1.f / D);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              a[i][j] = r * (c[i][j] - a[i][j] * dot);
              b[i][j] = r * (e[i][j] - b[i][j] * dot);
            }
          }
        }
        if (live) sl.store(y + (h + i) * sd.yh, a[i], b[i]);
      }
    }
  }

  if constexpr (OP == kNormTurnBwd) {
    // The block's rows of sums: lanes of a warp that hold the same elements
    // first, then the warps, in a fixed order.
    __shared__ float sums[kThreads / 32][D];
    const int warp = threadIdx.x >> 5;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
#pragma unroll
      for (int o = LPR; o < 32; o <<= 1) {
        ga[j] += __shfl_xor_sync(0xffffffffu, ga[j], o);
        gb[j] += __shfl_xor_sync(0xffffffffu, gb[j], o);
      }
      if ((threadIdx.x & 31) < LPR) {
        sums[warp][sl.element(j, 0)] = ga[j];
        sums[warp][sl.element(j, 1)] = gb[j];
      }
    }
    __syncthreads();
    if (threadIdx.x < D) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) s += sums[w][threadIdx.x];
      p.partial[(static_cast<long long>(blockIdx.y) * gridDim.x + blockIdx.x) * D + threadIdx.x] = s;
    }
  }
}

// dw[side][e] = sum of the side's rows of partial sums.  Block (e / 8, side):
// 8 elements, 32 threads each over every 32nd row; then a tree over those.
constexpr int kSumThreads = 256;
template <int D>
__global__ void __launch_bounds__(kSumThreads)
    rope_dw_kernel(const float *partial, float *dw0, float *dw1, int rows0, int rows1) {
  grid_dependency_wait();
  const int side = blockIdx.y;
  float *dw = side ? dw1 : dw0;
  const int rows = side ? rows1 : rows0;
  if (!dw) return;
  const float *src = partial + (side ? static_cast<long long>(rows0) * D : 0);
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
  long long tiles;
  int per[2], groups[2];
  int grid_x;
};

Cut cut(long long tokens, int Hq, int Hkv, int d, bool bwd) {
  Cut c;
  const int tt = kThreads / (d / 16);
  c.tiles = (tokens + tt - 1) / tt;
  // Heads per block: as many as leave about eight blocks for each SM (an
  // angle then serves all of them), at most 16.
  const long long want = c.tiles * (Hq + Hkv) / (kSMs * 8);
  const int per = static_cast<int>(want < 1 ? 1 : (want > 16 ? 16 : want));
  const int H[2] = {Hq, Hkv};
  for (int i = 0; i < 2; ++i) {
    c.groups[i] = H[i] ? (H[i] + per - 1) / per : 0;
    c.per[i] = c.groups[i] ? (H[i] + c.groups[i] - 1) / c.groups[i] : 0;
  }
  long long gx = c.tiles;
  if (bwd) {
    // A row of partial sums per block: a block takes several tiles, so that
    // there are at most about eight blocks per SM.
    const long long most = (kSMs * 8 + c.groups[0] + c.groups[1] - 1) / (c.groups[0] + c.groups[1]);
    if (gx > most) gx = most;
  }
  c.grid_x = gx > 0x7fffffffLL ? -1 : static_cast<int>(gx);
  return c;
}

template <typename T, int D, int OP>
attn_status_t launch_mode(const RopeParams &p, const Cut &c, bool interleaved, cudaStream_t stream) {
  const dim3 grid(c.grid_x, c.groups[0] + c.groups[1]);
  if (interleaved)
    rope_kernel<T, D, kPairs, OP><<<grid, kThreads, 0, stream>>>(p);
  else if (p.rot % 16 == 0)
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
  const Cut c = cut(tokens, Hq, Hkv, d, true);
  return static_cast<size_t>(c.grid_x) * (c.groups[0] + c.groups[1]) * d * sizeof(float);
}

attn_status_t launch_rope(const RopeSide &q, const RopeSide &k, const int *positions,
                          long long pos_stride, const double *inv_freq, int dtype, int op, int B,
                          int N, int d, int rot, int interleaved, float factor, int transpose,
                          float eps, void *workspace, cudaStream_t stream) {
  const bool bwd = op == kNormTurnBwd;
  RopeParams p{};
  p.tokens = static_cast<long long>(B) * N;
  const Cut c = cut(p.tokens, q.H, k.H, d, bwd);
  if (c.grid_x < 0 || c.groups[0] + c.groups[1] > 65535) return ATTN_ERR_INVALID_ARG;
  const RopeSide *in[2] = {&q, &k};
  for (int i = 0; i < 2; ++i) {
    const RopeSide &s = *in[i];
    Side &o = p.side[i];
    o = Side{s.x, s.dy, s.y, s.w, s.x_st.batch, s.x_st.head, s.x_st.token, s.y_st.batch, s.y_st.head,
             s.y_st.token, s.dy_st.batch, s.dy_st.head, s.dy_st.token, s.dw, s.H, c.groups[i], c.per[i]};
  }
  p.positions = positions;
  p.pos_stride = pos_stride;
  p.inv_freq = inv_freq;
  p.partial = static_cast<float *>(workspace);
  p.N = N;
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
  const int rows0 = c.grid_x * c.groups[0], rows1 = c.grid_x * c.groups[1];
  const cudaError_t err =
      d == 128 ? cudaLaunchKernelEx(&cfg, rope_dw_kernel<128>, partial, q.dw, k.dw, rows0, rows1)
               : cudaLaunchKernelEx(&cfg, rope_dw_kernel<64>, partial, q.dw, k.dw, rows0, rows1);
  if (err != cudaSuccess) return ATTN_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace exattn
