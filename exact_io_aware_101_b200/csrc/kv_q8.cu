// kv_q8.cu -- writing keys and values into an 8-bit paged cache, and reading
// them back.
//
// What it computes.  A (page, K/V head) slice of the cache holds 16 x d codes
// and one float32 scale; an element stands for scale * code.  A chunk's new
// tokens go to the last places of their sequence.  For every slice they touch:
//   s' = max(s if the page already holds earlier tokens of the sequence,
//            amax(new) / qmax, 2^-126)              (qmax: 448 E4M3, 127 INT8)
//   new codes     = x / s' rounded to the format,
//   earlier codes = code * s / s' rounded to the format (as they were if s' = s),
// each rounding to nearest, ties to even, of the exact quotient.  So the scale
// of a page only grows while it fills, a page whose first slot is written
// starts afresh, and writing the same tokens twice changes nothing.  A slice
// whose new tokens hold a NaN or an infinity gets the scale NaN: the sequence's
// attention then is NaN, as it would be over a 16-bit cache.
//
// Exact quotients without dividing: the product with inv = 1/s' (or s/s') is off
// by at most a few parts in 2^24, so each element is rounded twice, from x * lo
// and from x * hi with lo, hi = inv (1 -+ 2^-22), which enclose the quotient.
// Rounding is monotonic: where both give one code, it is the quotient's.
// Where they differ (a quotient within 2^-22 of a tie, a few in a million) the
// lane divides in 64 bits, where code * s and the comparison with a tie are
// exact.
//
// What bounds it: HBM for long chunks and for reading, one chain of dependent
// loads (lengths, block table, data) for a decode step.  One warp takes one
// slice (write: of K or of V; read: of both), so no two warps share a scale
// and a slice's maximum is one warp reduction; a lane moves 16-byte words of
// bf16 and has the slice's whole share (at most 8 of them) in flight.  Earlier
// codes are loaded along with the new rows, before it is known whether the
// scale grows.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "common.cuh"
#include "internal.h"

namespace exattn {
namespace {

constexpr int kPage = 16;
constexpr int kWarps = 4;  // per block

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
  return d;
}

// Four floats to four codes (element 0 in the low byte), rounded to nearest
// even.  E4M3 saturates at 448; INT8 takes |x * f| <= 127.5 - 2^-10 at most.
template <int FMT>
__device__ __forceinline__ uint32_t codes4(const float *x, float f) {
  if constexpr (FMT == ATTN_KV_E4M3) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(x[1] * f), "f"(x[0] * f));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(x[3] * f), "f"(x[2] * f));
    return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
  } else {
    // x * f + 1.5 * 2^23: the sum's unit is 1, so its low byte is the code.
    constexpr float kMagic = 12582912.f;
    const uint32_t a = __float_as_uint(fmaf(x[0], f, kMagic)), b = __float_as_uint(fmaf(x[1], f, kMagic));
    const uint32_t c = __float_as_uint(fmaf(x[2], f, kMagic)), d = __float_as_uint(fmaf(x[3], f, kMagic));
    return prmt(prmt(a, b, 0x0040u), prmt(c, d, 0x0040u), 0x5410u);
  }
}

// One code of x * num / den from the quotient in 64 bits.
template <int FMT>
__device__ __noinline__ uint32_t code_exact(float x, float num, float den) {
  const double q = static_cast<double>(x) * static_cast<double>(num) / static_cast<double>(den);
  if constexpr (FMT == ATTN_KV_E4M3) {
    // To 24 bits toward zero with the lost part kept as a set last bit, so that
    // the second rounding sees a tie only where there is one.
    float f = __double2float_rz(q);
    if (static_cast<double>(f) != q) f = __uint_as_float(__float_as_uint(f) | 1u);
    uint16_t h;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h) : "f"(0.f), "f"(f));
    return h & 0xffu;
  } else {
    return static_cast<uint32_t>(max(-127, min(127, __double2int_rn(q)))) & 0xffu;
  }
}

// Eight floats to eight codes of x * num / den; lo and hi enclose num / den.
template <int FMT>
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float lo, float hi, float num, float den) {
  uint2 c = make_uint2(codes4<FMT>(x, lo), codes4<FMT>(x + 4, lo));
  const uint2 e = make_uint2(codes4<FMT>(x, hi), codes4<FMT>(x + 4, hi));
  if (c.x != e.x || c.y != e.y) {
    c = make_uint2(0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      c.x |= code_exact<FMT>(x[i], num, den) << (8 * i);
      c.y |= code_exact<FMT>(x[4 + i], num, den) << (8 * i);
    }
  }
  return c;
}

// Four codes to floats (exact).
template <int FMT>
__device__ __forceinline__ void values4(uint32_t w, float *v) {
  if constexpr (FMT == ATTN_KV_E4M3) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t r;
      const uint16_t two = static_cast<uint16_t>(h ? (w >> 16) : (w & 0xffffu));
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(two));
      asm("{ .reg .f16 a, b; mov.b32 {a, b}, %2; cvt.f32.f16 %0, a; cvt.f32.f16 %1, b; }"
          : "=f"(v[2 * h]), "=f"(v[2 * h + 1])
          : "r"(r));
    }
  } else {
    // The byte with its sign flipped, under the exponent of 2^23, is
    // 2^23 + code + 128.
    const uint32_t b = w ^ 0x80808080u;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = __uint_as_float(prmt(b, 0x4b000000u, 0x7440u | i)) - 8388736.f;
  }
}

// The places of a sequence's chunk: new tokens ctx .. n-1, rows q0 .. of the
// token-major tensors.  False (and the status bit) where the lengths do not fit.
struct Chunk {
  int q0, nq, n, ctx;
};
__device__ __forceinline__ bool chunk_of(const int *seq_lens, const int *cu_q, int s, int T, int max_q,
                                         int max_blocks, Chunk &c) {
  c.q0 = cu_q[s];
  const int q1 = cu_q[s + 1];
  c.n = seq_lens[s];
  // (In 64 bits: a corrupt pair could wrap.)
  const long long nq = static_cast<long long>(q1) - c.q0;
  c.nq = static_cast<int>(nq);
  c.ctx = c.n - c.nq;
  return c.q0 >= 0 && nq >= 0 && nq <= max_q && q1 <= T && c.n >= nq &&
         c.n <= static_cast<long long>(max_blocks) * kPage;
}

struct WriteParams {
  const void *x[2];            // k, v (bf16)
  long long xt[2], xh[2];      // their token and head strides
  uint8_t *pages[2];
  float *scales[2];
  const int *block_table, *seq_lens, *cu_q;
  unsigned *status;
  int Hkv, T, max_q, max_blocks, num_pages, pages_per_seq;
};

// Block: sequence and page of its chunk (x), four of the 2 * Hkv slices (y).
template <int D, int FMT>
__global__ void __launch_bounds__(kWarps * 32) kv_write_kernel(const WriteParams p) {
  constexpr int LPR = D / 8, RPP = 32 / LPR, PASSES = kPage / RPP;  // lanes per row, rows per pass
  constexpr float kQmax = FMT == ATTN_KV_E4M3 ? 448.f : 127.f;
  const int lane = threadIdx.x & 31;
  const int item = blockIdx.y * kWarps + (threadIdx.x >> 5);  // 2 * head + (0: K, 1: V)
  const int s = blockIdx.x / p.pages_per_seq, j = blockIdx.x % p.pages_per_seq;
  if (item >= 2 * p.Hkv) return;
  Chunk c;
  if (!chunk_of(p.seq_lens, p.cu_q, s, p.T, p.max_q, p.max_blocks, c)) {
    if (threadIdx.x == 0 && j == 0 && blockIdx.y == 0) atomicOr(p.status, ATTN_DEV_BAD_PAGE);
    return;
  }
  const int page = c.ctx / kPage + j;
  if (c.nq == 0 || page * kPage >= c.n) return;
  const int pid = p.block_table[static_cast<size_t>(s) * p.max_blocks + page];
  if (pid < 0 || pid >= p.num_pages) {
    if (threadIdx.x == 0 && blockIdx.y == 0) atomicOr(p.status, ATTN_DEV_BAD_PAGE);
    return;
  }
  const int lo = max(c.ctx - page * kPage, 0), hi = min(kPage, c.n - page * kPage);
  const int kv = item & 1, head = item >> 1;
  const int row = lane / LPR, col = (lane % LPR) * 8;
  // Row r of the page is row q0 + page*16 + r - ctx of x.
  const __nv_bfloat16 *x = static_cast<const __nv_bfloat16 *>(p.x[kv]) +
                           (c.q0 + static_cast<long long>(page) * kPage - c.ctx) * p.xt[kv] +
                           head * p.xh[kv] + col;
  const size_t slice = static_cast<size_t>(pid) * p.Hkv + head;
  uint8_t *codes = p.pages[kv] + slice * (kPage * D) + col;

  uint4 in[PASSES];   // new rows
  uint2 was[PASSES];  // earlier rows' codes
  const float s_old = lo > 0 ? p.scales[kv][slice] : 0.f;
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int r = i * RPP + row;
    in[i] = make_uint4(0, 0, 0, 0);
    if (r >= lo && r < hi) in[i] = *reinterpret_cast<const uint4 *>(x + r * p.xt[kv]);
    if (r < lo) was[i] = *reinterpret_cast<const uint2 *>(codes + r * D);
  }
  // Largest magnitude as 15-bit patterns, two at a time: NaN above infinity
  // above every finite value.
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < PASSES; ++i)
    top = __vmaxu2(top, __vmaxu2(__vmaxu2(in[i].x & 0x7fff7fffu, in[i].y & 0x7fff7fffu),
                                 __vmaxu2(in[i].z & 0x7fff7fffu, in[i].w & 0x7fff7fffu)));
  top = __reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16));
  float s_new = fmaxf(__uint_as_float(top << 16) / kQmax, 1.17549435e-38f);
  const bool odd = top >= 0x7f80u || !(fabsf(s_old) <= 3.4028235e38f);  // a NaN or infinity
  if (lo > 0) s_new = fmaxf(s_new, s_old);
  if (odd) s_new = __uint_as_float(0x7fc00000u);
  if (lane == 0) p.scales[kv][slice] = s_new;

  const float inv = 1.f / s_new;
  const float inv_lo = inv * (1.f - 0x1p-22f), inv_hi = inv * (1.f + 0x1p-22f);
  const bool again = lo > 0 && s_new != s_old && !odd;
  float ratio_lo = 0.f, ratio_hi = 0.f;
  if (again) {
    const float ratio = s_old / s_new;
    ratio_lo = ratio * (1.f - 0x1p-22f);
    ratio_hi = ratio * (1.f + 0x1p-22f);
  }
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int r = i * RPP + row;
    float v[8];
    if (r >= lo && r < hi) {
      const uint32_t w[4] = {in[i].x, in[i].y, in[i].z, in[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[2 * e] = __uint_as_float(w[e] << 16);
        v[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
      }
      *reinterpret_cast<uint2 *>(codes + r * D) =
          odd ? make_uint2(0, 0) : codes8<FMT>(v, inv_lo, inv_hi, 1.f, s_new);
    } else if (r < lo && again) {
      values4<FMT>(was[i].x, v);
      values4<FMT>(was[i].y, v + 4);
      *reinterpret_cast<uint2 *>(codes + r * D) = codes8<FMT>(v, ratio_lo, ratio_hi, s_old, s_new);
    }
  }
}

struct ReadParams {
  const uint8_t *pages[2];
  const float *scales[2];
  void *out[2];  // [T, Hkv, D]
  const int *block_table, *seq_lens, *cu_q;
  unsigned *status;
  int Hkv, T, max_q, max_blocks, num_pages, pages_per_seq;
};

__device__ __forceinline__ void store4(float *p, const float *v) {
  *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
}

// Block: sequence and page of its range (x), four K/V heads (y).
template <int D, int FMT, typename T>
__global__ void __launch_bounds__(kWarps * 32) kv_read_kernel(const ReadParams p) {
  constexpr int LPR = D / 8, RPP = 32 / LPR, PASSES = kPage / RPP;
  const int lane = threadIdx.x & 31;
  const int head = blockIdx.y * kWarps + (threadIdx.x >> 5);
  const int s = blockIdx.x / p.pages_per_seq, j = blockIdx.x % p.pages_per_seq;
  if (head >= p.Hkv) return;
  Chunk c;
  if (!chunk_of(p.seq_lens, p.cu_q, s, p.T, p.max_q, p.max_blocks, c)) {
    if (threadIdx.x == 0 && j == 0 && blockIdx.y == 0) atomicOr(p.status, ATTN_DEV_BAD_PAGE);
    return;
  }
  const int page = c.ctx / kPage + j;
  if (c.nq == 0 || page * kPage >= c.n) return;
  const int pid = p.block_table[static_cast<size_t>(s) * p.max_blocks + page];
  const bool bad = pid < 0 || pid >= p.num_pages;
  if (bad && threadIdx.x == 0 && blockIdx.y == 0) atomicOr(p.status, ATTN_DEV_BAD_PAGE);
  const int lo = max(c.ctx - page * kPage, 0), hi = min(kPage, c.n - page * kPage);
  const int row = lane / LPR, col = (lane % LPR) * 8;
  const size_t slice = static_cast<size_t>(bad ? 0 : pid) * p.Hkv + head;
  uint2 in[2][PASSES];
  float scale[2];
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    scale[kv] = bad ? __uint_as_float(0x7fc00000u) : p.scales[kv][slice];
    const uint8_t *codes = p.pages[kv] + slice * (kPage * D) + col;
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      const int r = i * RPP + row;
      in[kv][i] = make_uint2(0, 0);
      if (r >= lo && r < hi && !bad) in[kv][i] = *reinterpret_cast<const uint2 *>(codes + r * D);
    }
  }
#pragma unroll
  for (int kv = 0; kv < 2; ++kv)
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      const int r = i * RPP + row;
      if (r < lo || r >= hi) continue;
      float v[8];
      values4<FMT>(in[kv][i].x, v);
      values4<FMT>(in[kv][i].y, v + 4);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= scale[kv];
      T *out = static_cast<T *>(p.out[kv]) +
               ((c.q0 + static_cast<long long>(page) * kPage - c.ctx + r) * p.Hkv + head) * D + col;
      if constexpr (sizeof(T) == 2) {
        *reinterpret_cast<uint4 *>(out) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                     pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
      } else {
        store4(out, v);
        store4(out + 4, v + 4);
      }
    }
}

// Pages a chunk of at most max_q tokens can touch: one token touches one, and
// every further one may open another at most every 16th time.
long long pages_touched(int max_q, int max_blocks) {
  const long long n = (static_cast<long long>(max_q) + kPage - 2) / kPage + 1;
  return n < max_blocks ? n : max_blocks;
}

}  // namespace

attn_status_t launch_kv_write_q8(const void *k, const void *v, const long long (&strides)[4],
                                 void *k_pages, void *v_pages, float *k_scales, float *v_scales,
                                 int kv_format, const int *block_table, const int *seq_lens,
                                 const int *cu_q, int S, int Hkv, int T, int max_q, int d,
                                 int max_blocks, int num_pages, cudaStream_t stream,
                                 unsigned *status) {
  WriteParams p{};
  p.x[0] = k;
  p.x[1] = v;
  p.xt[0] = strides[0];
  p.xh[0] = strides[1];
  p.xt[1] = strides[2];
  p.xh[1] = strides[3];
  p.pages[0] = static_cast<uint8_t *>(k_pages);
  p.pages[1] = static_cast<uint8_t *>(v_pages);
  p.scales[0] = k_scales;
  p.scales[1] = v_scales;
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.cu_q = cu_q;
  p.status = status;
  p.Hkv = Hkv;
  p.T = T;
  p.max_q = max_q;
  p.max_blocks = max_blocks;
  p.num_pages = num_pages;
  p.pages_per_seq = static_cast<int>(pages_touched(max_q, max_blocks));
  const long long gx = static_cast<long long>(S) * p.pages_per_seq;
  const long long gy = (2LL * Hkv + kWarps - 1) / kWarps;
  if (gx > 0x7fffffffLL || gy > 65535) return ATTN_ERR_INVALID_ARG;
  const dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>(gy));
  if (d == 128) {
    if (kv_format == ATTN_KV_E4M3) kv_write_kernel<128, ATTN_KV_E4M3><<<grid, kWarps * 32, 0, stream>>>(p);
    else kv_write_kernel<128, ATTN_KV_INT8><<<grid, kWarps * 32, 0, stream>>>(p);
  } else {
    if (kv_format == ATTN_KV_E4M3) kv_write_kernel<64, ATTN_KV_E4M3><<<grid, kWarps * 32, 0, stream>>>(p);
    else kv_write_kernel<64, ATTN_KV_INT8><<<grid, kWarps * 32, 0, stream>>>(p);
  }
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

template <int D, int FMT>
static void launch_read(const ReadParams &p, int dtype, dim3 grid, cudaStream_t stream) {
  if (dtype == ATTN_DTYPE_BF16) kv_read_kernel<D, FMT, __nv_bfloat16><<<grid, kWarps * 32, 0, stream>>>(p);
  else kv_read_kernel<D, FMT, float><<<grid, kWarps * 32, 0, stream>>>(p);
}

attn_status_t launch_kv_read_q8(const void *k_pages, const void *v_pages, const float *k_scales,
                                const float *v_scales, int kv_format, const int *block_table,
                                const int *seq_lens, const int *cu_q, void *k, void *v, int dtype,
                                int S, int Hkv, int T, int max_q, int d, int max_blocks,
                                int num_pages, cudaStream_t stream, unsigned *status) {
  ReadParams p{};
  p.pages[0] = static_cast<const uint8_t *>(k_pages);
  p.pages[1] = static_cast<const uint8_t *>(v_pages);
  p.scales[0] = k_scales;
  p.scales[1] = v_scales;
  p.out[0] = k;
  p.out[1] = v;
  p.block_table = block_table;
  p.seq_lens = seq_lens;
  p.cu_q = cu_q;
  p.status = status;
  p.Hkv = Hkv;
  p.T = T;
  p.max_q = max_q;
  p.max_blocks = max_blocks;
  p.num_pages = num_pages;
  p.pages_per_seq = static_cast<int>(pages_touched(max_q, max_blocks));
  const long long gx = static_cast<long long>(S) * p.pages_per_seq;
  const long long gy = (static_cast<long long>(Hkv) + kWarps - 1) / kWarps;
  if (gx > 0x7fffffffLL || gy > 65535) return ATTN_ERR_INVALID_ARG;
  const dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>(gy));
  if (d == 128) {
    if (kv_format == ATTN_KV_E4M3) launch_read<128, ATTN_KV_E4M3>(p, dtype, grid, stream);
    else launch_read<128, ATTN_KV_INT8>(p, dtype, grid, stream);
  } else {
    if (kv_format == ATTN_KV_E4M3) launch_read<64, ATTN_KV_E4M3>(p, dtype, grid, stream);
    else launch_read<64, ATTN_KV_INT8>(p, dtype, grid, stream);
  }
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace exattn
