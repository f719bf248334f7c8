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
// Exact quotients.  bf16 values meet ties often: x = amax / 2 is 63.5 steps of INT8
// but for the scale's own rounding, and every power of two times 3/4 amax may lie
// half way between two E4M3 codes.  Two ways, chosen for a slice as a whole:
//  * s' is the rounded amax / qmax of these very tokens, and not exact.  x and amax
//    have 8 bits, qmax and a tie t at most 8: x qmax and t amax, whole numbers but
//    for powers of two, are equal or at least 2^-16 apart.  Where they are equal
//    the quotient lies on the side of the tie that the rounding of s' put it on,
//    one side for all elements.  So one product with 1 / s', moved by 2^-22 to
//    that side (more than its own errors, far less than 2^-16), rounds right.
//  * Otherwise (an earlier scale stays, amax / qmax is exact, a rescaled code) each
//    quotient's remainder decides (see codes8).
// (For 16 chunks of 512 tokens of 8 heads, d = 128: a division in 64 bits near ties
// took 24 us (INT8) and 36 us (E4M3), the remainder for every element 17 and 18,
// five integer operations an element, the integer unit the busiest.)
//
// What bounds it: HBM for long chunks and for reading, one chain of dependent
// loads (lengths, block table, data) for a decode step.  Measured (B200, 8 heads,
// d = 128): writing 16 x 512 tokens 13 us (INT8) and 14.5 us (E4M3), 3.8 and 3.5
// TB/s of bf16 in and codes out, a third of it start and end; 16 x 4096 tokens 79
// us, 5.1 TB/s; 64 sequences' one token 3.2 us; reading 64 sequences of up to 8192
// tokens as bf16 281 us, 6.4 TB/s (98 % of the measured copy rate).  One warp takes one
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
// even.  E4M3 saturates at 448; INT8 takes -128.5 < q < 127.5.
template <int FMT>
__device__ __forceinline__ uint32_t codes4(const float *q) {
  if constexpr (FMT == ATTN_KV_E4M3) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(q[1]), "f"(q[0]));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(q[3]), "f"(q[2]));
    return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
  } else {
    // q + 1.5 * 2^23: the sum's unit is 1, so its low byte is the code.
    constexpr float kMagic = 12582912.f;
    const uint32_t a = __float_as_uint(q[0] + kMagic), b = __float_as_uint(q[1] + kMagic);
    const uint32_t c = __float_as_uint(q[2] + kMagic), d = __float_as_uint(q[3] + kMagic);
    return prmt(prmt(a, b, 0x0040u), prmt(c, d, 0x0040u), 0x5410u);
  }
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

// A division by den, scaled by a power of two so that den lies in [1, 2) and no
// remainder that matters underflows.
struct Divide {
  float num, den, inv;  // num / den = the factor; inv = 1 / den
  __device__ __forceinline__ Divide(float n, float d) {
    const int e = static_cast<int>(__float_as_uint(d) >> 23) - 127;  // d: normal, positive
    // 2^-e in two factors: e = 127 has no float of its own.
    const float a = __uint_as_float(static_cast<uint32_t>(127 - (e >> 1)) << 23);
    const float b = __uint_as_float(static_cast<uint32_t>(127 - (e - (e >> 1))) << 23);
    // A negative earlier scale may be any multiple of the new one: from 2^20 on every
    // code but 0 passes the format's largest alike.
    num = fmaxf(n * a * b, -0x1p20f);
    den = d * a * b;
    inv = 1.f / den;
  }
};

// Eight codes of x * num / den.  The quotient q of x' = x * num, its remainder r
// and q1 = q + r * inv, which is within one unit of the exact quotient; the
// remainder of q1 is exact, and its sign says on which side of q1 the quotient
// lies.  Cut toward zero, with the last bit set where anything was cut, it then
// rounds to the format as the exact quotient would: no value of the format and
// none half way between two has that bit.  kPair: x' does not fit one float (a
// code times a scale), and is taken as two; an earlier scale may have been
// negative, and the quotient then beyond INT8.
template <int FMT, bool kPair>
__device__ __forceinline__ uint2 codes8(const float (&x)[8], const Divide &by) {
  float q[8];
  const float2 n2 = make_float2(by.num, by.num), i2 = make_float2(by.inv, by.inv);
  const float2 d2 = make_float2(-by.den, -by.den), z2 = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float2 x2 = make_float2(x[i], x[i + 1]);
    const float2 xp = fma2(x2, n2, z2);
    const float2 xe = kPair ? fma2(x2, n2, make_float2(-xp.x, -xp.y)) : z2;
    const float2 q0 = fma2(xp, i2, z2);
    float2 r = fma2(q0, d2, xp);
    if (kPair) r = add2(r, xe);
    const float2 q1 = fma2(r, i2, q0);
    float2 left = fma2(q1, d2, xp);
    if (kPair) left = add2(left, xe);
    const float l[2] = {left.x, left.y}, g[2] = {q1.x, q1.y};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      uint32_t u = __float_as_uint(g[k]);
      const bool some = l[k] != 0.f;
      if (some && static_cast<int>(u ^ __float_as_uint(l[k])) < 0) --u;
      if (some) u |= 1u;
      q[i + k] = __uint_as_float(u);
      if (kPair && FMT == ATTN_KV_INT8) q[i + k] = fminf(fmaxf(q[i + k], -128.f), 127.f);
    }
  }
  return make_uint2(codes4<FMT>(q), codes4<FMT>(q + 4));
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

// Eight codes of x * f, f one product's factor.
template <int FMT>
__device__ __forceinline__ uint2 codes8_by_product(const float (&x)[8], float f) {
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float2 y = fma2(make_float2(x[i], x[i + 1]), make_float2(f, f), make_float2(0.f, 0.f));
    q[i] = y.x;
    q[i + 1] = y.y;
  }
  return make_uint2(codes4<FMT>(q), codes4<FMT>(q + 4));
}

struct WriteParams {
  const void *x[2];            // k, v (bf16)
  long long xt[2], xh[2];      // their token and head strides
  uint8_t *pages[2];
  float *scales[2];
  const int *block_table, *seq_lens, *cu_q;
  unsigned *status;
  int Hkv, T, max_q, max_blocks, num_pages, pages_per_seq, parts;
};

// Block: sequence and page of its chunk, and four of the 2 * Hkv slices (K's heads,
// then V's).
template <int D, int FMT>
__global__ void __launch_bounds__(kWarps * 32, 6) kv_write_kernel(const WriteParams p) {
  constexpr int LPR = D / 8, RPP = 32 / LPR, PASSES = kPage / RPP;  // lanes per row, rows per pass
  constexpr float kQmax = FMT == ATTN_KV_E4M3 ? 448.f : 127.f;
  const int lane = threadIdx.x & 31;
  const int pages = gridDim.x / p.parts;
  const int part = blockIdx.x / pages, at = blockIdx.x % pages;
  const int s = at / p.pages_per_seq, j = at % p.pages_per_seq;
  const int item = part * kWarps + (threadIdx.x >> 5);
  if (item >= 2 * p.Hkv) return;
  Chunk c;
  if (!chunk_of(p.seq_lens, p.cu_q, s, p.T, p.max_q, p.max_blocks, c)) {
    if (threadIdx.x == 0 && j == 0 && part == 0) atomicOr(p.status, ATTN_DEV_BAD_PAGE);
    return;
  }
  const int page = c.ctx / kPage + j;
  if (c.nq == 0 || page * kPage >= c.n) return;
  const int pid = p.block_table[static_cast<size_t>(s) * p.max_blocks + page];
  const int lo = max(c.ctx - page * kPage, 0), hi = min(kPage, c.n - page * kPage);
  const int kv = item >= p.Hkv, head = item - kv * p.Hkv;
  const int row = lane / LPR, col = (lane % LPR) * 8;
  // Row r of the page is row q0 + page*16 + r - ctx of x.  The new rows come
  // along with the page's number, which they do not hang on.
  const __nv_bfloat16 *x = static_cast<const __nv_bfloat16 *>(p.x[kv]) +
                           (c.q0 + static_cast<long long>(page) * kPage - c.ctx) * p.xt[kv] +
                           head * p.xh[kv] + col;
  uint4 in[PASSES];
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int r = i * RPP + row;
    in[i] = make_uint4(0, 0, 0, 0);
    if (r >= lo && r < hi) in[i] = *reinterpret_cast<const uint4 *>(x + r * p.xt[kv]);
  }
  if (pid < 0 || pid >= p.num_pages) {
    if (threadIdx.x == 0 && part == 0) atomicOr(p.status, ATTN_DEV_BAD_PAGE);
    return;
  }
  const size_t slice = static_cast<size_t>(pid) * p.Hkv + head;
  uint8_t *codes = p.pages[kv] + slice * (kPage * D) + col;
  uint2 was[PASSES];  // earlier rows' codes
  const float s_old = lo > 0 ? p.scales[kv][slice] : 0.f;
  if (lo > 0) {
#pragma unroll
    for (int i = 0; i < PASSES; ++i)
      if (i * RPP + row < lo) was[i] = *reinterpret_cast<const uint2 *>(codes + (i * RPP + row) * D);
  }
  // Largest magnitude, two at a time, as bits: NaN above infinity above every
  // finite value.
  __nv_bfloat162 most = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const uint32_t w[4] = {in[i].x, in[i].y, in[i].z, in[i].w};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      most = __hmax2_nan(most, __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&w[e])));
  }
  uint32_t top = *reinterpret_cast<const uint32_t *>(&most) & 0x7fff7fffu;
  top = __reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16));
  const float amax = __uint_as_float(top << 16);
  const float s_own = amax / kQmax;
  float s_new = fmaxf(s_own, 1.17549435e-38f);
  const bool odd = top >= 0x7f80u || !(fabsf(s_old) <= 3.4028235e38f);  // a NaN or infinity
  if (lo > 0) s_new = fmaxf(s_new, s_old);
  if (odd) s_new = __uint_as_float(0x7fc00000u);
  if (lane == 0) p.scales[kv][slice] = s_new;

  // On which side of amax / qmax its rounding put the scale (exact: a multiple of
  // the scale's last bit, of 8 bits at most).
  const float left = fmaf(-s_new, kQmax, amax);
  const bool by_product = s_new == s_own && left != 0.f;
  const float factor = (1.f / s_new) * (left > 0.f ? 1.f + 0x1p-22f : 1.f - 0x1p-22f);
  const bool again = lo > 0 && s_new != s_old && !odd;
  const Divide by(1.f, odd ? 1.f : s_new), rescale(again ? s_old : 0.f, odd ? 1.f : s_new);
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
          odd ? make_uint2(0, 0)
              : (by_product ? codes8_by_product<FMT>(v, factor) : codes8<FMT, false>(v, by));
    } else if (r < lo && again) {
      values4<FMT>(was[i].x, v);
      values4<FMT>(was[i].y, v + 4);
      *reinterpret_cast<uint2 *>(codes + r * D) = codes8<FMT, true>(v, rescale);
    }
  }
}

struct ReadParams {
  const uint8_t *pages[2];
  const float *scales[2];
  void *out[2];  // [T, Hkv, D]
  const int *block_table, *seq_lens, *cu_q;
  unsigned *status;
  int Hkv, T, max_q, max_blocks, num_pages, pages_per_seq, parts;
};

// A code times a scale, for a rounding to bf16 as of the exact product.  (Rounded to
// float32 first, a product next to a tie lands on it: 27 of 4 million INT8 ones.)
// A scale of at most 9 bits, trailing zeros aside, has products of at most 17, which
// float32 holds (but for some below 2^-136, which are zeros in bf16 either way).  The
// products of a longer scale are longer than 9 bits too, and so none of them is a
// bf16 value or half way between two: cut toward zero and with the last bit set,
// they lie on the same side of all of those.  (Reading 64 sequences of up to 8192
// tokens: E4M3 281 us as before, INT8 293 instead of 289.  Of the two float32 values
// around each product the one with the last bit set: 282 and 302, and in a run of
// calls 303 against 285.)
__device__ __forceinline__ uint32_t last_bit(float scale) {
  const uint32_t u = __float_as_uint(scale) & 0x7fffffffu;
  const uint32_t digits = (u & 0x7fffffu) | (u >= 0x800000u ? 0x800000u : 0u);
  return 32 - __clz(digits) - (__ffs(digits) - 1) > 9 ? 1u : 0u;
}

__device__ __forceinline__ void store4(float *p, const float *v) {
  *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
}

// Block: sequence and page of its range, and four K/V heads.
template <int D, int FMT, typename T>
__global__ void __launch_bounds__(kWarps * 32) kv_read_kernel(const ReadParams p) {
  constexpr int LPR = D / 8, RPP = 32 / LPR, PASSES = kPage / RPP;
  const int lane = threadIdx.x & 31;
  const int part = blockIdx.x % p.parts;
  const int at = blockIdx.x / p.parts;
  const int s = at / p.pages_per_seq, j = at % p.pages_per_seq;
  const int head = part * kWarps + (threadIdx.x >> 5);
  if (head >= p.Hkv) return;
  Chunk c;
  if (!chunk_of(p.seq_lens, p.cu_q, s, p.T, p.max_q, p.max_blocks, c)) {
    if (threadIdx.x == 0 && j == 0 && part == 0) atomicOr(p.status, ATTN_DEV_BAD_PAGE);
    return;
  }
  const int page = c.ctx / kPage + j;
  if (c.nq == 0 || page * kPage >= c.n) return;
  const int pid = p.block_table[static_cast<size_t>(s) * p.max_blocks + page];
  const bool bad = pid < 0 || pid >= p.num_pages;
  if (bad && threadIdx.x == 0 && part == 0) atomicOr(p.status, ATTN_DEV_BAD_PAGE);
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
  for (int kv = 0; kv < 2; ++kv) {
    const uint32_t last = last_bit(scale[kv]);
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      const int r = i * RPP + row;
      if (r < lo || r >= hi) continue;
      float v[8];
      values4<FMT>(in[kv][i].x, v);
      values4<FMT>(in[kv][i].y, v + 4);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        v[e] = sizeof(T) == 2 ? __uint_as_float(__float_as_uint(__fmul_rz(v[e], scale[kv])) | last) : v[e] * scale[kv];
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
  const long long parts = (2LL * Hkv + kWarps - 1) / kWarps;
  const long long blocks = static_cast<long long>(S) * p.pages_per_seq;
  if (blocks > 0x7fffffffLL / parts) return ATTN_ERR_INVALID_ARG;
  p.parts = static_cast<int>(parts);
  const dim3 grid(static_cast<unsigned>(blocks * parts));
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
  const long long parts = (static_cast<long long>(Hkv) + kWarps - 1) / kWarps;
  const long long blocks = static_cast<long long>(S) * p.pages_per_seq;
  if (blocks > 0x7fffffffLL / parts) return ATTN_ERR_INVALID_ARG;
  p.parts = static_cast<int>(parts);
  const dim3 grid(static_cast<unsigned>(blocks * parts));
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
