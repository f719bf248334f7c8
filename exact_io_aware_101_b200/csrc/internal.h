// internal.h -- launchers shared between the kernel files and the C ABI layer.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stddef.h>

#include "../../include/exattn.h"

namespace exattn {

// window > 0: sliding window; slopes (device, one per query head) or nullptr: ALiBi.
attn_status_t launch_prefill_bf16(const void *q, const void *k, const void *v, void *o, float *lse,
                                  int B, int Hq, int Hkv, int N, int d, float scale, int causal,
                                  int window, const float *slopes, cudaStream_t stream,
                                  unsigned *status);

// Chunked prefill over a paged cache (causal from the end of each sequence).
attn_status_t launch_prefill_paged(const void *q, const void *k_pages, const void *v_pages,
                                   const int *block_table, const int *seq_lens, const int *cu_q,
                                   void *o, float *lse, int S, int Hq, int Hkv, int T, int max_q,
                                   int d, int max_blocks, int num_pages, float scale, int window,
                                   const float *slopes, cudaStream_t stream, unsigned *status);

attn_status_t launch_prefill_f32(const float *q, const float *k, const float *v, float *o,
                                 float *lse, int B, int Hq, int Hkv, int N, int d, float scale,
                                 int causal, int window, const float *slopes,
                                 cudaStream_t stream);

// Number of key chunks (pages per chunk fixed) a sequence of max_blocks pages
// can be split into, and the workspace layout that follows from it.  The
// workspace starts with a 256-byte block whose first word is the call's
// ATTN_DEV_* status (read by attn_decode_read_status), then the chunk partials.
constexpr size_t kDecodeStatusBytes = 256;
struct DecodeWs {
  unsigned *status;  // the call's status word (cleared by the split kernel)
  float *o_part;     // [S][Hq][nsplit][d] normalised chunk outputs
  float *l2_part;    // [S][Hq][nsplit] chunk log2-sum-exps (tagged NaN: failed chunk)
};
int decode_max_splits(int max_blocks);
size_t decode_workspace_bytes(int S, int Hq, int d, int max_blocks);
DecodeWs decode_ws_layout(void *workspace, int S, int Hq, int d, int max_blocks);

// dev_status: nullptr, or a second word (the per-device one) that also gets
// the call's bits.
attn_status_t launch_decode_paged(const void *q, const void *k_pages, const void *v_pages,
                                  const int *block_table, const int *seq_lens, void *o, float *lse,
                                  int S, int Hq, int Hkv, int d, int max_blocks, int num_pages,
                                  float scale, void *workspace, cudaStream_t stream,
                                  unsigned *dev_status);

// Merge the chunk partials of a split decode into O (bf16) and L; chunks hold
// pages_per_split pages.  Failed chunks' bits go to ws.status (and dev_status).
attn_status_t launch_decode_combine(const DecodeWs &ws, const int *seq_lens, void *o, float *lse,
                                    int S, int Hq, int d, int max_blocks, int nsplit,
                                    int pages_per_split, cudaStream_t stream,
                                    unsigned *dev_status);

// The same decode over 8-bit pages (kv_format ATTN_KV_E4M3 or ATTN_KV_INT8) with
// per-(page, K/V head) fp32 scales; same workspace.
attn_status_t launch_decode_paged_q8(const void *q, const void *k_pages, const void *v_pages,
                                     const float *k_scales, const float *v_scales, int kv_format,
                                     const int *block_table, const int *seq_lens, void *o,
                                     float *lse, int S, int Hq, int Hkv, int d, int max_blocks,
                                     int num_pages, float scale, void *workspace,
                                     cudaStream_t stream);

// Chunked prefill over the 8-bit pages; workspace: the parts of a call whose keys
// are split (0 bytes where it is not).
size_t prefill_q8_workspace_bytes(int S, int Hq, int Hkv, int T, int max_q, int d, int max_blocks);
attn_status_t launch_prefill_paged_q8(const void *q, const void *k_pages, const void *v_pages,
                                      const float *k_scales, const float *v_scales, int kv_format,
                                      const int *block_table, const int *seq_lens, const int *cu_q,
                                      void *o, float *lse, int S, int Hq, int Hkv, int T, int max_q,
                                      int d, int max_blocks, int num_pages, float scale, int window,
                                      const float *slopes, void *workspace, cudaStream_t stream,
                                      unsigned *status);

// Writing a chunk's keys and values into the 8-bit pages (strides: k's token and
// head stride, then v's, in elements) and reading a range of tokens back.
attn_status_t launch_kv_write_q8(const void *k, const void *v, const long long (&strides)[4],
                                 void *k_pages, void *v_pages, float *k_scales, float *v_scales,
                                 int kv_format, const int *block_table, const int *seq_lens,
                                 const int *cu_q, int S, int Hkv, int T, int max_q, int d,
                                 int max_blocks, int num_pages, cudaStream_t stream,
                                 unsigned *status);
attn_status_t launch_kv_read_q8(const void *k_pages, const void *v_pages, const float *k_scales,
                                const float *v_scales, int kv_format, const int *block_table,
                                const int *seq_lens, const int *cu_q, void *k, void *v, int dtype,
                                int S, int Hkv, int T, int max_q, int d, int max_blocks,
                                int num_pages, cudaStream_t stream, unsigned *status);

// Rotary positions (op 0), a norm of each head before them (1), the gradient of
// that (2).  One side is q, the other k (H = 0: none).
struct RopeSide {
  const void *x, *dy;
  void *y;        // output, or dx
  const void *w;  // norm weights
  float *dw;
  attn_strides_t x_st, y_st, dy_st;
  int H;
};
size_t norm_rope_bwd_workspace_bytes(long long tokens, int Hq, int Hkv, int d);
attn_status_t launch_rope(const RopeSide &q, const RopeSide &k, const int *positions,
                          long long pos_stride, const double *inv_freq, int dtype, int op, int B,
                          int N, int d, int rot, int interleaved, float factor, int transpose,
                          float eps, void *workspace, cudaStream_t stream);

// Backward: workspace (L*log2e and rowsum(dO*O) per query row, padded to whole
// 128-row tiles) and the three-kernel launch.
size_t bwd_workspace_bytes(int B, int Hq, int N);
attn_status_t launch_attn_bwd(const void *q, const void *k, const void *v, const void *o,
                              const float *lse, const void *dout, void *dq, void *dk, void *dv,
                              int B, int Hq, int Hkv, int N, int d, float scale, int causal,
                              int window, const float *slopes, void *workspace,
                              cudaStream_t stream, unsigned *status);

// cuTensorMapEncodeTiled, or nullptr if the driver does not provide it.
PFN_cuTensorMapEncodeTiled_v12000 encode_fn();

// Device address of the fixed scratch array used by attn_decode_paged_noalloc
// (ATTN_DECODE_NOALLOC_SCRATCH_BYTES bytes) on the current device.
attn_status_t noalloc_scratch_address(void **addr);

}  // namespace exattn
