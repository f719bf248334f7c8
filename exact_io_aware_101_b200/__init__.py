"""exact_io_aware_101_b200 -- exact, IO-aware attention on NVIDIA B200 (sm_100a).

A thin ctypes binding over ``libexattn.so`` (C ABI in ``include/exattn.h``).
Every step of the computation runs in the library's CUDA kernels; this module
only checks tensors, allocates outputs with PyTorch and passes device pointers
and the current CUDA stream.  There is no fallback: if the library is missing
or the device is not sm_100, calls raise.

    o, lse = attn_fwd(q, k, v, causal=True)                  # bf16 prefill
    o, lse = attn_fwd_f32(q, k, v)                           # fp32 prefill
    o, lse = attn_decode_paged(q, k_pages, v_pages, block_table, seq_lens)

and, around them, the rotation of queries and keys by their positions (with or
without a norm of each head, and its gradients) and the 8-bit paged cache:

    inv_freq, factor = rope_frequencies(128)
    q, k = attn_norm_rope(q, k, q_weight, k_weight, positions, inv_freq)
    attn_kv_write_paged_q8(k, v, k_pages, v_pages, k_scales, v_scales, block_table,
                           seq_lens, cu_q, max_q)
    o, lse = attn_prefill_paged_q8(q, k_pages, v_pages, k_scales, v_scales, block_table,
                                   seq_lens, cu_q, max_q)

Device-side failures (a corrupt block table, a bounded wait that ran out) are
reported as ATTN_DEV_* bits: a decode given a ``workspace`` reports into that
workspace (``decode_read_status``), every other call into the device's word
(``device_status``).
"""
from __future__ import annotations

import ctypes
import math
import os
import struct

import torch

__all__ = [
    "attn_fwd", "attn_fwd_f32", "attn_decode_paged", "attn_decode_paged_noalloc",
    "attn_decode_paged_q8", "KV_FORMATS", "decode_workspace_bytes", "attn_bwd",
    "attn_prefill_paged",
    "rope_frequencies", "attn_rope", "attn_norm_rope", "attn_norm_rope_bwd",
    "norm_rope_bwd_workspace_bytes", "attn_kv_write_paged_q8", "attn_kv_read_paged_q8",
    "attn_prefill_paged_q8", "prefill_q8_workspace_bytes",
    "bwd_workspace_bytes", "DECODE_NOALLOC_SCRATCH_BYTES",
    "device_status", "decode_read_status", "status_string", "version", "library", "LIB_PATH", "EXPORTED_SYMBOLS",
    "ATTN_DEV_BAD_PAGE", "ATTN_DEV_TIMEOUT", "ATTN_DEV_LAYOUT", "AttnError",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libexattn.so")
EXPORTED_SYMBOLS = ("attn_fwd", "attn_fwd_f32", "attn_fwd_ext", "attn_fwd_f32_ext",
                    "attn_bwd_workspace_bytes", "attn_bwd", "attn_prefill_paged",
                    "attn_decode_workspace_bytes",
                    "attn_decode_paged", "attn_decode_paged_noalloc", "attn_decode_paged_q8",
                    "attn_kv_write_paged_q8", "attn_kv_read_paged_q8",
                    "attn_prefill_q8_workspace_bytes", "attn_prefill_paged_q8",
                    "attn_rope", "attn_norm_rope", "attn_norm_rope_bwd_workspace_bytes",
                    "attn_norm_rope_bwd",
                    "attn_decode_read_status", "attn_device_status",
                    "attn_status_string", "attn_version")
# Size of the library's fixed per-device scratch used by attn_decode_paged_noalloc.
DECODE_NOALLOC_SCRATCH_BYTES = 32 << 20
ATTN_DEV_BAD_PAGE = 0x1
ATTN_DEV_TIMEOUT = 0x2
ATTN_DEV_LAYOUT = 0x4
# kv_format codes of attn_decode_paged_q8 and the torch dtypes accepted for each.
KV_FORMATS = {"e4m3": 0, "int8": 1}
_KV_DTYPES = {"e4m3": (torch.float8_e4m3fn, torch.uint8), "int8": (torch.int8,)}
# Element types of the rotations and of attn_kv_read_paged_q8 (ATTN_DTYPE_*).
_DTYPES = {torch.bfloat16: 0, torch.float32: 1}
_STATUS = {0: "ATTN_OK", 1: "ATTN_ERR_INVALID_ARG", 2: "ATTN_ERR_UNSUPPORTED", 3: "ATTN_ERR_CUDA"}

_lib = None


class AttnError(RuntimeError):
    def __init__(self, code: int, what: str):
        super().__init__("%s failed: %s" % (what, _STATUS.get(code, "status %d" % code)))
        self.code = code


def load_library(path: str) -> ctypes.CDLL:
    """Load a build of the C ABI at ``path`` and declare every entry point's types."""
    if not os.path.exists(path):
        raise ImportError("%s is not built; run `python -m exact_io_aware_101_b200.build`" % path)
    lib = ctypes.CDLL(path)
    _declare(lib)
    return lib


def library() -> ctypes.CDLL:
    """Load libexattn.so (built by ``python -m exact_io_aware_101_b200.build``)."""
    global _lib
    if _lib is None:
        _lib = load_library(LIB_PATH)
    return _lib


def _declare(lib: ctypes.CDLL) -> None:
    vp, ci, cf = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    lib.attn_fwd.argtypes = [vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, cf, ci, vp]
    lib.attn_fwd.restype = ci
    lib.attn_fwd_f32.argtypes = [vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, cf, ci, vp]
    lib.attn_fwd_f32.restype = ci
    lib.attn_fwd_ext.argtypes = [vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, cf, ci, ci, vp, vp]
    lib.attn_fwd_ext.restype = ci
    lib.attn_fwd_f32_ext.argtypes = [vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, cf, ci, ci, vp, vp]
    lib.attn_fwd_f32_ext.restype = ci
    lib.attn_prefill_paged.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, ci,
                                       ci, ci, ci, cf, ci, vp, vp]
    lib.attn_prefill_paged.restype = ci
    lib.attn_bwd_workspace_bytes.argtypes = [ci, ci, ci]
    lib.attn_bwd_workspace_bytes.restype = ctypes.c_size_t
    lib.attn_bwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, cf, ci, ci,
                             vp, vp, ctypes.c_size_t, vp]
    lib.attn_bwd.restype = ci
    lib.attn_decode_workspace_bytes.argtypes = [ci, ci, ci, ci, ci]
    lib.attn_decode_workspace_bytes.restype = ctypes.c_size_t
    lib.attn_decode_paged.argtypes = [vp, vp, vp, vp, vp, vp, vp, ci, ci, ci, ci, ci, ci, ci,
                                      cf, vp, ctypes.c_size_t, vp]
    lib.attn_decode_paged.restype = ci
    lib.attn_decode_paged_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, ci, ci, ci, ci, ci,
                                              ci, ci, cf, vp]
    lib.attn_decode_paged_noalloc.restype = ci
    lib.attn_decode_paged_q8.argtypes = [vp, vp, vp, vp, vp, ci, vp, vp, vp, vp, ci, ci, ci,
                                         ci, ci, ci, ci, cf, vp, ctypes.c_size_t, vp]
    lib.attn_decode_paged_q8.restype = ci
    i64, st, sz = ctypes.c_int64, vp, ctypes.c_size_t  # st: attn_strides_t, three int64
    lib.attn_kv_write_paged_q8.argtypes = [vp, i64, i64, vp, i64, i64, vp, vp, vp, vp, ci, vp, vp,
                                           vp, ci, ci, ci, ci, ci, ci, ci, ci, vp]
    lib.attn_kv_write_paged_q8.restype = ci
    lib.attn_kv_read_paged_q8.argtypes = [vp, vp, vp, vp, ci, vp, vp, vp, vp, vp, ci, ci, ci, ci,
                                          ci, ci, ci, ci, ci, vp]
    lib.attn_kv_read_paged_q8.restype = ci
    lib.attn_prefill_q8_workspace_bytes.argtypes = [ci] * 8
    lib.attn_prefill_q8_workspace_bytes.restype = sz
    lib.attn_prefill_paged_q8.argtypes = [vp, vp, vp, vp, vp, ci, vp, vp, vp, vp, vp, ci, ci, ci,
                                          ci, ci, ci, ci, ci, ci, cf, ci, vp, vp, sz, vp]
    lib.attn_prefill_paged_q8.restype = ci
    lib.attn_rope.argtypes = [vp, st, vp, st, vp, st, vp, st, vp, i64, vp, ci, ci, ci, ci, ci, ci,
                              ci, ci, cf, ci, vp]
    lib.attn_rope.restype = ci
    lib.attn_norm_rope.argtypes = [vp, st, vp, vp, st, vp, st, vp, vp, st, vp, i64, vp, ci, ci, ci,
                                   ci, ci, ci, ci, ci, cf, cf, vp]
    lib.attn_norm_rope.restype = ci
    lib.attn_norm_rope_bwd_workspace_bytes.argtypes = [ci] * 5
    lib.attn_norm_rope_bwd_workspace_bytes.restype = sz
    lib.attn_norm_rope_bwd.argtypes = [vp, st, vp, vp, st, vp, st, vp, vp, st, vp, vp, st, vp, st,
                                       vp, vp, i64, vp, ci, ci, ci, ci, ci, ci, ci, ci, cf, cf, vp,
                                       sz, vp]
    lib.attn_norm_rope_bwd.restype = ci
    lib.attn_decode_read_status.argtypes = [vp, ctypes.POINTER(ctypes.c_uint)]
    lib.attn_decode_read_status.restype = ci
    lib.attn_device_status.argtypes = [ctypes.POINTER(ctypes.c_uint), ci, vp]
    lib.attn_device_status.restype = ci
    lib.attn_status_string.argtypes = [ci]
    lib.attn_status_string.restype = ctypes.c_char_p
    lib.attn_version.argtypes = []
    lib.attn_version.restype = ctypes.c_char_p


def status_string(code: int) -> str:
    return library().attn_status_string(int(code)).decode()


def version() -> str:
    return library().attn_version().decode()


def _stream(t: torch.Tensor) -> int:
    # (current_stream(device).cuda_stream makes a Stream object on the way: 2.4 us a call.)
    return torch._C._cuda_getCurrentRawStream(t.get_device())


def _check(t: torch.Tensor, name: str, dtype, ndim: int):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.dim() != ndim:
        raise ValueError("%s must have %d dims, got shape %s" % (name, ndim, tuple(t.shape)))
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _dims(t, name: str, ndim: int):
    """Type and rank of one argument, checked before its dtype or device so that
    shape errors are reported the same way on any device."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dim() != ndim:
        raise ValueError("%s must have %d dims, got shape %s" % (name, ndim, tuple(t.shape)))


def _same_device(device, **tensors):
    """Every tensor of one call must live on the device the call runs on: the
    kernel is launched there, and another GPU's pointer is not valid in it."""
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError("%s is on %s but q is on %s" % (name, t.device, device))


def _is(t, dtype, ndim: int, index: int) -> bool:
    """Whether a tensor is a dense one of this type and rank on this GPU: what _check and
    _same_device ask, in a few attribute reads (they name what is wrong where it is not)."""
    return (t.dtype is dtype and t.dim() == ndim and t.is_contiguous() and
            t.get_device() == index >= 0)  # (-1: not on a GPU)


class _Call:
    """One entry point of the library, called with the tensors' device current (switched only
    where another is) and its error raised."""

    def __init__(self, name: str):
        self.name = name

    def __call__(self, index: int, *args):
        fn = getattr(library(), self.name)
        if torch._C._cuda_getDevice() == index:
            rc = fn(*args)
        else:
            with torch.cuda.device(index):
                rc = fn(*args)
        if rc != 0:
            raise AttnError(rc, self.name)


def _raise(rc: int, what: str):
    if rc != 0:
        raise AttnError(rc, what)


def _prefill(fn, what, q, k, v, causal, scale, out, lse, dtype, window=0, alibi_slopes=None):
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _dims(t, n, 4)
    B, Hq, N, d = q.shape
    if k.shape != v.shape or k.shape[0] != B or k.shape[2] != N or k.shape[3] != d:
        raise ValueError("k/v must be [B, Hkv, N, d] matching q %s" % (tuple(q.shape),))
    Hkv = k.shape[1]
    if out is not None:
        _dims(out, "out", 4)
    if lse is not None:
        _dims(lse, "lse", 3)
    if (out is not None and tuple(out.shape) != tuple(q.shape)) or \
            (lse is not None and tuple(lse.shape) != (B, Hq, N)):
        raise ValueError("out/lse shapes do not match q")
    if alibi_slopes is not None:
        _dims(alibi_slopes, "alibi_slopes", 1)
        if alibi_slopes.numel() != Hq:
            raise ValueError("alibi_slopes needs one value per query head")
    for t, n in ((q, "q"), (k, "k"), (v, "v")):
        _check(t, n, dtype, 4)
    _same_device(q.device, k=k, v=v, out=out, lse=lse, alibi_slopes=alibi_slopes)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, Hq, N), dtype=torch.float32, device=q.device)
    _check(out, "out", dtype, 4)
    _check(lse, "lse", torch.float32, 3)
    if tuple(out.shape) != tuple(q.shape) or tuple(lse.shape) != (B, Hq, N):
        raise ValueError("out/lse shapes do not match q")
    if window or alibi_slopes is not None:
        slopes_ptr = None
        if alibi_slopes is not None:
            _check(alibi_slopes, "alibi_slopes", torch.float32, 1)
            slopes_ptr = alibi_slopes.data_ptr()
        ext = getattr(library(), fn.__name__ + "_ext")
        with torch.cuda.device(q.device):
            rc = ext(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                     B, Hq, Hkv, N, d, float(scale), int(bool(causal)), int(window), slopes_ptr,
                     _stream(q))
    else:
        with torch.cuda.device(q.device):
            rc = fn(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                    B, Hq, Hkv, N, d, float(scale), int(bool(causal)), _stream(q))
    _raise(rc, what)
    return out, lse


def attn_fwd(q, k, v, causal: bool = False, scale: float | None = None, out=None, lse=None,
             window: int = 0, alibi_slopes=None):
    """bf16 prefill: q [B,Hq,N,d], k/v [B,Hkv,N,d] -> (O bf16 [B,Hq,N,d], L fp32 [B,Hq,N]).

    window > 0 (with causal): keys with i - j >= window are masked.  alibi_slopes:
    a CUDA float32 tensor [Hq]; slope_h * (j - i) is added to the scaled scores.
    """
    return _prefill(library().attn_fwd, "attn_fwd", q, k, v, causal, scale, out, lse,
                    torch.bfloat16, window, alibi_slopes)


def attn_fwd_f32(q, k, v, causal: bool = False, scale: float | None = None, out=None, lse=None,
                 window: int = 0, alibi_slopes=None):
    """fp32 prefill with fp32 arithmetic throughout (same options as attn_fwd)."""
    return _prefill(library().attn_fwd_f32, "attn_fwd_f32", q, k, v, causal, scale, out, lse,
                    torch.float32, window, alibi_slopes)


def attn_prefill_paged(q, k_pages, v_pages, block_table, seq_lens, cu_q, max_q: int,
                       scale: float | None = None, window: int = 0, alibi_slopes=None,
                       out=None, lse=None):
    """Chunked prefill over the paged cache.

    q [T,Hq,d] bf16 token-major (sequence s: rows cu_q[s]..cu_q[s+1]-1, the
    last tokens of its seq_lens[s]); pages [num_pages,Hkv,16,d] bf16;
    block_table [S,max_blocks], seq_lens [S], cu_q [S+1] int32 (GPU).  max_q
    bounds every chunk length.  Returns (O bf16 [T,Hq,d], L fp32 [T,Hq]).
    """
    for name, t, nd in (("q", q, 3), ("k_pages", k_pages, 4), ("v_pages", v_pages, 4),
                        ("block_table", block_table, 2), ("seq_lens", seq_lens, 1),
                        ("cu_q", cu_q, 1)):
        _dims(t, name, nd)
    T, Hq, d = q.shape
    num_pages, Hkv, page_size, d2 = k_pages.shape
    S = seq_lens.shape[0]
    if d2 != d or tuple(v_pages.shape) != tuple(k_pages.shape):
        raise ValueError("page pools must be [num_pages, Hkv, page_size, d]")
    if block_table.shape[0] != S or cu_q.shape[0] != S + 1:
        raise ValueError("block_table needs S rows and cu_q S+1 entries")
    if out is not None:
        _dims(out, "out", 3)
    if lse is not None:
        _dims(lse, "lse", 2)
    if (out is not None and tuple(out.shape) != tuple(q.shape)) or \
            (lse is not None and tuple(lse.shape) != (T, Hq)):
        raise ValueError("out must be [T, Hq, d] and lse [T, Hq]")
    if alibi_slopes is not None:
        _dims(alibi_slopes, "alibi_slopes", 1)
        if alibi_slopes.numel() != Hq:
            raise ValueError("alibi_slopes needs one value per query head")
    _check(q, "q", torch.bfloat16, 3)
    _check(k_pages, "k_pages", torch.bfloat16, 4)
    _check(v_pages, "v_pages", torch.bfloat16, 4)
    _check(block_table, "block_table", torch.int32, 2)
    _check(seq_lens, "seq_lens", torch.int32, 1)
    _check(cu_q, "cu_q", torch.int32, 1)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    out = torch.empty_like(q) if out is None else out
    lse = torch.empty((T, Hq), dtype=torch.float32, device=q.device) if lse is None else lse
    _check(out, "out", torch.bfloat16, 3)
    _check(lse, "lse", torch.float32, 2)
    slopes_ptr = None
    if alibi_slopes is not None:
        _check(alibi_slopes, "alibi_slopes", torch.float32, 1)
        slopes_ptr = alibi_slopes.data_ptr()
    _same_device(q.device, k_pages=k_pages, v_pages=v_pages, block_table=block_table,
                 seq_lens=seq_lens, cu_q=cu_q, out=out, lse=lse, alibi_slopes=alibi_slopes)
    with torch.cuda.device(q.device):
        rc = library().attn_prefill_paged(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
                                          block_table.data_ptr(), seq_lens.data_ptr(),
                                          cu_q.data_ptr(), out.data_ptr(), lse.data_ptr(), S, Hq,
                                          Hkv, T, int(max_q), d, page_size, block_table.shape[1],
                                          num_pages, float(scale), int(window), slopes_ptr,
                                          _stream(q))
    _raise(rc, "attn_prefill_paged")
    return out, lse


def bwd_workspace_bytes(B: int, Hq: int, N: int) -> int:
    return int(library().attn_bwd_workspace_bytes(B, Hq, N))


def attn_bwd(q, k, v, o, lse, dout, causal: bool = False, scale: float | None = None,
             window: int = 0, alibi_slopes=None, dq=None, dk=None, dv=None, workspace=None):
    """Gradients (dQ, dK, dV) of sum(dout * O) for the bf16 attention.

    q, o, dout [B,Hq,N,d] bf16; k, v [B,Hkv,N,d] bf16; lse [B,Hq,N] fp32 as
    attn_fwd returned them for the same inputs and options.  Returns bf16
    (dQ [B,Hq,N,d], dK [B,Hkv,N,d], dV [B,Hkv,N,d]).
    """
    for name, t in (("q", q), ("k", k), ("v", v), ("o", o), ("dout", dout)):
        _dims(t, name, 4)
    _dims(lse, "lse", 3)
    B, Hq, N, d = q.shape
    Hkv = k.shape[1]
    if tuple(o.shape) != tuple(q.shape) or tuple(dout.shape) != tuple(q.shape):
        raise ValueError("o and dout must have q's shape")
    if tuple(k.shape) != (B, Hkv, N, d) or tuple(v.shape) != tuple(k.shape):
        raise ValueError("k and v must be [B, Hkv, N, d]")
    if tuple(lse.shape) != (B, Hq, N):
        raise ValueError("lse must be [B, Hq, N]")
    for name, t, like in (("dq", dq, q), ("dk", dk, k), ("dv", dv, v)):
        if t is not None:
            _dims(t, name, 4)
            if tuple(t.shape) != tuple(like.shape):
                raise ValueError("dq must have q's shape, dk and dv k's shape")
    for name, t in (("q", q), ("o", o), ("dout", dout)):
        _check(t, name, torch.bfloat16, 4)
    _check(k, "k", torch.bfloat16, 4)
    _check(v, "v", torch.bfloat16, 4)
    _check(lse, "lse", torch.float32, 3)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    _check(dq, "dq", torch.bfloat16, 4)
    _check(dk, "dk", torch.bfloat16, 4)
    _check(dv, "dv", torch.bfloat16, 4)
    slopes_ptr = None
    if alibi_slopes is not None:
        alibi_slopes = torch.as_tensor(alibi_slopes, dtype=torch.float32, device=q.device).contiguous()
        if alibi_slopes.numel() != Hq:
            raise ValueError("need one ALiBi slope per query head")
        slopes_ptr = alibi_slopes.data_ptr()
    need = bwd_workspace_bytes(B, Hq, N)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    _check(workspace, "workspace", torch.uint8, 1)
    _same_device(q.device, k=k, v=v, o=o, lse=lse, dout=dout, dq=dq, dk=dk, dv=dv,
                 alibi_slopes=alibi_slopes, workspace=workspace)
    with torch.cuda.device(q.device):
        rc = library().attn_bwd(q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(),
                                lse.data_ptr(), dout.data_ptr(), dq.data_ptr(), dk.data_ptr(),
                                dv.data_ptr(), B, Hq, Hkv, N, d, float(scale), int(bool(causal)),
                                int(window), slopes_ptr, workspace.data_ptr(), workspace.numel(),
                                _stream(q))
    _raise(rc, "attn_bwd")
    return dq, dk, dv


def decode_workspace_bytes(S: int, Hq: int, d: int, max_blocks: int, page_size: int = 16) -> int:
    return int(library().attn_decode_workspace_bytes(S, Hq, d, max_blocks, page_size))


def _decode_dims(q, k_pages, v_pages, block_table, seq_lens):
    """Shapes of a paged decode's tensors, checked against one another before any
    dtype or device check: the library gets no tensor sizes, so a block_table or
    seq_lens with fewer than S rows would be read past its end on the device."""
    for name, t, nd in (("q", q, 3), ("k_pages", k_pages, 4), ("v_pages", v_pages, 4),
                        ("block_table", block_table, 2), ("seq_lens", seq_lens, 1)):
        _dims(t, name, nd)
    S, Hq, d = q.shape
    num_pages, Hkv, page_size, d2 = k_pages.shape
    if d2 != d or tuple(v_pages.shape) != tuple(k_pages.shape):
        raise ValueError("page pools must be [num_pages, Hkv, page_size, d] with q's d, and "
                         "v_pages must match k_pages")
    if block_table.shape[0] != S or seq_lens.shape[0] != S:
        raise ValueError("block_table/seq_lens must have S rows")
    return S, Hq, d, num_pages, Hkv, page_size, block_table.shape[1]


def _decode_out_dims(q, S, Hq, out, lse):
    """Caller-given outputs of a decode, checked for shape before any device check."""
    if out is not None:
        _dims(out, "out", 3)
    if lse is not None:
        _dims(lse, "lse", 2)
    if (out is not None and tuple(out.shape) != tuple(q.shape)) or \
            (lse is not None and tuple(lse.shape) != (S, Hq)):
        raise ValueError("out must be [S, Hq, d] and lse [S, Hq]")


def _decode_outputs(q, S, Hq, out, lse):
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((S, Hq), dtype=torch.float32, device=q.device)
    _check(out, "out", torch.bfloat16, 3)
    _check(lse, "lse", torch.float32, 2)
    if tuple(out.shape) != tuple(q.shape) or tuple(lse.shape) != (S, Hq):
        raise ValueError("out must be [S, Hq, d] and lse [S, Hq]")
    return out, lse


def attn_decode_paged(q, k_pages, v_pages, block_table, seq_lens, scale: float | None = None,
                      out=None, lse=None, workspace=None):
    """Paged single-token decode.

    q [S,Hq,d] bf16; k_pages/v_pages [num_pages,Hkv,page_size,d] bf16;
    block_table [S,max_blocks] int32; seq_lens [S] int32 (all on the GPU).
    Returns (O bf16 [S,Hq,d], L fp32 [S,Hq]).  ``workspace`` (uint8, at least
    decode_workspace_bytes(...) bytes) is allocated when not given; pass one to
    read the call's status afterwards with ``decode_read_status(workspace)``.
    """
    S, Hq, d, num_pages, Hkv, page_size, max_blocks = _decode_dims(q, k_pages, v_pages,
                                                                   block_table, seq_lens)
    _decode_out_dims(q, S, Hq, out, lse)
    _check(q, "q", torch.bfloat16, 3)
    _check(k_pages, "k_pages", torch.bfloat16, 4)
    _check(v_pages, "v_pages", torch.bfloat16, 4)
    _check(block_table, "block_table", torch.int32, 2)
    _check(seq_lens, "seq_lens", torch.int32, 1)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    out, lse = _decode_outputs(q, S, Hq, out, lse)
    need = decode_workspace_bytes(S, Hq, d, max_blocks, page_size)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    _check(workspace, "workspace", torch.uint8, 1)
    _same_device(q.device, k_pages=k_pages, v_pages=v_pages, block_table=block_table,
                 seq_lens=seq_lens, out=out, lse=lse, workspace=workspace)
    with torch.cuda.device(q.device):
        rc = library().attn_decode_paged(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
                                         block_table.data_ptr(), seq_lens.data_ptr(),
                                         out.data_ptr(), lse.data_ptr(), S, Hq, Hkv, d, page_size,
                                         max_blocks, num_pages, float(scale), workspace.data_ptr(),
                                         workspace.numel(), _stream(q))
    _raise(rc, "attn_decode_paged")
    return out, lse


def attn_decode_paged_q8(q, k_pages, v_pages, k_scales, v_scales, block_table, seq_lens,
                         kv_format: str = "e4m3", scale: float | None = None, out=None, lse=None,
                         workspace=None):
    """Paged single-token decode over an 8-bit KV cache.

    k_pages/v_pages [num_pages,Hkv,page_size,d]: E4M3 codes (torch.float8_e4m3fn,
    or their bytes as uint8) for kv_format "e4m3", torch.int8 for "int8";
    k_scales/v_scales [num_pages,Hkv] float32, one per (page, K/V head): the
    element is scale * code.  Everything else (the workspace and its status
    word included) as attn_decode_paged.
    """
    if kv_format not in KV_FORMATS:
        raise ValueError("kv_format must be one of %s" % sorted(KV_FORMATS))
    S, Hq, d, num_pages, Hkv, page_size, max_blocks = _decode_dims(q, k_pages, v_pages,
                                                                   block_table, seq_lens)
    _decode_out_dims(q, S, Hq, out, lse)
    for name, t in (("k_scales", k_scales), ("v_scales", v_scales)):
        _dims(t, name, 2)
        if tuple(t.shape) != (num_pages, Hkv):
            raise ValueError("scales must be [num_pages, Hkv]")
    _check(q, "q", torch.bfloat16, 3)
    for name, t in (("k_pages", k_pages), ("v_pages", v_pages)):
        if t.dtype not in _KV_DTYPES[kv_format]:
            raise TypeError("%s must be one of %s for kv_format %r"
                            % (name, _KV_DTYPES[kv_format], kv_format))
        _check(t, name, t.dtype, 4)
    _check(k_scales, "k_scales", torch.float32, 2)
    _check(v_scales, "v_scales", torch.float32, 2)
    _check(block_table, "block_table", torch.int32, 2)
    _check(seq_lens, "seq_lens", torch.int32, 1)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    out, lse = _decode_outputs(q, S, Hq, out, lse)
    need = decode_workspace_bytes(S, Hq, d, max_blocks, page_size)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    _check(workspace, "workspace", torch.uint8, 1)
    _same_device(q.device, k_pages=k_pages, v_pages=v_pages, k_scales=k_scales,
                 v_scales=v_scales, block_table=block_table, seq_lens=seq_lens, out=out, lse=lse,
                 workspace=workspace)
    with torch.cuda.device(q.device):
        rc = library().attn_decode_paged_q8(q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(),
                                            k_scales.data_ptr(), v_scales.data_ptr(),
                                            KV_FORMATS[kv_format], block_table.data_ptr(),
                                            seq_lens.data_ptr(), out.data_ptr(), lse.data_ptr(), S,
                                            Hq, Hkv, d, page_size, max_blocks, num_pages,
                                            float(scale), workspace.data_ptr(), workspace.numel(),
                                            _stream(q))
    _raise(rc, "attn_decode_paged_q8")
    return out, lse


def attn_decode_paged_noalloc(q, k_pages, v_pages, block_table, seq_lens,
                              scale: float | None = None, out=None, lse=None):
    """Paged decode that allocates no device memory inside the library.

    For callers that may not call cudaMalloc (for example a plugin whose host
    program owns all device memory, or a decode loop that must not wait on the
    allocator): the chunk partials live in the library's fixed per-device scratch
    (DECODE_NOALLOC_SCRATCH_BYTES), shared by every such call on the device, so
    calls that overlap on the GPU race.  Pass ``out`` and ``lse`` to avoid torch
    allocating the outputs here.  Arguments as for attn_decode_paged; a bad page
    id or length is reported in the device's word (``device_status``).
    """
    S, Hq, d, num_pages, Hkv, page_size, max_blocks = _decode_dims(q, k_pages, v_pages,
                                                                   block_table, seq_lens)
    _decode_out_dims(q, S, Hq, out, lse)
    _check(q, "q", torch.bfloat16, 3)
    _check(k_pages, "k_pages", torch.bfloat16, 4)
    _check(v_pages, "v_pages", torch.bfloat16, 4)
    _check(block_table, "block_table", torch.int32, 2)
    _check(seq_lens, "seq_lens", torch.int32, 1)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    out, lse = _decode_outputs(q, S, Hq, out, lse)
    _same_device(q.device, k_pages=k_pages, v_pages=v_pages, block_table=block_table,
                 seq_lens=seq_lens, out=out, lse=lse)
    with torch.cuda.device(q.device):
        rc = library().attn_decode_paged_noalloc(
            q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), block_table.data_ptr(),
            seq_lens.data_ptr(), out.data_ptr(), lse.data_ptr(), S, Hq, Hkv, d, page_size,
            max_blocks, num_pages, float(scale), _stream(q))
    _raise(rc, "attn_decode_paged_noalloc")
    return out, lse


def _q8_cache(k_pages, v_pages, k_scales, v_scales, block_table, seq_lens, cu_q, kv_format):
    """The 8-bit cache and the chunks of a call, checked against one another; shapes first, so
    that they are reported the same way on any device."""
    if kv_format not in KV_FORMATS:
        raise ValueError("kv_format must be one of %s" % sorted(KV_FORMATS))
    try:
        fine = (k_pages.dim() == 4 and k_scales.dim() == 2 and block_table.dim() == 2 and
                seq_lens.dim() == 1 and cu_q.dim() == 1 and v_pages.shape == k_pages.shape and
                v_scales.shape == k_scales.shape)
    except AttributeError:
        fine = False
    if not fine:
        for name, t, nd in (("k_pages", k_pages, 4), ("v_pages", v_pages, 4),
                            ("k_scales", k_scales, 2), ("v_scales", v_scales, 2),
                            ("block_table", block_table, 2), ("seq_lens", seq_lens, 1),
                            ("cu_q", cu_q, 1)):
            _dims(t, name, nd)
        if v_pages.shape != k_pages.shape:
            raise ValueError("v_pages must match k_pages, [num_pages, Hkv, page_size, d]")
    num_pages, Hkv, page_size, d = k_pages.shape
    S, max_blocks = block_table.shape
    if k_scales.shape != (num_pages, Hkv) or v_scales.shape != (num_pages, Hkv):
        raise ValueError("scales must be [num_pages, Hkv]")
    if seq_lens.numel() != S or cu_q.numel() != S + 1:
        raise ValueError("block_table needs S rows and cu_q S+1 entries")
    return num_pages, Hkv, page_size, d, S, max_blocks


def _q8_types(k_pages, v_pages, k_scales, v_scales, block_table, seq_lens, cu_q, kv_format,
              device, index):
    codes = _KV_DTYPES[kv_format]
    f32, i32 = torch.float32, torch.int32
    if (k_pages.dtype in codes and v_pages.dtype in codes and k_scales.dtype is f32 and
            v_scales.dtype is f32 and block_table.dtype is i32 and seq_lens.dtype is i32 and
            cu_q.dtype is i32 and k_pages.is_contiguous() and v_pages.is_contiguous() and
            k_scales.is_contiguous() and v_scales.is_contiguous() and
            block_table.is_contiguous() and seq_lens.is_contiguous() and cu_q.is_contiguous() and
            0 <= index == k_pages.get_device() == v_pages.get_device() == k_scales.get_device() ==
            v_scales.get_device() == block_table.get_device() == seq_lens.get_device() ==
            cu_q.get_device()):
        return
    for name, t in (("k_pages", k_pages), ("v_pages", v_pages)):
        if t.dtype not in codes:
            raise TypeError("%s must be one of %s for kv_format %r" % (name, codes, kv_format))
        _check(t, name, t.dtype, 4)
    _check(k_scales, "k_scales", f32, 2)
    _check(v_scales, "v_scales", f32, 2)
    _check(block_table, "block_table", i32, 2)
    _check(seq_lens, "seq_lens", i32, 1)
    _check(cu_q, "cu_q", i32, 1)
    _same_device(device, k_pages=k_pages, v_pages=v_pages, k_scales=k_scales, v_scales=v_scales,
                 block_table=block_table, seq_lens=seq_lens, cu_q=cu_q)


def _bound(number, most: int) -> int:
    """A count as a C int: what passes most (and changes nothing there) as most, anything negative
    as -1, which the library refuses."""
    return max(-1, min(int(number), most))


_kv_write, _kv_read, _prefill_q8 = (_Call("attn_kv_write_paged_q8"), _Call("attn_kv_read_paged_q8"),
                                    _Call("attn_prefill_paged_q8"))
_rope, _norm_rope, _norm_rope_bwd = (_Call("attn_rope"), _Call("attn_norm_rope"),
                                     _Call("attn_norm_rope_bwd"))


def attn_kv_write_paged_q8(k, v, k_pages, v_pages, k_scales, v_scales, block_table, seq_lens, cu_q,
                           max_q: int, kv_format: str = "e4m3"):
    """Write a chunk's keys and values into the 8-bit cache, in place.

    k, v [T,Hkv,d] bf16 token-major (sequence s: rows cu_q[s]..cu_q[s+1]-1, the
    last tokens of its seq_lens[s], as for attn_prefill_paged_q8); they may be
    views, such as slices of one projection's output, with consecutive elements
    in a row.  Pages, scales, block_table, seq_lens and kv_format as for
    attn_decode_paged_q8; cu_q [S+1] int32; max_q bounds every chunk length.
    A page's scale grows with its tokens, and its earlier tokens are then rounded
    to the new one; a page whose first slot is written starts afresh.  A page
    that is written must belong to one sequence alone.
    """
    num_pages, Hkv, page_size, d, S, max_blocks = _q8_cache(
        k_pages, v_pages, k_scales, v_scales, block_table, seq_lens, cu_q, kv_format)
    if not (isinstance(k, torch.Tensor) and isinstance(v, torch.Tensor) and k.dim() == 3):
        _dims(k, "k", 3)
        _dims(v, "v", 3)
    T = k.shape[0]
    if k.shape != (T, Hkv, d) or v.shape != (T, Hkv, d):
        raise ValueError("k and v must be [T, Hkv, d] as the pages are")
    _rows(k, "k", torch.bfloat16)
    _rows(v, "v", torch.bfloat16)
    device, index = k.device, k.get_device()
    if v.get_device() != index:
        _same_device(device, v=v)
    _q8_types(k_pages, v_pages, k_scales, v_scales, block_table, seq_lens, cu_q, kv_format, device,
              index)
    kh, kt = _row_strides(k)
    vh, vt = _row_strides(v)
    _kv_write(index, k.data_ptr(), kt, kh, v.data_ptr(), vt, vh, k_pages.data_ptr(),
              v_pages.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(), KV_FORMATS[kv_format],
              block_table.data_ptr(), seq_lens.data_ptr(), cu_q.data_ptr(), S, Hkv, T,
              _bound(max_q, T), d, page_size, max_blocks, num_pages, _stream(k))


def attn_kv_read_paged_q8(k_pages, v_pages, k_scales, v_scales, block_table, seq_lens, cu_q,
                          tokens: int, max_q: int, kv_format: str = "e4m3",
                          dtype=torch.bfloat16, k=None, v=None):
    """The last cu_q[s+1] - cu_q[s] tokens of each sequence out of the 8-bit cache.

    Returns (k, v) [tokens,Hkv,d] of dtype (bfloat16 or float32), the element
    scale * code; tokens is cu_q's last entry, or more: rows of no sequence are
    not written.  max_q bounds every sequence's count.  Other arguments as for
    attn_kv_write_paged_q8.
    """
    num_pages, Hkv, page_size, d, S, max_blocks = _q8_cache(
        k_pages, v_pages, k_scales, v_scales, block_table, seq_lens, cu_q, kv_format)
    if dtype not in _DTYPES:
        raise TypeError("dtype must be torch.bfloat16 or torch.float32")
    T = int(tokens)
    shape = (T, Hkv, d)
    for name, t in (("k", k), ("v", v)):
        if t is not None:
            _dims(t, name, 3)
            if t.shape != shape:
                raise ValueError("k and v must be [tokens, Hkv, d]")
    device, index = k_pages.device, k_pages.get_device()
    _q8_types(k_pages, v_pages, k_scales, v_scales, block_table, seq_lens, cu_q, kv_format, device,
              index)
    if k is None:
        k = torch.empty(shape, dtype=dtype, device=device)
    if v is None:
        v = torch.empty_like(k)
    if not (_is(k, dtype, 3, index) and _is(v, dtype, 3, index)):
        _check(k, "k", dtype, 3)
        _check(v, "v", dtype, 3)
        _same_device(device, k=k, v=v)
    _kv_read(index, k_pages.data_ptr(), v_pages.data_ptr(), k_scales.data_ptr(),
             v_scales.data_ptr(), KV_FORMATS[kv_format], block_table.data_ptr(),
             seq_lens.data_ptr(), cu_q.data_ptr(), k.data_ptr(), v.data_ptr(), _DTYPES[dtype], S,
             Hkv, T, _bound(max_q, T), d, page_size, max_blocks, num_pages, _stream(k))
    return k, v


def prefill_q8_workspace_bytes(S: int, Hq: int, Hkv: int, T: int, max_q: int, d: int,
                               max_blocks: int, page_size: int = 16) -> int:
    return int(library().attn_prefill_q8_workspace_bytes(S, Hq, Hkv, T, _bound(max_q, T), d,
                                                         max_blocks, page_size))


def attn_prefill_paged_q8(q, k_pages, v_pages, k_scales, v_scales, block_table, seq_lens, cu_q,
                          max_q: int, kv_format: str = "e4m3", scale: float | None = None,
                          window: int = 0, alibi_slopes=None, out=None, lse=None, workspace=None):
    """Chunked prefill over the 8-bit paged cache.

    q [T,Hq,d] bf16 token-major, cu_q, max_q, window and alibi_slopes as for
    attn_prefill_paged; pages, scales and kv_format as for attn_decode_paged_q8.
    Returns (O bf16 [T,Hq,d], L fp32 [T,Hq]); rows of no sequence are not
    written.  ``workspace`` (uint8, at least prefill_q8_workspace_bytes(...) bytes)
    is allocated when not given; calls that may run at the same time need one each.
    """
    num_pages, Hkv, page_size, d, S, max_blocks = _q8_cache(
        k_pages, v_pages, k_scales, v_scales, block_table, seq_lens, cu_q, kv_format)
    _dims(q, "q", 3)
    T, Hq = q.shape[:2]
    if q.shape[2] != d or Hkv == 0 or Hq % Hkv != 0:
        raise ValueError("q must be [T, Hq, d] with the pages' d and a multiple of their heads")
    _decode_out_dims(q, T, Hq, out, lse)
    if alibi_slopes is not None:
        _dims(alibi_slopes, "alibi_slopes", 1)
        if alibi_slopes.numel() != Hq:
            raise ValueError("alibi_slopes needs one value per query head")
    _check(q, "q", torch.bfloat16, 3)
    device, index = q.device, q.get_device()
    _q8_types(k_pages, v_pages, k_scales, v_scales, block_table, seq_lens, cu_q, kv_format, device,
              index)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    out, lse = _decode_outputs(q, T, Hq, out, lse)
    slopes_ptr = None
    if alibi_slopes is not None:
        _check(alibi_slopes, "alibi_slopes", torch.float32, 1)
        slopes_ptr = alibi_slopes.data_ptr()
    max_q = _bound(max_q, T)  # (no chunk is longer)
    need = prefill_q8_workspace_bytes(S, Hq, Hkv, T, max_q, d, max_blocks, page_size)
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    if workspace is not None:
        _check(workspace, "workspace", torch.uint8, 1)
    _same_device(device, out=out, lse=lse, alibi_slopes=alibi_slopes, workspace=workspace)
    _prefill_q8(index, q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), k_scales.data_ptr(),
                v_scales.data_ptr(), KV_FORMATS[kv_format], block_table.data_ptr(),
                seq_lens.data_ptr(), cu_q.data_ptr(), out.data_ptr(), lse.data_ptr(), S, Hq, Hkv,
                T, max_q, d, page_size, max_blocks, num_pages, float(scale),
                _bound(window, 2**31 - 1), slopes_ptr,
                workspace.data_ptr() if workspace is not None else None,
                workspace.numel() if workspace is not None else 0, _stream(q))
    return out, lse


def rope_frequencies(rot: int, base: float = 10000.0, scaling: str | None = None,
                     factor: float = 1.0, original_length: int = 8192, beta_fast: float = 32.0,
                     beta_slow: float = 1.0, device="cuda"):
    """(inv_freq, attention_factor) for the rotations: inv_freq float64 [rot/2] on device.

    Pair i turns by base^(-2i/rot) radians a position.  For contexts ``factor``
    times the original_length: "linear" divides every frequency by factor (all
    positions are interpolated); "ntk" raises the base so that the slowest pair
    alone is divided by factor and the fastest keeps its pace; "yarn" keeps pairs
    that turn at least beta_fast times over the original length, divides those
    that turn at most beta_slow times, blends in between, linearly in the number
    of turns, and asks for the attention factor 0.1 ln(factor) + 1.  That is the
    method as its paper defines it.  Models trained with a blend that is linear in
    the pair's index, between two rounded indices, have other frequencies for the
    pairs in between: give the calls those as inv_freq.
    """
    if rot < 2 or rot % 2:
        raise ValueError("rot must be even and at least 2")
    if not (math.isfinite(base) and base > 0 and math.isfinite(factor) and factor >= 1.0):
        raise ValueError("base must be positive and factor at least 1")
    i = torch.arange(rot // 2, dtype=torch.float64)
    attention_factor = 1.0
    if scaling == "ntk" and rot > 2:
        base = base * factor ** (rot / (rot - 2.0))
    freq = torch.pow(torch.tensor(base, dtype=torch.float64), -2.0 * i / rot)
    if scaling == "linear":
        freq = freq / factor
    elif scaling == "yarn":
        if not (beta_fast > beta_slow and original_length > 0):
            raise ValueError("yarn needs beta_fast > beta_slow and a positive original_length")
        turns = original_length * freq / (2.0 * math.pi)
        keep = ((turns - beta_slow) / (beta_fast - beta_slow)).clamp(0.0, 1.0)
        freq = freq * keep + freq / factor * (1.0 - keep)
        attention_factor = 0.1 * math.log(factor) + 1.0
    elif scaling not in (None, "ntk"):
        raise ValueError("scaling must be None, 'linear', 'ntk' or 'yarn'")
    return freq.to(device), attention_factor


def _rows(t, name: str, dtype):
    """A tensor of rows: any strides, but consecutive elements in a row."""
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.stride(-1) != 1:
        raise ValueError("%s must have consecutive elements in its last dimension" % name)


def _row_strides(t):
    """(head, token) strides of a [T, H, d] tensor, 0 along an extent of one (where torch may
    report any number)."""
    (T, H, _), (token, head, _) = t.shape, t.stride()
    return head if H > 1 else 0, token if T > 1 else 0


_three = struct.Struct("3q").pack  # an attn_strides_t


def _strides(t):
    """A tensor's attn_strides_t as bytes, which ctypes passes by address."""
    if t is None:
        return None
    n, st = t.shape, t.stride()
    if len(n) == 3:
        return _three(0, st[1] if n[1] > 1 else 0, st[0] if n[0] > 1 else 0)
    return _three(st[0] if n[0] > 1 else 0, st[1] if n[1] > 1 else 0, st[2] if n[2] > 1 else 0)


def _rope_args(q, k, positions, inv_freq, like_q, like_k):
    """Shapes, types and devices of a rotation's tensors.  like_q, like_k: names and tensors
    (or None) that must look like q and k.  Returns B, Hq, Hkv, N, d and the position stride."""
    if not isinstance(q, torch.Tensor):
        raise TypeError("q must be a torch.Tensor")
    nd, qs = q.dim(), q.shape
    if nd == 3:
        N, Hq, d = qs
        B = 1
    elif nd == 4:
        B, Hq, N, d = qs
    else:
        raise ValueError("q must be [B, Hq, N, d] or token-major [T, Hq, d], got shape %s"
                         % (tuple(qs),))
    Hkv = 0
    if k is not None:
        _dims(k, "k", nd)
        ks = k.shape
        Hkv = ks[1]
        if ks != ((N, Hkv, d) if nd == 3 else (B, Hkv, N, d)):
            raise ValueError("k must be %s matching q %s"
                             % ("[T, Hkv, d]" if nd == 3 else "[B, Hkv, N, d]", tuple(qs)))
        if Hkv == 0:
            raise ValueError("k has no heads; None stands for no keys")
    elif any(t is not None for _, t in like_k):
        raise ValueError("%s given without k" % like_k[0][0])
    if not isinstance(positions, torch.Tensor) or not isinstance(inv_freq, torch.Tensor):
        raise TypeError("positions and inv_freq must be torch.Tensors")
    ps = positions.shape
    if ps != (N,) and (nd == 3 or ps != (B, N)):
        raise ValueError("positions must be [T] or [N], or [B, N] with a batch")
    _dims(inv_freq, "inv_freq", 1)
    if not 1 <= inv_freq.shape[0] <= d // 2:
        raise ValueError("inv_freq needs one value per pair, at most d/2")
    for like, ref, what in ((like_q, q, "q"), (like_k, k, "k")):
        for name, t in like:
            if t is not None:
                _dims(t, name, nd)
                if t.shape != ref.shape:
                    raise ValueError("%s must have %s's shape" % (name, what))
    dtype, index = q.dtype, q.get_device()
    if dtype not in _DTYPES:
        raise TypeError("q must be bfloat16 or float32, got %s" % dtype)
    _rows(q, "q", dtype)
    if k is not None:
        _rows(k, "k", dtype)
        if k.get_device() != index:
            _same_device(q.device, k=k)
    for name, t in like_q + like_k:
        if t is not None:
            _rows(t, name, dtype)
            _same_device(q.device, **{name: t})
    if not (_is(positions, torch.int32, len(ps), index) and _is(inv_freq, torch.float64, 1, index)):
        _check(positions, "positions", torch.int32, len(ps))
        _check(inv_freq, "inv_freq", torch.float64, 1)
        _same_device(q.device, positions=positions, inv_freq=inv_freq)
    return B, Hq, Hkv, N, d, N if len(ps) == 2 else 0


def _ptr(t):
    return None if t is None else t.data_ptr()


def _empty_rows(t):
    return None if t is None else torch.empty_like(t, memory_format=torch.contiguous_format)


def attn_rope(q, k, positions, inv_freq, interleaved: bool = False, attention_factor: float = 1.0,
              transpose: bool = False, q_out=None, k_out=None):
    """Rotary positions of q and k: returns (q_out, k_out).

    q [B,Hq,N,d] and k [B,Hkv,N,d], or token-major [T,Hq,d] and [T,Hkv,d]; bf16 or
    float32; k may be None.  They may be views (slices of one projection's
    output, transposed layouts) with consecutive elements in a row; given outputs
    too, and an output may be its input.  positions int32 [N] or [B,N] ([T]);
    inv_freq float64 [rot/2] (see rope_frequencies): the first rot elements of
    each row turn, pairs (i, i + rot/2) or, interleaved, (2i, 2i+1), times
    attention_factor; the others pass.  transpose applies the transposed map, the
    gradient of the other.
    """
    B, Hq, Hkv, N, d, pos_stride = _rope_args(q, k, positions, inv_freq, [("q_out", q_out)],
                                              [("k_out", k_out)])
    q_out = _empty_rows(q) if q_out is None else q_out
    k_out = _empty_rows(k) if k_out is None else k_out
    _rope(q.get_device(), _ptr(q), _strides(q), _ptr(q_out), _strides(q_out), _ptr(k), _strides(k),
          _ptr(k_out), _strides(k_out), positions.data_ptr(), pos_stride, inv_freq.data_ptr(),
          _DTYPES[q.dtype], B, Hq, Hkv, N, d, 2 * inv_freq.shape[0], int(bool(interleaved)),
          float(attention_factor), int(bool(transpose)), _stream(q))
    return q_out, k_out


def _norm_weights(q, k, q_weight, k_weight):
    if (k is None) != (k_weight is None):
        raise ValueError("k and k_weight go together")
    for name, t in (("q_weight", q_weight), ("k_weight", k_weight)):
        if t is not None or name == "q_weight":
            _dims(t, name, 1)
            if t.shape[0] != q.shape[-1]:
                raise ValueError("%s must be [d]" % name)
            if not _is(t, q.dtype, 1, q.get_device()):
                _check(t, name, q.dtype, 1)
                _same_device(q.device, **{name: t})


def attn_norm_rope(q, k, q_weight, k_weight, positions, inv_freq, eps: float = 1e-6,
                   interleaved: bool = False, attention_factor: float = 1.0, q_out=None,
                   k_out=None):
    """RMS norm of every head's row, times its weights, then attn_rope: (q_out, k_out).

    q_weight, k_weight [d] of q's dtype, shared by the heads (k_weight None without
    k).  Other arguments as for attn_rope.
    """
    B, Hq, Hkv, N, d, pos_stride = _rope_args(q, k, positions, inv_freq, [("q_out", q_out)],
                                              [("k_out", k_out)])
    _norm_weights(q, k, q_weight, k_weight)
    q_out = _empty_rows(q) if q_out is None else q_out
    k_out = _empty_rows(k) if k_out is None else k_out
    _norm_rope(q.get_device(), _ptr(q), _strides(q), _ptr(q_weight), _ptr(q_out), _strides(q_out),
               _ptr(k), _strides(k), _ptr(k_weight), _ptr(k_out), _strides(k_out),
               positions.data_ptr(), pos_stride, inv_freq.data_ptr(), _DTYPES[q.dtype], B, Hq, Hkv,
               N, d, 2 * inv_freq.shape[0], int(bool(interleaved)), float(attention_factor),
               float(eps), _stream(q))
    return q_out, k_out


def norm_rope_bwd_workspace_bytes(B: int, Hq: int, Hkv: int, N: int, d: int) -> int:
    return int(library().attn_norm_rope_bwd_workspace_bytes(B, Hq, Hkv, N, d))


def attn_norm_rope_bwd(q, k, q_weight, k_weight, dq_out, dk_out, positions, inv_freq,
                       eps: float = 1e-6, interleaved: bool = False,
                       attention_factor: float = 1.0, dq=None, dk=None, dq_weight=None,
                       dk_weight=None, workspace=None):
    """Gradients of attn_norm_rope: (dq, dk, dq_weight, dk_weight).

    q, k and the options as given to attn_norm_rope; dq_out, dk_out the gradients of
    its outputs.  dq, dk have q's dtype (dq may be dq_out or q); dq_weight,
    dk_weight are float32 [d].  Without k its parts are None.
    """
    if (k is None) != (dk_out is None):
        raise ValueError("k and dk_out go together")
    if dq_out is None:
        raise TypeError("dq_out must be a torch.Tensor")
    B, Hq, Hkv, N, d, pos_stride = _rope_args(q, k, positions, inv_freq,
                                              [("dq_out", dq_out), ("dq", dq)],
                                              [("dk_out", dk_out), ("dk", dk)])
    _norm_weights(q, k, q_weight, k_weight)
    index = q.get_device()
    for name, t in (("dq_weight", dq_weight), ("dk_weight", dk_weight)):
        if t is not None:
            _dims(t, name, 1)
            if t.shape[0] != d or k is None and name == "dk_weight":
                raise ValueError("%s must be [d], and None without k" % name)
            if not _is(t, torch.float32, 1, index):
                _check(t, name, torch.float32, 1)
                _same_device(q.device, **{name: t})
    dq = _empty_rows(q) if dq is None else dq
    dk = _empty_rows(k) if dk is None else dk
    if dq_weight is None:
        dq_weight = torch.empty(d, dtype=torch.float32, device=q.device)
    if dk_weight is None and k is not None:
        dk_weight = torch.empty_like(dq_weight)
    if workspace is None:
        need = norm_rope_bwd_workspace_bytes(B, Hq, Hkv, N, d)
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    elif not _is(workspace, torch.uint8, 1, index):
        _check(workspace, "workspace", torch.uint8, 1)
        _same_device(q.device, workspace=workspace)
    _norm_rope_bwd(index, _ptr(q), _strides(q), _ptr(q_weight), _ptr(dq_out), _strides(dq_out),
                   _ptr(dq), _strides(dq), _ptr(dq_weight), _ptr(k), _strides(k), _ptr(k_weight),
                   _ptr(dk_out), _strides(dk_out), _ptr(dk), _strides(dk), _ptr(dk_weight),
                   positions.data_ptr(), pos_stride, inv_freq.data_ptr(), _DTYPES[q.dtype], B, Hq,
                   Hkv, N, d, 2 * inv_freq.shape[0], int(bool(interleaved)),
                   float(attention_factor), float(eps), workspace.data_ptr(), workspace.numel(),
                   _stream(q))
    return dq, dk, dq_weight, dk_weight


def decode_read_status(workspace: torch.Tensor) -> int:
    """ATTN_DEV_* bits of the last workspace decode that used ``workspace`` (0: none).

    Synchronises nothing: first synchronise the stream the decode ran on (or an
    event recorded after it)."""
    _check(workspace, "workspace", torch.uint8, 1)
    st = ctypes.c_uint(0)
    with torch.cuda.device(workspace.device):
        rc = library().attn_decode_read_status(workspace.data_ptr(), ctypes.byref(st))
    _raise(rc, "attn_decode_read_status")
    return int(st.value)


def device_status(clear: bool = False, device=None) -> int:
    """Status bits (ATTN_DEV_*) that calls without a decode workspace raised on a device.

    Waits for the work enqueued so far on that device's current stream (and only
    for it)."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    st = ctypes.c_uint(0)
    with torch.cuda.device(dev):
        rc = library().attn_device_status(ctypes.byref(st), int(bool(clear)),
                                          torch.cuda.current_stream(dev).cuda_stream)
    _raise(rc, "attn_device_status")
    return int(st.value)
