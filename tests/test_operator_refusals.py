"""What the rotations and the 8-bit cache's calls refuse, on the CPU: through the C
ABI with addresses that validation turns away before any use, and through the
binding with CPU tensors that never reach the library.  Also the rotations'
frequencies, which need no GPU, against their formulas."""
from __future__ import annotations

import ctypes
import math
import struct

import numpy as np
import pytest
import torch

import exact_io_aware_101_b200 as ea
from exact_io_aware_101_b200 import build as eabuild

INVALID, UNSUPPORTED = 1, 2
A = 1 << 20  # a fake, 16-byte-aligned address: validation fails before any use
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    eabuild.build()
    return ea.library()


def st(b=1 << 16, h=1 << 12, t=128):
    return struct.pack("3q", b, h, t)


# ------------------------------------------------------------------- C ABI

ROPE = dict(q=A, qs=None, qo=A, qos=None, k=A, ks=None, ko=A, kos=None, pos=A, ps=0, f=A, dt=0, B=1, Hq=4, Hkv=2,
            N=16, d=128, rot=128, inter=0, factor=1.0)


def rope(lib, **kw):
    a = dict(ROPE, **kw)
    return lib.attn_rope(a["q"], a["qs"], a["qo"], a["qos"], a["k"], a["ks"], a["ko"], a["kos"], a["pos"], a["ps"],
                         a["f"], a["dt"], a["B"], a["Hq"], a["Hkv"], a["N"], a["d"], a["rot"], a["inter"],
                         a["factor"], 0, None)


def norm_rope(lib, qw=A, kw_=A, eps=1e-6, **kw):
    a = dict(ROPE, **kw)
    return lib.attn_norm_rope(a["q"], a["qs"], qw, a["qo"], a["qos"], a["k"], a["ks"], kw_, a["ko"], a["kos"],
                              a["pos"], a["ps"], a["f"], a["dt"], a["B"], a["Hq"], a["Hkv"], a["N"], a["d"],
                              a["rot"], a["inter"], a["factor"], eps, None)


def norm_rope_bwd(lib, qw=A, kw_=A, eps=1e-6, dqo=A, dko=A, dqw=A, dkw=A, ws=A, ws_bytes=1 << 30, dqs=None, **kw):
    a = dict(ROPE, **kw)
    return lib.attn_norm_rope_bwd(a["q"], a["qs"], qw, dqo, dqs, a["qo"], a["qos"], dqw, a["k"], a["ks"], kw_, dko,
                                  None, a["ko"], a["kos"], dkw, a["pos"], a["ps"], a["f"], a["dt"], a["B"], a["Hq"],
                                  a["Hkv"], a["N"], a["d"], a["rot"], a["inter"], a["factor"], eps, ws, ws_bytes,
                                  None)


COMMON = [
    (dict(q=None), INVALID), (dict(q=A + 8), INVALID), (dict(qo=None), INVALID), (dict(k=None), INVALID),
    (dict(ko=A + 4), INVALID), (dict(pos=None), INVALID), (dict(pos=A + 2), INVALID), (dict(f=None), INVALID),
    (dict(f=A + 4), INVALID), (dict(ps=-1), INVALID), (dict(dt=2), INVALID), (dict(dt=-1), INVALID),
    (dict(B=-1), INVALID), (dict(N=-1), INVALID), (dict(Hq=0), INVALID), (dict(Hkv=-1), INVALID),
    (dict(Hkv=0), INVALID),  # with k given
    (dict(rot=0), INVALID), (dict(rot=3), INVALID), (dict(rot=130), INVALID), (dict(factor=NAN), INVALID),
    (dict(factor=INF), INVALID), (dict(d=96, rot=96), UNSUPPORTED), (dict(d=256), UNSUPPORTED),
    (dict(B=1 << 16, N=1 << 15), INVALID), (dict(Hq=1 << 17), INVALID),
    (dict(qs=st(t=4)), INVALID), (dict(ks=st(h=-8)), INVALID),      # not of 16 bytes, negative
    (dict(qos=st(t=0)), INVALID), (dict(kos=st(h=0)), INVALID),     # outputs on one place
    (dict(B=2, qos=st(b=0)), INVALID), (dict(qos=st(t=64)), INVALID),
    (dict(qs=st(b=1 << 50)), INVALID), (dict(dt=1, qs=st(t=130)), INVALID),
]


@pytest.mark.parametrize("call", [rope, norm_rope, norm_rope_bwd])
@pytest.mark.parametrize("kw,code", COMMON)
def test_rotations_refuse(lib, call, kw, code):
    assert call(lib, **kw) == code


@pytest.mark.parametrize("call", [norm_rope, norm_rope_bwd])
@pytest.mark.parametrize("kw", [dict(qw=None), dict(kw_=None), dict(qw=A + 2), dict(eps=0.0), dict(eps=-1.0),
                                dict(eps=NAN), dict(eps=INF)])
def test_norms_refuse(lib, call, kw):
    assert call(lib, **kw) == INVALID


@pytest.mark.parametrize("kw", [dict(dqo=None), dict(dko=A + 8), dict(dqw=None), dict(dkw=A + 2), dict(ws=None),
                                dict(ws=A + 8), dict(ws_bytes=16), dict(dqs=st(t=4))])
def test_norm_gradient_refuses(lib, kw):
    assert norm_rope_bwd(lib, **kw) == INVALID


def test_norm_gradient_workspace(lib):
    f = lib.attn_norm_rope_bwd_workspace_bytes
    assert f(0, 4, 2, 16, 128) == 0 and f(1, 4, 2, 0, 128) == 0 and f(1, 0, 2, 16, 128) == 0 and f(1, 4, 2, 16, 80) == 0
    # Rows of d floats for q and for k, one per block: at least one, and no more as the work grows
    # than there are blocks at a time.
    assert f(1, 1, 0, 1, 64) >= 2 * 64 * 4
    assert f(4, 32, 8, 4096, 128) <= 2 * 148 * 8 * 128 * 4
    assert f(64, 64, 64, 1 << 20, 128) <= 2 * 148 * 8 * 256 * 128 * 4


CACHE = dict(kp=A, vp=A, ks=A, vs=A, fmt=0, bt=A, sl=A, cu=A, S=4, Hkv=2, T=64, maxq=16, d=128, ps=16, maxb=8,
             npages=100)


def write(lib, k=A, v=A, kt=256, kh=128, vt=256, vh=128, **kw):
    a = dict(CACHE, **kw)
    return lib.attn_kv_write_paged_q8(k, kt, kh, v, vt, vh, a["kp"], a["vp"], a["ks"], a["vs"], a["fmt"], a["bt"],
                                      a["sl"], a["cu"], a["S"], a["Hkv"], a["T"], a["maxq"], a["d"], a["ps"],
                                      a["maxb"], a["npages"], None)


def read(lib, k=A, v=A, dt=0, **kw):
    a = dict(CACHE, **kw)
    return lib.attn_kv_read_paged_q8(a["kp"], a["vp"], a["ks"], a["vs"], a["fmt"], a["bt"], a["sl"], a["cu"], k, v,
                                     dt, a["S"], a["Hkv"], a["T"], a["maxq"], a["d"], a["ps"], a["maxb"],
                                     a["npages"], None)


def prefill(lib, q=A, o=A, lse=A, Hq=4, scale=0.1, window=0, slopes=None, ws=A, ws_bytes=1 << 30, **kw):
    a = dict(CACHE, **kw)
    return lib.attn_prefill_paged_q8(q, a["kp"], a["vp"], a["ks"], a["vs"], a["fmt"], a["bt"], a["sl"], a["cu"], o,
                                     lse, a["S"], Hq, a["Hkv"], a["T"], a["maxq"], a["d"], a["ps"], a["maxb"],
                                     a["npages"], scale, window, slopes, ws, ws_bytes, None)


@pytest.mark.parametrize("call", [write, read, prefill])
@pytest.mark.parametrize("kw,code", [
    (dict(kp=None), INVALID), (dict(vp=A + 8), INVALID), (dict(ks=A + 2), INVALID), (dict(vs=None), INVALID),
    (dict(fmt=2), INVALID), (dict(fmt=-1), INVALID), (dict(bt=A + 1), INVALID), (dict(sl=None), INVALID),
    (dict(cu=A + 2), INVALID), (dict(S=0), INVALID), (dict(Hkv=0), INVALID), (dict(T=-1), INVALID),
    (dict(maxq=-1), INVALID), (dict(maxb=0), INVALID), (dict(npages=0), INVALID), (dict(d=96), UNSUPPORTED),
    (dict(ps=32), UNSUPPORTED), (dict(maxb=(1 << 26) + 1), INVALID), (dict(npages=1 << 30, Hkv=4), INVALID),
    (dict(T=1 << 30, Hkv=4), INVALID),
])
def test_cache_calls_refuse(lib, call, kw, code):
    assert call(lib, **kw) == code


@pytest.mark.parametrize("kw", [dict(k=None), dict(v=A + 8), dict(kt=100), dict(vh=-8), dict(vt=1 << 50)])
def test_write_refuses(lib, kw):
    assert write(lib, **kw) == INVALID


@pytest.mark.parametrize("kw", [dict(k=None), dict(v=A + 8), dict(dt=2), dict(dt=-1)])
def test_read_refuses(lib, kw):
    assert read(lib, **kw) == INVALID


@pytest.mark.parametrize("kw", [dict(q=None), dict(o=A + 8), dict(lse=A + 2), dict(Hq=3), dict(Hq=0), dict(scale=0.0),
                                dict(scale=NAN), dict(window=-1), dict(slopes=A + 1), dict(ws=A + 8, maxb=64),
                                dict(ws_bytes=64, maxb=64), dict(ws=None, maxb=64), dict(T=1 << 29, Hq=8)])
def test_prefill_refuses(lib, kw):
    assert prefill(lib, **kw) == INVALID


@pytest.mark.parametrize("call", [write, read, prefill])
@pytest.mark.parametrize("kw", [dict(T=0), dict(maxq=0)])
def test_nothing_to_do(lib, call, kw):
    # No tokens: a no-op, whatever the token tensors' addresses, on any machine.
    args = dict(q=None, o=None, lse=None) if call is prefill else dict(k=None, v=None)
    assert call(lib, **args, **kw) == 0


def test_no_rows_to_turn(lib):
    assert rope(lib, N=0, q=None, qo=None, k=None, ko=None, pos=None) == 0
    assert norm_rope(lib, B=0, q=None, qo=None, k=None, ko=None, pos=None) == 0


def test_prefill_workspace(lib):
    f = ea.prefill_q8_workspace_bytes
    assert f(4, 32, 8, 20, 5, 128, 2048) > 0                 # few work items over long keys: split
    assert f(16, 32, 8, 8192, 512, 128, 512) == 0            # enough of them
    assert f(1, 32, 8, 5, 5, 128, 8) == 0                    # one key tile
    # A row of d + 1 floats for each row of a CTA of which there are 148, and the plan.
    assert f(1, 8, 8, 1, 1, 64, 4096) == 256 + 148 * 65 * 4
    assert f(4, 32, 8, 20, 5, 128, 2048) == 256 + 148 * 20 * 129 * 4
    for bad in (dict(S=0), dict(Hq=3), dict(Hkv=0), dict(T=0), dict(max_q=0), dict(d=80), dict(max_blocks=0),
                dict(page_size=8)):
        assert f(**dict(dict(S=4, Hq=8, Hkv=4, T=20, max_q=5, d=128, max_blocks=2048), **bad)) == 0


def test_prefill_workspace_of_a_loose_bound():
    """No chunk is longer than T: a bound past it asks for what T does."""
    f = ea.prefill_q8_workspace_bytes
    for S, T in ((1, 5), (3, 700), (100, 4000)):
        for most in (T + 1, 1 << 20, 2**31 - 256, 2**31 - 1):
            assert f(S, 8, 8, T, most, 128, 4096) == f(S, 8, 8, T, T, 128, 4096)


def test_dtype_codes_match_the_header():
    import os
    import re
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "exattn.h")).read()
    codes = dict(re.findall(r"#define\s+ATTN_DTYPE_(\w+)\s+(\d+)", text))
    assert codes == {"BF16": str(ea._DTYPES[torch.bfloat16]), "F32": str(ea._DTYPES[torch.float32])}


# ----------------------------------------------------------------- binding

BF = torch.bfloat16


def test_binding_rotations_check_shapes_first():
    q, k = torch.zeros(2, 4, 9, 64, dtype=BF), torch.zeros(2, 2, 9, 64, dtype=BF)
    pos, f = torch.zeros(9, dtype=torch.int32), torch.zeros(32, dtype=torch.float64)
    w = torch.zeros(64, dtype=BF)
    for fn in (lambda **kw: ea.attn_rope(**dict(dict(q=q, k=k, positions=pos, inv_freq=f), **kw)),
               lambda **kw: ea.attn_norm_rope(**dict(dict(q=q, k=k, q_weight=w, k_weight=w, positions=pos, inv_freq=f), **kw))):
        with pytest.raises(ValueError, match="k must be"):
            fn(k=k[:, :, :8])
        with pytest.raises(ValueError, match="dims"):
            fn(k=k[0])
        with pytest.raises(ValueError, match="q must be"):
            fn(q=q[0, 0])
        with pytest.raises(ValueError, match="positions"):
            fn(positions=pos[:8])
        with pytest.raises(ValueError, match="positions"):
            fn(positions=torch.zeros(3, 9, dtype=torch.int32))
        with pytest.raises(ValueError, match="inv_freq"):
            fn(inv_freq=torch.zeros(33, dtype=torch.float64))
        with pytest.raises(ValueError, match="inv_freq"):
            fn(inv_freq=f[:0])
        with pytest.raises(ValueError, match="q_out must have q's shape"):
            fn(q_out=q[:, :2])
        with pytest.raises(TypeError, match="bfloat16 or float32"):
            fn(q=q.half())
        with pytest.raises(ValueError, match="CUDA tensor"):
            fn()
    with pytest.raises(ValueError, match="given without k"):
        ea.attn_rope(q, None, pos, f, k_out=k)
    with pytest.raises(ValueError, match="k and dk_out go together"):
        ea.attn_norm_rope_bwd(q, k, w, w, q, None, pos, f)
    with pytest.raises(TypeError, match="dq_out"):
        ea.attn_norm_rope_bwd(q, None, w, None, None, None, pos, f)
    with pytest.raises(ValueError, match="dk_out must have k's shape"):
        ea.attn_norm_rope_bwd(q, k, w, w, q, q, pos, f)


def test_binding_refuses_keys_without_heads():
    """(Their weights' gradient would be left as it was allocated.)"""
    q, k, pos, f = torch.zeros(2, 4, 8, 64), torch.zeros(2, 0, 8, 64), torch.zeros(8, dtype=torch.int32), \
        torch.zeros(32, dtype=torch.float64)
    w = torch.zeros(64)
    for call in (lambda: ea.attn_rope(q, k, pos, f), lambda: ea.attn_norm_rope(q, k, w, w, pos, f),
                 lambda: ea.attn_norm_rope_bwd(q, k, w, w, q, k, pos, f)):
        with pytest.raises(ValueError, match="no heads"):
            call()


def test_binding_cache_calls_check_shapes_first():
    P, Hkv, d, S = 6, 2, 64, 3
    kp = torch.zeros(P, Hkv, 16, d, dtype=torch.int8)
    sc = torch.ones(P, Hkv)
    bt, sl = torch.zeros(S, 4, dtype=torch.int32), torch.zeros(S, dtype=torch.int32)
    cu = torch.zeros(S + 1, dtype=torch.int32)
    kv = torch.zeros(5, Hkv, d, dtype=BF)
    q = torch.zeros(5, 4, d, dtype=BF)
    base = dict(k_pages=kp, v_pages=kp, k_scales=sc, v_scales=sc, block_table=bt, seq_lens=sl, cu_q=cu, max_q=5,
                kv_format="int8")
    calls = (lambda **kw: ea.attn_kv_write_paged_q8(**dict(dict(base, k=kv, v=kv), **kw)),
             lambda **kw: ea.attn_kv_read_paged_q8(**dict(dict(base, tokens=5), **kw)),
             lambda **kw: ea.attn_prefill_paged_q8(**dict(dict(base, q=q), **kw)))
    for fn in calls:
        with pytest.raises(ValueError, match="kv_format"):
            fn(kv_format="int4")
        with pytest.raises(ValueError, match="v_pages must match"):
            fn(v_pages=kp[:5])
        with pytest.raises(ValueError, match="scales must be"):
            fn(k_scales=sc[:5], v_scales=sc[:5])
        with pytest.raises(ValueError, match="S rows"):
            fn(block_table=bt[:2])
        with pytest.raises(ValueError, match="S rows"):
            fn(cu_q=cu[:3])
        with pytest.raises(ValueError, match="dims"):
            fn(seq_lens=bt)
        with pytest.raises(TypeError, match="torch.Tensor"):
            fn(seq_lens=[1, 2, 3])
        with pytest.raises((ValueError, TypeError), match="CUDA tensor|must be one of"):
            fn()
    with pytest.raises(ValueError, match="as the pages are"):
        calls[0](v=kv[:4])
    with pytest.raises(ValueError, match="as the pages are"):
        calls[0](k=torch.zeros(5, Hkv, 128, dtype=BF))
    with pytest.raises(TypeError, match="dtype"):
        calls[1](dtype=torch.float16)
    with pytest.raises(ValueError, match=r"\[tokens, Hkv, d\]"):
        calls[1](k=kv[:4])
    with pytest.raises(ValueError, match="multiple of their heads"):
        calls[2](q=torch.zeros(5, 3, d, dtype=BF))
    with pytest.raises(ValueError, match="out must be"):
        calls[2](out=q[:4])
    with pytest.raises(ValueError, match="one value per query head"):
        calls[2](alibi_slopes=torch.zeros(3))


# ------------------------------------------------------------- frequencies

def test_frequencies():
    f, a = ea.rope_frequencies(64, base=500000.0, device="cpu")
    i = np.arange(32)
    assert f.dtype == torch.float64 and a == 1.0
    assert np.allclose(f.numpy(), 500000.0 ** (-i / 32.0), rtol=1e-14)
    g, a = ea.rope_frequencies(64, base=500000.0, scaling="linear", factor=4.0, device="cpu")
    assert a == 1.0 and torch.equal(g, f / 4)
    # A raised base: the fastest pair keeps its pace, the slowest is divided by the factor.
    g, a = ea.rope_frequencies(64, scaling="ntk", factor=8.0, device="cpu")
    f, _ = ea.rope_frequencies(64, device="cpu")
    assert a == 1.0 and g[0] == f[0] and abs(g[-1] * 8 / f[-1] - 1) < 1e-12 and (g[1:] < f[1:]).all()
    # By parts: pairs of at least 32 turns over the original length stay, those of at most one are divided.
    g, a = ea.rope_frequencies(128, scaling="yarn", factor=16.0, original_length=4096, device="cpu")
    f, _ = ea.rope_frequencies(128, device="cpu")
    turns = 4096 * f / (2 * math.pi)
    assert a == 0.1 * math.log(16.0) + 1.0
    assert torch.equal(g[turns >= 32], f[turns >= 32])
    assert torch.allclose(g[turns <= 1], f[turns <= 1] / 16, rtol=1e-14, atol=0)
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and (g[mid] < f[mid]).all() and (g[mid] > f[mid] / 16).all()
    for bad in (dict(rot=0), dict(rot=7), dict(base=0.0), dict(base=INF), dict(factor=0.5), dict(factor=NAN),
                dict(scaling="other"), dict(scaling="yarn", original_length=0),
                dict(scaling="yarn", beta_fast=1.0, beta_slow=1.0)):
        with pytest.raises(ValueError):
            ea.rope_frequencies(**dict(dict(rot=64, device="cpu"), **bad))
