"""GPU parity of attn_rope, attn_norm_rope and attn_norm_rope_bwd against plain
64-bit forms, through the binding.

Bounds, element by element.  A stored value is rounded once: half a step of its
type.  Before that, in float32, an element's error is relative to F (|x| + |x'|)
of its pair ("size"): the reduced turn, at most half a turn, is rounded to
float32 (2^-26 of a turn, 2^-23.3 radians), sincospi is within 2 units (2^-23),
and the factor, the two products and their sum round once each (3 * 2^-24):
together below 2^-21.  A norm adds its sum of squares (an element passes at most
16 + 4 additions, 20 * 2^-24, halved by the root), the root, and two products:
below 2^-20 in all, 2^-19 with the rotation.  The gradient's dx has two such
factors and the row's second sum (at most another 20 * 2^-24): 2^-18 of its size.
A weight's gradient adds n terms, each off by 2^-19 of its size: an element passes
at most 48 additions over heads here, 3 over a block's tiles, 6 across the block
and 24 across the blocks, 81 * 2^-24: together below 2^-17 of the sum of sizes.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import exact_io_aware_101_b200 as ea
import operator_reference as ref
from operator_reference import f64, half_step

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS = 1e-6


def within(got, want, size, dtype, rel, what=""):
    got = f64(got)
    assert np.isfinite(got).all(), what
    lim = half_step(dtype) * np.abs(want) * (1 + rel) + rel * size + 1e-37
    worst = float((np.abs(got - want) / lim).max()) if got.size else 0.0
    assert worst <= 1.0, (what, worst)


def make(layout, B, N, Hq, Hkv, d, dtype, seed, far=5000):
    g = torch.Generator().manual_seed(seed)
    rows = lambda H: torch.randn(B, H, N, d, generator=g).to(dtype).to(DEV)
    q, k = rows(Hq), rows(Hkv) if Hkv else None
    pos = torch.randint(-far, far, (B, N), generator=g, dtype=torch.int32).to(DEV)
    if layout == "tokens":
        assert B == 1
        q, k, pos = q[0].transpose(0, 1).contiguous(), k[0].transpose(0, 1).contiguous() if Hkv else None, pos[0]
    w = [(1 + 0.3 * torch.randn(d, generator=g)).to(dtype).to(DEV) for _ in range(2)]
    return q, k, pos, w[0], w[1] if Hkv else None


def freqs(rot, seed=0):
    f, _ = ea.rope_frequencies(rot, device=DEV)
    return f


def heads_last(t, layout):
    """[..., N, d] with the token axis next to the last, and positions to match."""
    return f64(t).transpose(1, 0, 2) if layout == "tokens" else f64(t)


def pos64(pos, layout):
    p = pos.cpu().numpy().astype(np.float64)
    return p if layout == "tokens" or p.ndim == 1 else p[:, None]


CASES = [
    # layout, B, N, Hq, Hkv, d, rot, interleaved, dtype
    ("heads", 2, 37, 4, 2, 128, 128, False, torch.bfloat16),
    ("heads", 1, 1, 1, 1, 64, 64, False, torch.float32),
    ("heads", 3, 65, 5, 1, 64, 32, True, torch.bfloat16),
    ("heads", 2, 16, 3, 3, 128, 2, True, torch.float32),
    ("tokens", 1, 100, 8, 2, 128, 64, False, torch.bfloat16),
    ("tokens", 1, 7, 12, 4, 128, 128, True, torch.bfloat16),
    ("tokens", 1, 33, 2, 1, 64, 24, False, torch.bfloat16),   # half of rot is no multiple of 8
    ("tokens", 1, 19, 6, 2, 128, 2, False, torch.float32),
    ("heads", 1, 50, 2, 2, 128, 126, False, torch.float32),
    ("heads", 1, 50, 2, 2, 128, 90, True, torch.bfloat16),    # a lane turns some of its pairs
    ("tokens", 1, 300, 20, 0, 128, 96, False, torch.bfloat16),  # queries alone
    ("heads", 1, 2500, 40, 8, 64, 64, False, torch.bfloat16),   # several heads and tiles a block
]


@pytest.mark.parametrize("layout,B,N,Hq,Hkv,d,rot,inter,dtype", CASES)
@pytest.mark.parametrize("transpose", [False, True])
def test_rope(layout, B, N, Hq, Hkv, d, rot, inter, dtype, transpose):
    q, k, pos, _, _ = make(layout, B, N, Hq, Hkv, d, dtype, seed=N + rot)
    f = freqs(rot)
    got = ea.attn_rope(q, k, pos, f, interleaved=inter, attention_factor=1.25, transpose=transpose)
    torch.cuda.synchronize()
    assert (got[1] is None) == (k is None)
    for x, y in zip((q, k), got):
        if x is None:
            continue
        want, size = ref.rotate(heads_last(x, layout), pos64(pos, layout), f64(f), inter, 1.25, transpose)
        within(torch.from_numpy(heads_last(y, layout)), want, size, dtype, 2.0 ** -21)
        if rot < d:  # the rest of each row passes bit for bit
            assert torch.equal(y[..., rot:], x[..., rot:])
    assert ea.device_status() == 0


@pytest.mark.parametrize("layout,B,N,Hq,Hkv,d,rot,inter,dtype", CASES)
def test_norm_rope(layout, B, N, Hq, Hkv, d, rot, inter, dtype):
    q, k, pos, qw, kw = make(layout, B, N, Hq, Hkv, d, dtype, seed=2 * N + rot)
    f = freqs(rot)
    got = ea.attn_norm_rope(q, k, qw, kw, pos, f, eps=EPS, interleaved=inter, attention_factor=0.75)
    torch.cuda.synchronize()
    for x, w, y in zip((q, k), (qw, kw), got):
        if x is None:
            continue
        want, size = ref.norm_rotate(heads_last(x, layout), f64(w), pos64(pos, layout), f64(f), inter, 0.75,
                                     float(np.float32(EPS)))
        within(torch.from_numpy(heads_last(y, layout)), want, size, dtype, 2.0 ** -19)


@pytest.mark.parametrize("layout,B,N,Hq,Hkv,d,rot,inter,dtype", CASES)
def test_norm_rope_bwd(layout, B, N, Hq, Hkv, d, rot, inter, dtype):
    q, k, pos, qw, kw = make(layout, B, N, Hq, Hkv, d, dtype, seed=3 * N + rot)
    dq_out, dk_out, _, _, _ = make(layout, B, N, Hq, Hkv, d, dtype, seed=4 * N + rot)
    f = freqs(rot)
    how = dict(eps=EPS, interleaved=inter, attention_factor=1.5)
    got = ea.attn_norm_rope_bwd(q, k, qw, kw, dq_out, dk_out, pos, f, **how)
    torch.cuda.synchronize()
    for x, w, dy, dx, dw in ((q, qw, dq_out, got[0], got[2]), (k, kw, dk_out, got[1], got[3])):
        if x is None:
            assert dx is None and dw is None
            continue
        want, size, wantw, sizew = ref.norm_rotate_bwd(heads_last(x, layout), f64(w), heads_last(dy, layout),
                                                       pos64(pos, layout), f64(f), inter, 1.5, float(np.float32(EPS)))
        within(torch.from_numpy(heads_last(dx, layout)), want, size, dtype, 2.0 ** -18)
        within(dw, wantw, sizew, torch.float32, 2.0 ** -17)
    again = ea.attn_norm_rope_bwd(q, k, qw, kw, dq_out, dk_out, pos, f, **how)
    for a, b in zip(got, again):
        assert a is None or torch.equal(a, b)  # no order of blocks shows


def test_gradient_against_differences():
    # The 64-bit form, by central differences of the loss sum(dy * y) in x and w: the formulas
    # that the kernels are held to are the gradients of the forward form.
    r = np.random.RandomState(5)
    x, w, dy = r.randn(3, 64), 1 + 0.2 * r.randn(64), r.randn(3, 64)
    pos, f = np.array([0.0, 7.0, 901.0]), 10000.0 ** (-np.arange(16) / 16)
    loss = lambda x, w: (ref.norm_rotate(x, w, pos, f, False, 1.5, 1e-6)[0] * dy).sum()
    dx, _, dw, _ = ref.norm_rotate_bwd(x, w, dy, pos, f, False, 1.5, 1e-6)
    h = 1e-6
    for i, j in ((0, 0), (1, 17), (2, 31), (2, 32), (1, 63)):
        e = np.zeros_like(x)
        e[i, j] = h
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * h) - dx[i, j]) < 1e-6
        e = np.zeros_like(w)
        e[j] = h
        assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * h) - dw[j]) < 1e-6


@pytest.mark.parametrize("inter", [False, True])
def test_far_positions(inter):
    pos = torch.tensor([0, 1, -1, 123456, 1 << 20, (1 << 24) + 1, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device=DEV)
    g = torch.Generator().manual_seed(9)
    q = torch.randn(8, 2, 64, generator=g).to(DEV)
    f = freqs(64)
    y, _ = ea.attn_rope(q, None, pos, f, interleaved=inter)
    want, size = ref.rotate(heads_last(q, "tokens"), pos64(pos, "tokens"), f64(f), inter, 1.0)
    # 2^31 * f / 2 pi has an error of 2^-53 of itself twice over: at most 2^-23 radians more.
    within(torch.from_numpy(heads_last(y, "tokens")), want, size, torch.float32, 2.0 ** -20.5)


def test_views_in_place_and_shared_positions():
    g = torch.Generator().manual_seed(11)
    T, Hq, Hkv, d = 45, 4, 2, 128
    x = torch.randn(T, Hq + 2 * Hkv, d, generator=g).to(torch.bfloat16).to(DEV)
    keep = x.clone()
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    f = freqs(d)
    want = ea.attn_rope(x[:, :Hq].contiguous(), x[:, Hq:Hq + Hkv].contiguous(), pos, f)
    # In place in the fused projection's output; the values are not touched.
    q, k = x[:, :Hq], x[:, Hq:Hq + Hkv]
    ea.attn_rope(q, k, pos, f, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(x[:, Hq + Hkv:], keep[:, Hq + Hkv:])
    # Token-major rows seen as [1, H, T, d], positions [N] shared by a batch, outputs transposed.
    xb = torch.stack([keep, keep.flip(0)])  # [2, T, H, d]
    qb = xb[:, :, :Hq].transpose(1, 2)
    out = torch.full((2, T, Hq, d), 7.0, dtype=torch.bfloat16, device=DEV).transpose(1, 2)
    ea.attn_rope(qb, None, pos, f, q_out=out)
    assert torch.equal(out[0].transpose(0, 1), want[0])
    one, _ = ea.attn_rope(qb[1].transpose(0, 1), None, pos, f)
    assert torch.equal(out[1].transpose(0, 1), one)
    # A row repeated over the batch as an input (stride 0).
    rep, _ = ea.attn_rope(keep[:, :Hq].transpose(0, 1)[None].expand(3, Hq, T, d), None, pos, f)
    assert all(torch.equal(rep[i].transpose(0, 1), want[0]) for i in range(3))


def test_gradient_in_place_and_strided():
    q, k, pos, qw, kw = make("heads", 2, 40, 4, 2, 64, torch.bfloat16, seed=21)
    dq, dk, _, _, _ = make("heads", 2, 40, 4, 2, 64, torch.bfloat16, seed=22)
    f = freqs(64)
    want = ea.attn_norm_rope_bwd(q, k, qw, kw, dq, dk, pos, f)
    dq2, dk2 = dq.clone(), dk.clone()
    got = ea.attn_norm_rope_bwd(q, k, qw, kw, dq2, dk2, pos, f, dq=dq2, dk=dk2)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    # The same through strided views of every tensor.
    t = lambda x: x.transpose(1, 2).contiguous().transpose(1, 2)
    got = ea.attn_norm_rope_bwd(t(q), t(k), qw, kw, t(dq), t(dk), pos, f)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_rows_that_are_not_numbers():
    # A NaN or an infinity stays in its row, and what does not turn stays as it is.
    q, _, pos, _, _ = make("tokens", 1, 20, 3, 1, 64, torch.float32, seed=31)
    f = freqs(16)
    clean, _ = ea.attn_rope(q, None, pos, f)
    q[4, 1, 3], q[5, 2, 40], q[6, 0, 60] = float("nan"), float("inf"), float("nan")
    y, _ = ea.attn_rope(q, None, pos, f)
    same = torch.ones_like(q, dtype=torch.bool)
    same[4, 1, 3] = same[4, 1, 11] = same[5, 2, 40] = same[6, 0, 60] = False
    assert torch.equal(y[same], clean[same])
    assert y[4, 1, 3].isnan() and y[4, 1, 11].isnan() and y[5, 2, 40].isinf() and y[6, 0, 60].isnan()
    # Rows of zeros: the norm leaves zeros.
    z = torch.zeros(5, 2, 64, dtype=torch.bfloat16, device=DEV)
    one = torch.ones(64, dtype=torch.bfloat16, device=DEV)
    pos = torch.arange(5, dtype=torch.int32, device=DEV)
    assert not ea.attn_norm_rope(z, None, one, None, pos, f)[0].any()


def test_empty():
    f = freqs(64)
    q = torch.empty(0, 4, 64, dtype=torch.bfloat16, device=DEV)
    pos = torch.empty(0, dtype=torch.int32, device=DEV)
    w = torch.ones(64, dtype=torch.bfloat16, device=DEV)
    assert ea.attn_rope(q, None, pos, f)[0].shape == (0, 4, 64)
    dq, dk, dqw, dkw = ea.attn_norm_rope_bwd(q, q, w, w, q, q, pos, f)
    assert dq.shape == q.shape and not dqw.any() and not dkw.any()


def test_streams_and_graph():
    q, k, pos, qw, kw = make("heads", 2, 200, 8, 2, 128, torch.bfloat16, seed=41)
    dq, dk, _, _, _ = make("heads", 2, 200, 8, 2, 128, torch.bfloat16, seed=42)
    f = freqs(128)
    want = ea.attn_norm_rope_bwd(q, k, qw, kw, dq, dk, pos, f)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = ea.attn_norm_rope_bwd(q, k, qw, kw, dq, dk, pos, f)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    outs = [torch.empty_like(t) for t in want]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ea.attn_norm_rope_bwd(q, k, qw, kw, dq, dk, pos, f, dq=outs[0], dk=outs[1], dq_weight=outs[2], dk_weight=outs[3])
    for seed in (41, 43):
        q2, k2, _, _, _ = make("heads", 2, 200, 8, 2, 128, torch.bfloat16, seed=seed)
        q.copy_(q2)
        k.copy_(k2)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ea.attn_norm_rope_bwd(q, k, qw, kw, dq, dk, pos, f), outs))
