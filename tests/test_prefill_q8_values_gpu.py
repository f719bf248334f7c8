"""attn_prefill_paged_q8 over values of far-apart sizes and values that are no numbers:
what a row gets hangs on the keys that it sees, and on nothing else.

Bounds.  O is rounded to bf16 once: 2^-8 of it at most.  The rest is relative to the
row's size, the sum of p |V scale| |code|: P times the V scale is rounded to f16,
2^-11 of each term; the row's largest term without its code (p |V scale|) is at least
2^4 there, so that one below f16's normal numbers is off by 2^-25 of them at most,
2^-29 of the largest: 2^-18 of it added to every term, which counts with 2^-11.
Scores are float32 sums of d products, off by 2^-18 of their absolute sum, below 16
here: 2^-14, which moves p and the row sum: 2^-13.  2^x and the weights are within
2^-20.  2^-11 + 2^-13 + the small ones is below 2^-10.6.  L: 2^-13 + 2^-20 |L|.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import exact_io_aware_101_b200 as ea
import operator_reference as ref
from operator_reference import f64
from test_kv_q8_gpu import on_gpu
from test_prefill_paged_q8_gpu import make, run

pytestmark = pytest.mark.gpu
DEV = "cuda"
HQ, HKV, D = 4, 2, 64

# Ways a call is cut: rows of at most a warp, of one row tile and of more; with few
# sequences the keys are split over CTAs, with many they are not.
CUTS = [(5, 0), (5, 80), (60, 0), (60, 80), (140, 0), (140, 80)]


def reference(st, fmt, window=0):
    """(o, lse, size) of the first sequence's chunk; size as the bounds take it."""
    nq, n = int(st["cu_q"][1]), int(st["seq_lens"][0])
    table = st["block_table"][0].tolist()
    q = f64(st["q"][:nq])
    kc, vc = (ref.code_values(st[m + "_pages"], fmt) for m in ("k", "v"))
    page = np.array(table)[np.arange(n) // 16]
    k = kc[page, :, np.arange(n) % 16] * f64(st["k_scales"])[page][:, :, None]
    vcode, vscale = vc[page, :, np.arange(n) % 16], f64(st["v_scales"])[page]
    pos, key = n - nq + np.arange(nq)[:, None], np.arange(n)[None]
    see = (key <= pos) & ((key > pos - window) if window else True)
    o, lse, size = np.zeros((nq, HQ, D)), np.zeros((nq, HQ)), np.zeros((nq, HQ, D))
    for h in range(HQ):
        g = h // (HQ // HKV)
        x = np.where(see, q[:, h] @ k[:, g].T * D ** -0.5, -np.inf)
        m = x.max(1, keepdims=True)
        p = np.exp(x - m)
        lse[:, h] = m[:, 0] + np.log(p.sum(1))
        p /= p.sum(1, keepdims=True)
        w = p * np.abs(vscale[:, g])
        c = vcode[:, g]
        o[:, h] = (p * vscale[:, g]) @ c
        size[:, h] = (w + see * 2.0 ** -18 * w.max(1, keepdims=True)) @ np.abs(c)
    return o, lse, size


def check(o, lse, want, rows=slice(None), wide=0.0):
    wo, wl, size = (x[rows] for x in want)
    o, lse = f64(o)[:len(want[0])][rows], f64(lse)[:len(want[0])][rows]
    lim = 2.0 ** -8 * np.abs(wo) + (2.0 ** -10.6 + wide) * size
    err = np.abs(o - wo)
    assert (err <= lim).all(), float(np.nanmax(err / np.maximum(lim, 1e-300)))  # (no NaN passes)
    assert (np.abs(lse - wl) <= 2.0 ** -13 + wide + 2.0 ** -20 * np.abs(wl)).all()


def sequences(nq, ctx, copies, fmt, seed):
    return make([nq] + [1] * copies, [ctx] + [20] * copies, HQ, HKV, D, fmt, seed=seed)


@pytest.mark.parametrize("nq,copies", CUTS)
@pytest.mark.parametrize("far", [24, 32, 100])
def test_a_later_large_value_changes_no_earlier_row(nq, copies, far):
    # The chunk's last token alone lies on a page whose V scale is 2^far times the others'.
    n = 16 * 40 + 1
    st = sequences(nq, n - nq, copies, "e4m3", seed=far)
    st["v_scales"][int(st["block_table"][0, 40])] *= 2.0 ** far
    check(*run(on_gpu(st), "e4m3"), reference(st, "e4m3"))


@pytest.mark.parametrize("nq,copies", CUTS)
def test_a_large_value_behind_the_window_changes_no_row(nq, copies):
    ctx, window = 600, 40
    st = sequences(nq, ctx, copies, "int8", seed=3)
    first = ctx - window + 1  # the first key that any row sees; pages that end before it
    for b in range(first // 16):
        st["v_scales"][int(st["block_table"][0, b])] *= 2.0 ** 60
    check(*run(on_gpu(st), "int8", window=window), reference(st, "int8", window))


@pytest.mark.parametrize("nq,copies", CUTS)
@pytest.mark.parametrize("far", [24, 40, 60])
def test_a_large_value_barely_attended(nq, copies, far):
    # One page's keys score 28 below the others' (2^-40 of their weight): at 2^24 times their
    # values it adds nothing to speak of, at 2^40 as much as they do, at 2^60 all.
    n = 16 * 40
    st = sequences(nq, n - nq, copies, "e4m3", seed=far)
    st["q"][..., 0] = 8.0
    st["k_pages"].view(torch.uint8)[..., 0] = 0
    p = int(st["block_table"][0, 17])
    st["k_pages"][p] = torch.zeros_like(st["k_pages"][p])
    st["k_pages"][p, :, :, 0] = torch.full((HKV, 16), -112.0).to(st["k_pages"].dtype)
    st["k_scales"][p] = 0.25
    st["v_scales"][p] *= 2.0 ** far
    # (Scores of 28 are off by 2^-18 of that, which moves p and the row sum.)
    check(*run(on_gpu(st), "e4m3"), reference(st, "e4m3"), wide=2.0 ** -12.1)


@pytest.mark.parametrize("nq,copies", CUTS)
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("order", ["up", "down", "mixed"])
def test_scales_over_the_whole_range(nq, copies, fmt, order):
    # Page by page up or down by 2^5, or in no order: rows see some of it, up to their own place.
    n = 16 * 40 - 3
    st = sequences(nq, n - nq, copies, fmt, seed=nq)
    e = torch.linspace(-100.0, 100.0, 40)
    if order == "down":
        e = e.flip(0)
    elif order == "mixed":
        e = e[torch.randperm(40, generator=torch.Generator().manual_seed(copies))]
    for b in range(40):
        st["v_scales"][int(st["block_table"][0, b])] *= 2.0 ** float(e[b])
    st["v_scales"][::3] *= -1
    check(*run(on_gpu(st), fmt), reference(st, fmt))


@pytest.mark.parametrize("nq,copies", CUTS)
@pytest.mark.parametrize("scale", [2.0 ** -126, 2.0 ** -110, 2.0 ** 113])
def test_all_scales_small_or_large(nq, copies, scale):
    st = sequences(nq, 300, copies, "int8", seed=5)
    st["v_scales"][:] = scale
    check(*run(on_gpu(st), "int8"), reference(st, "int8"))


@pytest.mark.parametrize("nq,copies", CUTS)
def test_scales_of_zero(nq, copies):
    # Some pages of zeros (the smallest scale, or 0), then all of them.
    st = sequences(nq, 300, copies, "e4m3", seed=6)
    st["v_scales"][::3] = 0.0
    st["v_scales"][1::3] = 2.0 ** -126
    check(*run(on_gpu(st), "e4m3"), reference(st, "e4m3"))
    st["v_scales"][:] = 0.0
    o, lse = run(on_gpu(st), "e4m3")
    assert not o.any() and lse.isfinite().all()


@pytest.mark.parametrize("nq,copies", [(5, 0), (5, 80), (60, 0), (60, 80), (300, 0), (300, 80)])
@pytest.mark.parametrize("window", [0, 40, 500])
def test_a_code_that_is_no_number_reaches_its_element_only(nq, copies, window):
    # NaN codes of V, one at a time: in tiles that every row sees whole, at the window's ends, on
    # the diagonal, in the last page.  Rows that see the token get NaN in that element of O.
    ctx, fmt = 1000, "e4m3"
    n = ctx + nq
    st = sequences(nq, ctx, copies, fmt, seed=nq + window)
    want = reference(st, fmt, window)
    pos = ctx + np.arange(nq)
    toks = [3, 300, ctx - 300, ctx - 20, ctx, ctx + nq // 2, n - 1]
    if window:
        toks += [ctx - window, ctx - window + 1, ctx - window + nq // 2, n - window]
    for i, tok in enumerate(toks):
        col = (5, 40, 63, 0)[i % 4]
        sick = dict(st, v_pages=st["v_pages"].clone())
        p = int(st["block_table"][0, tok // 16])
        sick["v_pages"].view(torch.uint8)[p, 1, tok % 16, col] = (0x7F, 0xFF)[i % 2]
        o, lse = run(on_gpu(sick), fmt, window=window)
        hit = (pos >= tok) & ((pos - window < tok) if window else True)
        nan = np.zeros((nq, HQ, D), bool)
        nan[hit, HQ // HKV:, col] = True
        got = f64(o)[:nq]
        assert np.array_equal(np.isnan(got), nan), tok
        lim = 2.0 ** -8 * np.abs(want[0]) + 2.0 ** -10.6 * want[2]
        assert (np.abs(got - want[0]) <= lim)[~nan].all(), tok
        assert (np.abs(f64(lse)[:nq] - want[1]) <= 2.0 ** -13 + 2.0 ** -20 * np.abs(want[1])).all()
    # Several at once, two of them in one element, one in a page of its own.
    sick = dict(st, v_pages=st["v_pages"].clone())
    nan = np.zeros((nq, HQ, D), bool)
    for tok, col in ((ctx, 7), (ctx + nq // 2, 7), (n - 1, 8), (ctx - 20, 33), (3, 34)):
        sick["v_pages"].view(torch.uint8)[int(st["block_table"][0, tok // 16]), 0, tok % 16, col] = 0x7F
        hit = (pos >= tok) & ((pos - window < tok) if window else True)
        nan[hit, :HQ // HKV, col] = True
    assert np.array_equal(np.isnan(f64(run(on_gpu(sick), fmt, window=window)[0])[:nq]), nan)


@pytest.mark.parametrize("nq,copies", CUTS)
def test_a_row_whose_scores_are_all_minus_infinity(nq, copies):
    # K scales of infinity over negative codes: 0 / 0 by the formula, whichever way the call is cut;
    # L is -inf, and the other heads' rows are what they were.
    st = sequences(nq, 300, copies, "int8", seed=9)
    st["q"] = st["q"].abs() + 0.5
    st["k_pages"] = -st["k_pages"].abs().clamp(1, 127)
    n = int(st["seq_lens"][0])
    want = reference(st, "int8")
    for b in range(-(-n // 16)):
        st["k_scales"][int(st["block_table"][0, b]), 1] = float("inf")
    o, lse = run(on_gpu(st), "int8")
    assert o[:nq, HQ // HKV:].isnan().all()
    assert (lse[:nq, HQ // HKV:] == float("-inf")).all()
    own = (slice(None), slice(0, HQ // HKV))
    # (Scores of one sign add up: their absolute sums reach 50, 2^-18 of which moves p and L.)
    check(o, lse, want, rows=own, wide=2.0 ** -11)


@pytest.mark.parametrize("nq,copies", CUTS)
@pytest.mark.parametrize("window", [1, 40, 130])
def test_pages_given_back_behind_the_window(nq, copies, window):
    # Pages that end before the first key that any row sees are no longer the sequence's: their
    # entries name no page, and are not looked at.
    ctx = 600
    st = sequences(nq, ctx, copies, "e4m3", seed=11)
    want = reference(st, "e4m3", window)
    st["block_table"][0, :(ctx - window + 1) // 16] = -1
    check(*run(on_gpu(st), "e4m3", window=window), want)
    assert ea.device_status(clear=True) == 0
    st["block_table"][0, (ctx - window + 1) // 16] = -1  # the first that is seen
    o, _ = run(on_gpu(st), "e4m3", window=window)
    assert ea.device_status(clear=True) == ea.ATTN_DEV_BAD_PAGE
    assert o[0].isnan().all() and o[nq:].isfinite().all()


@pytest.mark.parametrize("nq,copies", CUTS)
@pytest.mark.parametrize("far", [116, 122, 128])
def test_a_weight_at_the_end_of_float32(nq, copies, far):
    # One page's keys score 84 below the others' (2^-122 of their weight) and hold values 2^far times
    # theirs: a sixty-fourth of the sum, as much as the others, 64 times as much.
    n = 16 * 40
    st = sequences(nq, n - nq, copies, "e4m3", seed=far)
    st["v_scales"] *= 2.0 ** -60
    st["q"][..., 0] = 8.0
    st["k_pages"].view(torch.uint8)[..., 0] = 0
    p = int(st["block_table"][0, 17])
    st["k_pages"][p] = torch.zeros_like(st["k_pages"][p])
    st["k_pages"][p, :, :, 0] = torch.full((HKV, 16), -112.0).to(st["k_pages"].dtype)
    st["k_scales"][p] = 0.75
    st["v_scales"][p] *= 2.0 ** (far // 2)
    st["v_scales"][p] *= 2.0 ** (far // 2)
    # (Scores of 84 are off by 2^-18 of that, which moves p and the row sum.)
    check(*run(on_gpu(st), "e4m3"), reference(st, "e4m3"), wide=2.0 ** -10.6)
