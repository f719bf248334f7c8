"""GPU parity of attn_prefill_paged_q8 against a plain 64-bit form.

Bounds.  O is rounded to bf16 once: half a step, 2^-8 of it at most (bf16 keeps 8
bits, a step is up to 2^-7 of a value).  The rest is relative to the row's "size",
the sum of p |v|: P is rounded to f16 (half a step of 11 bits, 2^-11 of each
term; one below 2^-14 of the row's largest by 2^-25 of that, f16's last place: so
the size has 2^-15 of the largest p added to every p, 2^-9.7 of which is above
2^-25) and each element of
V too (2^-11, and its scale to 22 bits); scores are float32 sums of d products
(2^-18 of their absolute sum at most, which scaled is below 16 here: 2^-14, which
moves p by twice that, in the row sum too); 2^x is within 2^-22.  2^-11 + 2^-11 +
2^-13 + the small ones is below 1.2 * 2^-10, below 2^-9.7: |dO| <= 2^-8 |O| +
2^-9.7 size.  L carries the scores' error and float32's: 2^-13 + 2^-20 |L|.
(Scores above 16 in size, where a test makes them, widen both by 2^-18 of that
size.)
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import exact_io_aware_101_b200 as ea
import operator_reference as ref
from operator_reference import f64
from test_kv_q8_gpu import CACHE, make as make_cache, on_gpu

pytestmark = pytest.mark.gpu
DEV = "cuda"


def make(qlens, ctxs, Hq, Hkv, d, fmt, seed, **kw):
    st = make_cache(qlens, ctxs, Hkv, d, fmt, seed, **kw)
    for n in ("k", "v"):  # codes of size about 100 over scales that make values of size about 1
        st[n + "_scales"] = (0.5 + torch.rand(st[n + "_scales"].shape, generator=torch.Generator().manual_seed(seed))) / 100
    g = torch.Generator().manual_seed(seed + 1)
    st["q"] = torch.randn(sum(qlens), Hq, d, generator=g).to(torch.bfloat16)
    return st


def run(dv, fmt, **kw):
    lens = (dv["cu_q"][1:] - dv["cu_q"][:-1]).tolist()
    kw.setdefault("max_q", max(lens))
    o, lse = ea.attn_prefill_paged_q8(dv["q"], *(dv[n] for n in CACHE), kv_format=fmt, **kw)
    torch.cuda.synchronize()
    return o, lse


def reference(st, fmt, scale=None, window=0, slopes=None, rows=None):
    """(o, lse, size) of every sequence's chunk, concatenated."""
    out = []
    cu, lens = st["cu_q"].tolist(), st["seq_lens"].tolist()
    d = st["q"].shape[-1]
    for s, n in enumerate(lens):
        q = f64(st["q"][cu[s]:cu[s + 1]])
        k, v = (ref.tokens_of(ref.code_values(st[m + "_pages"], fmt), f64(st[m + "_scales"]),
                              st["block_table"][s].tolist(), n) for m in ("k", "v"))
        out.append(ref.prefill(q, k, v, d ** -0.5 if scale is None else scale, window, slopes))
    return tuple(np.concatenate([x[i] for x in out]) for i in range(3))


def check(o, lse, want, wide=0.0):
    wo, wl, size = want
    assert np.isfinite(f64(o)).all() and np.isfinite(f64(lse)).all()
    lim = 2.0 ** -8 * np.abs(wo) + (2.0 ** -9.7 + wide) * size + 1e-30
    worst = float((np.abs(f64(o) - wo) / lim).max())
    assert worst <= 1, worst
    assert (np.abs(f64(lse) - wl) <= 2.0 ** -13 + wide + 2.0 ** -20 * np.abs(wl)).all()


CASES = [
    # qlens, ctxs, Hq, Hkv, d
    ([1], [0], 1, 1, 64),
    ([5], [0], 4, 2, 128),
    ([1, 1], [127, 128], 8, 1, 128),
    ([40], [90], 3, 3, 64),
    ([20, 0, 33], [0, 7, 250], 6, 2, 128),   # three heads a token: rows left idle
    ([70], [300], 8, 2, 128),                # a pair of tiles, and one token over
    ([129], [10], 2, 2, 64),
    ([17, 64, 3], [500, 64, 1000], 8, 8, 64),
    ([9], [700], 40, 8, 64),                 # five heads a token
    ([2, 3], [40, 17], 160, 1, 64),          # more heads a token than a tile has rows
]


@pytest.mark.parametrize("qlens,ctxs,Hq,Hkv,d", CASES)
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_small(qlens, ctxs, Hq, Hkv, d, fmt):
    st = make(qlens, ctxs, Hq, Hkv, d, fmt, seed=sum(qlens) + d)
    check(*run(on_gpu(st), fmt), reference(st, fmt))
    assert ea.device_status() == 0


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_not_split(fmt):
    # As many work items as SMs: the keys are not split over CTAs.
    qlens, ctxs = [3] * 80, [i % 37 * 4 for i in range(80)]
    st = make(qlens, ctxs, 4, 2, 64, fmt, seed=3)
    assert ea.prefill_q8_workspace_bytes(80, 4, 2, 240, 3, 64, st["block_table"].shape[1]) == 0
    check(*run(on_gpu(st), fmt), reference(st, fmt))


# The ways a call is cut: chunks that fit one row tile of 128 rows (twin tiles over
# halves of the keys) or not, as many work items as SMs or fewer (keys split over
# CTAs, by each sequence's length), one key tile for all.
@pytest.mark.parametrize("qlens,ctxs,Hq,Hkv,d,split", [
    ([4, 1, 4], [3000, 100, 1290], 8, 2, 128, True),          # twin, split
    ([1], [9000], 4, 1, 64, True),                            # one work item over all SMs
    ([32, 31], [1000, 127], 8, 2, 64, True),                  # a full tile of rows
    ([33, 20, 1], [1500, 900, 2600], 8, 2, 64, True),         # one row tile and a bit: not twin
    ([140], [2000], 4, 2, 128, True),                         # three tiles, the keys split
    ([2] * 40, [37 * i for i in range(40)], 8, 4, 64, False),         # twin, enough work items
    ([50] * 40, [150 + 11 * i for i in range(40)], 8, 4, 64, False),  # neither
    ([0] * 30 + [3] + [0] * 40, [500] * 71, 2, 2, 64, True),  # most sequences have no chunk
])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_every_cut(qlens, ctxs, Hq, Hkv, d, split, fmt):
    st = make(qlens, ctxs, Hq, Hkv, d, fmt, seed=len(qlens) + d)
    need = ea.prefill_q8_workspace_bytes(len(qlens), Hq, Hkv, sum(qlens), max(qlens), d, st["block_table"].shape[1])
    assert (need > 0) == split
    dv = on_gpu(st)
    ws = torch.full((max(need, 16),), 0xFF, dtype=torch.uint8, device=DEV)  # NaN wherever nothing is written
    check(*run(dv, fmt, workspace=ws), reference(st, fmt))
    # A table far wider than the lengths cuts the call otherwise; so does a larger bound.
    wide = torch.full((len(qlens), dv["block_table"].shape[1] + 300), -1, dtype=torch.int32, device=DEV)
    wide[:, :dv["block_table"].shape[1]] = dv["block_table"]
    dv["block_table"] = wide
    check(*run(dv, fmt, max_q=max(qlens) + 70), reference(st, fmt))
    assert ea.device_status() == 0


@pytest.mark.parametrize("qlens,ctxs,d", [([1, 5], [700, 0], 128), ([200, 3], [0, 400], 64)])
def test_loose_bounds(qlens, ctxs, d):
    """A chunk bound past T is T, and a window past every length is none."""
    st = make(qlens, ctxs, 4, 2, d, "int8", seed=d)
    dv = on_gpu(st)
    want = run(dv, "int8", max_q=sum(qlens))
    check(*want, reference(st, "int8"))
    for kw in (dict(max_q=2**31 - 1), dict(max_q=2**32 + 1), dict(max_q=sum(qlens), window=2**31 - 1),
               dict(max_q=2**31 - 1, window=2**32 + 3)):
        for got, w in zip(run(dv, "int8", **kw), want):
            assert torch.equal(got, w), kw
    k = [ea.attn_kv_read_paged_q8(*(dv[n] for n in CACHE), tokens=sum(qlens), max_q=m, kv_format="int8")
         for m in (max(qlens), 2**31 - 1)]
    assert torch.equal(k[0][0], k[1][0]) and torch.equal(k[0][1], k[1][1])
    assert ea.device_status() == 0


def test_many_splits_join():
    # Long keys whose parts differ by far in weight: the last keys' scores dominate.
    st = make([3], [6000], 4, 1, 128, "e4m3", seed=19)
    st["k_scales"] *= torch.linspace(0.2, 3.0, st["k_scales"].shape[0])[:, None]
    check(*run(on_gpu(st), "e4m3"), reference(st, "e4m3"), wide=2.0 ** -12)


@pytest.mark.parametrize("window", [0, 40, 500])
@pytest.mark.parametrize("qlen,copies", [(5, 0), (5, 80), (90, 0), (90, 80)])
def test_nan_scale_reaches_its_rows_only(window, qlen, copies):
    # Twin tiles and others, split keys and not: a page whose V scale is NaN, in the tile of the
    # diagonal and in an earlier one.
    ctx = 700
    st = make([qlen] + [1] * copies, [ctx] + [200] * copies, 4, 2, 64, "int8", seed=23)
    want = reference(st, "int8", window=window)
    for tok in (ctx, 300):
        sick = dict(st, v_scales=st["v_scales"].clone())
        sick["v_scales"][int(st["block_table"][0, tok // 16]), 1] = float("nan")
        o, lse = run(on_gpu(sick), "int8", window=window)
        pos = ctx + np.arange(qlen)
        page = tok // 16 * 16
        hit = pos >= page
        if window:
            hit &= pos - window + 1 <= page + 15
        rows = np.zeros((qlen + copies, 4), bool)
        rows[:qlen, 2:] = hit[:, None]
        assert o[torch.from_numpy(rows).to(DEV)].isnan().all()
        assert lse.isfinite().all()
        keep = ~rows
        got = f64(o)[keep]
        lim = 2.0 ** -8 * np.abs(want[0][keep]) + 2.0 ** -9.7 * want[2][keep] + 1e-30
        assert (np.abs(got - want[0][keep]) <= lim).all()


def test_more_sequences_than_are_ranked():
    qlens, ctxs = [1] * 600, [i % 23 for i in range(600)]
    st = make(qlens, ctxs, 2, 1, 64, "int8", seed=4)
    check(*run(on_gpu(st), "int8"), reference(st, "int8"))


@pytest.mark.parametrize("window", [1, 16, 100, 128, 1000])
@pytest.mark.parametrize("d", [64, 128])
def test_window(window, d):
    st = make([90, 4], [300, 700], 4, 2, d, "e4m3", seed=window)
    check(*run(on_gpu(st), "e4m3", window=window), reference(st, "e4m3", window=window))


@pytest.mark.parametrize("window", [0, 60])
@pytest.mark.parametrize("copies", [1, 75])  # split over keys, and not
def test_alibi(window, copies):
    st = make([30] + [2] * copies, [200] + [50] * copies, 4, 2, 64, "int8", seed=6)
    slopes = [0.5, 0.1, 0.02, 0.0]
    o, lse = run(on_gpu(st), "int8", window=window, alibi_slopes=torch.tensor(slopes, device=DEV))
    check(o, lse, reference(st, "int8", window=window, slopes=slopes))


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("jump", [3.0, 30.0])
def test_score_jump(fmt, jump):
    # One key far above all before it, in a tile behind the first: the running
    # reference moves and the accumulator is rescaled.
    qlens, ctxs = [100] * 10, [600] * 10
    st = make(qlens, ctxs, 16, 8, 128, fmt, seed=7)
    st["q"] = st["q"].float().abs().to(torch.bfloat16)
    for s in range(10):
        p = int(st["block_table"][s, 400 // 16])
        st["k_pages"][p, :, 400 % 16] = torch.full((128,), 100.0).to(st["k_pages"].dtype)
        st["k_scales"][p] = jump / 100
    big = jump * 0.8 * 128 * 128 ** -0.5 * 1.5
    rows = [0, 99, 500, 999]
    o, lse = run(on_gpu(st), fmt)
    cu = st["cu_q"].tolist()
    for r in rows:
        s = r // 100
        k, v = (ref.tokens_of(ref.code_values(st[m + "_pages"], fmt), f64(st[m + "_scales"]), st["block_table"][s].tolist(), 600 + r % 100 + 1)
                for m in ("k", "v"))
        check(o[r:r + 1], lse[r:r + 1], ref.prefill(f64(st["q"][r:r + 1]), k, v, 128 ** -0.5), wide=2.0 ** -18 * big)


def test_uneven_value_scales():
    # Pages whose V scales lie 2^12 apart, the largest ones barely attended.
    st = make([40], [400], 4, 2, 64, "e4m3", seed=8)
    P = st["v_scales"].shape[0]
    st["v_scales"] *= torch.exp2(torch.arange(P) % 13 - 6.0)[:, None]
    st["k_scales"] *= torch.exp2(-(torch.arange(P) % 13) / 4.0)[:, None]
    check(*run(on_gpu(st), "e4m3"), reference(st, "e4m3"))
    # Negative and zero scales are scales too.
    st["v_scales"][::3] *= -1
    st["k_scales"][::5] *= -1
    st["k_scales"][1], st["v_scales"][2] = 0.0, 0.0
    check(*run(on_gpu(st), "e4m3"), reference(st, "e4m3"))


@pytest.mark.parametrize("copies", [0, 80])
def test_rows_behind_the_last_sequence(copies):
    st = make([5] + [1] * copies, [20] + [3] * copies, 4, 2, 64, "int8", seed=9)
    T = 5 + copies
    dv = on_gpu(st)
    dv["q"] = torch.cat([dv["q"], torch.full((7, 4, 64), float("nan"), dtype=torch.bfloat16, device=DEV)])
    out = torch.full((T + 7, 4, 64), 3.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((T + 7, 4), 3.0, device=DEV)
    run(dv, "int8", out=out, lse=lse, max_q=11)
    check(out[:T], lse[:T], reference(st, "int8"))
    assert (out[T:] == 3).all() and (lse[T:] == 3).all()


@pytest.mark.parametrize("copies", [0, 80])
def test_values_that_are_not_numbers(copies):
    # Slots behind the sequence's end and unused pages hold NaN; a token's V is
    # NaN: rows before it do not see it, rows from it on are NaN.
    fmt, nq, ctx = "e4m3", 60, 100
    st = make([nq] + [1] * copies, [ctx] + [0] * copies, 4, 2, 64, fmt, seed=10)
    want = reference(st, fmt)
    used = torch.zeros(st["k_pages"].shape[0], dtype=torch.bool)
    for s, n in enumerate(st["seq_lens"].tolist()):
        for b in range(-(-n // 16)):
            p = int(st["block_table"][s, b])
            used[p] = True
            for m in ("k", "v"):
                st[m + "_pages"].view(torch.uint8)[p, :, n - 16 * b if n < 16 * b + 16 else 16:] = 0x7F
    for m in ("k", "v"):
        st[m + "_pages"].view(torch.uint8)[~used] = 0x7F
        st[m + "_scales"][~used] = float("nan")
    check(*run(on_gpu(st), fmt), want)
    # The K of token 130 and the V of token 140 become NaN for K/V head 1.
    for m, tok in (("k", 130), ("v", 140)):
        p = int(st["block_table"][0, tok // 16])
        st[m + "_pages"].view(torch.uint8)[p, 1, tok % 16, 5] = 0x7F
    o, lse = run(on_gpu(st), fmt)
    clean = [slice(0, nq), slice(0, 130 - ctx)]  # rows of heads 0-1, and 2-3
    for hs, rows in ((slice(0, 2), clean[0]), (slice(2, 4), clean[1])):
        check(o[rows, hs], lse[rows, hs], tuple(x[rows, hs] for x in want))
    assert o[130 - ctx:nq, 2:].isnan().all()
    # A page whose V scale is infinite: rows that see it are not finite, those before it are.
    st = make([nq] + [1] * copies, [ctx] + [0] * copies, 4, 2, 64, fmt, seed=10)
    st["v_scales"][int(st["block_table"][0, 9]), 0] = float("inf")  # tokens 144 ..
    o, lse = run(on_gpu(st), fmt)
    check(o[:44, :2], lse[:44, :2], tuple(x[:44, :2] for x in want))
    check(o[:, 2:], lse[:, 2:], tuple(x[:, 2:] for x in want))
    assert o[44:nq, :2].isnan().all()


def test_bad_pages_and_lengths():
    for copies in (0, 80):
        st = make([10, 10] + [1] * copies, [300, 300] + [3] * copies, 4, 2, 64, "int8", seed=11)
        want = reference(st, "int8")
        dv = on_gpu(st)
        dv["block_table"][1, 4] = dv["k_pages"].shape[0]
        o, lse = run(dv, "int8")
        assert ea.device_status(clear=True) == ea.ATTN_DEV_BAD_PAGE
        assert o[10:20].isnan().all() and lse[10:20].isnan().all()
        keep = np.r_[0:10, 20:20 + copies]
        check(o[keep], lse[keep], tuple(x[keep] for x in want))
        # With a window that does not reach the bad page the rows are whole.
        o, lse = run(dv, "int8", window=100)
        assert ea.device_status(clear=True) == 0
        check(o, lse, reference(st, "int8", window=100))
        dv = on_gpu(st)
        dv["seq_lens"][1] = 9
        out = torch.full_like(dv["q"], 3.0)
        o, lse = run(dv, "int8", out=out)
        assert ea.device_status(clear=True) == ea.ATTN_DEV_BAD_PAGE
        assert (o[10:20] == 3).all()
        check(o[keep], lse[keep], tuple(x[keep] for x in want))


def test_waits_run_out():
    """The library's test build stops the copies early: the kernels' waits run out, the call
    returns and the status says so; the product library then works on the same device."""
    from exact_io_aware_101_b200 import build as eabuild
    import ctypes
    tlib = ea.load_library(eabuild.build_test_lib())
    for qlens, ctxs in (([4, 4], [700, 900]), ([100], [900]), ([4] * 80, [300] * 80)):
        st = make(qlens, ctxs, 4, 2, 128, "e4m3", seed=17)
        dv = on_gpu(st)
        T, mb, P = sum(qlens), dv["block_table"].shape[1], dv["k_pages"].shape[0]
        need = ea.prefill_q8_workspace_bytes(len(qlens), 4, 2, T, max(qlens), 128, mb)
        ws = torch.empty(max(need, 16), dtype=torch.uint8, device=DEV)
        o, lse = torch.empty_like(dv["q"]), torch.empty(T, 4, device=DEV)
        rc = tlib.attn_prefill_paged_q8(
            dv["q"].data_ptr(), *(dv[n].data_ptr() for n in CACHE[:4]), 0, *(dv[n].data_ptr() for n in CACHE[4:]),
            o.data_ptr(), lse.data_ptr(), len(qlens), 4, 2, T, max(qlens), 128, 16, mb, P, 128 ** -0.5, 0, None,
            ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
        assert rc == 0
        torch.cuda.synchronize()
        word = ctypes.c_uint(0)
        assert tlib.attn_device_status(ctypes.byref(word), 1, torch.cuda.current_stream().cuda_stream) == 0
        assert word.value == ea.ATTN_DEV_TIMEOUT
        check(*run(dv, "e4m3"), reference(st, "e4m3"))
    assert ea.device_status() == 0


def test_large_query_values():
    st = make([30], [100], 4, 2, 128, "int8", seed=12)
    st["q"][0] *= 2.0 ** 60
    st["q"][1] *= 2.0 ** -60
    st["q"][2] = 0
    o, lse = run(on_gpu(st), "int8", scale=2.0 ** -62)
    want = reference(st, "int8", scale=2.0 ** -62)
    check(o, lse, want)


def test_streams_and_graph():
    # Two captured graphs with workspaces of their own, and calls on other streams.
    fmt = "e4m3"
    sts = [make([6, 2], [900, 1500], 8, 2, 128, fmt, seed=s) for s in (13, 14)]
    dvs = [on_gpu(s) for s in sts]
    want = [run(d, fmt) for d in dvs]
    graphs, outs = [], []
    for d in dvs:
        o, lse = torch.empty_like(d["q"]), torch.empty(8, 8, device=DEV)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ea.attn_prefill_paged_q8(d["q"], *(d[n] for n in CACHE), max_q=6, kv_format=fmt, out=o, lse=lse)
        graphs.append(g)
        outs.append((o, lse))
    streams = [torch.cuda.Stream() for _ in dvs]
    for _ in range(3):
        for o, lse in outs:
            o.zero_(), lse.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for (o, lse), (wo, wl) in zip(outs, want):
            assert torch.equal(o, wo) and torch.equal(lse, wl)
    with torch.cuda.stream(streams[0]):
        o, lse = ea.attn_prefill_paged_q8(dvs[0]["q"], *(dvs[0][n] for n in CACHE), max_q=6, kv_format=fmt)
    streams[0].synchronize()
    assert torch.equal(o, want[0][0]) and torch.equal(lse, want[0][1])


def test_a_serving_step():
    """Projections to answers: norm and rotation, the cache's new tokens, the chunk's attention;
    then a decode step of one token the same way.  Each call is held to the 64-bit form of what
    the one before it left."""
    fmt, Hq, Hkv, d = "int8", 8, 2, 64
    qlens, ctxs = [50, 7], [0, 30]
    st = make(qlens, ctxs, Hq, Hkv, d, fmt, seed=15, extra_blocks=2)
    for s in range(2):  # room for the decode step's tokens
        st["block_table"][s, -(-(qlens[s] + ctxs[s]) // 16)] = st["k_pages"].shape[0] - 1 - s
    dv = on_gpu(st)
    g = torch.Generator().manual_seed(16)
    inv_freq, factor = ea.rope_frequencies(d, scaling="yarn", factor=4.0, original_length=64, device=DEV)
    w = (1 + 0.1 * torch.randn(2, d, generator=g)).to(torch.bfloat16).to(DEV)
    for qlens in ([50, 7], [1, 1]):
        T = sum(qlens)
        x = torch.randn(T, Hq + 2 * Hkv, d, generator=g).to(torch.bfloat16).to(DEV)
        if qlens == [1, 1]:
            dv["seq_lens"] += 1
        dv["cu_q"] = torch.tensor([0, qlens[0], T], dtype=torch.int32, device=DEV)
        lens = dv["seq_lens"].tolist()
        pos = torch.cat([torch.arange(n - a, n, dtype=torch.int32) for n, a in zip(lens, qlens)]).to(DEV)
        q, k = ea.attn_norm_rope(x[:, :Hq], x[:, Hq:Hq + Hkv], w[0], w[1], pos, inv_freq, attention_factor=factor)
        before = {n: dv[n].cpu() for n in CACHE[:4]}
        ea.attn_kv_write_paged_q8(k, x[:, Hq + Hkv:], *(dv[n] for n in CACHE), max_q=max(qlens), kv_format=fmt)
        for n, new in (("k", k), ("v", x[:, Hq + Hkv:])):
            codes, scales = ref.write(n, f64(new), ref.code_values(before[n + "_pages"], fmt), f64(before[n + "_scales"]),
                                      dv["block_table"].cpu().numpy(), np.array(lens), dv["cu_q"].cpu().numpy(), fmt)
            assert np.array_equal(ref.code_values(dv[n + "_pages"], fmt), codes)
            assert np.array_equal(f64(dv[n + "_scales"]), scales)
        dv["q"] = q
        o, lse = run(dv, fmt)
        now = {n: t.cpu() for n, t in dv.items()}
        check(o, lse, reference(now, fmt))
        if qlens == [1, 1]:  # the library's decode says the same of one token
            o2, l2 = ea.attn_decode_paged_q8(q, *(dv[n] for n in CACHE[:6]), kv_format=fmt)
            wo, wl, size = reference(now, fmt)
            assert (np.abs(f64(o2) - wo) <= 2.0 ** -8 * np.abs(wo) + 2.0 ** -9 * size).all()
            assert np.abs(f64(l2) - wl).max() < 1e-3
    assert ea.device_status() == 0
