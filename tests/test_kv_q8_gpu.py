"""GPU parity of attn_kv_write_paged_q8 and attn_kv_read_paged_q8.

Codes and scales are whole decisions: they equal the 64-bit form's bit for bit
(the scale is one float32 division, each code the nearest value of an exact
quotient, ties to even).  What is read is scale * code rounded once; the product
is rounded to float32 on the way to bf16, 2^-24 beside bf16's 2^-8.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import exact_io_aware_101_b200 as ea
import operator_reference as ref
from operator_reference import f64

pytestmark = pytest.mark.gpu
DEV = "cuda"
CODES = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}


def make(qlens, ctxs, Hkv, d, fmt, seed, spare=3, extra_blocks=1, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    lens = [a + b for a, b in zip(qlens, ctxs)]
    blocks = [-(-n // 16) for n in lens]
    P, mb = sum(blocks) + spare, max(blocks + [1]) + extra_blocks
    perm = torch.randperm(P, generator=g).tolist()
    table = torch.full((len(lens), mb), -1, dtype=torch.int32)
    for s, b in enumerate(blocks):
        table[s, :b] = torch.tensor(perm[:b], dtype=torch.int32)
        perm = perm[b:]
    cu = torch.tensor([0] + list(np.cumsum(qlens)), dtype=torch.int32)
    st = dict(block_table=table, seq_lens=torch.tensor(lens, dtype=torch.int32), cu_q=cu)
    for n in ("k", "v"):
        x = torch.randn(P, Hkv, 16, d, generator=g, dtype=torch.float64).numpy() * 100
        st[n + "_pages"] = torch.from_numpy(ref.nearest(x, fmt)).float().to(CODES[fmt])
        # Scales around those that new tokens bring, some above and some below.
        st[n + "_scales"] = torch.exp(2 * torch.randn(P, Hkv, generator=g)) * 2.5 / ref.QMAX[fmt]
        st[n] = (spread * torch.randn(sum(qlens), Hkv, d, generator=g)).to(torch.bfloat16)
    return st


def on_gpu(st):
    return {n: t.to(DEV) for n, t in st.items()}


CACHE = ("k_pages", "v_pages", "k_scales", "v_scales", "block_table", "seq_lens", "cu_q")


def write(dv, fmt, max_q=None):
    lens = (dv["cu_q"][1:] - dv["cu_q"][:-1]).tolist()
    ea.attn_kv_write_paged_q8(dv["k"], dv["v"], *(dv[n] for n in CACHE), max_q=max(lens) if max_q is None else max_q,
                              kv_format=fmt)
    torch.cuda.synchronize()


def check_written(st, dv, fmt):
    for n in ("k", "v"):
        codes, scales = ref.write(n, f64(st[n]), ref.code_values(st[n + "_pages"], fmt), f64(st[n + "_scales"]),
                                  st["block_table"].numpy(), st["seq_lens"].numpy(), st["cu_q"].numpy(), fmt)
        assert np.array_equal(f64(dv[n + "_scales"]), scales, equal_nan=True)
        assert np.array_equal(ref.code_values(dv[n + "_pages"], fmt), codes, equal_nan=True)


CASES = [
    # qlens, ctxs, Hkv, d
    ([1], [0], 1, 64),
    ([1], [16], 2, 128),
    ([1, 1, 1, 1, 1], [15, 1, 31, 0, 7], 8, 128),
    ([0, 3, 17], [5, 14, 16], 3, 64),
    ([16, 32, 33], [0, 16, 8], 2, 128),
    ([40, 0, 2, 100], [3, 0, 15, 29], 5, 128),
    ([250], [1000], 4, 64),
]


@pytest.mark.parametrize("qlens,ctxs,Hkv,d", CASES)
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_write(qlens, ctxs, Hkv, d, fmt):
    st = make(qlens, ctxs, Hkv, d, fmt, seed=sum(ctxs) + d)
    dv = on_gpu(st)
    write(dv, fmt)
    check_written(st, dv, fmt)
    # The same call again leaves what it left.
    first = {n: dv[n].clone() for n in CACHE[:4]}
    write(dv, fmt)
    assert all(torch.equal(first[n].view(torch.uint8), dv[n].view(torch.uint8)) for n in CACHE[:4])
    assert ea.device_status() == 0


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_write_token_by_token(fmt):
    # A sequence written one token a call, its amplitude growing: every page is
    # rounded again and again, as the 64-bit form does it.
    n, Hkv, d = 37, 2, 64
    g = torch.Generator().manual_seed(3)
    x = (torch.randn(2, n, Hkv, d, generator=g) * torch.linspace(0.1, 5, n)[None, :, None, None]).to(torch.bfloat16)
    st = make([1], [n - 1], Hkv, d, fmt, seed=8)
    dv = on_gpu(st)
    for t in range(n):
        st["seq_lens"][0] = dv["seq_lens"][0] = t + 1
        for i, name in enumerate(("k", "v")):
            st[name] = x[i, t:t + 1]
            dv[name] = x[i, t:t + 1].to(DEV)
        want = {name: ref.write(name, f64(st[name]), ref.code_values(st[name + "_pages"], fmt), f64(st[name + "_scales"]),
                                st["block_table"].numpy(), st["seq_lens"].numpy(), st["cu_q"].numpy(), fmt)
                for name in ("k", "v")}
        write(dv, fmt)
        for name in ("k", "v"):
            assert np.array_equal(f64(dv[name + "_scales"]), want[name][1])
            assert np.array_equal(ref.code_values(dv[name + "_pages"], fmt), want[name][0])
            st[name + "_pages"], st[name + "_scales"] = dv[name + "_pages"].cpu(), dv[name + "_scales"].cpu()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_write_ties(fmt):
    # Quotients that lie on ties and next to them: scales that are powers of two
    # times 1 (the slice's largest is qmax) and every half step of the format.
    q = ref.QMAX[fmt]
    vals = sorted(set(np.abs(ref.nearest(np.linspace(0, q, 4000), fmt))))
    mids = [(a + b) / 2 for a, b in zip(vals, vals[1:])]
    x = torch.tensor([s * m for m in mids for s in (1, -1)], dtype=torch.float64)
    x = x[x.to(torch.bfloat16).double() == x]  # those that bf16 holds
    d = 128
    x = torch.cat([x, torch.zeros((-len(x)) % (15 * d), dtype=torch.float64)]).view(-1, 15, d)
    n = x.shape[0] * 16
    rows = torch.zeros(x.shape[0], 16, d, dtype=torch.float64)
    rows[:, :15] = x
    rows[:, 15] = q  # the slice's largest: scale 1
    for mul in (1.0, 2.0 ** -20):
        st = make([n], [0], 1, d, fmt, seed=1)
        st["k"] = st["v"] = (rows.view(n, 1, d) * mul).to(torch.bfloat16)
        dv = on_gpu(st)
        write(dv, fmt)
        check_written(st, dv, fmt)
    # Earlier codes halved (the scale doubles): odd codes land on ties.
    st = make([1], [15], 1, d, fmt, seed=2)
    for name in ("k", "v"):
        p = int(st["block_table"][0, 0])
        st[name + "_scales"][p] = 1.0
        st[name] = torch.full((1, 1, d), 2 * q, dtype=torch.bfloat16)
        c = torch.arange(16 * d, dtype=torch.float64).remainder(126) - 63
        st[name + "_pages"][p, 0] = torch.from_numpy(ref.nearest(c.numpy(), fmt)).view(16, d).float().to(CODES[fmt])
    dv = on_gpu(st)
    write(dv, fmt)
    check_written(st, dv, fmt)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_write_every_pair_of_mantissas(fmt):
    # A slice for every 8-bit mantissa of its largest value, holding every mantissa at 16
    # exponents: all the ties that bf16 values can meet, and how the scale's rounding breaks them.
    d, n = 128, 128
    amax = torch.arange(128, 256, dtype=torch.float64)
    x = torch.arange(128, 256, dtype=torch.float64)[None, :] * torch.exp2(-torch.arange(1, 17, dtype=torch.float64))[:, None]
    x = x[None].repeat(n, 1, 1)                      # [slice, 16 tokens, d]
    x[:, 0, 0] = amax
    x[:, 1::2] *= -1
    for mul in (1.0, 2.0 ** 60, 2.0 ** -90):
        st = make([16 * n], [0], 1, d, fmt, seed=1)
        st["k"] = st["v"] = (x * mul).view(16 * n, 1, d).to(torch.bfloat16)
        assert torch.equal(st["k"].double(), (x * mul).view(16 * n, 1, d))
        dv = on_gpu(st)
        write(dv, fmt)
        check_written(st, dv, fmt)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_write_small_large_zero_and_not_numbers(fmt):
    st = make([16] * 7, [0] * 7, 2, 64, fmt, seed=5)
    for name in ("k", "v"):
        x = st[name].view(7, 16, 2, 64)
        x[0] = 0
        x[1] *= 1e-38
        x[2] *= 1e37
        x[3, 4, 0, 9] = float("nan")
        x[4, 15, 1, 63] = float("-inf")
        x[5, :, :, 1:] = 0
        x[6] *= 2.0 ** -133  # bf16's subnormals
    dv = on_gpu(st)
    write(dv, fmt)
    check_written(st, dv, fmt)
    k, v = ea.attn_kv_read_paged_q8(*(dv[n] for n in CACHE), tokens=112, max_q=16, kv_format=fmt)
    k = k.view(7, 16, 2, 64)
    assert not k[0].any() and k[3, :, 0].isnan().all() and k[4, :, 1].isnan().all()
    assert k[3, :, 1].isfinite().all() and k[4, :, 0].isfinite().all()
    # A token behind a page whose scale is NaN leaves it NaN.
    dv["seq_lens"] += 0
    nxt = {n: dv[n] for n in CACHE}
    nxt["cu_q"] = torch.arange(8, dtype=torch.int32, device=DEV)
    ea.attn_kv_write_paged_q8(dv["k"].view(7, 16, 2, 64)[:, 0], dv["v"].view(7, 16, 2, 64)[:, 0], *nxt.values(), max_q=1,
                              kv_format=fmt)
    torch.cuda.synchronize()
    p = dv["block_table"][3, 0]
    assert dv["k_scales"][p, 0].isnan() and dv["k_scales"][p, 1].isfinite()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_write_from_a_projection(fmt):
    # k and v as slices of one [T, Hq + 2 Hkv, d] output.
    st = make([30, 5], [3, 100], 2, 128, fmt, seed=6)
    x = torch.randn(35, 8, 128).to(torch.bfloat16)
    x[:, 4:6], x[:, 6:] = st["k"], st["v"]
    dv = on_gpu(st)
    x = x.to(DEV)
    dv["k"], dv["v"] = x[:, 4:6], x[:, 6:]
    write(dv, fmt)
    check_written(st, dv, fmt)


def test_write_bad_lengths_and_pages():
    fmt = "int8"
    st = make([20, 20, 20, 20], [5, 5, 5, 5], 2, 64, fmt, seed=7)
    good = on_gpu(st)
    write(good, fmt)
    for what in ("page high", "page negative", "length", "bound"):
        dv = on_gpu(st)
        s, max_q = 1, 20
        if what == "page high":
            dv["block_table"][s, 1] = dv["k_pages"].shape[0]
        elif what == "page negative":
            dv["block_table"][s, 1] = -1
        elif what == "length":
            dv["seq_lens"][s] = 16 * dv["block_table"].shape[1] + 1
        else:
            dv["cu_q"] = torch.tensor([0, 0, 41, 41, 41], dtype=torch.int32, device=DEV)
        write(dv, fmt, max_q=max_q)
        assert ea.device_status(clear=True) == ea.ATTN_DEV_BAD_PAGE, what
        if what == "bound":
            assert torch.equal(dv["k_pages"], on_gpu(st)["k_pages"])
            continue
        for o in (0, 2, 3):  # the other sequences are written
            for p in st["block_table"][o, :2].tolist():
                assert torch.equal(dv["k_pages"][p], good["k_pages"][p])
        p = int(st["block_table"][s, 1])  # and nothing else is
        assert torch.equal(dv["k_pages"][p].cpu(), st["k_pages"][p])
    assert ea.device_status() == 0


@pytest.mark.parametrize("qlens,ctxs,Hkv,d", CASES)
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_read(qlens, ctxs, Hkv, d, fmt, dtype):
    st = make(qlens, ctxs, Hkv, d, fmt, seed=sum(qlens) + d)
    dv = on_gpu(st)
    T = sum(qlens)
    out = [torch.full((T + 2, Hkv, d), 7.0, dtype=dtype, device=DEV) for _ in range(2)]
    ea.attn_kv_read_paged_q8(*(dv[n] for n in CACHE), tokens=T + 2, max_q=max(qlens), kv_format=fmt, dtype=dtype,
                             k=out[0], v=out[1])
    torch.cuda.synchronize()
    for n, got in zip(("k", "v"), out):
        want = np.concatenate([ref.tokens_of(ref.code_values(st[n + "_pages"], fmt), f64(st[n + "_scales"]),
                                             st["block_table"][s].tolist(), a + b)[b:]
                               for s, (a, b) in enumerate(zip(qlens, ctxs))])
        assert (got[T:] == 7).all()  # rows of no sequence
        err = np.abs(f64(got[:T]) - want)
        lim = ref.half_step(dtype) * (1 + 2.0 ** -7) + (2.0 ** -24 if dtype == torch.bfloat16 else 0)
        assert (err <= lim * np.abs(want)).all()
    assert ea.device_status() == 0


def test_read_bad_page():
    st = make([20, 20], [5, 5], 2, 64, "e4m3", seed=9)
    dv = on_gpu(st)
    dv["block_table"][1, 1] = 1 << 30
    k, v = ea.attn_kv_read_paged_q8(*(dv[n] for n in CACHE), tokens=40, max_q=20)
    assert ea.device_status(clear=True) == ea.ATTN_DEV_BAD_PAGE
    assert k[:20].isfinite().all() and k[20:31].isfinite().all() and k[31:].isnan().all() and v[31:].isnan().all()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_written_cache_is_the_decodes(fmt):
    # A sequence written in two chunks and a token, then decoded by the library's 8-bit decode:
    # the same as the 64-bit attention over what is read back.
    Hkv, Hq, d, n = 2, 8, 128, 75
    g = torch.Generator().manual_seed(13)
    x = torch.randn(2, n, Hkv, d, generator=g).to(torch.bfloat16).to(DEV)
    st = make([n], [0], Hkv, d, fmt, seed=14)
    dv = on_gpu(st)
    done = 0
    for step in (50, 24, 1):
        dv["k"], dv["v"] = x[0, done:done + step], x[1, done:done + step]
        done += step
        dv["seq_lens"].fill_(done)
        dv["cu_q"] = torch.tensor([0, step], dtype=torch.int32, device=DEV)
        write(dv, fmt)
    q = torch.randn(1, Hq, d, generator=g).to(torch.bfloat16).to(DEV)
    o, lse = ea.attn_decode_paged_q8(q, *(dv[m] for m in CACHE[:6]), kv_format=fmt)
    dv["cu_q"] = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    k, v = ea.attn_kv_read_paged_q8(*(dv[m] for m in CACHE), tokens=n, max_q=n, kv_format=fmt, dtype=torch.float32)
    # One step of a grown scale is at most amax / qmax (int8) and 2^-4 of a value (E4M3); a token
    # is rounded at most three times here.
    step = 3 * (5.0 / 127 if fmt == "int8" else 5.0 / 16)
    assert (k - x[0].float()).abs().max() < step and (v - x[1].float()).abs().max() < step
    wo, wl, size = ref.prefill(f64(q), f64(k), f64(v), d ** -0.5)
    assert (np.abs(f64(o) - wo) <= 2.0 ** -8 * np.abs(wo) + 2.0 ** -9 * size).all()
    assert np.abs(f64(lse) - wl).max() < 1e-3
