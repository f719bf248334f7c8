"""Values that attn_kv_read_paged_q8 gives out and codes that attn_kv_write_paged_q8 rounds again,
where one rounding and two differ: whole decisions, equal to the 64-bit form's."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import exact_io_aware_101_b200 as ea
import operator_reference as ref
from operator_reference import f64
from test_kv_q8_gpu import CACHE, CODES, check_written, make, on_gpu, write

pytestmark = pytest.mark.gpu
DEV = "cuda"


def to_bf16(x: np.ndarray) -> np.ndarray:
    """The bf16 value nearest to a product of a float32 and a code (at most 32 bits, exact in 64),
    ties to even: half-way cases decided on the exact value."""
    m, e = np.frexp(np.abs(x))                      # m in [1/2, 1)
    unit = np.exp2(np.maximum(e - 8, -133.0))       # bf16's last place there
    return np.copysign(np.rint(np.abs(x) / unit) * unit, x)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_read_rounds_once(fmt, dtype):
    # Every code over scales whose products fall on bf16's ties and a float32 step beside them,
    # and over random ones; sizes from bf16's subnormals up.
    codes = torch.arange(256, dtype=torch.uint8).view(CODES[fmt])
    if fmt == "e4m3":
        codes = codes[~codes.float().isnan()]
    codes = torch.cat([codes, codes[:-len(codes) % 256 or len(codes)]])[:256]
    g = torch.Generator().manual_seed(4)
    vals = codes.double()
    scales = []
    for c in vals[vals != 0].abs().unique()[::3].tolist():
        # A bf16 tie t = (2k + 1) 2^-9 over the code, rounded to float32, and its neighbours.
        k = torch.randint(128, 256, (6,), generator=g).double()
        near = ((2 * k + 1) / 512 / c).float()
        scales += [near, torch.nextafter(near, torch.tensor(0.0)), torch.nextafter(near, torch.tensor(9.0))]
    scales = torch.cat(scales + [torch.randn(1000, generator=g) * 0.01])
    d, Hkv, per = 64, 1, 16 * 64 // 256
    for mul in (1.0, 2.0 ** -120, 2.0 ** -131, 2.0 ** 100):
        sc = (scales * mul).float()
        P = sc.numel()
        pages = codes.view(1, 1, 1, 256).expand(P, Hkv, per, 256).reshape(P, Hkv, 16, d).contiguous()
        dv = on_gpu(dict(k_pages=pages, v_pages=pages, k_scales=sc.view(P, 1), v_scales=-sc.view(P, 1),
                         block_table=torch.arange(P, dtype=torch.int32).view(1, P),
                         seq_lens=torch.tensor([16 * P], dtype=torch.int32),
                         cu_q=torch.tensor([0, 16 * P], dtype=torch.int32)))
        k, v = ea.attn_kv_read_paged_q8(*(dv[n] for n in CACHE), tokens=16 * P, max_q=16 * P, kv_format=fmt, dtype=dtype)
        exact = f64(pages.float()).reshape(P, 16 * d) * f64(sc)[:, None]
        with np.errstate(over="ignore"):
            want = to_bf16(exact) if dtype == torch.bfloat16 else exact.astype(np.float32).astype(np.float64)
        assert np.array_equal(f64(k).reshape(P, -1), want)
        assert np.array_equal(f64(v).reshape(P, -1), -want)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("old", [-1.0, -0.013, -300.0, -3e38, -1e-40, 0.0, -0.0])
def test_earlier_codes_under_a_negative_scale(fmt, old):
    # A page whose scale was negative: its earlier codes change sign, and those that the new scale
    # cannot hold become the format's largest.
    d, Hkv = 64, 2
    st = make([3], [9], Hkv, d, fmt, seed=31)
    p = int(st["block_table"][0, 0])
    for n in ("k", "v"):
        st[n + "_scales"][p] = old
    dv = on_gpu(st)
    write(dv, fmt)
    lo, hi = (-128.0, 127.0) if fmt == "int8" else (-448.0, 448.0)
    for n in ("k", "v"):
        new = np.maximum(np.abs(f64(st[n])).max((0, 2)).astype(np.float32) / np.float32(ref.QMAX[fmt]), np.float32(2.0 ** -126))
        assert np.array_equal(f64(dv[n + "_scales"])[p], new.astype(np.float64))
        was = ref.code_values(st[n + "_pages"], fmt)[p, :, :9]
        x = was * float(np.float32(old)) / new.astype(np.float64)[:, None, None]
        want = np.clip(np.rint(x), lo, hi) if fmt == "int8" else ref.nearest(x, fmt)
        got = ref.code_values(dv[n + "_pages"], fmt)[p]
        assert np.array_equal(got[:, :9], want)
        rows = ref.nearest(f64(st[n]).transpose(1, 0, 2) / new.astype(np.float64)[:, None, None], fmt)
        assert np.array_equal(got[:, 9:12], rows)
