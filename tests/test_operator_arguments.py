"""Numbers that a call of the 8-bit cache's entry points cannot take: refused with the call's own
errors, not taken for others."""
from __future__ import annotations

import pytest
import torch

import exact_io_aware_101_b200 as ea

CACHE = ("k_pages", "v_pages", "k_scales", "v_scales", "block_table", "seq_lens", "cu_q")


def tensors(Hkv=2, device="cpu"):
    i32 = dict(dtype=torch.int32, device=device)
    return dict(q=torch.zeros(3, 4, 64, dtype=torch.bfloat16, device=device),
                k=torch.zeros(3, Hkv, 64, dtype=torch.bfloat16, device=device),
                k_pages=torch.zeros(5, Hkv, 16, 64, dtype=torch.int8, device=device),
                v_pages=torch.zeros(5, Hkv, 16, 64, dtype=torch.int8, device=device),
                k_scales=torch.ones(5, Hkv, device=device), v_scales=torch.ones(5, Hkv, device=device),
                block_table=torch.zeros(1, 4, **i32), seq_lens=torch.tensor([3], **i32),
                cu_q=torch.tensor([0, 3], **i32))


def test_pages_without_heads():
    t = tensors(Hkv=0)
    with pytest.raises(ValueError):
        ea.attn_prefill_paged_q8(t["q"], *(t[n] for n in CACHE), max_q=3, kv_format="int8")


# (Past the C int: -2^32 + 3 is 3 in 32 bits, and -2^32 is 0.)
@pytest.mark.gpu
@pytest.mark.parametrize("number", [-1, -2**31, -2**32, -2**32 + 3, -2**63])
def test_negative_bounds_and_windows(number):
    t = tensors(device="cuda")
    cache = [t[n] for n in CACHE]
    for call in (lambda: ea.attn_prefill_paged_q8(t["q"], *cache, max_q=number, kv_format="int8"),
                 lambda: ea.attn_prefill_paged_q8(t["q"], *cache, max_q=3, window=number, kv_format="int8"),
                 lambda: ea.attn_kv_write_paged_q8(t["k"], t["k"], *cache, max_q=number, kv_format="int8"),
                 lambda: ea.attn_kv_read_paged_q8(*cache, tokens=3, max_q=number, kv_format="int8")):
        with pytest.raises(ea.AttnError):
            call()
