"""How a chunk call over the 8-bit cache is cut into blocks, at numbers of heads that no model has:
an answer, at once, whatever they are.  Asked in a process of its own, which has to live."""
from __future__ import annotations

import json
import subprocess
import sys

import pytest

import exact_io_aware_101_b200 as ea
from exact_io_aware_101_b200 import build as eabuild


@pytest.fixture(scope="module", autouse=True)
def built():
    eabuild.build()


def ask(calls):
    code = "import json, exact_io_aware_101_b200 as ea\nlib = ea.library()\nprint(json.dumps([%s]))" % ", ".join(calls)
    out = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=120)
    assert out.returncode == 0, (out.returncode, out.stderr[-500:])
    return json.loads(out.stdout)


def test_any_number_of_heads():
    # Primes (one head a group, as many groups as heads), the largest int, sums past it.
    # More work items than SMs, or rows past the limit of a call: no workspace.
    heads = [2**31 - 1, 2**31 - 19, 2**31 - 128, 2**31 - 127, 1000003, 2**30]
    assert not any(ask("ea.prefill_q8_workspace_bytes(1, %d, 1, %d, %d, 128, 4096)" % (h, T, T)
                       for h in heads for T in (1, 2, 1000)))
    a = 1 << 20  # never read: the sizes (or a missing GPU) turn the calls away
    for rc in ask("lib.attn_prefill_paged_q8(%d, %d, %d, %d, %d, 0, %d, %d, %d, %d, %d, 1, %d, 1, 1, 1, 128, 16, "
                  "4096, 1, 0.1, 0, None, %d, 1 << 30, None)" % ((a,) * 10 + (h, a)) for h in heads[:2]):
        assert rc in (1, 3)


def test_heads_of_a_block():
    # The largest divisor of the group that a tile holds, and a token's rows in so many groups.
    f = ea.prefill_q8_workspace_bytes
    for group, heads in ((1, 1), (5, 5), (128, 128), (129, 43), (130, 65), (160, 80), (254, 127), (256, 128),
                         (131, 1)):  # a prime past the tile: one head a block
        assert f(1, group, 1, 1, 1, 64, 4096) == 256 + 148 * heads * 65 * 4
