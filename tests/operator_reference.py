"""Plain 64-bit forms of the rotations and of the 8-bit paged cache, for the
parity tests: numpy, one row, page or sequence at a time, no code of the
package."""
from __future__ import annotations

import math

import numpy as np
import torch

PAGE = 16
QMAX = {"e4m3": 448.0, "int8": 127.0}


def half_step(t: torch.dtype) -> float:
    """Largest rounding error of a value to t, relative to the value."""
    return torch.finfo(t).eps / 2


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().double().numpy()


# ------------------------------------------------------------------ rotations

def rotate(x, positions, inv_freq, interleaved, factor, transpose=False):
    """x [..., N, d], positions broadcast to x[..., 0]: (rotated, |x| of the pair summed, times
    factor: what an error bound of each element is relative to)."""
    r = 2 * len(inv_freq)
    a = positions.astype(np.float64)[..., None] * inv_freq
    c, s = np.cos(a) * factor, np.sin(a) * factor * (-1.0 if transpose else 1.0)
    first = np.arange(0, r, 2) if interleaved else np.arange(r // 2)
    second = np.arange(1, r, 2) if interleaved else np.arange(r // 2, r)
    y, size = x.copy(), np.abs(x)
    p, q = x[..., first], x[..., second]
    y[..., first], y[..., second] = p * c - q * s, p * s + q * c
    size[..., first] = size[..., second] = (np.abs(p) + np.abs(q)) * factor
    return y, size


def norm_rotate(x, w, positions, inv_freq, interleaved, factor, eps):
    r = 1.0 / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps)
    return rotate(x * r * w, positions, inv_freq, interleaved, factor)


def norm_rotate_bwd(x, w, dy, positions, inv_freq, interleaved, factor, eps):
    """(dx, size of dx, dw, size of dw)."""
    u, us = rotate(dy, positions, inv_freq, interleaved, factor, transpose=True)
    r = 1.0 / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps)
    h = x * r
    dx = r * (w * u - h * (w * u * h).mean(-1, keepdims=True))
    sx = r * (np.abs(w) * us + np.abs(h) * (np.abs(w) * us * np.abs(h)).mean(-1, keepdims=True))
    d = x.shape[-1]
    return dx, sx, (u * h).reshape(-1, d).sum(0), (us * np.abs(h)).reshape(-1, d).sum(0)


# -------------------------------------------------------------- the 8-bit cache

_E4M3 = np.array([torch.tensor([c], dtype=torch.uint8).view(torch.float8_e4m3fn).double().item()
                  for c in range(256)])
_MAGS = _E4M3[:127]  # non-negative values, code by code


def code_values(codes: torch.Tensor, fmt: str) -> np.ndarray:
    raw = codes.detach().cpu().contiguous().view(torch.uint8).numpy()
    return raw.view(np.int8).astype(np.float64) if fmt == "int8" else _E4M3[raw]


def nearest(x: np.ndarray, fmt: str) -> np.ndarray:
    """The format's value nearest to x, ties to the even code, kept within it."""
    if fmt == "int8":
        return np.clip(np.rint(x), -127, 127)
    mag = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(_MAGS, mag), 1, 126)
    lo = hi - 1
    up, down = _MAGS[hi] - mag, mag - _MAGS[lo]
    pick = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return np.copysign(_MAGS[pick], x)


def write(kind, x, codes, scales, table, seq_lens, cu_q, fmt):
    """One of K and V: x [T, Hkv, d]; codes [P, Hkv, 16, d] and scales [P, Hkv] as 64-bit values.
    Returns the new (codes, scales)."""
    codes, scales = codes.copy(), scales.copy()
    for s in range(len(seq_lens)):
        t, end = int(cu_q[s]), int(cu_q[s + 1])
        pos = int(seq_lens[s]) - (end - t)
        while t < end:
            n = min(PAGE - pos % PAGE, end - t)
            pg, at = int(table[s][pos // PAGE]), pos % PAGE
            for g in range(x.shape[1]):
                rows = x[t:t + n, g]
                if not np.isfinite(rows).all() or (at and not np.isfinite(scales[pg, g])):
                    scales[pg, g] = np.nan
                    codes[pg, g, at:at + n] = 0.0
                    continue
                new = max(float(np.float32(np.abs(rows).max()) / np.float32(QMAX[fmt])), 2.0 ** -126)
                if at:
                    new = max(new, scales[pg, g])
                    if new != scales[pg, g]:
                        codes[pg, g, :at] = nearest(codes[pg, g, :at] * scales[pg, g] / new, fmt)
                codes[pg, g, at:at + n] = nearest(rows / new, fmt)
                scales[pg, g] = new
            t, pos = t + n, pos + n
    return codes, scales


def tokens_of(codes, scales, table, n):
    """The n tokens of one sequence, [n, Hkv, d]."""
    return np.stack([codes[table[t // PAGE], :, t % PAGE] * scales[table[t // PAGE]][:, None]
                     for t in range(n)]) if n else np.zeros((0,) + codes.shape[1:2] + codes.shape[3:])


def prefill(q, k, v, scale, window=0, slopes=None):
    """One sequence's chunk: q [nq, Hq, d] at the end of k, v [n, Hkv, d].  Returns o, lse and the
    size of o: the sum of (p + 2^-15 of the row's largest p) |v|, the second part for terms that
    a 16-bit p of its own no longer holds."""
    nq, hq, d = q.shape
    n, group = k.shape[0], hq // k.shape[1]
    o, lse, size = np.zeros((nq, hq, d)), np.zeros((nq, hq)), np.zeros((nq, hq, d))
    for h in range(hq):
        for t in range(nq):
            pos = n - nq + t
            first = max(0, pos - window + 1) if window else 0
            x = k[first:pos + 1, h // group] @ q[t, h] * scale
            if slopes is not None:
                x = x + slopes[h] * (np.arange(first, pos + 1) - pos)
            m = x.max()
            p = np.exp(x - m)
            lse[t, h] = m + math.log(p.sum())
            p /= p.sum()
            o[t, h] = p @ v[first:pos + 1, h // group]
            size[t, h] = (p + 2.0 ** -15 * p.max()) @ np.abs(v[first:pos + 1, h // group])
    return o, lse, size
