"""Plain restatement of the paged cache's three calls: one token, one head, one group at a time,
in fp64 (the 4-bit format's own roundings in fp32, as its definition has them).

The cache is held here as Python lists of rows per sequence, so nothing of the pages, the stored
nibble order or the kernels' tiling appears in the arithmetic; ``nibble_order_*`` restate the
stored order on their own.
"""
from __future__ import annotations

import math

import torch

GROUP = 32


def rotate(x, cos_sin_row, interleaved=False):
    """x [h, d] rotated by one table row (cosines, then sines), fp64, not rounded."""
    x = x.double()
    out = x.clone()
    n = cos_sin_row.numel() // 2
    for j in range(n):
        c, s = float(cos_sin_row[j]), float(cos_sin_row[n + j])
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + n)
        out[:, a] = x[:, a] * c - x[:, b] * s
        out[:, b] = x[:, b] * c + x[:, a] * s
    return out


def quantise(x):
    """x [..., 32] (bf16 values) -> codes [..., 32], s, z [...], every operation in fp32."""
    f = x.float()
    lo, hi = f.amin(-1), f.amax(-1)
    third = torch.tensor(1.0 / 15.0, dtype=torch.float32)
    s = ((hi - lo) * third).to(torch.bfloat16).float()
    s = torch.where(s < 2.0 ** -100, torch.zeros_like(s), s)
    z = (lo + 8 * s).to(torch.bfloat16).float()
    inv = torch.where(s > 0, torch.ones_like(s) / s, torch.zeros_like(s))
    codes = (torch.round((f - z[..., None]) * inv[..., None]) + 8).clamp(0, 15)
    bad = ~(torch.isfinite(f).all(-1) & torch.isfinite(hi - lo))
    s[bad], z[bad], codes[bad] = math.nan, math.nan, 8
    return codes.to(torch.uint8), s, z


def dequantise(codes, s, z):
    """fp64 values that codes [..., 32] with s, z [...] stand for."""
    return s.double()[..., None] * (codes.double() - 8) + z.double()[..., None]


def through_4_bits(x):
    """fp64 values that a row x [..., d] (bf16) has after it went through the 4-bit format."""
    g = x.unflatten(-1, (-1, GROUP))
    return dequantise(*quantise(g)).flatten(-2)


def nibble_order_keys(d):
    """value index held by each nibble of a stored key row, in order."""
    order = [0] * d
    for word in range(d // 8):
        g, i = word // 4, word % 4
        place = i * (d // 32) + g
        for e in range(8):
            order[8 * place + e] = 8 * word + e
    return order


def nibble_order_values(d):
    order = [0] * d
    for half in range(d // 4):
        g, i = half // 8, half % 8
        place = i * (d // 32) + g
        for e in range(4):
            order[4 * place + e] = 4 * half + e
    return order


def attend(q, k, v, *, scale=0.0, softcap=0.0, slopes=None, window=0, seen=None):
    """The newest n queries q [n, h_q, d_k] of one sequence over its k [L, h_kv, d_k], v [L, h_kv, d_v]
    (fp64): out [n, h_q, d_v], lse [n, h_q], and sum_u P |v_u| [n, h_q, d_v] (for error bounds).
    seen: optional [L] truth values, tokens that exist."""
    n, h_q, d_k = q.shape
    L, h_kv, d_v = v.shape
    scale = scale or 1.0 / math.sqrt(d_k)
    out = torch.zeros((n, h_q, d_v), dtype=torch.float64)
    mag = torch.zeros_like(out)
    lse = torch.full((n, h_q), -math.inf, dtype=torch.float64)
    for i in range(n):
        p = L - n + i
        us = [u for u in range(max(0, p - window + 1) if window else 0, p + 1) if seen is None or bool(seen[u])]
        if not us:
            continue
        for h in range(h_q):
            kh, vh = k[us, h // (h_q // h_kv)].double(), v[us, h // (h_q // h_kv)].double()
            x = kh @ q[i, h].double() * scale
            if softcap > 0:
                x = softcap * torch.tanh(x / softcap)
            if slopes is not None:
                x = x + float(slopes[h]) * (torch.tensor(us, dtype=torch.float64) - p)
            m = x.max()
            e = torch.exp(x - m)
            lse[i, h] = m + torch.log(e.sum())
            w = e / e.sum()
            out[i, h] = w @ vh
            mag[i, h] = w @ vh.abs()
    return out, lse, mag
