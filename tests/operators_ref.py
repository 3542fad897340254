"""Plain 64-bit forms for the tests of rotary positions, 4-bit pools and modified scores (CPU, torch and
numpy), written from the formulas in include/hswa.h.

Tolerances. A rounding to bf16 is off by at most half a step, 2^-8 of the value; f16 2^-11. An attention
output sum_j w_j v_j is rounded once (2^-8 |o|), and its weights w_j are rounded once on their way into
the tensor cores (bf16: 2^-8 sum w|v|; f16 on the codes of a 4-bit pool: 2^-11 sum w step code). The rest
(fp32 scores and exponentials) stays below 1e-4 of sum w|v| for the score sizes used here (|score| < 60:
60 * 2^-23 * a few). `Attention.tol` is that sum.
"""
from __future__ import annotations

import math
from dataclasses import dataclass

import numpy as np
import torch

BF16, F16 = 2.0 ** -8, 2.0 ** -11


# ------------------------------------------------------------------ 4-bit rows

def int4_rows(x: torch.Tensor):
    """Codes (uint8), step and minimum (bf16) of each row x [..., d] (bf16, CPU)."""
    f = x.float().numpy()
    lo, hi = f.min(-1, keepdims=True), f.max(-1, keepdims=True)
    with np.errstate(all="ignore"):
        rng = (hi - lo).astype(np.float32)
        step = torch.from_numpy((rng * np.float32(1.0 / 15.0)).astype(np.float32)).to(torch.bfloat16)
        bad = ~np.isfinite(f).all(-1, keepdims=True) | ~(rng <= np.finfo(np.float32).max)
        step[step.float() < 2.0 ** -120] = 0
        sf = step.float().numpy()
        inv = np.where(sf > 0, np.float32(1.0) / np.where(sf > 0, sf, np.float32(1.0)), np.float32(0.0)).astype(np.float32)
        t = ((f - lo).astype(np.float32) * inv).astype(np.float32)
        codes = np.where(bad, 0, np.clip(np.rint(np.where(bad, 0, t)), 0, 15)).astype(np.uint8)
    low = torch.from_numpy(lo.copy()).to(torch.bfloat16)
    step[torch.from_numpy(bad)] = float("nan")
    low[torch.from_numpy(bad)] = float("nan")
    return torch.from_numpy(codes), step, low


def int4_values(x: torch.Tensor) -> torch.Tensor:
    """What the rows stand for, in 64 bits (code * step + lo is exact in fp32 up to its last rounding)."""
    codes, step, low = int4_rows(x)
    return (codes.float() * step.float() + low.float()).double()


def int4_blocks(blocks: torch.Tensor, rows: int, d: int):
    """(codes [..., rows, d] uint8, pairs [..., rows, 2] int16 bit patterns) of raw pool blocks."""
    b = blocks.cpu()
    packed = b[..., : rows * d // 2].reshape(*b.shape[:-1], rows, d // 2)
    codes = torch.stack([packed & 15, packed >> 4], -1).reshape(*b.shape[:-1], rows, d)
    pairs = b[..., rows * d // 2: rows * d // 2 + rows * 4].contiguous().view(torch.int16)
    return codes, pairs.reshape(*b.shape[:-1], rows, 2)


# ------------------------------------------------------------------ attention

@dataclass
class Attention:
    o: torch.Tensor      # [n, Hq, d]
    tol: torch.Tensor


def attention(q, k, v, lo, hi, pos0=0, q_pos=None, cap=0.0, slope=None, weight_eps=BF16, v_range=None):
    """Row i of q [n, Hq, d] sees the keys at positions [lo[i], hi[i]) of k, v [m, Hkv, d] (positions
    pos0 ..). All double. A row without keys gives zeros. v_range [m, Hkv]: the range of 4-bit V rows,
    whose weights multiply codes."""
    q, k, v = q.double(), k.double(), v.double()
    n, hq, d = q.shape
    m, hkv = k.shape[0], k.shape[1]
    pos = torch.arange(pos0, pos0 + m)
    see = (pos[None] >= lo[:, None]) & (pos[None] < hi[:, None])
    o, tol = torch.zeros_like(q), torch.zeros_like(q)
    any_row = see.any(-1)
    for h in range(hq):
        g = h // (hq // hkv)
        z = (q[:, h] @ k[:, g].T) / math.sqrt(d)
        if cap:
            z = cap * torch.tanh(z / cap)
        if slope is not None:
            z = z - float(slope[h]) * (q_pos[:, None] - pos[None]).abs().double()
        z = torch.where(see, z, torch.tensor(-math.inf, dtype=torch.float64))
        w = torch.exp(z - torch.where(any_row, z.amax(-1), torch.zeros(n, dtype=torch.float64))[:, None])
        w = torch.where(see, w, torch.zeros_like(w))
        w = w / torch.where(any_row, w.sum(-1), torch.ones(n, dtype=torch.float64))[:, None]
        vv = torch.where(torch.isfinite(v[:, g]), v[:, g], torch.zeros_like(v[:, g]))
        o[:, h] = w @ vv
        scale = w @ vv.abs()
        if v_range is not None:
            scale = scale + (w @ v_range[:, g].double())[:, None]
        tol[:, h] = BF16 * o[:, h].abs() + (weight_eps + 1e-4) * scale
    return Attention(o, tol)


def check(got: torch.Tensor, ref: Attention, what=""):
    g = got.detach().cpu().double()
    assert g.shape == ref.o.shape, (g.shape, ref.o.shape)
    assert torch.isfinite(g).all(), f"{what}: non-finite output"
    bad = (g - ref.o).abs() > ref.tol + 1e-30
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} off, worst "
                           f"{float(((g - ref.o).abs() / (ref.tol + 1e-30)).max()):.2f} tolerances")


def ranges(n_q, start, end_all, window=0, key_begin=None, key_end=None):
    """Visible [lo, hi) of the query rows at positions start .. start + n_q - 1."""
    i = torch.arange(start, start + n_q)
    lo, hi = torch.zeros_like(i), i + 1
    if key_end is not None:
        hi = torch.clamp(key_end, max=end_all)
    if key_begin is not None:
        lo = torch.maximum(lo, key_begin)
    if window:
        lo = torch.maximum(lo, i - window + 1)
        hi = torch.minimum(hi, i + window)
    return lo, hi


# ------------------------------------------------------------------ rotary positions

def rope(x, pos, inv_freq, axis, interleaved):
    """x [n, heads, d] (bf16), pos [n_axes, n]: the turned values in 64 bits and their tolerance (one bf16
    rounding; an fp32 sine and cosine of an angle good to 2^-24 turns)."""
    n, h, d = x.shape
    half = len(inv_freq)
    f = torch.tensor(inv_freq, dtype=torch.float64)
    ang = pos.double()[torch.tensor(axis)].T * f[None]      # [n, half]
    c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
    y = x.double().clone()
    size = x.double().abs().clone()
    a = slice(0, 2 * half, 2) if interleaved else slice(0, half)
    b = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
    xa, xb = x.double()[..., a], x.double()[..., b]
    y[..., a], y[..., b] = xa * c - xb * s, xb * c + xa * s
    size[..., a] = size[..., b] = xa.abs() + xb.abs()
    return y, BF16 * y.abs() + 2e-6 * size
