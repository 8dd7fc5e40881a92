"""Microscaled 4-bit values and the grouped product on them in fp64 (torch, on whatever device the
inputs are): the definitions that the GPU kernels are checked against.

A block of 32 values: the smallest power of two 2^e, e >= -127, with max|x| <= 6 2^e (LightLLM PR
#1687, walkthrough row "Grouped MoE kernel support": block scales are exact powers of two), and the
nearest of +-{0, 0.5, 1, 1.5, 2, 3, 4, 6} times it, ties to the even code.
"""
from __future__ import annotations

import torch

from . import grouped

F64 = torch.float64
BLOCK = 32
LEVELS = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=F64)


def quantize(x):
    """(codes [..., C / 2], scales [..., C / 32]) of x [..., C]."""
    lead, C = x.shape[:-1], x.shape[-1]
    b = x.to(F64).reshape(*lead, C // BLOCK, BLOCK)
    bad = ~torch.isfinite(b).all(-1)
    b = torch.where(bad[..., None], torch.zeros_like(b), b)
    top = b.abs().amax(-1)
    e = torch.full_like(top, -127.0)
    for p in range(-126, 127):  # one power at a time
        e = torch.where(top > 6 * 2.0 ** (p - 1), torch.full_like(e, float(p)), e)
    e = torch.where(top == 0, torch.zeros_like(e), e)
    v = (b * torch.exp2(-e)[..., None]).abs()
    levels = LEVELS.to(x.device)
    d = (v[..., None] - levels).abs()
    best = d.amin(-1, keepdim=True)
    # of two levels equally near, the even code
    rank = torch.where(d == best, torch.arange(8, device=x.device) % 2, 2)
    q = rank.argmin(-1).to(torch.uint8) | (torch.signbit(x).reshape(b.shape).to(torch.uint8) << 3)
    q = torch.where(bad[..., None], torch.zeros_like(q), q).reshape(*lead, C)
    s = torch.where(bad, torch.full_like(e, 255.0), e + 127).to(torch.uint8)
    return q[..., 0::2] | (q[..., 1::2] << 4), s


def dequantize(codes, scales):
    """What codes and scale bytes stand for, in fp64."""
    levels = torch.cat((LEVELS, -LEVELS)).to(codes.device)
    v = torch.stack((levels[(codes & 15).long()], levels[(codes >> 4).long()]), -1)
    v = v.reshape(*codes.shape[:-1], -1)
    f = torch.exp2(scales.to(F64) - 127)
    f = torch.where(scales == 255, torch.full_like(f, float("nan")), f)
    return v * f.repeat_interleave(BLOCK, -1)


def dequantize8(codes, scales):
    f = torch.exp2(scales.to(F64) - 127)
    f = torch.where(scales == 255, torch.full_like(f, float("nan")), f)
    return codes.view(torch.float8_e4m3fn).to(F64) * f.repeat_interleave(BLOCK, -1)


def linear(x, w, segs, bias=None, row_token=None):
    """(z, sum of |terms|) of the live rows: x [., K] and w [E, N, K] in fp64 (dequantised)."""
    return grouped.linear(x, w.transpose(1, 2), segs, bias, row_token)
