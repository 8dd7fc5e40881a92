"""The grouped linear products, their gradients and the 8-bit checkpoints in fp64 (torch, on
whatever device the inputs are): the definitions that the GPU kernels are checked against.

  linear   z = x W[e] + b[e], y = act(z) + residual   over the rows of each expert
  dx       dx = (dz W[e]^T) act'(z), a = act(z)
  dw       dW[e] = x_e^T dz_e, db[e] = sum dz_e
  checkpoint: E4M3 values times one power of two per 32 columns, the smallest 2^e with
  max|z| <= 448 2^e (LightLLM PR #1687, walkthrough row "Grouped MoE kernel support": UE8M0
  block scales, exact powers of two)

Every product also returns the same sum over absolute values, which bounds the rounding of an
fp32 accumulation in any order.
"""
from __future__ import annotations

import torch

F64 = torch.float64
BLOCK = 32
SQRT_2_PI = 0.7978845608028654


def act(z, name):
    """(act(z), act'(z))"""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        return z.clamp(min=0), (z > 0).to(z.dtype)
    if name == "relu2":
        return z.clamp(min=0) ** 2, 2 * z.clamp(min=0)
    if name == "silu":
        s = torch.sigmoid(z)
        return z * s, s + z * s * (1 - s)
    if name == "gelu_tanh":
        # z (1 + tanh u) / 2 = z sigma(2 u), without the cancellation at negative z
        s = torch.sigmoid(2 * SQRT_2_PI * (z + 0.044715 * z ** 3))
        du2 = 2 * SQRT_2_PI * (1 + 3 * 0.044715 * z ** 2)
        return z * s, s + z * s * (1 - s) * du2
    raise ValueError(name)


def segments(offsets, R, E):
    if offsets is None:
        return [(0, R)]
    o = [int(v) for v in offsets.tolist()]
    return list(zip(o[:E], o[1:E + 1]))


def rows_of(x, row_token, lo, hi):
    """x[row_token[lo:hi]] in fp64; a token outside x reads as zeros."""
    if row_token is None:
        return x[lo:hi].to(F64)
    t = row_token[lo:hi].long()
    ok = (t >= 0) & (t < x.shape[0])
    return torch.where(ok[:, None], x[t.clamp(0, max(0, x.shape[0] - 1))].to(F64),
                       torch.zeros((), dtype=F64, device=x.device))


def linear(x, w, segs, bias=None, row_token=None):
    """(z, abs): the pre-activations of the live rows and sum |x||w| + |b|."""
    N = w.shape[2]
    z, m = [], []
    for e, (lo, hi) in enumerate(segs):
        if lo == hi:
            continue
        xr, we = rows_of(x, row_token, lo, hi), w[e].to(F64)
        ze, me = xr @ we, xr.abs() @ we.abs()
        if bias is not None:
            ze, me = ze + bias[e].to(F64), me + bias[e].to(F64).abs()
        z.append(ze)
        m.append(me)
    if not z:
        return (torch.zeros(0, N, dtype=F64, device=w.device),) * 2
    return torch.cat(z), torch.cat(m)


def dx(dz, w, segs):
    """(dz W^T, its sum of absolute values) of the live rows."""
    wt = [w[e].to(F64).t() for e in range(len(segs))]
    d = [dz[lo:hi].to(F64) @ wt[e] for e, (lo, hi) in enumerate(segs) if lo < hi]
    m = [dz[lo:hi].to(F64).abs() @ wt[e].abs() for e, (lo, hi) in enumerate(segs) if lo < hi]
    if not d:
        return (torch.zeros(0, w.shape[1], dtype=F64, device=w.device),) * 2
    return torch.cat(d), torch.cat(m)


def dw(x, dz, segs, row_token=None):
    """(dW [E, K, N], db [E, N], and their sums of absolute values)."""
    out = ([], [], [], [])
    for lo, hi in segs:
        xr, d = rows_of(x, row_token, lo, hi), dz[lo:hi].to(F64)
        for o, v in zip(out, (xr.t() @ d, d.sum(0), xr.abs().t() @ d.abs(), d.abs().sum(0))):
            o.append(v)
    return tuple(torch.stack(o) for o in out)


def quantize(z):
    """(values, scales) of the checkpoint of z: what its codes and scale bytes stand for."""
    R, N = z.shape
    b = z.reshape(R, N // BLOCK, BLOCK)  # both given: R may be 0
    finite = torch.isfinite(b)
    top = torch.where(finite, b.abs(), torch.zeros_like(b)).amax(-1)
    m, x = torch.frexp(top)
    e = torch.where(top > 0, x - 9 + (m > 0.875), torch.zeros_like(x)).clamp(-127, 127).to(F64)
    v = b * torch.exp2(-e)[..., None]
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    q = torch.round(v / step) * step
    q = torch.where(finite, q, torch.full_like(q, float("nan")))
    return (q * torch.exp2(e)[..., None]).reshape(R, N), torch.exp2(e)


def dequantize(codes, scales):
    """What the bytes of a checkpoint stand for."""
    c = codes.view(torch.float8_e4m3fn).to(F64)
    s = torch.exp2(scales.to(F64) - 127)
    return c * s.repeat_interleave(BLOCK, 1)
