"""Shared by the tests of the 4-bit values and the product on them."""
import torch

from grouped_common import BF16_HALF, U24, act_tol, moe, stored, sum_tol
from oracle import fp4, grouped as og

F64 = torch.float64
DEV = "cuda"
PATTERN = 0x5A


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def offsets_of(counts, first=0):
    o = torch.zeros(len(counts) + 1, dtype=torch.int32)
    o[0] = first
    o[1:] = first + torch.cumsum(torch.tensor(counts, dtype=torch.int32), 0)
    return o.to(DEV)


def codes4(g, rows, K, spread=4):
    """Random 4-bit rows: any code, scales of a few powers of two; no block is NaN."""
    c = torch.randint(0, 256, (*rows, K // 2), generator=g, device=DEV, dtype=torch.uint8)
    s = torch.randint(127 - spread, 128, (*rows, K // 32), generator=g, device=DEV,
                      dtype=torch.uint8)
    return c, s


def codes8(g, rows, K, narrow):
    """Random 8-bit rows (E4M3).  narrow: magnitudes 16 .. 448 and zeros, whose products with E2M1
    codes (0.5 .. 6) have no bit more than 13 below a block's largest: 448 * 6 < 2^12 against the
    last bit of 16 * 0.5, 2^0; the matrix cores then drop nothing."""
    if narrow:
        c = torch.randint(0x58, 0x7F, (*rows, K), generator=g, device=DEV, dtype=torch.uint8)
        c |= torch.randint(0, 2, c.shape, generator=g, device=DEV, dtype=torch.uint8) << 7
        c *= torch.rand(c.shape, generator=g, device=DEV) < 0.9
    else:
        x = torch.randn(*rows, K, generator=g, device=DEV).bfloat16()
        c, s = moe().quantize_fp8(x.reshape(-1, K))
        return c.reshape(*rows, K), s.reshape(*rows, K // 32)
    s = torch.randint(117, 121, (*rows, K // 32), generator=g, device=DEV, dtype=torch.uint8)
    return c, s


def shifted(t):
    """A copy of a byte tensor that begins one byte behind an aligned place."""
    flat = torch.empty(t.numel() + 1, dtype=torch.uint8, device=t.device)
    out = flat[1:].view(t.shape)
    out.copy_(t)
    return out


class Case:
    """A product with its inputs; rows that no expert owns have NaN scales and a patterned y, as
    have the tokens that no row names."""

    def __init__(self, counts, K, N, x="fp4", act="none", gated=False, bias=False, residual=False,
                 gather=False, behind=0, front=0, T=None, seed=1, wild=False, shift=False):
        self.m = m = moe()
        g = gen(seed)
        E, live = len(counts), sum(counts)
        self.K, self.N, self.act, self.eight = K, N, act, x != "fp4"
        self.wide = x == "fp8 wide"
        R = front + live + behind
        self.lo, self.hi = front, front + live
        self.offsets = offsets_of(counts, front) if E > 1 or behind or front else None
        self.segs = og.segments(self.offsets, R, E)
        self.row_token = None
        rows = R
        if gather:
            rows = T if T is not None else max(1, R // 2)
            t = torch.randint(0, rows, (R,), generator=g, device=DEV, dtype=torch.int32)
            if wild and live > 2:  # rows that name no token read as zeros
                t[front], t[front + 1], t[front + 2] = -1, rows, 2 ** 31 - 1
            t[:front] = 2 ** 30
            t[front + live:] = 2 ** 30
            self.row_token = t
        if self.eight:
            self.xq = codes8(g, (rows,), K, not self.wide)
        else:
            self.xq = codes4(g, (rows,), K)
        if shift:  # scales need no alignment
            self.xq = self.xq[0], shifted(self.xq[1])
        if gather:
            named = torch.zeros(rows, dtype=torch.bool, device=DEV)
            t = self.row_token[front:front + live].long()
            named[t[(t >= 0) & (t < rows)]] = True
            self.xq[1][~named] = 255
        else:
            self.xq[1][:front] = 255
            self.xq[1][front + live:] = 255
        self.w = codes4(g, (E, N), K, 3)
        self.up = codes4(g, (E, N), K, 3) if gated else None
        if shift:
            self.w = self.w[0], shifted(self.w[1])
        if gated or act != "none":  # pre-activations of a few units: scales down by a power of two
            down = max(0, (K * (2 if not self.eight else 40)).bit_length() // 2)
            for q in (self.w, self.up) if gated else (self.w,):
                q[1].sub_(down)
        rnd = lambda *s: torch.randn(*s, generator=g, device=DEV).bfloat16()  # noqa: E731
        self.bias = rnd(E, N) if bias else None
        self.up_bias = rnd(E, N) if bias and gated else None
        self.residual = rnd(R, N) if residual else None
        if residual:
            self.residual[:front] = float("nan")
            self.residual[front + live:] = float("nan")
        self.p = m.GroupedProblem(R=R, K=K, N=N, E=E, T=rows if gather else None)
        self.R = R

    def new_y(self):
        return torch.full((self.R * self.N * 2,), PATTERN, dtype=torch.uint8,
                          device=DEV).view(torch.bfloat16).view(self.R, self.N)

    def run(self, y=None, ws=None):
        y = self.new_y() if y is None else y
        self.m.grouped_linear_fp4(self.p, self.xq, self.w, self.offsets, up=self.up,
                                  bias=self.bias, up_bias=self.up_bias, act=self.act,
                                  residual=self.residual, row_token=self.row_token, out=y, ws=ws)
        return y

    def product(self, q, bias):
        """(z, bound of its error) of the live rows, expert by expert"""
        x_of = fp4.dequantize8 if self.eight else fp4.dequantize
        zs, tols = [torch.zeros(0, self.N, dtype=F64, device=DEV)], []
        tols.append(zs[0])
        for e, (lo, hi) in enumerate(self.segs):
            if lo >= hi:
                continue
            rows, dead = slice(lo, hi), None
            if self.row_token is not None:
                t = self.row_token[lo:hi].long()
                dead = (t < 0) | (t >= self.xq[0].shape[0])
                rows = torch.where(dead, torch.zeros_like(t), t)
            x, w = x_of(self.xq[0][rows], self.xq[1][rows]), fp4.dequantize(q[0][e], q[1][e])
            if dead is not None:
                x = torch.where(dead[:, None], torch.zeros_like(x), x)
            z, size = x @ w.t(), x.abs() @ w.abs().t()
            tol = sum_tol(self.K, size)
            if self.wide:  # each of a block's 32 products loses what is 2^-13 of the largest
                top = lambda v: v.abs().reshape(v.shape[0], -1, 32).amax(-1)  # noqa: E731
                tol = tol + 32 * 2.0 ** -13 * (top(x) @ top(w).t())
            if bias is not None:
                z, tol = z + bias[e].to(F64), tol + U24 * (size + bias[e].to(F64).abs())
            zs.append(z)
            tols.append(tol)
        return torch.cat(zs), torch.cat(tols)

    def check(self, y):
        z, zt = self.product(self.w, self.bias)
        f = og.act(z, self.act)[0]
        tol = act_tol(z, f, zt, self.act) if self.act != "none" else zt
        if self.up is not None:
            u, ut = self.product(self.up, self.up_bias)
            tol = tol * u.abs() + f.abs() * ut + tol * ut + U24 * (f * u).abs()
            f = f * u
        if self.residual is not None:
            f = f + self.residual[self.lo:self.hi].to(F64)
            tol = tol + U24 * f.abs()
        got = y[self.lo:self.hi].to(F64)
        tol = stored(f, tol)
        err = (got - f).abs()
        if f.numel():
            print(f"  worst error/tolerance {float((err / tol).max()):.3f}", flush=True)
        assert bool((err <= tol).all()), (float((err - tol).max()), int((err > tol).sum()))
        for part in (y[:self.lo], y[self.hi:]):
            assert bool((part.contiguous().view(torch.uint8) == PATTERN).all())
