"""GPU parity of the grouped linear products, their gradients and the 8-bit checkpoints with
the fp64 definitions (oracle/grouped.py), element by element, with the rounding bounds of
tests/grouped_common.py.

Rows behind the last expert hold NaN in every input and a pattern in every output: they are
neither read nor written.  So do the token rows that no row names."""
import ctypes
import itertools

import pytest
import torch

from grouped_common import act_tol, dact_tol, moe, stored, sum_tol
from oracle import grouped as og

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF, F64 = torch.bfloat16, torch.float64
PATTERN = 0x5A


def say(*a):
    print(*a, flush=True)


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def rand(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(BF)


def offsets_of(counts):
    o = torch.zeros(len(counts) + 1, dtype=torch.int32)
    o[1:] = torch.cumsum(torch.tensor(counts, dtype=torch.int32), 0)
    return o.to(DEV)


def patterned(*shape, dtype):
    """A buffer of the byte PATTERN."""
    n = torch.empty(0, dtype=dtype).element_size()
    for s in shape:
        n *= s
    return torch.full((n,), PATTERN, dtype=torch.uint8, device=DEV).view(dtype).view(shape)


def untouched(t):
    return bool((t.contiguous().view(torch.uint8) == PATTERN).all())


def within(what, got, ref, tol):
    err = (got.to(F64) - ref).abs()
    ok = err <= tol
    if ref.numel():
        say(f"  {what}: worst error/tolerance {float((err / tol.clamp(min=1e-300)).max()):.3f}")
    assert bool(ok.all()), (what, float(err[~ok].max()), int((~ok).sum()))


class Case:
    """Inputs of a layout with `counts` rows per expert and `extra` rows behind them."""

    def __init__(self, counts, K, N, extra=0, tokens=None, seed=0, dense=False):
        g = self.g = gen(1000 + seed)
        self.E, self.K, self.N = len(counts), K, N
        self.n = sum(counts)
        self.R = self.n + extra
        self.offsets = None if dense else offsets_of(counts)
        self.segs = list(zip(*(lambda o: (o[:-1], o[1:]))(
            [0] + list(itertools.accumulate(counts)))))
        self.tokens = tokens
        rows = self.R if tokens is None else tokens
        self.x = rand(g, rows, K)
        if tokens is None:
            self.row_token = None
            self.x[self.n:] = float("nan")
        else:
            self.row_token = torch.randint(0, tokens, (self.R,), generator=g, device=DEV,
                                           dtype=torch.int32)
            named = torch.zeros(rows, dtype=torch.bool, device=DEV)
            named[self.row_token[:self.n].long()] = True
            self.x[~named] = float("nan")
        self.w = rand(g, self.E, K, N, scale=max(K, N) ** -0.5)
        self.w[[e for e, c in enumerate(counts) if c == 0]] = float("nan")
        self.bias = rand(g, self.E, N)
        self.residual = rand(g, self.R, N)
        self.dz = rand(g, self.R, N)
        self.residual[self.n:] = float("nan")
        self.dz[self.n:] = float("nan")
        self.p = moe().GroupedProblem(R=self.R, K=K, N=N, E=self.E, T=tokens)

    def checkpoint(self, cols, scale=1.0):
        """A checkpoint of random pre-activations; NaN codes behind the last row."""
        v, s = og.quantize(torch.randn(self.R, cols, generator=self.g, device=DEV, dtype=F64) *
                           scale)
        codes = (v / s.repeat_interleave(32, 1)).float().to(torch.float8_e4m3fn).view(torch.uint8)
        scales = (torch.log2(s) + 127).to(torch.uint8)
        codes[self.n:] = 0x7F
        return codes.contiguous(), scales.contiguous()


def check_linear(c, act="none", bias=False, residual=False, ckpt=False):
    m = moe()
    y = patterned(c.R, c.N, dtype=BF)
    ck = None
    if ckpt:
        ck = (patterned(c.R, c.N, dtype=torch.uint8), patterned(c.R, c.N // 32, dtype=torch.uint8))
    m.grouped_linear(c.p, c.x, c.w, c.offsets, bias=c.bias if bias else None, act=act,
                     residual=c.residual if residual else None, row_token=c.row_token,
                     checkpoint=ck, out=y)
    torch.cuda.synchronize()
    z, mag = og.linear(c.x, c.w, c.segs, c.bias if bias else None, c.row_token)
    dz = sum_tol(c.K, mag)
    f, _ = og.act(z, act)
    ref, tol = f, act_tol(z, f, dz, act)
    if residual:
        r = c.residual[:c.n].to(F64)
        ref = ref + r
        tol = tol + 2.0 ** -23 * (f.abs() + r.abs())
    within("y", y[:c.n], ref, stored(ref, tol))
    assert untouched(y[c.n:])
    if ckpt:
        check_checkpoint(ck, z, dz)
        assert untouched(ck[0][c.n:]) and untouched(ck[1][c.n:])
    return y, ck


def check_checkpoint(ck, z, dz):
    """The codes are nearest values (half a step at most) of a z that is off by dz, under the
    scale of a maximum that is off by dz."""
    n = z.shape[0]
    if n == 0:
        return
    v = og.dequantize(ck[0][:n], ck[1][:n])
    s = torch.exp2(ck[1][:n].to(F64) - 127)
    blocks = z.abs().reshape(n, -1, 32)
    off = dz.reshape(n, -1, 32)
    _, lo = og.quantize((blocks - off).clamp(min=0).amax(-1, keepdim=True)
                        .expand_as(blocks).reshape(z.shape))
    _, hi = og.quantize((blocks + off).amax(-1, keepdim=True).expand_as(blocks).reshape(z.shape))
    zero = blocks.amax(-1) == 0
    assert bool(((s >= lo) & (s <= hi) | zero & (s == 1)).all())
    sz = s.repeat_interleave(32, 1)
    half = sz * torch.exp2(torch.floor(torch.log2(((z.abs() + dz) / sz).clamp(min=2.0 ** -6))) - 4)
    within("z", v, z, dz + half)


def check_dx(c, act="none", ckpt=False, want_a=True, scale=1.0):
    m = moe()
    ck = c.checkpoint(c.K, scale) if ckpt else None
    dx = patterned(c.R, c.K, dtype=BF)
    a = patterned(c.R, c.K, dtype=BF) if ckpt and want_a else None
    m.grouped_linear_dx(c.p, c.dz, c.w, c.offsets, act=act, checkpoint=ck, out=dx, a=a)
    torch.cuda.synchronize()
    d, mag = og.dx(c.dz, c.w, c.segs)
    tol = sum_tol(c.N, mag)
    ref = d
    if ckpt:
        z = og.dequantize(*ck)[:c.n]
        f, df = og.act(z, act)
        e = dact_tol(z, df, act)
        ref, tol = d * df, tol * (df.abs() + e) + d.abs() * e + 2.0 ** -23 * (d * df).abs()
        if a is not None:
            within("a", a[:c.n], f, stored(f, act_tol(z, f, 0 * z, act)))
            assert untouched(a[c.n:])
    within("dx", dx[:c.n], ref, stored(ref, tol))
    assert untouched(dx[c.n:])
    return dx, a


def check_dw(c, bias=False, accumulate=False):
    m = moe()
    dw = patterned(c.E, c.K, c.N, dtype=torch.float32)
    db = patterned(c.E, c.N, dtype=torch.float32) if bias else None
    w0 = b0 = 0
    if accumulate:
        dw.copy_(torch.randn(dw.shape, generator=c.g, device=DEV))
        w0 = dw.to(F64)
        if bias:
            db.copy_(torch.randn(db.shape, generator=c.g, device=DEV))
            b0 = db.to(F64)
    m.grouped_linear_dw(c.p, c.x, c.dz, c.offsets, row_token=c.row_token, dw=dw, dbias=db,
                        accumulate=accumulate)
    torch.cuda.synchronize()
    rw, rb, mw, mb = og.dw(c.x, c.dz, c.segs, c.row_token)
    rows = torch.tensor([hi - lo for lo, hi in c.segs], device=DEV, dtype=F64)
    tw = sum_tol(rows[:, None, None], mw) + 2.0 ** -23 * (rw + w0).abs()
    within("dw", dw, rw + w0, tw + 1e-300)
    if bias:
        within("db", db, rb + b0, sum_tol(rows[:, None], mb) + 2.0 ** -23 * (rb + b0).abs() + 1e-300)
    return dw, db


# Row counts around every tile height, experts without rows, all rows on one expert.
LAYOUTS = {
    "one row": [1],
    "few": [0, 1, 0, 3, 2, 0],
    "tile edges": [63, 64, 65, 0, 127, 128, 129],
    "large edges": [255, 256, 257, 1, 0, 513],
    "skewed": [0, 0, 700, 0, 5, 0, 0, 33],
    "no rows": [0, 0, 0],
    "many experts": [(7 * i) % 5 for i in range(300)],
}
WIDTHS = [(8, 8), (64, 128), (72, 520), (264, 136), (520, 40), (1000, 264)]


@pytest.mark.parametrize("K,N", WIDTHS)
@pytest.mark.parametrize("name", LAYOUTS)
def test_products_on_every_layout(name, K, N):
    say(f"case {name} K={K} N={N}")
    if len(LAYOUTS[name]) > 100 and K * N > 64 * 128:
        K, N = 64, 136
    c = Case(LAYOUTS[name], K, N, extra=5, seed=K + N)
    check_linear(c)
    check_dx(c)
    check_dw(c, bias=True)


@pytest.mark.parametrize("act", ["none", "relu", "relu2", "silu", "gelu_tanh"])
@pytest.mark.parametrize("K,N", [(96, 160), (264, 512), (512, 96)])
def test_epilogues(act, K, N):
    say(f"case {act} K={K} N={N}")
    for tokens, counts in ((None, [130, 0, 64, 7]), (37, [5, 1, 0, 90, 300])):
        c = Case(counts, K, N, extra=3, tokens=tokens, seed=7)
        check_linear(c, act, bias=True, residual=True, ckpt=True)
        check_linear(c, act, bias=True, ckpt=True)
        check_linear(c, act, residual=True)
        c = Case(counts, N, K, extra=3, seed=8)
        check_dx(c, act, ckpt=True)
        check_dx(c, act, ckpt=True, want_a=False, scale=20.0)


@pytest.mark.parametrize("tokens", [1, 9, 400])
def test_gathered_rows(tokens):
    say(f"case tokens={tokens}")
    c = Case([40, 0, 129, 300, 2], 136, 264, extra=9, tokens=tokens, seed=tokens)
    check_linear(c, "silu", bias=True)
    check_dw(c, bias=True)


@pytest.mark.parametrize("rows", [1, 2, 15, 16, 17, 33, 100, 1003, 4100])
@pytest.mark.parametrize("K,N", [(2048, 768), (1416, 2056), (128, 4096)])
def test_dense(rows, K, N):
    """One expert without offsets: few tiles, long reductions."""
    say(f"case rows={rows} K={K} N={N}")
    c = Case([rows], K, N, seed=rows, dense=True)
    check_linear(c, "gelu_tanh", bias=True, residual=True)
    check_dx(c)
    check_dw(c, bias=True)


def test_no_live_rows_of_a_filled_buffer():
    c = Case([0, 0], 64, 64, extra=300, seed=3)
    check_linear(c, "silu", bias=True, ckpt=True)
    check_dx(c, "silu", ckpt=True)
    check_dw(c, bias=True)
    check_dw(c, bias=True, accumulate=True)


def test_no_rows_at_all():
    m = moe()
    p = m.GroupedProblem(R=0, K=64, N=96, E=2)
    e = torch.empty(0, 64, dtype=BF, device=DEV)
    dz = torch.empty(0, 96, dtype=BF, device=DEV)
    w = rand(gen(1), 2, 64, 96)
    off = offsets_of([0, 0])
    assert m.grouped_linear(p, e, w, off).shape == (0, 96)
    assert m.grouped_linear_dx(p, dz, w, off).shape == (0, 64)
    dw, db = m.grouped_linear_dw(p, e, dz, off, want_bias=True)
    torch.cuda.synchronize()
    assert not dw.any() and not db.any()
    dw.fill_(3.0)
    rt = torch.empty(0, dtype=torch.int32, device=DEV)
    m.grouped_linear_dw(p, e, dz, off, row_token=rt, dw=dw)
    torch.cuda.synchronize()
    assert not dw.any()
    dw.fill_(3.0)
    m.grouped_linear_dw(p, e, dz, off, dw=dw, accumulate=True)
    torch.cuda.synchronize()
    assert bool((dw == 3.0).all())
    ck = m.checkpoint_buffers(0, 96)
    assert m.activation_backward(dz, ck, "silu").shape == (0, 96)


@pytest.mark.parametrize("counts,K,N", [([70, 0, 300, 5], 136, 264), ([3000], 256, 128)])
def test_accumulated_weight_gradients(counts, K, N):
    c = Case(counts, K, N, extra=2, seed=11)
    check_dw(c, bias=True, accumulate=True)
    check_dw(c, accumulate=True)


# Sizes that reach each kernel and each way of splitting the reduction, with rows that are
# unevenly spread, widths that end inside a tile and a partial last stage.
FULL = [1300, 0, 900, 2, 700]          # many rows per expert
PART = [300, 299, 0, 511, 1, 640, 97, 400]
SPARSE = [(37 * i) % 101 for i in range(64)]  # less than a tile's rows per expert
LONE = [0] * 20 + [400] + [0] * 11     # few rows, all of them one expert's


@pytest.mark.parametrize("counts,K,N", [
    (FULL, 264, 6176), (FULL, 6176, 264), (PART, 264, 2208), (PART, 2208, 264), (SPARSE, 264, 800),
    (SPARSE, 800, 264), (LONE, 1096, 544), (LONE, 544, 1096), ([1], 4104, 1056),
    ([16], 4104, 1056), ([1], 1056, 4104), ([100], 4104, 1056), ([100], 1056, 4104)])
def test_products_of_every_size(counts, K, N):
    say(f"case {counts[:8]} K={K} N={N}")
    c = Case(counts, K, N, extra=7, seed=K + len(counts))
    check_linear(c, "silu", bias=True, residual=True, ckpt=N % 32 == 0)
    check_dx(c, "gelu_tanh" if K % 32 == 0 else "none", ckpt=K % 32 == 0)
    c = Case(counts, K, N, extra=7, seed=K + len(counts) + 1, tokens=333)
    check_linear(c, "relu2", bias=True, ckpt=N % 32 == 0)


@pytest.mark.parametrize("tokens", [None, 333])
@pytest.mark.parametrize("counts,K,N", [
    (PART, 1288, 1032), (PART, 520, 1032), (SPARSE, 136, 264), ([3000], 264, 136),
    ([5, 9000], 136, 520)])
def test_weight_gradients_of_every_size(counts, K, N, tokens):
    say(f"case {counts[:8]} K={K} N={N} tokens={tokens}")
    c = Case(counts, K, N, extra=7, seed=K + len(counts), tokens=tokens)
    check_dw(c, bias=True)
    check_dw(c, bias=True, accumulate=True)


def test_rows_behind_four_gigabytes():
    """Byte offsets past 32 bits in x (gathered), z's row buffers, the weights and their
    gradients; every value of a buffer's first and last rows, or of its last expert."""
    m = moe()
    g = gen(77)

    def big(*shape):  # one block repeated: random bits of that many values take too long
        t = torch.empty(*shape, dtype=BF, device=DEV)
        rows = t.view(-1, shape[-1])
        block = rand(g, 1021, shape[-1])
        for r in range(0, rows.shape[0], 1021):
            rows[r:r + 1021] = block[:rows.shape[0] - r]
        return t

    say("x")  # 600001 x 4096: 4.9 GB
    T, R, K, N = 600001, 300, 4096, 136
    x, w = big(T, K), rand(g, 2, K, N, scale=K ** -0.5)
    rt = torch.randint(T - 1000, T, (R,), generator=g, device=DEV, dtype=torch.int32)
    dz = rand(g, R, N)
    p = m.GroupedProblem(R=R, K=K, N=N, E=2, T=T)
    off = offsets_of([170, 130])
    y = m.grouped_linear(p, x, w, off, row_token=rt)
    dw, _ = m.grouped_linear_dw(p, x, dz, off, row_token=rt)
    for e, (lo, hi) in enumerate(((0, 170), (170, 300))):
        xe, we, de = x[rt[lo:hi].long()].to(F64), w[e].to(F64), dz[lo:hi].to(F64)
        ref = xe @ we
        within("y", y[lo:hi], ref, stored(ref, sum_tol(K, xe.abs() @ we.abs())))
        within("dw", dw[e], xe.T @ de, sum_tol(hi - lo, xe.abs().T @ de.abs()))
    del x, y, dw
    say("rows")  # the same height in the layout, and y of 4.9 GB
    R, K, N = 600001, 64, 4096
    x, w = rand(g, R, K), rand(g, 2, K, N, scale=K ** -0.5)
    off = offsets_of([R - 600, 600])
    p = m.GroupedProblem(R=R, K=K, N=N, E=2)
    y = m.grouped_linear(p, x, w, off)
    dx = m.grouped_linear_dx(p, y, w, off)
    for e, rows in ((0, slice(0, 500)), (0, slice(R - 700, R - 600)), (1, slice(R - 600, R))):
        xe, we, ye = x[rows].to(F64), w[e].to(F64), y[rows].to(F64)
        ref = xe @ we
        within("y", y[rows], ref, stored(ref, sum_tol(K, xe.abs() @ we.abs())))
        ref = ye @ we.T
        within("dx", dx[rows], ref, stored(ref, sum_tol(N, ye.abs() @ we.abs().T)))
    del y, dx, x
    say("weights")  # 136 x 4096 x 4608: 5.1 GB of weights, 10.3 GB of gradients
    E, K, N = 136, 4096, 4608
    w = big(E, K, N)
    for rows in (5, 70):
        off = offsets_of([rows] * E)
        p = m.GroupedProblem(R=rows * E, K=K, N=N, E=E)
        x, dz = rand(g, rows * E, K), rand(g, rows * E, N)
        y = m.grouped_linear(p, x, w, off)
        dx = m.grouped_linear_dx(p, dz, w, off)
        dw, _ = m.grouped_linear_dw(p, x, dz, off)
        for e in (0, E - 1):
            s = slice(rows * e, rows * (e + 1))
            xe, we, de = x[s].to(F64), w[e].to(F64), dz[s].to(F64)
            ref = xe @ we
            within("y", y[s], ref, stored(ref, sum_tol(K, xe.abs() @ we.abs())))
            ref = de @ we.T
            within("dx", dx[s], ref, stored(ref, sum_tol(N, de.abs() @ we.abs().T)))
            within("dw", dw[e], xe.T @ de, sum_tol(rows, xe.abs().T @ de.abs()))


@pytest.mark.parametrize("act", ["none", "relu", "relu2", "silu", "gelu_tanh"])
@pytest.mark.parametrize("rows,cols", [(1, 32), (61, 768), (300, 1408), (7, 4128)])
def test_activation_backward(act, rows, cols):
    say(f"case {act} {rows}x{cols}")
    m = moe()
    for live in (None, 0, rows // 2, rows, rows + 9):
        n = rows if live is None else min(live, rows)
        c = Case([n], 8, cols, extra=rows - n, seed=rows)
        ck = c.checkpoint(cols, 3.0)
        dz, a = patterned(rows, cols, dtype=BF), patterned(rows, cols, dtype=BF)
        lt = None if live is None else torch.tensor([live], dtype=torch.int32, device=DEV)
        m.activation_backward(c.dz, ck, act, live_rows=lt, out=dz, a=a)
        torch.cuda.synchronize()
        z = og.dequantize(*ck)[:n]
        f, df = og.act(z, act)
        d = c.dz[:n].to(F64)
        tol = d.abs() * (dact_tol(z, df, act) + 2.0 ** -23 * df.abs())
        within("dz", dz[:n], d * df, stored(d * df, tol))
        within("a", a[:n], f, stored(f, act_tol(z, f, 0 * z, act)))
        assert untouched(dz[n:]) and untouched(a[n:])
        dz2 = m.activation_backward(c.dz, ck, act, live_rows=lt)
        torch.cuda.synchronize()
        assert torch.equal(dz2[:n], dz[:n])


def test_every_code_and_scale_reads_back():
    """All 256 codes under scales from the smallest to the largest, through the identity."""
    m = moe()
    codes = torch.arange(256, dtype=torch.uint8, device=DEV).repeat(64, 1)
    scales = torch.arange(0, 256, 4, dtype=torch.uint8, device=DEV)[:, None].repeat(1, 8)
    scales = scales.contiguous()
    a = torch.empty(64, 256, dtype=BF, device=DEV)
    m.activation_backward(torch.zeros_like(a), (codes, scales), "none", a=a)
    torch.cuda.synchronize()
    ref = og.dequantize(codes, scales).to(torch.float32).to(BF)
    assert torch.equal(torch.isnan(a), torch.isnan(ref))
    ok = ~torch.isnan(ref)
    assert torch.equal(a[ok], ref[ok])


def test_extreme_values_reach_the_checkpoint():
    """A tiny, a huge, an infinite and a NaN pre-activation in otherwise ordinary blocks (an
    identity product): the codes of the values that are not finite are NaN, the other values
    of their blocks keep an ordinary scale."""
    m = moe()
    K = N = 64
    w = torch.eye(K, device=DEV, dtype=BF)[None]
    x = rand(gen(5), 6, K)
    x[0, 3], x[1, 40], x[2, 5], x[3, 6] = 1e30, -1e-30, float("inf"), float("nan")
    x[4] = 0
    # an infinite input times the identity's zeros is NaN in every column: through the bias
    # instead
    bias = torch.zeros(1, N, dtype=BF, device=DEV)
    ck = m.checkpoint_buffers(6, N)
    p = m.GroupedProblem(R=6, K=K, N=N)
    fin = x.clone()
    fin[2], fin[3] = 1.0, 2.0
    m.grouped_linear(p, fin, w, bias=bias, checkpoint=ck)
    torch.cuda.synchronize()
    v, _ = og.quantize(fin.to(F64))
    assert torch.equal(og.dequantize(*ck), v)
    bias[0, 5], bias[0, 36] = float("inf"), float("nan")
    y = m.grouped_linear(p, fin, w, bias=bias, act="silu", checkpoint=ck)
    torch.cuda.synchronize()
    v, s = og.quantize(fin.to(F64) + bias.to(F64))
    got = og.dequantize(*ck)
    assert torch.equal(torch.isnan(got), torch.isnan(v))
    assert torch.equal(got[~torch.isnan(v)], v[~torch.isnan(v)])
    assert bool(torch.isnan(y[:, 36]).all()) and bool(torch.isinf(y[:, 5]).all())
    g = m.activation_backward(torch.ones(6, N, dtype=BF, device=DEV), ck, "silu")
    torch.cuda.synchronize()
    assert torch.equal(torch.isnan(g), torch.isnan(v))


def test_rows_named_outside_the_tokens_read_zeros():
    c = Case([20, 30], 64, 64, tokens=16, seed=21)
    c.x = rand(gen(9), 16, 64)
    c.row_token[3], c.row_token[25], c.row_token[40] = -1, 16, 2 ** 31 - 1
    check_linear(c, bias=True)
    check_dw(c)


def test_offsets_beyond_the_rows_are_cut():
    """offsets past R, negative or decreasing name only rows inside the buffers."""
    m = moe()
    c = Case([10, 10, 10], 64, 64, seed=22)
    off = torch.tensor([-5, 8, 4, 99], dtype=torch.int32, device=DEV)
    y = m.grouped_linear(c.p, c.x, c.w, off)
    dw, _ = m.grouped_linear_dw(c.p, c.x, c.dz, off)
    torch.cuda.synchronize()
    for e, (lo, hi) in enumerate([(0, 8), (8, 8), (4, 30)]):
        ref = c.x[lo:hi].to(F64).t() @ c.dz[lo:hi].to(F64)
        mag = c.x[lo:hi].to(F64).abs().t() @ c.dz[lo:hi].to(F64).abs()
        within(f"dw[{e}]", dw[e], ref, sum_tol(hi - lo, mag) + 1e-300)
    ref = c.x[8:30].to(F64) @ c.w[2].to(F64)  # rows 4 .. 7 belong to two experts
    mag = c.x[8:30].to(F64).abs() @ c.w[2].to(F64).abs()
    within("y", y[8:30], ref, stored(ref, sum_tol(64, mag)))


def test_results_do_not_depend_on_the_run():
    c = Case([300, 0, 77, 1000], 264, 520, extra=4, tokens=200, seed=31)
    m = moe()

    def go():
        y = m.grouped_linear(c.p, c.x, c.w, c.offsets, act="silu", row_token=c.row_token)
        dx = m.grouped_linear_dx(c.p, c.dz, c.w, c.offsets)
        dw, db = m.grouped_linear_dw(c.p, c.x, c.dz, c.offsets, row_token=c.row_token,
                                     want_bias=True)
        return y[:c.n], dx[:c.n], dw, db

    first = go()
    for _ in range(3):
        for a, b in zip(first, go()):
            assert torch.equal(a, b)


def all_calls(c, ck, bufs):
    m = moe()
    m.grouped_linear(c.p, c.x, c.w, c.offsets, bias=c.bias, act="silu", row_token=c.row_token,
                     checkpoint=(bufs["zc"], bufs["zs"]), out=bufs["y"], ws=bufs["ws0"])
    m.grouped_linear_dx(c.p, c.dz, c.w, c.offsets, act="gelu_tanh", checkpoint=ck,
                        out=bufs["dx"], a=bufs["a"], ws=bufs["ws1"])
    m.grouped_linear_dw(c.p, c.x, c.dz, c.offsets, row_token=c.row_token, dw=bufs["dw"],
                        dbias=bufs["db"], ws=bufs["ws2"])
    m.activation_backward(c.residual, (bufs["zc"], bufs["zs"]), "silu",
                          live_rows=None if c.offsets is None else c.offsets[-1:],
                          out=bufs["g"])


def all_buffers(c):
    m = moe()
    b = dict(y=patterned(c.R, c.N, dtype=BF), dx=patterned(c.R, c.K, dtype=BF),
             a=patterned(c.R, c.K, dtype=BF), g=patterned(c.R, c.N, dtype=BF),
             zc=patterned(c.R, c.N, dtype=torch.uint8),
             zs=patterned(c.R, c.N // 32, dtype=torch.uint8),
             dw=patterned(c.E, c.K, c.N, dtype=torch.float32),
             db=patterned(c.E, c.N, dtype=torch.float32))
    for op in range(3):
        b[f"ws{op}"] = m.grouped_workspace(c.p, op, DEV)
    return b


def same(a, b):
    return all(torch.equal(a[n].view(torch.uint8), b[n].view(torch.uint8)) for n in a
               if not n.startswith("ws"))


@pytest.mark.parametrize("counts,dense", [([300, 0, 77, 5], False), ([24], True), ([2500], True)])
def test_graph_replays_equal_eager(counts, dense):
    """Captured once, replayed with changed inputs and eager calls in between."""
    say(f"case {counts}")
    c = Case(counts, 256, 512, extra=0 if dense else 4, seed=41, dense=dense)
    ck = c.checkpoint(c.K)
    eager, cap = all_buffers(c), all_buffers(c)
    all_calls(c, ck, eager)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        all_calls(c, ck, cap)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        all_calls(c, ck, cap)
    for i in range(4):
        c.x[:c.n] = rand(c.g, c.n, c.K)
        c.dz[:c.n] = rand(c.g, c.n, c.N)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        all_calls(c, ck, eager)
        torch.cuda.synchronize()
        assert same(eager, cap), f"replay {i}"


def test_calls_on_two_streams_at_once():
    """Each stream with its own buffers and workspaces."""
    cs = [Case([300, 0, 77, 5], 256, 512, extra=4, seed=51),
          Case([24], 1024, 512, seed=52, dense=True)]
    cks = [c.checkpoint(c.K) for c in cs]
    ref = [all_buffers(c) for c in cs]
    for c, ck, b in zip(cs, cks, ref):
        all_calls(c, ck, b)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    for _ in range(5):
        bufs = [all_buffers(c) for c in cs]
        torch.cuda.synchronize()
        for s, c, ck, b in zip(streams, cs, cks, bufs):
            with torch.cuda.stream(s):
                all_calls(c, ck, b)
        torch.cuda.synchronize()
        for b, r in zip(bufs, ref):
            assert same(b, r)


def test_layer_of_biased_experts_trains():
    """The operators together, as a layer of GELU experts is trained: routing and layout by the
    layer's own calls, two grouped products, the combine; then the gradients from the 8-bit
    checkpoint (the expert activation itself is not kept).  Every stage is held to its
    definition on the inputs that it got; the gradient of x as a whole to the exact one within
    what the checkpoint's rounding allows."""
    m = moe()
    T, H, E, k, I, act = 333, 128, 6, 2, 192, "gelu_tanh"
    g = gen(61)
    lp = m.Problem(T=T, H=H, E=E, k=k, I=I)
    x, dy = rand(g, T, H), rand(g, T, H)
    logits = torch.randn(T, E, generator=g, device=DEV)
    w1, w2 = rand(g, E, H, I, scale=H ** -0.5), rand(g, E, I, H, scale=I ** -0.5)
    b1, b2 = rand(g, E, I, scale=0.3), rand(g, E, H, scale=0.3)
    ids, wt, keep = m.route(lp, logits)
    d = m.dispatch(lp, x, ids, keep, rows=False)
    off, rt, R = d["offsets"], d["row_token"], T * k
    p1 = m.GroupedProblem(R=R, K=H, N=I, E=E, T=T)
    p2 = m.GroupedProblem(R=R, K=I, N=H, E=E)
    ck = m.checkpoint_buffers(R, I)
    h = m.grouped_linear(p1, x, w1, off, bias=b1, act=act, row_token=rt, checkpoint=ck)
    yp = m.grouped_linear(p2, h, w2, off, bias=b2)
    y = m.combine(lp, yp, wt, d["slot_to_row"])
    # backward
    row_w = torch.zeros(R, device=DEV)
    row_w[d["slot_to_row"].reshape(-1).long()] = wt.reshape(-1)
    dyp = (dy[rt.long()].float() * row_w[:, None]).to(BF)
    a = torch.empty(R, I, dtype=BF, device=DEV)
    dz1 = m.grouped_linear_dx(p2, dyp, w2, off, act=act, checkpoint=ck, a=a)
    dw2, db2 = m.grouped_linear_dw(p2, a, dyp, off, want_bias=True)
    dw1, db1 = m.grouped_linear_dw(p1, x, dz1, off, row_token=rt, want_bias=True)
    dxp = m.grouped_linear_dx(p1, dz1, w1, off)
    dx = m.combine(lp, dxp, torch.ones_like(wt), d["slot_to_row"])
    torch.cuda.synchronize()

    segs = og.segments(off, R, E)
    z, mag = og.linear(x, w1, segs, b1, rt)
    f, df = og.act(z, act)
    within("h", h, f, stored(f, act_tol(z, f, sum_tol(H, mag), act)))
    check_checkpoint(ck, z, sum_tol(H, mag))
    ref, mag = og.linear(h, w2, segs, b2)
    within("yp", yp, ref, stored(ref, sum_tol(I, mag)))
    zq = og.dequantize(*ck)
    fq, dfq = og.act(zq, act)
    within("a", a, fq, stored(fq, act_tol(zq, fq, 0 * zq, act)))
    da, mag = og.dx(dyp, w2, segs)
    e = dact_tol(zq, dfq, act)
    within("dz1", dz1, da * dfq,
           stored(da * dfq, sum_tol(H, mag) * (dfq.abs() + e) + da.abs() * e +
                  2.0 ** -23 * (da * dfq).abs()))
    rows = torch.tensor([hi - lo for lo, hi in segs], device=DEV, dtype=F64)
    for got_w, got_b, xin, din, rtk in ((dw2, db2, a, dyp, None), (dw1, db1, x, dz1, rt)):
        rw, rb, mw, mb = og.dw(xin, din, segs, rtk)
        within("dw", got_w, rw, sum_tol(rows[:, None, None], mw) + 1e-300)
        within("db", got_b, rb, sum_tol(rows[:, None], mb) + 1e-300)
    ref, mag = og.dx(dz1, w1, segs)
    within("dxp", dxp, ref, stored(ref, sum_tol(I, mag)))
    # the whole gradient of x against the exact chain: z off by half an E4M3 step (2^-4 of it,
    # or 2^-10 of its block's scale) moves act' by at most max|act''| times that (gelu:
    # |act''| <= 1.13); dyp, dz1 and dxp are each rounded once more
    exact_dz = da * df
    s = torch.exp2(ck[1].to(F64) - 127).repeat_interleave(32, 1)
    dz_off = da.abs() * 1.13 * torch.maximum(2.0 ** -4 * z.abs(), 2.0 ** -10 * s) * 1.01 + \
        1.01 * 2.0 ** -8 * exact_dz.abs() + 1e-5
    want, _ = og.dx(exact_dz.float().to(F64), w1.to(F64), segs)
    lim, _ = og.dx(dz_off, w1.abs(), segs)
    lim = lim + 2.0 ** -8 * (want.abs() + lim)
    tok = torch.zeros(T, H, dtype=F64, device=DEV).index_add_(0, rt.long(), want)
    tl = torch.zeros(T, H, dtype=F64, device=DEV).index_add_(0, rt.long(), lim)
    within("dx", dx, tok, stored(tok, tl))


def test_python_checks_on_the_device():
    m = moe()
    c = Case([4, 4], 64, 64, seed=71)
    good = dict(x=c.x, w=c.w, offsets=c.offsets)
    for kw, msg in ((dict(w=c.w.float()), "dtype"), (dict(w=c.w[:1]), "shape"),
                    (dict(x=c.x.t().contiguous().t()), "contiguous"),
                    (dict(offsets=None), "one expert"), (dict(offsets=c.offsets.cpu()), "GPU"),
                    (dict(offsets=c.offsets.long()), "dtype"),
                    (dict(bias=c.bias[:, :32]), "shape"),
                    (dict(checkpoint=(torch.empty(8, 64, dtype=torch.uint8, device=DEV),
                                      torch.empty(8, 3, dtype=torch.uint8, device=DEV))), "shape"),
                    (dict(act="swish"), "activation"),
                    (dict(ws=torch.empty(8, device=DEV)), "uint8")):
        with pytest.raises(ValueError, match=msg):
            m.grouped_linear(c.p, **{**good, **kw})
    with pytest.raises(ValueError, match="accumulate"):
        m.grouped_linear_dw(c.p, c.x, c.dz, c.offsets, accumulate=True)
    with pytest.raises(m.MoeError):
        m.grouped_linear_dx(c.p, c.dz, c.w, c.offsets, act="silu")  # no checkpoint to read
    with pytest.raises(m.MoeError):
        m.grouped_linear(c.p, c.x, c.w, c.offsets, out=c.x)  # output over an input


def test_debug_library_reports_bad_layouts():
    m = moe()
    dl = m.debug_lib()
    c = Case([20, 30], 64, 64, tokens=16, seed=81)
    y = torch.empty(50, 64, dtype=BF, device=DEV)
    ws = m.grouped_workspace(c.p, 0, DEV)
    m.debug_status()

    def go(off, rt):
        g = c.p.c()
        m._call_on(dl, "moe_grouped_linear", ctypes.byref(g), m._ptr(c.x), m._ptr(rt),
                   m._ptr(off), m._ptr(c.w), None, 0, None, m._ptr(y), None, None, m._ptr(ws),
                   0 if ws is None else ws.numel(), m._stream())
        return m.debug_status()

    assert go(c.offsets, c.row_token) == 0
    assert go(torch.tensor([0, 30, 20], dtype=torch.int32, device=DEV), c.row_token) == 4
    assert go(torch.tensor([0, 30, 51], dtype=torch.int32, device=DEV), c.row_token) == 4
    bad = c.row_token.clone()
    bad[7] = 16
    assert go(c.offsets, bad) == 8
