"""Paths through the grouped kernels that the layouts of test_gpu_grouped.py do not take."""
import pytest
import torch

from grouped_common import moe
from grouped_paths import DW, DX, LINEAR, ONES, PATHS
from test_gpu_grouped import (BF, DEV, Case, check_dw, check_dx, check_linear, patterned, rand, say,
                              untouched)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("counts,K,N", [
    ([64, 128, 64, 0, 192, 64, 320, 64, 64, 128] * 4, 1024, 1024),  # several items per block
    ([64, 192, 128, 64, 256, 64, 0, 128, 64], 1032, 1024),          # the same on smaller tiles
    ([64, 63, 64, 65, 128, 1, 64, 127] * 3, 1032, 520)])            # whole and partial last stages
def test_gathered_weight_gradients_of_whole_stages(counts, K, N):
    """Experts whose rows are a multiple of a stage: the copies go from one item's last whole
    stage straight on to the next item's token list."""
    say(f"case {counts[:10]} K={K} N={N}")
    c = Case(counts, K, N, extra=3, tokens=301, seed=len(counts))
    check_dw(c, bias=True)
    check_dw(c, accumulate=True)


def of(p):
    return dict(argvalues=[q for q in PATHS if q.mode == p], ids=lambda q: q.name)


def case(p, tokens, seed):
    c = Case(p.counts, p.K, p.N, extra=p.extra, tokens=tokens, seed=seed)
    if tokens is not None:  # rows that name no token read zeros: a first, a last and one between
        c.row_token[0], c.row_token[c.n - 1], c.row_token[c.n // 2] = -1, tokens, 2 ** 31 - 1
    return c


@pytest.mark.parametrize("tokens", [None, 333])
@pytest.mark.parametrize("p", **of(LINEAR))
def test_linear_on_every_kernel(p, tokens):
    say(f"case {p.name} tokens={tokens}")
    c = case(p, tokens, 1)
    check_linear(c)
    check_linear(c, "silu", bias=True, residual=True)
    if p.N % 32 == 0:
        check_linear(c, "gelu_tanh", bias=True, residual=True, ckpt=True)


@pytest.mark.parametrize("p", **of(DX))
def test_dx_on_every_kernel(p):
    say(f"case {p.name}")
    c = case(p, None, 2)
    check_dx(c)
    check_dx(c, "gelu_tanh", ckpt=True)
    check_dx(c, "relu2", ckpt=True, want_a=False)


@pytest.mark.parametrize("tokens", [None, 333])
@pytest.mark.parametrize("p", **of(DW))
def test_dw_on_every_kernel(p, tokens):
    say(f"case {p.name} tokens={tokens}")
    c = case(p, tokens, 3)
    check_dw(c)
    check_dw(c, bias=True)
    check_dw(c, bias=True, accumulate=True)


@pytest.mark.parametrize("p", [q for q in PATHS if q.counts is not ONES], ids=lambda q: q.name)
def test_rows_before_the_first_expert_are_left_alone(p):
    """Offsets that start behind row 0 (the experts of a slice of a layout): the same values as
    from row 0, bit for bit, and nothing read or written in front of them."""
    say(f"case {p.name}")
    m, lead = moe(), 5
    c = Case(p.counts, p.K, p.N, extra=p.extra, seed=4)
    off = c.offsets + lead

    def moved(t):  # the same rows, NaN (or its code) around them
        s = torch.full_like(t, 0x7F if t.dtype == torch.uint8 else float("nan"))
        s[lead:lead + c.n] = t[:c.n]
        return s

    def compare(a, b):
        assert torch.equal(a[:c.n].view(torch.uint8), b[lead:lead + c.n].view(torch.uint8))
        assert untouched(b[:lead]) and untouched(b[lead + c.n:])

    if p.mode == LINEAR:
        width, wide = (p.N, p.N // 32 if p.N % 32 == 0 else 0)

        def run(x, res, off):
            y = patterned(c.R, width, dtype=BF)
            ck = (patterned(c.R, width, dtype=torch.uint8),
                  patterned(c.R, wide, dtype=torch.uint8)) if wide else None
            m.grouped_linear(c.p, x, c.w, off, bias=c.bias, act="silu", residual=res,
                             checkpoint=ck, out=y)
            return (y, *(ck or ()))

        outs = run(c.x, c.residual, c.offsets), run(moved(c.x), moved(c.residual), off)
    elif p.mode == DX:
        ck = c.checkpoint(p.K)

        def run(dz, ck, off):
            dx, a = patterned(c.R, p.K, dtype=BF), patterned(c.R, p.K, dtype=BF)
            m.grouped_linear_dx(c.p, dz, c.w, off, act="gelu_tanh", checkpoint=ck, out=dx, a=a)
            return dx, a

        outs = run(c.dz, ck, c.offsets), run(moved(c.dz), tuple(map(moved, ck)), off)
    else:
        got = [m.grouped_linear_dw(c.p, x, dz, o, want_bias=True)
               for x, dz, o in ((c.x, c.dz, c.offsets), (moved(c.x), moved(c.dz), off))]
        for a, b in zip(*got):
            assert torch.equal(a, b)
        return
    for a, b in zip(*outs):
        compare(a, b)


def test_the_most_experts():
    counts = [(5 * i) % 7 % 4 for i in range(1024)]
    c = Case(counts, 64, 96, extra=3, seed=5)
    check_linear(c, "silu", bias=True, ckpt=True)
    check_dx(c, "silu", ckpt=True)
    check_dw(c, bias=True)
    c = Case([130 if i % 97 == 3 else 0 for i in range(1024)], 72, 64, extra=3, tokens=50, seed=6)
    check_linear(c, "relu", bias=True)
    check_dw(c, bias=True)


def test_captured_graphs_that_share_a_workspace():
    """Two graphs of split calls with one workspace, replayed in turn with eager calls on the
    same workspace between them."""
    m = moe()
    p = m.GroupedProblem(R=16, K=4104, N=512)
    q = m.GroupedProblem(R=16, K=512, N=4104)
    n = max(p.workspace_bytes(m.OP_GROUPED_LINEAR), q.workspace_bytes(m.OP_GROUPED_DX))
    assert p.workspace_bytes(m.OP_GROUPED_LINEAR) and q.workspace_bytes(m.OP_GROUPED_DX)
    ws = patterned(n, dtype=torch.uint8)
    g = torch.Generator(device=DEV)
    g.manual_seed(7)
    x, w1, w2 = rand(g, 16, 4104), rand(g, 1, 4104, 512), rand(g, 1, 512, 4104)
    y, dx = torch.empty(16, 512, dtype=BF, device=DEV), torch.empty(16, 512, dtype=BF, device=DEV)

    def lin(out):
        m.grouped_linear(p, x, w1, act="silu", out=out, ws=ws)

    def back(out):
        m.grouped_linear_dx(q, x, w2, out=out, ws=ws)

    s = torch.cuda.Stream()
    graphs = []
    for f, out in ((lin, y), (back, dx)):
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            f(out)
        s.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=s):
            f(out)
    for i in range(4):
        x.copy_(rand(g, 16, 4104))
        for graph in (graphs if i % 2 else reversed(graphs)):
            graph.replay()
        ey, ed = torch.empty_like(y), torch.empty_like(dx)
        lin(ey)
        back(ed)
        torch.cuda.synchronize()
        assert torch.equal(y, ey) and torch.equal(dx, ed), f"replay {i}"
