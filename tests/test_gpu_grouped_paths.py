"""Paths through the grouped kernels that the layouts of test_gpu_grouped.py do not take."""
import pytest

from grouped_paths import DW, DX, LINEAR, PATHS
from test_gpu_grouped import Case, check_dw, check_dx, check_linear, say

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
