"""The grouped product on 4-bit weights at the ends of its range: blocks whose scales are far apart,
what the matrix cores drop of 8-bit codes, and outputs past 4 GB."""
import pytest
import torch

from fp4_common import DEV, Case, gen
from grouped_common import BF16_HALF, sum_tol
from oracle import fp4

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("x", ["fp4", "fp8"])
@pytest.mark.parametrize("spread", [12, 20, 40])
@pytest.mark.parametrize("counts,K,N", [([40], 64, 64), ([9, 0, 11], 480, 72), ([300, 0, 80], 1120, 264),
                                        ([33], 7200, 520), ([700], 4096, 16400)])
def test_blocks_with_scales_far_apart(counts, K, N, spread, x):
    """Neighbouring blocks' products differ by up to 2^(2 spread): each block keeps its own bits."""
    case = Case(counts, K, N, x=x, seed=spread)
    g = gen(spread)
    for q in (case.xq, case.w):
        q[1].copy_(torch.randint(127 - spread, 127, q[1].shape, generator=g, device=DEV,
                                 dtype=torch.uint8))
    case.check(case.run())


def dropped(x, w):
    """The most that the products of x and w's rows lose where what lies more than 13 bits below
    (the power of two in) a block's largest product is dropped.  A product of E4M3 and E2M1 values
    has 6 bits, so that one of 64 times the last bit kept, or more, loses nothing."""
    loss = torch.zeros(x.shape[0], w.shape[0], dtype=torch.float64, device=x.device)
    for n in range(w.shape[0]):
        p = (x * w[n]).abs().reshape(x.shape[0], -1, 32)
        top = p.amax(-1, keepdim=True)
        last = torch.exp2(torch.floor(torch.log2(top.clamp(min=2.0 ** -300))) - 13)
        lost = torch.where(p < 64 * last, torch.minimum(p, last), torch.zeros_like(p))
        loss[:, n] = lost.sum((-1, -2))
    return loss


@pytest.mark.parametrize("counts,K,N,seed", [([64], 32, 64, 1), ([3], 32, 64, 2), ([300], 64, 136, 3),
                                             ([40], 96, 64, 4), ([64], 256, 64, 5)])
def test_eight_bit_products_keep_13_bits(counts, K, N, seed):
    """Quantized normal values: the residual takes away the rounded product, so that what is stored
    shows the sum's own error."""
    case = Case(counts, K, N, x="fp8 wide", residual=True, seed=seed)
    x, w = fp4.dequantize8(*case.xq), fp4.dequantize(case.w[0][0], case.w[1][0])
    z, size = x @ w.t(), x.abs() @ w.abs().t()
    case.residual.copy_((-z).to(torch.bfloat16))
    rest = z + case.residual.double()
    err = (case.run().double() - rest).abs()
    tol = sum_tol(K, size) + dropped(x, w)
    tol = tol + BF16_HALF * (rest.abs() + tol)
    print(f"  worst error/tolerance {float((err / tol).max()):.3f}", flush=True)
    assert bool((err <= tol).all())


@pytest.mark.parametrize("x", ["fp4", "fp8"])
def test_outputs_and_residuals_behind_4_gb(x):
    case = Case([300, 0, 41], 96, 2056, x=x, bias=True, residual=True, front=1050000, behind=5,
                act="silu", seed=3)
    assert case.R * case.N * 2 > 1 << 32
    case.check(case.run())


@pytest.mark.parametrize("x,T", [("fp4", 600000), ("fp8", 300000)])
@pytest.mark.parametrize("counts", [[70, 30], [3, 1], [300, 0, 200]])
def test_gathered_rows_behind_4_gb(counts, x, T):
    case = Case(counts, 16384, 72, x=x, gather=True, wild=True, T=T, gated=True, act="silu")
    assert case.xq[0].numel() > 1 << 32
    assert int(case.row_token[case.lo:case.hi].clamp(max=T - 1).max()) > T - T // 8
    case.check(case.run())
