"""The fp64 definitions of the grouped linear products (oracle/grouped.py): the activations
against their textbook forms, the gradients against central differences, the checkpoint
against a search over the E4M3 values."""
import math

import pytest
import torch

from oracle import grouped as og

ACTS = ["none", "relu", "relu2", "silu", "gelu_tanh"]


def gen(seed):
    return torch.Generator().manual_seed(seed)


@pytest.mark.parametrize("name", ACTS)
def test_activation_and_derivative(name):
    z = torch.randn(400, generator=gen(1), dtype=torch.float64) * 3
    f, df = og.act(z, name)
    ref = {"none": z, "relu": torch.relu(z), "relu2": torch.relu(z) ** 2,
           "silu": torch.nn.functional.silu(z),
           "gelu_tanh": torch.nn.functional.gelu(z, approximate="tanh")}[name]
    assert torch.allclose(f, ref, rtol=1e-13, atol=1e-15)
    h = 1e-6
    diff = (og.act(z + h, name)[0] - og.act(z - h, name)[0]) / (2 * h)
    # a central difference is off by h^2 |f'''| / 6 (below 1e-11 here), by the rounding of its
    # two values, 2 * 2^-53 |f| / (2 h), and next to relu2's jump of f'' by at most h
    assert ((diff - df).abs() <= 1e-11 + 2.0 ** -52 * (f.abs() + 1) / h + h).all()


@pytest.mark.parametrize("name", ACTS)
def test_gradients_against_differences(name):
    g = gen(2)
    E, K, N, T = 3, 6, 64, 5
    offsets = torch.tensor([0, 4, 4, 7])
    segs = og.segments(offsets, 7, E)
    row_token = torch.tensor([0, 2, 3, 4, 1, 2, 2])
    x = torch.randn(T, K, generator=g, dtype=torch.float64)
    w = torch.randn(E, K, N, generator=g, dtype=torch.float64)
    b = torch.randn(E, N, generator=g, dtype=torch.float64)
    c = torch.randn(7, N, generator=g, dtype=torch.float64)  # loss = sum(c * y)

    def loss(x, w, b):
        z, _ = og.linear(x, w, segs, b, row_token)
        return (c * og.act(z, name)[0]).sum()

    z, _ = og.linear(x, w, segs, b, row_token)
    dz = c * og.act(z, name)[1]
    dw, db, _, _ = og.dw(x, dz, segs, row_token)
    drow, _ = og.dx(dz, w, segs)
    dx = torch.zeros_like(x).index_add_(0, row_token, drow)
    h = 1e-6
    for t, grad in ((x, dx), (w, dw), (b, db)):
        d = torch.randn(t.shape, generator=g, dtype=torch.float64)
        args = {id(x): x, id(w): w, id(b): b}
        up = [v + h * d if v is t else v for v in args.values()]
        dn = [v - h * d if v is t else v for v in args.values()]
        diff = (loss(*up) - loss(*dn)) / (2 * h)
        assert abs(diff - (grad * d).sum()) <= 1e-6 * (1 + abs(diff))
    assert dw[1].abs().max() == 0 and db[1].abs().max() == 0  # an expert without rows


def test_checkpoint_is_the_nearest_value():
    vals = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).to(torch.float64)
    z = torch.randn(6, 64, generator=gen(3), dtype=torch.float64) * torch.tensor(
        [[1e-3], [1.0], [40.0], [448.0], [0.0], [1e-30]])
    z[3, 0], z[3, 40] = 448.0, 449.0
    q, s = og.quantize(z)
    for r in range(6):
        for blk in range(2):
            v = z[r, 32 * blk:32 * blk + 32]
            sc = float(s[r, blk])
            top = float(v.abs().max())
            if top == 0:
                assert sc == 1.0
            else:
                assert top <= 448 * sc and top > 448 * sc / 2 and math.log2(sc) % 1 == 0
            near = (v.abs()[:, None] / sc - vals[None]).abs().min(1).values * sc
            assert torch.allclose((q[r, 32 * blk:32 * blk + 32] - v).abs(), near, rtol=1e-12,
                                  atol=0)
    z = torch.ones(1, 32, dtype=torch.float64)
    z[0, 5], z[0, 6] = float("inf"), float("nan")
    q, s = og.quantize(z)
    assert torch.isnan(q[0, 5:7]).all() and torch.isfinite(q[0, 7:]).all() and s[0, 0] == 2.0 ** -8
