"""The grouped operators at the sizes where a single launch or a 32-bit count would end."""
import pytest
import torch

from grouped_common import act_tol, dact_tol, moe, stored
from oracle import grouped as og
from test_gpu_grouped import BF, DEV, F64, gen, patterned, rand, say, untouched, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("log_values,with_a", [(32, True), (35, False)])
def test_activation_backward_beyond_one_launch(log_values, with_a):
    """More values than a launch has threads for (2^32 threads of 8 values): inputs that repeat
    every 1021 rows, so that the first rows, held to their definition, say what all others
    have to be, bit for bit."""
    cols, period, behind = 4128, 1021, 5
    rows = (1 << log_values) // cols + 2 * period
    need = rows * cols * (5 + (2 if with_a else 0)) * 1.06
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < need:
        pytest.skip(f"needs {need / 2 ** 30:.0f} GiB of device memory")
    say(f"case {rows} x {cols}")
    m, g = moe(), gen(log_values)
    dy = rand(g, period, cols)
    v, s = og.quantize(torch.randn(period, cols, generator=g, device=DEV, dtype=F64) * 3)
    codes = (v / s.repeat_interleave(32, 1)).float().to(torch.float8_e4m3fn).view(torch.uint8)
    scales = (torch.log2(s) + 127).to(torch.uint8)

    def repeated(block):
        t = torch.empty(rows, block.shape[1], dtype=block.dtype, device=DEV)
        n = rows // period * period
        t[:n].view(-1, period, block.shape[1])[:] = block
        t[n:] = block[:rows - n]
        return t

    live = rows - behind
    out = torch.empty(rows, cols, dtype=BF, device=DEV)
    a = torch.empty(rows, cols, dtype=BF, device=DEV) if with_a else None
    outs = [t for t in (out, a) if t is not None]
    tail = patterned(behind, cols, dtype=BF)
    for t in outs:
        t[live:] = tail
    m.activation_backward(repeated(dy), (repeated(codes), repeated(scales)), "silu", out=out, a=a,
                          live_rows=torch.tensor([live], dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    z = og.dequantize(codes, scales)
    f, df = og.act(z, "silu")
    d = dy.to(F64)
    within("dz", out[:period], d * df,
           stored(d * df, d.abs() * (dact_tol(z, df, "silu") + 2.0 ** -23 * df.abs())))
    if with_a:
        within("a", a[:period], f, stored(f, act_tol(z, f, 0 * z, "silu")))
    for t in outs:
        assert untouched(t[live:])
        first = t[:period].clone()
        whole = t[:live // period * period].view(-1, period, cols)
        for i in range(0, whole.shape[0], 128):
            assert bool((whole[i:i + 128] == first).all()), i
        rest = live % period
        assert torch.equal(t[live - rest:live], first[:rest])
