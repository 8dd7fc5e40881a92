"""The 4-bit values bit for bit, and the grouped product on them element by element, against the
fp64 definitions (oracle/fp4.py); tolerances as in tests/grouped_common.py."""
import pytest
import torch

from fp4_common import DEV, PATTERN, Case, codes4, gen, moe
from fp4_paths import PATHS
from oracle import fp4

pytestmark = pytest.mark.gpu


def patterned(*shape, dtype=torch.uint8):
    n = torch.empty(0, dtype=dtype).element_size()
    for s in shape:
        n *= s
    return torch.full((n,), PATTERN, dtype=torch.uint8, device=DEV).view(dtype).view(shape)


def every_bf16():
    """Blocks that hold every bf16 value next to maxima from far below to far above it."""
    v = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    v = v[torch.isfinite(v.float())]
    v = v[: v.numel() // 30 * 30].reshape(-1, 30)  # neighbours share a block
    tops = [0.0, 1.0, 6.0, 6.03125, 2.0 ** -120, 3.0e38]
    out = []
    for t in tops:
        b = torch.zeros(v.shape[0], 32, dtype=torch.bfloat16)
        b[:, 1:31] = v
        b[:, 0] = t
        out.append(b)
    return torch.cat(out)


def same4(x, codes, scales):
    want = fp4.quantize(x)
    assert torch.equal(scales.cpu(), want[1])
    assert torch.equal(codes.cpu(), want[0])


def test_quantize_every_value():
    x = every_bf16()
    same4(x, *moe().quantize_fp4(x.cuda()))


@pytest.mark.parametrize("rows,cols", [(1, 32), (1, 7168), (3, 96), (37, 1440), (130, 2048),
                                       (1025, 160)])
def test_quantize_rows(rows, cols):
    g = torch.Generator().manual_seed(rows)
    x = (torch.randn(rows, cols, generator=g)
         * torch.exp2(torch.randint(-140, 60, (rows, 1), generator=g).float())).bfloat16()
    x[0, :32] = 0
    x[rows // 2, 5] = float("inf")
    x[rows - 1, cols - 1] = float("nan")
    m = moe()
    codes, scales = m.quantize_fp4(x.cuda())
    same4(x, codes, scales)
    back = m.dequantize_fp4(codes, scales).cpu()
    want = fp4.dequantize(*fp4.quantize(x))
    nan = want.isnan()
    assert torch.equal(back.isnan(), nan) and nan[rows - 1, cols - 1]
    assert torch.equal(back.double()[~nan], want[~nan])
    # three dimensions, and rows behind live_rows
    live = rows // 3
    out = (patterned(rows, cols // 2), patterned(rows, cols // 32))
    n = torch.tensor([live], dtype=torch.int32, device=DEV)
    m.quantize_fp4(x.cuda(), live_rows=n, out=out)
    for o, w in zip(out, (codes, scales)):
        assert torch.equal(o[:live], w[:live]) and bool((o[live:] == PATTERN).all())
    v = patterned(rows, cols, dtype=torch.bfloat16)
    m.dequantize_fp4(codes, scales, live_rows=n, out=v)
    assert torch.equal(v[:live].cpu().view(torch.int16), back[:live].view(torch.int16))
    assert bool((v[live:].contiguous().view(torch.uint8) == PATTERN).all())
    c3, s3 = m.quantize_fp4(x.cuda()[None])
    assert c3.shape == (1, rows, cols // 2) and torch.equal(c3[0], codes) and torch.equal(
        s3[0], scales)


def test_dequantize_every_byte():
    codes = torch.arange(256, dtype=torch.uint8).repeat(256, 1)  # 256 scales x 16 blocks
    scales = torch.arange(256, dtype=torch.uint8)[:, None].repeat(1, 16)
    got = moe().dequantize_fp4(codes.cuda(), scales.cuda()).cpu().float()
    want = fp4.dequantize(codes, scales).float()  # 2^128 and more: inf
    assert torch.equal(got.isnan(), want.isnan())
    assert torch.equal(torch.nan_to_num(got, nan=7.0), torch.nan_to_num(want, nan=7.0))


def test_live_rows_out_of_range():
    x = torch.randn(5, 64, device=DEV).bfloat16()
    m = moe()
    for n, live in ((-3, 0), (0, 0), (5, 5), (900, 5)):
        out = (patterned(5, 32), patterned(5, 2))
        m.quantize_fp4(x, live_rows=torch.tensor([n], dtype=torch.int32, device=DEV), out=out)
        want = m.quantize_fp4(x)
        assert torch.equal(out[0][:live], want[0][:live])
        assert bool((out[0][live:] == PATTERN).all()) and bool((out[1][live:] == PATTERN).all())


@pytest.mark.parametrize("E,K,N", [(1, 32, 8), (3, 96, 40), (2, 256, 128), (5, 1440, 136),
                                   (2, 2048, 768), (1, 288, 1000)])
def test_quantize_weights(E, K, N):
    g = torch.Generator().manual_seed(K)
    w = (torch.randn(E, K, N, generator=g) * K ** -0.5).bfloat16()
    w[0, 3, 1] = float("inf")
    w[E - 1, :32, N - 1] = 0
    m = moe()
    codes, scales = m.quantize_fp4_weights(w.cuda())
    want = fp4.quantize(w.transpose(1, 2).contiguous())
    assert torch.equal(codes.cpu(), want[0]) and torch.equal(scales.cpu(), want[1])
    rows = m.quantize_fp4(w.transpose(1, 2).contiguous().cuda())
    assert torch.equal(rows[0], codes) and torch.equal(rows[1], scales)


BIG = [300, 0, 1, 77, 513, 32]
CASES = [
    dict(counts=[1], K=32, N=8),
    dict(counts=[1], K=32, N=8, x="fp8"),
    dict(counts=[5], K=256, N=64),
    dict(counts=[5], K=256, N=64, x="fp8"),
    dict(counts=[33], K=1440, N=136, act="gelu_tanh", bias=True, residual=True),
    dict(counts=[33], K=1440, N=136, act="gelu_tanh", bias=True, residual=True, x="fp8"),
    dict(counts=[2, 0, 31, 1, 64, 0], K=288, N=72, behind=9, act="relu2", bias=True),
    dict(counts=[2, 0, 31, 1, 64, 0], K=288, N=72, behind=9, front=4, gather=True, wild=True,
         gated=True, act="silu", bias=True, residual=True),
    dict(counts=[2, 0, 31, 1, 64, 0], K=288, N=72, behind=9, front=4, gather=True, wild=True,
         gated=True, act="silu", bias=True, residual=True, x="fp8"),
    dict(counts=[0, 0, 0], K=64, N=16, behind=5),
    dict(counts=[1] * 8 + [0] * 120, K=2048, N=768, gather=True, T=1, gated=True, act="silu"),
    dict(counts=[3, 5, 0, 4] * 8, K=1024, N=384, gather=True, T=16, gated=True, act="silu",
         x="fp8"),
    dict(counts=[200], K=512, N=520, gated=True, act="relu"),
    dict(counts=[257], K=544, N=264, act="silu"),
    dict(counts=[700], K=800, N=328, x="fp8", residual=True),
    dict(counts=[1003], K=1440, N=2056, act="gelu_tanh", bias=True, residual=True),
    dict(counts=[1003], K=1440, N=2056, act="gelu_tanh", bias=True, residual=True, x="fp8"),
    dict(counts=BIG, K=736, N=648, behind=40, front=3, bias=True),
    dict(counts=BIG, K=736, N=648, behind=40, gather=True, wild=True, x="fp8", residual=True),
    dict(counts=BIG, K=2048, N=776, gather=True, T=128, gated=True, act="silu", bias=True,
         residual=True, behind=10),
    dict(counts=BIG, K=2048, N=776, gather=True, T=128, gated=True, act="silu", bias=True,
         residual=True, behind=10, x="fp8"),
    dict(counts=[40, 700, 3], K=512, N=256, x="fp8 wide"),
    dict(counts=[2100], K=256, N=4096),
    dict(counts=[1500, 900, 1200, 0, 600], K=1024, N=1536, gated=True, act="silu"),
    dict(counts=[1500, 900, 1200, 0, 600], K=1024, N=1536, x="fp8"),
]


@pytest.mark.parametrize("c", CASES, ids=str)
def test_grouped_linear_fp4(c):
    case = Case(**c)
    y = case.run()
    case.check(y)
    again = case.run()
    assert torch.equal(y.view(torch.int16), again.view(torch.int16))  # no order of its own


@pytest.mark.parametrize("x", ["fp4", "fp8"])
@pytest.mark.parametrize("i", range(len(PATHS)))
def test_every_kernel(i, x):
    case = Case(**PATHS[i][2], x=x, seed=i + 20)
    y = case.run()
    case.check(y)
    assert torch.equal(y.view(torch.int16), case.run().view(torch.int16))


@pytest.mark.parametrize("kw", [dict(counts=[300], K=864, N=136), dict(counts=[3], K=864, N=136),
                                dict(counts=[300, 0, 80], K=1120, N=264, gather=True, x="fp8")],
                         ids=str)
def test_scales_need_no_alignment(kw):
    case = Case(**kw, shift=True)
    assert case.w[1].data_ptr() % 2 == 1 and case.xq[1].data_ptr() % 2 == 1
    case.check(case.run())


@pytest.mark.parametrize("counts", [[70, 30], [9, 4]])
def test_rows_and_weights_behind_4_gb(counts):
    case = Case(counts, 16384, 72, front=600000)  # 4.9 GB of x
    assert case.xq[0].numel() > 1 << 32
    case.check(case.run())
    del case
    torch.cuda.empty_cache()
    case = Case([0] * 1022 + counts, 8224, 1048, act="silu")  # 4.4 GB of weights
    assert case.w[0].numel() > 1 << 32
    case.check(case.run())


def test_more_values_than_one_launch_takes():
    m = moe()
    cols, rows = 8192, (1 << 19) + 40  # 2^32 values and 40 rows more
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device=DEV)
    x[-50:] = torch.randn(50, cols, device=DEV).bfloat16()
    codes, scales = m.quantize_fp4(x)
    want = m.quantize_fp4(x[-50:].contiguous())
    assert torch.equal(codes[-50:], want[0]) and torch.equal(scales[-50:], want[1])
    x.fill_(1.0)
    m.dequantize_fp4(codes, scales, out=x)
    assert torch.equal(x[-50:], m.dequantize_fp4(*want)) and not x[:-50].any()


def test_two_calls_at_once_on_two_streams():
    cases = [Case([90, 0, 37, 130], 5600, 264, x=x, gated=True, act="silu", gather=True, seed=s)
             for s, x in ((3, "fp4"), (4, "fp8"))]
    ys = [c.new_y() for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for c, y, s in zip(cases, ys, streams):
            with torch.cuda.stream(s):
                c.run(y)
    torch.cuda.synchronize()
    for c, y in zip(cases, ys):
        c.check(y)


def test_two_graphs_that_share_a_workspace():
    m = moe()
    cases = [Case([90, 0, 37, 130], 5600, 264, seed=s, bias=True) for s in (5, 6)]
    ws = m.grouped_workspace(cases[0].p, m.OP_GROUPED_FP4)
    assert ws is not None
    ys = [c.new_y() for c in cases]
    graphs = []
    for c, y in zip(cases, ys):
        c.run(y, ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run(y, ws)
        graphs.append(g)
    for _ in range(3):
        for y in ys:
            y.view(torch.uint8).fill_(PATTERN)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for c, y in zip(cases, ys):
            c.check(y)


def test_debug_library_reports_bad_offsets_and_tokens():
    import ctypes
    m = moe()
    c = Case([40, 30, 20], 128, 64, gather=True)
    d = m.debug_lib()
    m.debug_status()

    def call():
        y = c.new_y()
        w = m.MoeFp4Weights(c.w[0].data_ptr(), c.w[1].data_ptr(), None)
        ptr = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
        st = d.moe_grouped_linear_fp4(c.p._ref, m.MOE_FP4, ptr(c.xq[0]), ptr(c.xq[1]),
                                      ptr(c.row_token), ptr(c.offsets), ctypes.byref(w), None, 0,
                                      None, ptr(y), None, 0, m._stream())
        assert st == m.MOE_OK
        return y

    c.check(call())
    assert m.debug_status() == 0
    c.offsets[3] = 4000
    c.row_token[5] = -7
    call()
    assert m.debug_status() == 12


def test_nan_scales_and_codes_poison_their_sums_only():
    c = Case([40], 512, 64, x="fp8")
    c.xq[1][3, 7] = 255
    c.xq[0][9, 100] = 0x7F
    c.w[1][0, 20, 2] = 255
    y = c.run()
    nan = torch.zeros(40, 64, dtype=torch.bool, device=DEV)
    nan[3] = nan[9] = True
    nan[:, 20] = True
    assert torch.equal(y.isnan(), nan)
    c = Case([400], 512, 320)
    c.xq[1][399, 15] = 255
    c.w[1][0, 319, 0] = 255
    y = c.run()
    nan = torch.zeros(400, 320, dtype=torch.bool, device=DEV)
    nan[399] = True
    nan[:, 319] = True
    assert torch.equal(y.isnan(), nan)


def test_offsets_out_of_range_stay_inside():
    c = Case([40, 30, 20], 128, 64)
    c.offsets = torch.tensor([-5, 40, 70, 4000], dtype=torch.int32, device=DEV)
    c.segs = [(0, 40), (40, 70), (70, 90)]
    c.check(c.run())


def test_the_layer_from_its_parts():
    """route_scored -> dispatch -> quantize -> gate/up -> quantize -> down -> combine, against the
    same chain in fp64 on the same codes."""
    from oracle import grouped as og
    m = moe()
    T, H, E, k, I = 200, 512, 16, 4, 256
    g = gen(4)
    x = torch.randn(T, H, generator=g, device=DEV).bfloat16()
    wg, wu = ((torch.randn(E, H, I, generator=g, device=DEV) * H ** -0.5).bfloat16()
              for _ in range(2))
    wd = (torch.randn(E, I, H, generator=g, device=DEV) * I ** -0.5).bfloat16()
    logits = torch.randn(T, E, generator=g, device=DEV)
    bias = 0.1 * torch.randn(E, generator=g, device=DEV)
    p = m.Problem(T=T, H=H, E=E, k=k, I=I, capacity=60)
    sc = m.Scoring("sigmoid", 4, 2, "top2", 2.5)
    ids, tw, keep = m.route_scored(p, logits, sc, bias=bias)
    d = m.dispatch(p, x, ids, keep, rows=False)
    offsets, row_token, slot_to_row = d["offsets"], d["row_token"], d["slot_to_row"]
    q = {n: m.quantize_fp4_weights(w) for n, w in (("g", wg), ("u", wu), ("d", wd))}
    p1 = m.GroupedProblem(R=T * k, K=H, N=I, E=E, T=T)
    p2 = m.GroupedProblem(R=T * k, K=I, N=H, E=E)
    for quant in (m.quantize_fp4, m.quantize_fp8):
        xq = quant(x)
        a = m.grouped_linear_fp4(p1, xq, q["g"], offsets, up=q["u"], act="silu",
                                 row_token=row_token, out=torch.zeros(T * k, I, device=DEV,
                                                                      dtype=torch.bfloat16))
        aq = quant(a)
        yp = m.grouped_linear_fp4(p2, aq, q["d"], offsets)
        y = m.combine(p, yp, tw, slot_to_row)
        deq = fp4.dequantize if quant is m.quantize_fp4 else fp4.dequantize8
        segs = og.segments(offsets, T * k, E)
        n = segs[-1][1]
        xs = deq(*xq)[row_token[:n].long()]
        z, _ = fp4.linear(xs, fp4.dequantize(*q["g"]), segs)
        u, _ = fp4.linear(xs, fp4.dequantize(*q["u"]), segs)
        want = z * torch.sigmoid(z) * u
        assert ((a[:n].double() - want).norm() / want.norm()) < 2.0 ** -8
        v, _ = fp4.linear(deq(*aq)[:n], fp4.dequantize(*q["d"]), segs)
        rows = torch.cat((v, torch.zeros(1, H, device=DEV, dtype=torch.float64)))
        s2r = slot_to_row.long()
        s2r = torch.where(s2r < 0, torch.full_like(s2r, n), s2r)
        want = (rows[s2r] * tw.double()[..., None]).sum(1)
        assert ((y.double() - want).norm() / want.norm()) < 2.0 ** -7


def test_capture_replays_on_new_inputs_and_other_streams():
    c = Case([60, 0, 200, 9], 768, 392, gather=True, gated=True, act="silu", bias=True)
    y = c.new_y()
    ws = c.m.grouped_workspace(c.p, c.m.OP_GROUPED_FP4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.run(y, ws)
    torch.cuda.current_stream().wait_stream(side)
    c.check(y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(y, ws)
    for seed in (1, 2, 3):
        g = gen(seed)
        c.xq[0].copy_(torch.randint(0, 256, c.xq[0].shape, generator=g, device=DEV,
                                    dtype=torch.uint8))
        y.view(torch.uint8).fill_(PATTERN)
        graph.replay()
        torch.cuda.synchronize()
        c.check(y)
