"""Routing by scores on the GPU against the fp64 definition: ids and keep flags equal, weights
rounded once, the gradient within its roundings."""
import numpy as np
import pytest
import torch

from oracle import scored
from scored_common import INF, bias as make_bias, logits as make_logits, numpy_of

pytestmark = pytest.mark.gpu


def moe():
    import expert_ffn_moe_amd

    return expert_ffn_moe_amd


# T, E, k, score, groups, taken, group score, bias, renorm, scale, capacity, logits
CASES = [
    (1, 256, 8, "sigmoid", 8, 4, "top2", "normal", True, 2.5, 0, "normal"),
    (1, 1, 1, "sigmoid", 1, 1, "max", None, True, 1.0, 0, "normal"),
    (1, 1, 1, "softmax", 1, 1, "max", "normal", False, 1.0, 0, "normal"),
    (67, 256, 8, "sigmoid", 8, 4, "top2", "ties", True, 2.5, 0, "ties"),
    (67, 256, 8, "softmax", 8, 3, "max", None, False, 1.0, 0, "ties"),
    (33, 64, 6, "softmax", 1, 1, "max", None, True, 1.0, 0, "ties"),
    (33, 64, 6, "softmax", 4, 2, "top2", None, True, 1.0, 0, "normal"),
    (50, 72, 4, "sigmoid", 8, 2, "top2", None, False, 1.5, 0, "normal"),
    (50, 72, 4, "softmax", 8, 5, "top2", "out", False, 1.0, 0, "masked"),
    (41, 160, 6, "softmax", 8, 3, "max", "normal", True, 16.0, 0, "masked"),
    (41, 160, 6, "sigmoid", 1, 1, "max", "out", True, 1.0, 7, "masked"),
    (19, 128, 32, "sigmoid", 1, 1, "max", "ties", True, 1.0, 0, "wide"),
    (19, 128, 8, "sigmoid", 16, 4, "top2", "normal", True, 1.0, 0, "wide"),
    (19, 128, 8, "softmax", 1, 1, "max", None, False, 1.0, 0, "wide"),
    (23, 64, 2, "sigmoid", 64, 5, "top2", "normal", True, 1.0, 0, "masked"),  # groups of one
    (23, 100, 3, "sigmoid", 50, 7, "top2", None, True, 1.0, 0, "ties"),
    (13, 384, 8, "sigmoid", 1, 1, "max", "normal", True, 2.5, 0, "normal"),
    (13, 512, 8, "sigmoid", 8, 4, "top2", "normal", True, 2.5, 0, "ties"),
    (9, 1000, 10, "softmax", 10, 3, "top2", "normal", False, 1.0, 0, "masked"),
    (9, 1024, 32, "sigmoid", 64, 9, "top2", "out", True, 1.0, 0, "normal"),
    (300, 48, 4, "softmax", 1, 1, "max", "normal", True, 1.0, 11, "ties"),
    (300, 48, 4, "sigmoid", 4, 2, "top2", None, False, 2.5, 20, "normal"),
    (65, 37, 5, "sigmoid", 1, 1, "max", "normal", True, 1.0, 0, "normal"),  # rows of odd length
    (65, 90, 8, "softmax", 3, 2, "top2", "normal", True, 1.0, 0, "ties"),
    (33, 250, 8, "sigmoid", 5, 2, "top2", "out", False, 1.0, 0, "masked"),
    (47, 256, 8, "sigmoid", 1, 1, "max", "same", True, 1.0, 0, "lane"),  # one lane's experts lead
    (47, 256, 7, "sigmoid", 1, 1, "max", None, True, 1.0, 0, "lane"),
    (5000, 128, 8, "softmax", 1, 1, "max", "normal", True, 1.0, 0, "close"),
    (5000, 256, 8, "sigmoid", 8, 4, "top2", "normal", True, 2.5, 0, "close"),
    (3001, 64, 8, "sigmoid", 8, 4, "max", "close", False, 2.5, 0, "close"),
]


def setup(c, seed=5):
    T, E, k, kind, G, taken, gs, b, renorm, scale, cap, lk = c
    m = moe()
    p = m.Problem(T=T, H=64, E=E, k=k, I=64, capacity=cap, renormalize=int(renorm))
    sc = m.Scoring(kind, G, taken, gs, scale)
    x, bias = make_logits(T, E, seed, lk), make_bias(E, seed, b)
    want = scored.route(numpy_of(x), k, kind, capacity=cap, bias=numpy_of(bias), n_group=G,
                        topk_group=taken, group_score=gs, renorm=renorm, scale=scale)
    return m, p, sc, x, bias, want


@pytest.mark.parametrize("c", CASES, ids=str)
def test_route_scored(c):
    m, p, sc, x, bias, (ids, w, keep) = setup(c)
    got = m.route_scored(p, x.cuda(), sc, bias=None if bias is None else bias.cuda())
    assert not (got[0].cpu().numpy() != ids).any()
    assert not (got[2].cpu().numpy() != keep).any()
    # a weight is an fp64 value (off by a few 2^-53) rounded to f32: half a step, 2^-24, of itself
    # from the other's where the two lie on different sides of a border: a whole step
    err = np.abs(got[1].cpu().numpy().astype(np.float64) - w)
    assert (err <= 2.0 ** -23 * np.abs(w) + 2.0 ** -149).all()


@pytest.mark.parametrize("c", CASES, ids=str)
def test_backward(c):
    m, p, sc, x, bias, (ids, w, keep) = setup(c)
    dw = torch.randn(p.T, p.k, generator=torch.Generator().manual_seed(9))
    dw[torch.from_numpy(keep) == 0] = 0
    dw[torch.from_numpy(w) == 0] = float("nan")  # slots without a weight are not read
    want, size = scored.backward(numpy_of(x), ids, w, numpy_of(dw), sc.score, bool(p.renormalize),
                                 sc.scale)
    got = m.route_scored_backward(p, x.cuda(), sc, torch.from_numpy(ids).cuda(),
                                  torch.from_numpy(w).cuda(), dw.cuda()).cpu().double().numpy()
    # the weights were rounded to f32 (2^-24 of themselves each, which moves every term by as
    # much, and a mean of terms by twice that), the result once more (2^-24); a weight below the
    # normal range is off by 2^-150
    g = np.nan_to_num(np.abs(dw.numpy())).sum(1, keepdims=True)
    tol = 4 * 2.0 ** -24 * size + 2.0 ** -24 * np.abs(want) + 2.0 ** -149 * (1 + 4 * g)
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= tol).all()
    assert (got[~(numpy_of(x) > -INF)] == 0).all()


def test_router_scored_selects_from_its_own_logits():
    m = moe()
    T, H, E, k = 300, 192, 96, 6
    g = torch.Generator().manual_seed(1)
    x = torch.randn(T, H, generator=g).bfloat16()
    wr = (torch.randn(E, H, generator=g) * H ** -0.5).bfloat16()
    b = make_bias(E, 4)
    for cap in (0, 15):
        p = m.Problem(T=T, H=H, E=E, k=k, I=64, capacity=cap)
        sc = m.Scoring("sigmoid", 8, 3, "top2", 2.5)
        ids, w, keep, lg = m.router_scored(p, x.cuda(), wr.cuda(), sc, bias=b.cuda(),
                                           want_logits=True)
        ref = x.double() @ wr.double().t()
        size = x.double().abs() @ wr.double().abs().t()
        assert ((lg.cpu().double() - ref).abs() <= 2 * H * 2.0 ** -24 * size).all()
        want = scored.route(lg.cpu().numpy(), k, "sigmoid", capacity=cap, bias=numpy_of(b),
                            n_group=8, topk_group=3, group_score="top2", scale=2.5)
        assert np.array_equal(ids.cpu().numpy(), want[0])
        assert np.array_equal(keep.cpu().numpy(), want[2])
        same = m.route_scored(p, lg, sc, bias=b.cuda())
        assert all(torch.equal(a, q) for a, q in zip((ids, w, keep), same))
        none = m.router_scored(p, x.cuda(), wr.cuda(), sc, bias=b.cuda())
        assert none[3] is None and torch.equal(none[0], ids)


def test_softmax_without_bias_is_route_grouped():
    m = moe()
    T, E, k = 500, 128, 8
    x = make_logits(T, E, 8, "ties").cuda()
    p = m.Problem(T=T, H=64, E=E, k=k, I=64, capacity=40)
    a = m.route_grouped(p, x, 8, 3)
    b = m.route_scored(p, x, m.Scoring("softmax", 8, 3, "max"))
    assert torch.equal(a[0], b[0])
    assert ((a[1] - b[1]).abs() <= 1e-6 * b[1]).all()


def test_logits_that_begin_between_words():
    m = moe()
    T, E, k = 40, 64, 4
    p = m.Problem(T=T, H=64, E=E, k=k, I=64)
    sc = m.Scoring("sigmoid", 4, 2, "top2")
    x, b = make_logits(T, E, 3), make_bias(E, 3)
    want = m.route_scored(p, x.cuda(), sc, bias=b.cuda())
    flat = torch.empty(T * E + 1, device="cuda")
    at = flat[1:].view(T, E)
    at.copy_(x)
    got = m.route_scored(p, at, sc, bias=b.cuda())
    assert all(torch.equal(a, q) for a, q in zip(got, want))
    dw = torch.randn(T, k, device="cuda")
    dl = torch.empty(T * E + 1, device="cuda")[1:].view(T, E)
    m.route_scored_backward(p, at, sc, got[0], got[1], dw, out=dl)
    assert torch.equal(dl, m.route_scored_backward(p, x.cuda(), sc, got[0], got[1], dw))


def test_more_than_2_31_logits():
    m = moe()
    E, k, n = 256, 8, 300
    T = (1 << 23) + n
    x = torch.zeros(T, E, device="cuda")
    x[-n:] = make_logits(n, E, 4).cuda()
    b = make_bias(E, 4).cuda()
    sc = m.Scoring("sigmoid", 8, 4, "top2", 2.5)
    big, small = (m.Problem(T=t, H=64, E=E, k=k, I=64) for t in (T, n))
    got = m.route_scored(big, x, sc, bias=b)
    tail = x[-n:].contiguous()
    want = m.route_scored(small, tail, sc, bias=b)
    assert all(torch.equal(a[-n:], q) for a, q in zip(got, want))
    dw = torch.zeros(T, k, device="cuda")
    dw[-n:] = torch.randn(n, k, device="cuda")
    dl = m.route_scored_backward(big, x, sc, got[0], got[1], dw)
    assert torch.equal(dl[-n:], m.route_scored_backward(small, tail, sc, want[0], want[1],
                                                        dw[-n:].contiguous()))
    assert not dl[:-n].any()


def test_debug_library_reports_bad_ids():
    import ctypes
    m = moe()
    T, E, k = 70, 16, 2
    p = m.Problem(T=T, H=64, E=E, k=k, I=64)
    sc = m.Scoring("sigmoid")
    x = make_logits(T, E, 2).cuda()
    ids, w, _ = m.route_scored(p, x, sc)
    dw, dl = torch.randn(T, k, device="cuda"), torch.empty(T, E, device="cuda")
    want = m.route_scored_backward(p, x, sc, ids, w, dw)
    d, c = m.debug_lib(), p.c()
    m.debug_status()
    ptr = lambda t: ctypes.c_void_p(t.data_ptr())  # noqa: E731
    run = lambda: d.moe_route_scored_backward(  # noqa: E731
        ctypes.byref(c), sc._ref, ptr(x), ptr(ids), ptr(w), ptr(dw), ptr(dl), m._stream())
    assert run() == m.MOE_OK and m.debug_status() == 0 and torch.equal(dl, want)
    ids[3, 1], ids[9, 0] = 99, -4
    assert run() == m.MOE_OK and m.debug_status() & 1
    keep = torch.ones(T, dtype=torch.bool)
    keep[[3, 9]] = False
    assert torch.equal(dl[keep.cuda()], want[keep.cuda()])


def test_large_batch_capture_and_streams():
    """A captured call replayed on new logits, and the call on another stream."""
    m = moe()
    T, E, k = 5000, 256, 8
    p = m.Problem(T=T, H=64, E=E, k=k, I=64, capacity=200)
    sc = m.Scoring("sigmoid", 8, 4, "top2", 2.5)
    b = make_bias(E, 2).cuda()
    x = make_logits(T, E, 3).cuda()
    ws = m.workspace(p, m.OP_ROUTE)
    dw = torch.randn(T, k, device="cuda")
    out = (torch.empty(T, k, dtype=torch.int32, device="cuda"),
           torch.empty(T, k, device="cuda"), torch.empty(T, k, dtype=torch.uint8, device="cuda"))
    dl = torch.empty(T, E, device="cuda")

    def call():
        m.route_scored(p, x, sc, bias=b, out=out, ws=ws)
        m.route_scored_backward(p, x, sc, out[0], out[1], dw, out=dl)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    first = [t.clone() for t in (*out, dl)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for seed in (3, 11, 12):
        x.copy_(make_logits(T, E, seed))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (*out, dl)]
        call()
        torch.cuda.synchronize()
        assert all(torch.equal(a, q) for a, q in zip(got, (*out, dl)))
        if seed == 3:
            assert all(torch.equal(a, q) for a, q in zip(got, first))


@pytest.mark.parametrize("kind", ["equal", "few", "normal", "wide"])
@pytest.mark.parametrize("T", [1, 2, 256, 257, 1025, 8192, 8193, 13001])
def test_capacity_of_one_crowded_expert(T, kind):
    """Nearly every token chooses expert 2: 256 candidates are ranked, more are selected by digits,
    8193 tokens and more through a layout, and 12288 candidates no longer fit on the chip."""
    import oracle

    m = moe()
    g = torch.Generator().manual_seed(T)
    x = {"equal": torch.zeros(T, 8), "few": torch.randint(0, 3, (T, 8), generator=g).float() / 4,
         "normal": torch.randn(T, 8, generator=g), "wide": 40 * torch.randn(T, 8, generator=g)}[kind]
    x[:, 2] += 6.0 * (torch.arange(T) % 29 != 0)
    for C in sorted({1, (T + 1) // 2, max(1, T - 1), T}):
        p = m.Problem(T=T, H=64, E=8, k=2, I=64, capacity=C)
        for sc in (None, m.Scoring("softmax"), m.Scoring("sigmoid", scale=2.5)):
            ids, w, keep = (m.route(p, x.cuda()) if sc is None else m.route_scored(p, x.cuda(), sc))
            want = oracle.capacity(ids.cpu().numpy(), w.cpu().numpy(), 8, C)
            assert (keep.cpu().numpy() == want).all(), (C, sc)


# (more than 8192 tokens, or more than 2^24 slots times experts: capacity through a layout)
LAYOUT_CASES = [
    (9001, 16, 6, "softmax", 4, 3, "top2", "out", True, 1.0, 1500, "masked"),
    (8192, 300, 8, "sigmoid", 1, 1, "max", "normal", False, 2.5, 190, "masked"),
]


@pytest.mark.parametrize("c", LAYOUT_CASES, ids=str)
def test_capacity_through_a_layout(c):
    """Slots whose expert is out do not count there either; captured and replayed, too."""
    m, p, sc, x, bias, (ids, w, keep) = setup(c)
    x, bias = x.cuda(), bias.cuda()
    ws = m.workspace(p, m.OP_ROUTE)
    out = tuple(torch.empty(p.T, p.k, dtype=t, device="cuda")
                for t in (torch.int32, torch.float32, torch.uint8))
    m.route_scored(p, x, sc, bias=bias, out=out, ws=ws)
    assert (out[0].cpu().numpy() == ids).all() and (out[2].cpu().numpy() == keep).all()
    assert (keep == 0).sum() > (w == 0).sum() > 0  # some by the capacity, some that are out
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        m.route_scored(p, x, sc, bias=bias, out=out, ws=ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.route_scored(p, x, sc, bias=bias, out=out, ws=ws)
    for step in range(3):
        x.copy_(x.roll(1, 0))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        want = m.route_scored(p, x, sc, bias=bias)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
