"""Refusals of the 4-bit values, the product on them and the routing by scores: reported before
anything is enqueued, so all of them run without a GPU."""
import copy
import ctypes
import pickle

import pytest

from fp4_paths import PATHS, plan
from grouped_common import fake, moe

INV, UNS, WS, OK = 1, 2, 3, 0


def at(p, n):
    return ctypes.c_void_p(p.value + n)


def test_quantize_refusals():
    m = moe()
    x, c, s, v = fake(4)
    q, d, i64, i32 = m.lib.moe_quantize_fp4, m.lib.moe_dequantize_fp4, ctypes.c_int64, ctypes.c_int32
    assert q(None, i64(0), i32(32), None, None, None, None) == OK
    assert d(None, None, i64(0), i32(64), None, None, None) == OK
    for rows, cols in ((-1, 32), (4, 0), (4, 48), (4, -32), (1 << 35, 32), (1 << 62, 1 << 20)):
        assert q(x, i64(rows), i32(cols), None, c, s, None) == INV
        assert d(c, s, i64(rows), i32(cols), None, v, None) == INV
    for a in ((None, c, s), (x, None, s), (x, c, None), (at(x, 8), c, s), (x, at(c, 4), s),
              (x, at(x, 64), s), (x, c, c), (x, c, at(x, 250))):
        assert q(a[0], i64(4), i32(32), None, a[1], a[2], None) == INV
    for a in ((None, s, v), (c, None, v), (c, s, None), (c, s, at(v, 2)), (c, s, c), (c, s, s)):
        assert d(a[0], a[1], i64(4), i32(32), None, a[2], None) == INV
    assert q(x, i64(4), i32(32), c, c, s, None) == INV  # live_rows inside an output


def test_quantize_weights_refusals():
    m = moe()
    w, c, s = fake(3)
    q = lambda E, K, N, a=(w, c, s): m.lib.moe_quantize_fp4_weights(  # noqa: E731
        a[0], ctypes.c_int32(E), ctypes.c_int32(K), ctypes.c_int32(N), a[1], a[2], None)
    for E, K, N in ((0, 32, 8), (1, 0, 8), (1, 32, 0), (-1, 32, 8)):
        assert q(E, K, N) == INV
    for E, K, N in ((1025, 32, 8), (1, 48, 8), (1, 32, 12), (1, (1 << 20) + 32, 8),
                    (1, 32, (1 << 20) + 8)):
        assert q(E, K, N) == UNS
    for a in ((None, c, s), (w, None, s), (w, c, None), (at(w, 2), c, s), (w, at(c, 8), s),
              (w, w, s), (w, c, c)):
        assert q(2, 64, 16, a) == INV


def call(m, g, p, **kw):
    """moe_grouped_linear_fp4 with the stand-ins p (a dict) and what kw replaces."""
    a = dict(p, xd=m.MOE_FP4, act=0, up=None, ub=None, uc=None, us=None, b=None, res=None, rt=None)
    a.update(kw)
    w = m.MoeFp4Weights(a["wc"], a["ws_"], a["b"])
    u = m.MoeFp4Weights(a["uc"], a["us"], a["ub"])
    return m.lib.moe_grouped_linear_fp4(
        None if g is None else ctypes.byref(g), a["xd"], a["xc"], a["xs"], a["rt"], a["off"],
        None if a.get("now") else ctypes.byref(w), ctypes.byref(u) if a["uc"] or a["us"] else None,
        a["act"], a["res"], a["y"], a.get("ws"), a.get("wsn", 0), None)


def test_grouped_linear_fp4_refusals():
    m = moe()
    names = ("xc", "xs", "off", "wc", "ws_", "y", "spare", "more", "rest")
    p = dict(zip(names, fake(len(names))))
    spare, more, rest = p.pop("spare"), p.pop("more"), p.pop("rest")
    G = lambda R=64, T=64, K=64, N=16, E=2: m.MoeGrouped(R, T, K, N, E)  # noqa: E731
    assert call(m, G(R=0), p) == OK
    assert call(m, G(R=0, T=0), dict(p, xc=None, xs=None, y=None)) == OK
    assert call(m, None, p) == INV
    for bad in (G(R=-1), G(K=0), G(N=0), G(E=0), G(T=-1)):
        assert call(m, bad, p) == INV
    for bad in (G(E=1025), G(K=40), G(N=12), G(R=(1 << 30) + 1)):
        assert call(m, bad, p) == UNS
    g = G()
    for kw in (dict(xc=None), dict(xs=None), dict(wc=None), dict(ws_=None), dict(y=None),
               dict(off=None), dict(now=True), dict(xd=m.MOE_BF16), dict(xd=9), dict(act=5),
               dict(act=-1), dict(xc=at(p["xc"], 8)), dict(wc=at(p["wc"], 8)),
               dict(y=at(p["y"], 8)), dict(b=at(spare, 2)), dict(res=at(spare, 4)),
               dict(uc=spare), dict(us=spare), dict(uc=at(spare, 4), us=more),
               dict(uc=spare, us=more, ub=at(rest, 8))):
        assert call(m, g, p, **kw) == INV, kw
    assert call(m, G(T=0), p, rt=spare) == INV  # rows through a list, and no rows to read
    for kw in (dict(y=p["xc"]), dict(y=at(p["xc"], 64 * 32 - 16)), dict(y=p["wc"]),
               dict(y=p["xs"]), dict(y=p["ws_"]), dict(y=p["off"]), dict(res=p["y"]),
               dict(b=p["y"]), dict(rt=p["y"]), dict(uc=p["y"], us=more),
               dict(uc=spare, us=p["y"]), dict(uc=spare, us=more, ub=p["y"])):
        assert call(m, g, p, **kw) == INV, kw
    # 8-bit codes are twice as long
    assert call(m, g, p, xd=m.MOE_FP8, y=at(p["xc"], 64 * 64 - 16)) == INV


def test_workspace_op():
    m = moe()
    assert m.GroupedProblem(R=8, K=40, N=16).workspace_bytes(m.OP_GROUPED_FP4) == 0
    assert m.GroupedProblem(R=8, K=64, N=16).workspace_bytes(4) == 0


def problem_of(kw):
    R = sum(kw["counts"]) + kw.get("front", 0) + kw.get("behind", 0)
    return R, kw["K"], kw["N"], len(kw["counts"])


@pytest.mark.parametrize("i", range(len(PATHS)))
def test_paths_reach_what_they_name(i):
    four, eight, kw = PATHS[i]
    gated = kw.get("gated", False)
    assert plan(*problem_of(kw), False, gated) == four
    assert plan(*problem_of(kw), True, gated) == eight


@pytest.mark.parametrize("R,K,N,E", [
    (1, 32, 8, 1), (16, 7168, 4096, 1), (17, 7168, 4096, 1), (64, 7168, 1024, 1),
    (128, 7168, 4096, 1), (512, 7168, 4096, 1), (1024, 7168, 4096, 1), (4096, 2048, 2048, 1),
    (100, 1 << 20, 64, 1), (300, 3584, 264, 4), (300, 3552, 264, 4), (4096, 2048, 768, 128),
    (32768, 2048, 768, 128), (131072, 7168, 2048, 256), (0, 7168, 64, 1)])
def test_workspace_holds_the_parts(R, K, N, E):
    m = moe()
    need = 0
    for eight in (False, True):
        for gated in (False, True):
            split = plan(R, K, N, E, eight, gated)[1]
            if split > 1:
                need = max(need, -(-split * R * N * (8 if gated else 4) // 256) * 256)
    assert m.GroupedProblem(R=R, K=K, N=N, E=E).workspace_bytes(m.OP_GROUPED_FP4) == need


def test_workspace_refusals():
    m = moe()
    names = ("xc", "xs", "off", "wc", "ws_", "y", "w")
    p = dict(zip(names, fake(len(names))))
    ws = p.pop("w")
    g = m.MoeGrouped(100, 100, 7168, 64, 1)
    need = m.GroupedProblem(R=100, K=7168, N=64).workspace_bytes(m.OP_GROUPED_FP4)
    assert need > 0
    assert call(m, g, p) == WS
    assert call(m, g, p, ws=ws, wsn=need - 1) == WS
    assert call(m, g, p, ws=at(ws, 16), wsn=need) == INV
    assert call(m, g, p, ws=p["y"], wsn=need) == INV


def test_scoring_refusals():
    m = moe()
    lg, ids, w, keep, b, dw, dl, x = fake(8)
    p = m.Problem(T=64, H=64, E=64, k=4, I=64)
    P = ctypes.byref(p.c())
    S = lambda **kw: ctypes.byref(m.MoeScoring(*[  # noqa: E731
        {**dict(score=1, n_group=8, topk_group=4, group_score=1, scale=1.0), **kw}[n]
        for n in ("score", "n_group", "topk_group", "group_score", "scale")]))
    r, rt, bw = (m.lib.moe_route_scored, m.lib.moe_router_scored,
                 m.lib.moe_route_scored_backward)
    bad = [S(score=2), S(score=-1), S(group_score=2), S(n_group=3), S(n_group=0), S(topk_group=0),
           S(topk_group=9), S(n_group=64, topk_group=3), S(n_group=128), S(scale=0.0),
           S(scale=-1.0), S(scale=float("nan")), S(scale=float("inf")), S(scale=1e300), None]
    for s in bad:
        assert r(P, s, lg, b, ids, w, keep, None, 0, None) == INV
        assert rt(P, s, x, dw, b, None, ids, w, keep, None, 0, None) == INV
        assert bw(P, s, lg, ids, w, dw, dl, None) == INV
    ok = S()
    for a in ((None, ids, w, keep), (lg, None, w, keep), (lg, ids, None, keep), (lg, ids, w, None),
              (lg, lg, w, keep), (lg, ids, ids, keep), (lg, ids, w, b)):
        assert r(P, ok, a[0], b, a[1], a[2], a[3], None, 0, None) == INV
    capped = ctypes.byref(m.Problem(T=64, H=64, E=64, k=4, I=64, capacity=3).c())
    assert r(capped, ok, lg, b, ids, w, keep, None, 0, None) == WS
    for a in ((None, ids, w, dw, dl), (lg, None, w, dw, dl), (lg, ids, None, dw, dl),
              (lg, ids, w, None, dl), (lg, ids, w, dw, None), (lg, ids, w, dw, lg),
              (lg, ids, w, dl, dl)):
        assert bw(P, ok, *a, None) == INV
    assert rt(P, ok, x, dw, b, None, ids, w, keep, None, 0, None) == WS
    assert rt(P, ok, at(x, 8), dw, b, None, ids, w, keep, None, 0, None) == INV
    f32 = ctypes.byref(m.Problem(T=64, H=64, E=64, k=4, I=64, dtype="f32").c())
    assert rt(f32, ok, x, dw, b, None, ids, w, keep, None, 0, None) == UNS
    assert r(ctypes.byref(m.Problem(T=0, H=64, E=64, k=4, I=64).c()), ok, lg, b, ids, w, keep,
             None, 0, None) == INV


def test_python_refusals():
    import torch
    m = moe()
    with pytest.raises(ValueError):
        m.Scoring(score="relu")
    with pytest.raises(ValueError):
        m.Scoring(group_score="sum")
    s = m.Scoring("sigmoid", 8, 4, "top2", 2.5)
    for c in (copy.copy(s), copy.deepcopy(s), pickle.loads(pickle.dumps(s))):
        assert c == s and c._c.scale == 2.5 and c._c.n_group == 8
    p = m.Problem(T=4, H=64, E=8, k=2, I=64)
    with pytest.raises(ValueError):
        m.route_scored(p, torch.zeros(4, 8), s)  # not on the GPU
    with pytest.raises(ValueError):
        m.quantize_fp4(torch.zeros(4, 40, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        m.quantize_fp4(torch.zeros(32, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        m.quantize_fp4_weights(torch.zeros(32, 8, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        m.dequantize_fp4(torch.zeros(4, 0, dtype=torch.uint8), torch.zeros(4, 0))
    with pytest.raises(ValueError):
        m.grouped_linear_fp4(m.GroupedProblem(R=4, K=64, N=8), (torch.zeros(4, 32), None),
                             (None, None))
