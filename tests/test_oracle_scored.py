"""The definitions of the routing by scores and of the 4-bit values: worked cases, autograd and
differences."""
import numpy as np
import pytest
import torch

from oracle import fp4, scored

INF = float("inf")


def test_bias_moves_the_choice_and_not_the_weights():
    l = np.log(np.array([1.0, 2.0, 3.0, 2.0]))
    ids, w, _ = scored.route_token(l, 2, "softmax")
    assert ids.tolist() == [2, 1] and np.allclose(w, [3 / 5, 2 / 5])
    ids, w, _ = scored.route_token(l, 2, "softmax", bias=np.array([0.5, 0, 0, 0.0]))
    assert ids.tolist() == [0, 2] and np.allclose(w, [1 / 4, 3 / 4])  # 0.625, 0.375 lead
    ids, w, _ = scored.route_token(l, 2, "softmax", renorm=False, scale=2.0)
    assert np.allclose(w, [2 * 3 / 8, 2 * 2 / 8])


def test_group_scores():
    # groups {0, 1}, {2, 3}, {4, 5}: the best expert is in the first, the best pair in the second
    s = np.array([0.9, 0.05, 0.6, 0.55, 0.4, 0.4])
    l = np.log(s / (1 - s))
    how = dict(n_group=3, topk_group=1)
    assert scored.route_token(l, 2, "sigmoid", group_score="max", **how)[0].tolist() == [0, 1]
    assert scored.route_token(l, 2, "sigmoid", group_score="top2", **how)[0].tolist() == [2, 3]
    l[2] = -INF  # one of a pair is out: the group counts for the other alone
    assert scored.route_token(l, 2, "sigmoid", group_score="top2", **how)[0].tolist() == [0, 1]


def test_experts_that_are_out_fill_the_last_slots():
    l = np.array([-INF, 0.0, float("nan"), -INF, 1.0])
    ids, w, live = scored.route_token(l, 4, "softmax")
    assert ids.tolist() == [4, 1, 0, 2] and live.tolist() == [True, True, False, False]
    assert w[2:].tolist() == [0, 0] and np.isclose(w.sum(), 1)
    ids, w, live = scored.route_token(np.full(4, -INF), 2, "sigmoid")
    assert ids.tolist() == [0, 1] and w.tolist() == [0, 0] and not live.any()
    low = np.full(3, -scored.BIG)  # the type's lowest value is a number
    assert np.allclose(scored.route_token(low, 3, "softmax")[1], 1 / 3)
    assert scored.route_token(low, 3, "sigmoid")[1].tolist() == [0, 0, 0]
    ids, w, live = scored.route_token(np.zeros(3), 2, "sigmoid", bias=np.array([-INF, 1.0, 0.0]))
    assert ids.tolist() == [1, 2] and live.all()
    assert np.isclose(scored.route_token(np.array([INF, 0.0]), 2, "softmax")[1][0], 1)


def test_capacity_does_not_count_experts_that_are_out():
    l = np.array([[-INF, 2.0], [1.0, 2.0], [0.5, 2.0]])
    ids, w, keep = scored.route(l, 2, "sigmoid", capacity=1)
    at0 = ids == 0
    assert keep[0][at0[0]] == 0 and keep[1][at0[1]] == 1 and keep[2][at0[2]] == 0


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_backward_is_the_gradient(kind, renorm):
    g = torch.Generator().manual_seed(3)
    T, E, k, scale = 5, 11, 3, 2.5
    l = torch.randn(T, E, generator=g, dtype=torch.float64)
    l[1, 4] = -INF
    l.requires_grad_()
    dw = torch.randn(T, k, generator=g, dtype=torch.float64)
    ids, _, _ = scored.route(l.detach().numpy(), k, kind, renorm=renorm, scale=scale)

    def weights(v):
        s = torch.softmax(v, 1) if kind == "softmax" else torch.sigmoid(v)
        w = s.gather(1, torch.from_numpy(ids).long())
        return scale * (w / w.sum(1, keepdim=True) if renorm else w)

    w = weights(l)
    (w * dw).sum().backward()
    got, size = scored.backward(l.detach().numpy(), ids, w.detach().numpy(), dw.numpy(), kind,
                                renorm, scale)
    want = torch.nan_to_num(l.grad).numpy()
    assert np.abs(got - want).max() < 1e-12 and (size + 1e-12 >= np.abs(got)).all()
    h = 1e-6
    for t, e in ((0, int(ids[0, 0])), (1, 2), (4, 10)):
        up, dn = l.detach().clone(), l.detach().clone()
        up[t, e] += h
        dn[t, e] -= h
        diff = ((weights(up) - weights(dn)) * dw).sum().item() / (2 * h)
        assert abs(diff - got[t, e]) < 1e-7


def test_fp4_levels_ties_and_scales():
    x = torch.zeros(1, 32, dtype=torch.float64)
    x[0, :17] = torch.tensor([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -0.75, -5, 0.26, 2.4,
                              -6, -0.0, 0.2, 5.01], dtype=torch.float64)
    c, s = fp4.quantize(x)
    assert s.tolist() == [[127]]
    v = fp4.dequantize(c, s)[0, :17].tolist()
    assert v == [6, 0, 1, 1, 2, 2, 4, 4, 0, -1, -4, 0.5, 2, -6, 0, 0, 6]
    assert c[0, 0].item() == 7 and (c[0, 7].item() & 15) == 8  # low half first; -0 keeps its sign
    for top, byte in ((6.0, 127), (6.0001, 128), (3.0, 126), (3.0001, 127), (0.0, 127),
                      (2.0 ** -133, 0), (6 * 2.0 ** -127, 0), (6.1 * 2.0 ** -127, 1),
                      (3.3e38, 253), (INF, 255), (float("nan"), 255)):
        x = torch.zeros(1, 32, dtype=torch.float64)
        x[0, 9] = -top
        c, s = fp4.quantize(x)
        assert s.item() == byte, top
        if byte == 255:
            assert c.eq(0).all() and fp4.dequantize(c, s).isnan().all()


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
def test_infinite_logits_get_no_gradient(kind, renorm):
    l = np.array([[0.5, INF, -1.0, INF, 2.0], [INF, 0.0, 1.0, scored.BIG, -INF]])
    ids, w, _ = scored.route(l, 3, kind, renorm=renorm)
    dw = np.array([[0.3, -1.2, 0.7], [1.1, 0.4, -0.9]])
    got, size = scored.backward(l, ids, w, dw, kind, renorm)
    assert (got[l == INF] == 0).all() and (size[l == INF] == 0).all()
    if kind == "softmax":  # as for the largest number in its place, but for itself
        low = np.minimum(l, scored.BIG)
        want = scored.backward(low, ids, w, dw, kind, renorm)[0]
        assert np.array_equal(got[l < INF], want[l < INF]) and want[1, 0] != 0 and got[1, 3] != 0
