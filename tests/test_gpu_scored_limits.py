"""Routing by scores at the ends of its range: biases far larger than the scores, which leave a group's
sum of two nothing but a small difference, or pass the range of 32 bits together."""
import numpy as np
import pytest
import torch

from oracle import scored
from scored_common import INF, logits as make_logits, numpy_of

pytestmark = pytest.mark.gpu


def moe():
    import expert_ffn_moe_amd

    return expert_ffn_moe_amd


def check(x, k, kind, bias, n_group, taken, group_score="top2", renorm=True):
    m = moe()
    T, E = x.shape
    p = m.Problem(T=T, H=64, E=E, k=k, I=64, renormalize=int(renorm))
    sc = m.Scoring(kind, n_group, taken, group_score)
    got = m.route_scored(p, x.cuda(), sc, bias=None if bias is None else bias.cuda())
    ids, w, keep = scored.route(numpy_of(x), k, kind, bias=numpy_of(bias), n_group=n_group,
                                topk_group=taken, group_score=group_score, renorm=renorm)
    wrong = (got[0].cpu().numpy() != ids).any(1)
    assert not wrong.any(), (int(wrong.sum()), int(wrong.argmax()))
    assert np.array_equal(got[2].cpu().numpy(), keep)
    # as in test_gpu_scored.py: two roundings of one fp64 value
    err = np.abs(got[1].cpu().numpy().astype(np.float64) - w)
    assert (err <= 2.0 ** -23 * np.abs(w) + 2.0 ** -149).all()


# E, groups: every number of experts per lane, groups of one lane and of several
SHAPES = [(64, 16), (64, 2), (128, 8), (128, 16), (256, 4), (256, 16)]


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("B", [16.0, 100.0, 1e4, 1e6, 1e20, "mixed"])
@pytest.mark.parametrize("E,G", SHAPES)
def test_biases_that_cancel_in_a_group(E, G, B, kind):
    """A group's two best have biases B and -B: its sum is that of two scores, behind values whose
    32 bits end far above them."""
    T, size = 1500, E // G
    g = torch.Generator().manual_seed(E + G)
    of = torch.full((G,), 0.0) + (torch.tensor([0.0, 10.0, 1e3, 1e5])[torch.arange(G) % 4]
                                  if B == "mixed" else B)
    b = (-4 * of[:, None] - 4).repeat(1, size)
    at = torch.rand(G, size, generator=g).argsort(1)[:, :2]  # which two
    b.scatter_(1, at, torch.stack((of, -of), 1))
    x = 2 * torch.randn(T, E, generator=g)
    check(x, 3, kind, b.reshape(-1), G, max(1, G // 2))


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,G", SHAPES)
def test_sums_beyond_the_range(E, G, kind):
    """Pairs that 32 bits hold and whose sums they do not, of both signs: as 64 bits order them."""
    T, size = 60, E // G
    x = make_logits(T, E, 6)
    for top in ((3.0e38, 2.9e38), (-3.0e38, -2.9e38), (INF, INF), (3.4e38, -3.4e38)):
        for step in (1.0, 0.8, 1.2):  # the first group ahead, or the last, or all equal
            b = torch.full((E,), -3.402e38)
            for q in range(G):
                f = 1.0 if step == 1.0 else (0.999 ** q if step < 1 else 0.999 ** (G - 1 - q))
                b[q * size] = top[0] * f if top[0] != INF else INF
                b[q * size + size // 2] = top[1] * f if top[1] != INF else INF
            check(x, 3, kind, b, G, 1)
            check(x, 3, kind, b, G, max(1, G - 1))


def test_two_groups_beyond_the_range():
    b = torch.zeros(64)
    b[0], b[1], b[32], b[33] = 3.0e38, 2.9e38, 2.5e38, 2.4e38
    check(make_logits(50, 64, 1), 3, "sigmoid", b, 2, 1)
    b[32:34], b[0:2] = b[0:2].clone(), b[32:34].clone()
    check(make_logits(50, 64, 1), 3, "sigmoid", b, 2, 1)


@pytest.mark.parametrize("kind", ["sigmoid", "softmax"])
@pytest.mark.parametrize("group_score", ["max", "top2"])
@pytest.mark.parametrize("by", ["logits", "bias", "logits alone"])
@pytest.mark.parametrize("E,G", SHAPES)
def test_groups_that_are_wholly_out(E, G, by, group_score, kind):
    """They are behind the others, take no part where enough are left, and fill the last slots (with
    their lowest experts, in the taken groups) where not."""
    T, size = 100, E // G
    for gone in sorted({1, G // 2, G - 1, G}):
        x = make_logits(T, E, gone)
        b = None if by == "logits alone" else 0.1 * torch.randn(
            E, generator=torch.Generator().manual_seed(gone))
        out = torch.randperm(G, generator=torch.Generator().manual_seed(E))[:gone]
        at = (out[:, None] * size + torch.arange(size)).reshape(-1)
        if by == "bias":
            b[at] = -INF
        else:
            x[:, at] = -INF
            x[1, at[0]] = 0.5  # one of a group is there after all
        for taken in sorted({1, max(1, G // 2), G - 1}):
            check(x, 3, kind, b, G, taken, group_score)


# T, E, k on both sides of the rules of the capacity's two ways: 8192 tokens, 98304 slots, 2^24 slots
# times experts
@pytest.mark.parametrize("T,E,k", [(8192, 32, 12), (8192, 32, 13), (3100, 40, 32), (3000, 40, 32),
                                   (8192, 16, 16), (8191, 34, 32), (8192, 170, 12), (8192, 171, 12)])
def test_capacity_by_slots_and_through_a_layout(T, E, k):
    import oracle

    m = moe()
    x = make_logits(T, E, k)
    for skew in (0, 2):
        xs = x + skew * torch.randn(E, generator=torch.Generator().manual_seed(E))
        for C in (1, max(1, T * k // E), T - 1):
            p = m.Problem(T=T, H=64, E=E, k=k, I=64, capacity=C)
            for sc in (None, m.Scoring("sigmoid", scale=2.5)):
                ids, w, keep = (m.route(p, xs.cuda()) if sc is None
                                else m.route_scored(p, xs.cuda(), sc))
                want = oracle.capacity(ids.cpu().numpy(), w.cpu().numpy(), E, C)
                assert (keep.cpu().numpy() == want).all(), (C, sc)


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k", [(8, 2), (64, 3), (72, 6), (256, 8), (300, 1), (520, 12)])
def test_infinite_logits_get_no_gradient(E, k, kind, renorm):
    """None, one, two or all of a token's logits +inf, beside the largest number and finite ones."""
    m = moe()
    T = 67
    x = make_logits(T, E, 3)
    for t in range(T):
        x[t, torch.randperm(E, generator=torch.Generator().manual_seed(t))[:t % 4]] = INF
    x[5], x[6, :] = INF, torch.finfo(torch.float32).max
    x[6, E // 2] = x[7, 0] = INF
    x[8] = 1.0  # equal weights without any
    p = m.Problem(T=T, H=64, E=E, k=k, I=64, renormalize=int(renorm))
    sc = m.Scoring(kind, scale=2.5)
    ids, w, _ = scored.route(numpy_of(x), k, kind, renorm=renorm, scale=2.5)
    dw = torch.randn(T, k, generator=torch.Generator().manual_seed(9))
    want, size = scored.backward(numpy_of(x), ids, w, numpy_of(dw), kind, renorm, 2.5)
    got = m.route_scored_backward(p, x.cuda(), sc, torch.from_numpy(ids).cuda(),
                                  torch.from_numpy(w).cuda(), dw.cuda()).cpu().double().numpy()
    assert (got[x.numpy() == np.inf] == 0).all()
    # as in test_gpu_scored.py
    g = dw.abs().numpy().sum(1, keepdims=True)
    tol = 4 * 2.0 ** -24 * size + 2.0 ** -24 * np.abs(want) + 2.0 ** -149 * (1 + 4 * g)
    assert (np.abs(got - want) <= tol).all()
