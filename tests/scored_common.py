"""Inputs shared by the tests of the routing by scores."""
import numpy as np
import torch

INF = float("inf")


def logits(T, E, seed, kind="normal"):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, E, generator=g)
    if kind == "ties":  # few distinct values: the order of equal ones shows
        x = torch.round(x * 2) / 2
        x[x == 0] = torch.where(torch.rand(int((x == 0).sum()), generator=g) < 0.5, 0.0, -0.0)
    if kind == "wide":  # scores that vanish and saturate
        x = x * 60
    if kind == "lane":  # 16 neighbours ahead of all others
        x[:, 32:48] += 9
    if kind == "close":  # pairs that 32 bits cannot tell apart, on both sides of a border
        half = E // 2
        pair = x[:, :half] * (1 + 2.0 ** -22 * torch.randint(-3, 4, (T, half), generator=g))
        x[:, half:2 * half] = pair
        x = x[:, torch.randperm(E, generator=g)]
    if kind == "masked":
        x[torch.rand(T, E, generator=g) < 0.4] = -INF
        x[torch.rand(T, E, generator=g) < 0.05] = float("nan")
        x[0] = -INF  # nothing left
        if T > 1:
            x[1] = -torch.finfo(torch.float32).max
        if T > 2:
            x[2, :] = -INF
            x[2, E // 2] = 0.25
        if T > 3:
            x[3, E - 1] = INF
    return x


def bias(E, seed, kind="normal"):
    if kind is None:
        return None
    b = 0.2 * torch.randn(E, generator=torch.Generator().manual_seed(seed + 1000))
    if kind == "ties":
        b = torch.round(b * 4) / 4
    if kind == "same":
        b = torch.full((E,), 0.125)
    if kind == "close":
        b[E // 2:2 * (E // 2)] = b[:E // 2]
    if kind == "out" and E > 2:
        b[E // 3] = -INF
    return b


def numpy_of(t):
    return None if t is None else t.numpy().astype(np.float64)
