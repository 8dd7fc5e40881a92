"""The choice of kernel for a product on 4-bit weights, written out from its documented rule, and
layouts that reach every kernel for both types of x, with several experts where it takes them."""
STREAM, TILE256, TILE128, TILE128_ONCE = range(4)


def up(a, b):
    return -(-a // b)


def plan(R, K, N, E, eight, gated):
    """(kernel, parts of the reduction)"""
    rows, active = R // E, min(E, max(R, 1))
    stages, big = up(K, 256), 128 if eight else 256

    def tiles(bm, bn):
        mt = max(active, R // bm + (active // 2 if E > 1 else 1))
        return mt * up(N, bn // 2 if gated else bn)

    n256, n128 = tiles(big, 256), tiles(big // 2, 128)
    if rows <= (4 if eight else 16) and (n128 < 256 or (not eight and stages <= 8)):
        return STREAM, 1
    if 16 * rows > 7 * big and n256 >= 192:
        return TILE256, 1
    if n128 >= 256:
        return (TILE128_ONCE if 8 * rows <= 3 * big else TILE128), 1
    return TILE128, max(1, min(stages // 7, 256 // n128))


RAGGED = [0, 700, 0, 1, 513, 1031, 255, 0]  # 2500 rows
FEW = [0, 3, 0, 0, 40, 1, 0, 0] * 8

# (what it reaches for x in 4 bits, in 8 bits) and the arguments of fp4_common.Case
PATHS = [
    ((TILE256, 1), (TILE256, 1), dict(counts=RAGGED, K=544, N=5000)),
    ((TILE256, 1), (TILE256, 1),
     dict(counts=RAGGED, K=1824, N=2504, gated=True, act="silu", bias=True, residual=True,
          gather=True, wild=True, T=900, behind=40)),
    ((TILE128, 1), (TILE128, 1), dict(counts=[300, 0, 1, 99], K=288, N=6664, behind=10)),
    ((TILE128, 1), (TILE128, 1),
     dict(counts=[300, 0, 1, 99], K=1056, N=3336, gated=True, act="gelu_tanh", gather=True,
          wild=True, front=2, residual=True)),
    ((TILE128_ONCE, 1), (TILE128_ONCE, 1), dict(counts=FEW, K=2336, N=648, behind=7, bias=True)),
    ((TILE128_ONCE, 1), (TILE128_ONCE, 1),
     dict(counts=FEW, K=2336, N=328, gated=True, act="silu", gather=True, wild=True, T=50)),
    ((TILE128, 1), (TILE128, 1), dict(counts=[90, 0, 37], K=160, N=136, act="relu", bias=True)),
    ((TILE128, 2), (TILE128, 2),
     dict(counts=[90, 0, 37, 5], K=3616, N=200, bias=True, residual=True, behind=9)),
    ((TILE128, 3), (TILE128, 3),
     dict(counts=[90, 0, 37, 130], K=5600, N=264, gated=True, act="silu", bias=True, gather=True,
          wild=True, front=3, behind=9)),
    ((TILE128, 4), (TILE128, 4), dict(counts=[33], K=7200, N=520, act="relu2")),
    ((STREAM, 1), (TILE128, 1), dict(counts=[9, 0, 11, 0], K=480, N=72, behind=3)),
    ((STREAM, 1), (STREAM, 1),
     dict(counts=[0, 2, 0, 1, 0] * 5, K=992, N=104, gated=True, act="silu", bias=True, gather=True,
          wild=True, residual=True)),
    ((STREAM, 1), (STREAM, 1), dict(counts=[1] + [0] * 1022 + [40], K=64, N=40)),
    ((STREAM, 1), (STREAM, 1), dict(counts=[0] * 200 + [70] + [0] * 100, K=288, N=72)),
    # scales by four stages: 16 stages, 17 with a partial one, 21 with several items of a block
    ((TILE256, 1), (TILE256, 1), dict(counts=[700], K=4096, N=16400)),
    ((TILE256, 1), (TILE256, 1), dict(counts=[390, 301], K=4320, N=16400, bias=True, behind=9)),
    ((TILE256, 1), (TILE256, 1),
     dict(counts=[1030], K=5376, N=16400, gated=True, act="silu", front=3)),
]
