"""Layouts that reach every kernel of the grouped products, with and without a split reduction,
each with several experts, experts without rows, widths that end inside a tile and rows behind
the last expert.  test_grouped_plan.py holds the library's choice to this table on the host;
test_gpu_grouped_paths.py runs it."""
from collections import namedtuple

STREAM, TILE256, TILE128, TILE64, TILE128_ONCE = range(5)
LINEAR, DX, DW = range(3)

MANY = [1300, 0, 900, 2, 700]                       # many rows per expert
SOME = [300, 299, 0, 511, 1, 640, 97, 400]          # some hundreds
FEW = [(37 * i) % 101 for i in range(64)]           # less than a tile's
LATE = [0] * 7 + [100]                              # few, all of them the last expert's
ONES = [1, 0, 2, 1, 0, 1, 1, 0, 1, 0, 0, 1, 0, 0, 0, 0]  # single tokens
LONG = [5, 9000]

Path = namedtuple("Path", "name mode counts extra K N kernel split")
PATHS = [
    Path("linear stream", LINEAR, LATE, 28, 544, 264, STREAM, 1),
    Path("linear stream parts", LINEAR, LATE, 28, 4104, 512, STREAM, 4),
    Path("linear stream parts, single rows", LINEAR, ONES, 0, 7168, 512, STREAM, 4),
    Path("linear 256", LINEAR, MANY, 7, 264, 6176, TILE256, 1),
    Path("linear 128", LINEAR, SOME, 7, 264, 2464, TILE128, 1),
    Path("linear 128 once", LINEAR, FEW, 7, 264, 800, TILE128_ONCE, 1),
    Path("linear 64", LINEAR, SOME, 7, 520, 1056, TILE64, 1),
    Path("linear 64 parts", LINEAR, SOME, 7, 4104, 288, TILE64, 4),
    Path("dx stream", DX, LATE, 28, 288, 520, STREAM, 1),
    Path("dx stream parts", DX, LATE, 28, 512, 4104, STREAM, 4),
    Path("dx stream parts, single rows", DX, ONES, 0, 512, 7168, STREAM, 4),
    Path("dx 256", DX, MANY, 7, 6176, 264, TILE256, 1),
    Path("dx 128", DX, SOME, 7, 2464, 264, TILE128, 1),
    Path("dx 128 once", DX, FEW, 7, 800, 264, TILE128_ONCE, 1),
    Path("dx 64", DX, SOME, 7, 1056, 520, TILE64, 1),
    Path("dx 64 parts", DX, SOME, 7, 288, 4104, TILE64, 4),
    Path("dw 256", DW, SOME, 7, 1288, 1032, TILE256, 1),
    Path("dw 128", DW, SOME, 7, 544, 1032, TILE128, 1),
    Path("dw 128 parts", DW, LONG, 7, 264, 160, TILE128, 8),
    Path("dw 64", DW, LATE, 28, 544, 264, TILE64, 1),
]
