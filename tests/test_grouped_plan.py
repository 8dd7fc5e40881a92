"""Which kernel and how many parts of the reduction a grouped call gets: the library's own
choice, called through its C++ symbols (not part of the C ABI).  Nothing is launched."""
import ctypes

import pytest

from grouped_common import moe
from grouped_paths import (DW, DX, LINEAR, PATHS, STREAM, TILE64, TILE128, TILE128_ONCE,
                           TILE256)


class Plan(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_int), ("split", ctypes.c_int), ("ws_bytes", ctypes.c_size_t)]


class Args(ctypes.Structure):
    """GroupedArgs of csrc/grouped.h"""
    _fields_ = ([(n, ctypes.c_void_p) for n in ("x", "w", "row_token", "offsets", "bias", "residual",
                                                "out", "a", "codes", "scales", "dw", "dbias")] +
                [(n, ctypes.c_int) for n in ("R", "T", "K", "N", "E", "act", "accumulate", "split")] +
                [("part", ctypes.c_void_p)])


def plan(R, K, N, E, mode):
    f = moe().lib["_ZN3moe12grouped_planERK11moe_groupedi"]
    f.restype, f.argtypes = Plan, [ctypes.c_void_p, ctypes.c_int]
    g = moe().MoeGrouped(R, R, K, N, E)
    p = f(ctypes.byref(g), mode)
    return p.kernel, p.split


@pytest.mark.parametrize("mode", [DW, -1, 3])
def test_streaming_kernel_takes_linear_and_dx_alone(mode):
    f = moe().lib["_ZN3moe21launch_grouped_streamERKNS_11GroupedArgsEiP12ihipStream_t"]
    f.restype, f.argtypes = ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p]
    g = Args(R=0, T=0, K=64, N=64, E=1, split=1)  # no rows: a launch would do nothing
    assert f(ctypes.byref(g), mode, None) == 1  # hipErrorInvalidValue


def test_weight_gradients_never_stream():
    for E in (1, 2, 8, 60, 256, 1024):
        for K, N in ((8, 8), (64, 128), (520, 1096), (2048, 768), (7168, 2048)):
            for R in (0, 1, 8, 100, 4096, 131072, 1 << 24):
                assert plan(R, K, N, E, DW)[0] in (TILE256, TILE128, TILE64), (E, K, N, R)


@pytest.mark.parametrize("p", PATHS, ids=lambda p: p.name)
def test_paths_reach_their_kernel(p):
    assert plan(sum(p.counts) + p.extra, p.K, p.N, len(p.counts), p.mode) == (p.kernel, p.split)


def test_paths_reach_every_kernel_and_split():
    tiles = {(m, k, False) for m in (LINEAR, DX) for k in (STREAM, TILE256, TILE128, TILE64,
                                                           TILE128_ONCE)}
    parts = {(m, k, True) for m in (LINEAR, DX) for k in (STREAM, TILE64)}
    dw = {(DW, TILE256, False), (DW, TILE128, False), (DW, TILE128, True), (DW, TILE64, False)}
    assert {(p.mode, p.kernel, p.split > 1) for p in PATHS} == tiles | parts | dw
    # and the choice knows no others
    seen = set()
    for mode in (LINEAR, DX, DW):
        for E in (1, 2, 8, 60, 256, 1024):
            for K in (8, 128, 520, 2048, 7168):
                for N in (8, 128, 520, 2048, 7168):
                    for R in (0, 1, 8, 100, 1000, 4096, 32768, 131072):
                        kernel, split = plan(R, K, N, E, mode)
                        seen.add((mode, kernel, split > 1))
    assert seen <= tiles | parts | dw
