"""Which kernel and how many parts of the reduction a grouped call gets: the library's own
choice, called through its C++ symbols (not part of the C ABI).  Nothing is launched."""
import ctypes

import pytest

from grouped_common import moe

STREAM, TILE256, TILE128, TILE64, TILE128_ONCE = range(5)
LINEAR, DX, DW = range(3)


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
