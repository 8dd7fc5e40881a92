"""Which kernel and how many parts of the reduction a product on 4-bit weights gets: the library's
own choice, called through its C++ symbol (not part of the C ABI), against the rule written out in
fp4_paths.py.  Nothing is launched."""
import ctypes
import random

import pytest

from fp4_paths import PATHS, STREAM, TILE128, TILE128_ONCE, TILE256, plan
from grouped_common import moe
from test_fp4_host import problem_of


class Plan(ctypes.Structure):
    _fields_ = [("kernel", ctypes.c_int), ("split", ctypes.c_int)]


def library_plan(R, K, N, E, eight, gated):
    f = moe().lib["_ZN3moe8fp4_planERK11moe_groupedbb"]
    f.restype, f.argtypes = Plan, [ctypes.c_void_p, ctypes.c_bool, ctypes.c_bool]
    p = f(ctypes.byref(moe().MoeGrouped(R, R, K, N, E)), eight, gated)
    return p.kernel, p.split


@pytest.mark.parametrize("i", range(len(PATHS)))
def test_paths_reach_their_kernel(i):
    four, eight, kw = PATHS[i]
    gated = kw.get("gated", False)
    assert library_plan(*problem_of(kw), False, gated) == four
    assert library_plan(*problem_of(kw), True, gated) == eight


def test_paths_reach_every_kernel():
    for x in (0, 1):
        got = {(p[x][0], p[x][1] > 1) for p in PATHS}
        assert got == {(STREAM, False), (TILE256, False), (TILE128, False), (TILE128, True),
                       (TILE128_ONCE, False)}


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("gated", [False, True])
def test_the_rule_is_the_librarys(eight, gated):
    """Random sizes, and both sides of each of the rule's comparisons."""
    rng, seen = random.Random(7), set()
    big = 128 if eight else 256
    log = lambda lo, hi: int(round(lo * (hi / lo) ** rng.random()))  # noqa: E731
    for _ in range(4000):
        E = rng.choice([1, 1, log(2, 1024), log(2, 1024)])
        K, N = 32 * log(1, 512), 8 * log(1, 2048)
        per = rng.choice([0, 4, 5, 16, 17, 7 * big // 16, 7 * big // 16 + 1, 3 * big // 8,
                          3 * big // 8 + 1, log(1, 4096)])
        R = max(0, per * E + rng.choice([0, -1, 1, rng.randrange(E)]))
        if rng.random() < 0.5:  # N where the tiles reach 192 or 256
            bn, bm, most = rng.choice([(256, big, 192), (128, big // 2, 256)])
            mt = max(min(E, max(R, 1)), R // bm + (min(E, max(R, 1)) // 2 if E > 1 else 1))
            edge = -(-most // mt) * (bn // 2 if gated else bn)
            N = min(1 << 20, max(8, edge - (bn // 2 if gated else bn) + rng.choice([0, 8, -8])))
        want = plan(R, K, N, E, eight, gated)
        assert library_plan(R, K, N, E, eight, gated) == want, (R, K, N, E)
        seen.add((want[0], want[1] > 1))
    assert len(seen) == 5
