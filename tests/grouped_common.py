"""Shared by the tests of the grouped linear products."""
import ctypes


def moe():
    import expert_ffn_moe_amd

    return expert_ffn_moe_amd


def fake(n, base=1 << 44):
    """n distinct aligned stand-ins for device pointers, far apart (see tests/test_abi.py);
    only for calls that return before launching anything."""
    return [ctypes.c_void_p(base + (i << 40)) for i in range(n)]


# Tolerances.  A sum of n products of bf16 values in fp32 (each product exact), in any order
# and split, is off by at most 2 n 2^-24 sum|a||b| (twice the standard bound: the matrix
# cores' own alignment of the addends is not documented).  A stored bf16 value is off by half
# a step more, 2^-8 of itself.
U24 = 2.0 ** -24
BF16_HALF = 2.0 ** -8


def sum_tol(n, abs_sum):
    return 2 * (n + 4) * U24 * abs_sum


def sigmoid_arg(z, act):
    """|argument| of the sigmoid inside the activation (0 where it has none)."""
    if act == "silu":
        return z.abs()
    if act == "gelu_tanh":
        return 1.5957691216057308 * (z.abs() + 0.044715 * z.abs() ** 3)
    return 0 * z


def flushed(z, act):
    """A sigmoid below the normal range, 2^-126, may be zero: that times the factors it has in
    act and act', z (and gelu's argument's slope, 2 r (1 + 3 c z^2))."""
    if act not in ("silu", "gelu_tanh"):
        return 0 * z
    return 2.0 ** -126 * (2 + z.abs() * (1.6 + 0.22 * z * z))


def act_tol(z, f, dz_tol, act):
    """Bound of act's error at z known up to dz_tol: its slope (at most 1.13 for silu and gelu,
    2 |z| for relu2) times dz_tol, and its own evaluation: the argument of exp is off by
    3 * 2^-23 of itself, which is the relative error that exp makes of it, and the ten
    roundings around it."""
    slope = 2 * (z.abs() + dz_tol) if act == "relu2" else 1.13
    return (slope * dz_tol + (3 * sigmoid_arg(z, act) + 16) * 2.0 ** -23 * f.abs() +
            flushed(z, act))


def dact_tol(z, df, act):
    """Bound of act'(z)'s evaluation error at an exact z: as act_tol; the terms of act' are at
    most |act'| + |z| + 1 in size."""
    if act in ("none", "relu"):
        return 0 * df
    big = df.abs() + 1 + z.abs() * (1 if act == "silu" else 0)
    if act == "gelu_tanh":  # the second term: z s (1 - s) 2 r (1 + 3 c z^2), bounded by 1.1
        big = df.abs() + 2.2
    return (3 * sigmoid_arg(z, act) + 32) * 2.0 ** -23 * big + flushed(z, act)


def stored(ref, tol):
    """Tolerance of a bf16 value whose unrounded error is at most tol (2^-133: the smallest
    step below the normal range)."""
    return tol + BF16_HALF * (ref.abs() + tol) + 2.0 ** -133
