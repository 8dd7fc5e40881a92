"""Host-side checks of the grouped linear entry points: shapes, pointers, aliasing and
workspaces are refused before anything is enqueued.  No kernel is launched here."""
import copy
import ctypes
import pickle

import pytest
import torch

from grouped_common import fake, moe


def call(m, name, p, *args):
    c = p.c()
    return getattr(m.lib, name)(ctypes.byref(c), *args)


@pytest.mark.parametrize("kw,status", [
    (dict(), 0), (dict(R=0), 0), (dict(T=0), 0), (dict(E=1024), 0), (dict(K=8, N=8), 0),
    (dict(R=-1), 1), (dict(T=-1), 1), (dict(K=0), 1), (dict(N=0), 1), (dict(E=0), 1),
    (dict(E=1025), 2), (dict(K=12), 2), (dict(N=4), 2), (dict(K=(1 << 20) + 8), 2),
    (dict(R=(1 << 30) + 1), 2), (dict(R=1 << 30, N=1 << 20), 2),
    (dict(E=1024, K=1 << 20, N=1 << 20), 2),
])
def test_grouped_check(kw, status):
    base = dict(R=64, K=128, N=64, E=4, T=32)
    base.update(kw)
    assert moe().GroupedProblem(**base).check() == status


def test_null_problem_and_unknown_op():
    m = moe()
    assert m.lib.moe_grouped_check(None) == m.MOE_ERR_INVALID_ARG
    p = m.GroupedProblem(64, 128, 64)
    for op in (-1, 3):
        assert p.workspace_bytes(op) == 0
    assert m.GroupedProblem(64, 12, 64).workspace_bytes(m.OP_GROUPED_DW) == 0


def ws_args(m, p, op, f):
    n = p.workspace_bytes(op)
    return (f, n) if n else (None, 0)


def test_linear_refusals():
    m = moe()
    p = m.GroupedProblem(R=64, K=128, N=96, E=4, T=32)
    x, rt, off, w, b, res, y, zc, zs, ws = fake(10)
    W = ws_args(m, p, m.OP_GROUPED_LINEAR, ws)

    def go(p=p, x=x, rt=rt, off=off, w=w, b=b, act=3, res=res, y=y, zc=zc, zs=zs, ws=W):
        return call(m, "moe_grouped_linear", p, x, rt, off, w, b, act, res, y, zc, zs, *ws, None)

    off8 = ctypes.c_void_p(x.value + 8)
    inv, uns = m.MOE_ERR_INVALID_ARG, m.MOE_ERR_UNSUPPORTED
    for kw in (dict(x=None), dict(w=None), dict(y=None), dict(act=5), dict(act=-1),
               dict(zs=None), dict(zc=None), dict(off=None), dict(x=off8), dict(w=off8),
               dict(b=off8), dict(res=off8), dict(y=off8), dict(zc=off8),
               dict(y=x), dict(y=w), dict(y=res), dict(y=zc), dict(zc=x), dict(zs=off),
               dict(y=ctypes.c_void_p(rt.value))):
        assert go(**kw) == inv, kw
    assert go(p=m.GroupedProblem(64, 128, 96, 4, 0)) == inv  # rows of no tokens
    assert go(p=m.GroupedProblem(64, 128, 72, 4, 32)) == uns  # a checkpoint of 72 columns
    assert go(p=m.GroupedProblem(64, 12, 96, 4, 32)) == uns
    # no rows: nothing to do, nothing enqueued
    assert go(p=m.GroupedProblem(0, 128, 96, 4, 32), ws=(None, 0)) == m.MOE_OK


def test_dx_refusals():
    m = moe()
    p = m.GroupedProblem(R=64, K=96, N=128, E=4)
    dz, off, w, zc, zs, dx, a, ws = fake(8)
    W = ws_args(m, p, m.OP_GROUPED_DX, ws)

    def go(p=p, dz=dz, off=off, w=w, act=3, zc=zc, zs=zs, dx=dx, a=a, ws=W):
        return call(m, "moe_grouped_linear_dx", p, dz, off, w, act, zc, zs, dx, a, *ws, None)

    off8 = ctypes.c_void_p(dz.value + 8)
    inv, uns = m.MOE_ERR_INVALID_ARG, m.MOE_ERR_UNSUPPORTED
    for kw in (dict(dz=None), dict(w=None), dict(dx=None), dict(act=9), dict(zs=None),
               dict(zc=None, zs=None), dict(zc=None, zs=None, act=0), dict(zc=None, zs=None, a=None),
               dict(off=None), dict(dz=off8), dict(w=off8), dict(zc=off8), dict(dx=off8),
               dict(a=off8), dict(dx=dz), dict(a=dx), dict(a=zc), dict(dx=w)):
        assert go(**kw) == inv, kw
    assert go(p=m.GroupedProblem(64, 72, 128, 4)) == uns
    assert go(p=m.GroupedProblem(0, 96, 128, 4), ws=(None, 0)) == m.MOE_OK


def test_dw_refusals():
    m = moe()
    p = m.GroupedProblem(R=64, K=96, N=128, E=4, T=16)
    x, rt, dz, off, dw, db, ws = fake(7)
    W = ws_args(m, p, m.OP_GROUPED_DW, ws)

    def go(p=p, x=x, rt=rt, dz=dz, off=off, acc=0, dw=dw, db=db, ws=W):
        return call(m, "moe_grouped_linear_dw", p, x, rt, dz, off, acc, dw, db, *ws, None)

    off8 = ctypes.c_void_p(x.value + 8)
    inv = m.MOE_ERR_INVALID_ARG
    for kw in (dict(x=None), dict(dz=None), dict(dw=None), dict(acc=2), dict(acc=-1),
               dict(off=None), dict(x=off8), dict(dz=off8), dict(dw=off8), dict(db=off8),
               dict(dw=x), dict(db=dz), dict(db=dw), dict(dw=rt)):
        assert go(**kw) == inv, kw
    assert go(p=m.GroupedProblem(64, 96, 128, 4, 0)) == inv  # rows of no tokens


def test_activation_backward_refusals():
    m = moe()
    dy, zc, zs, dz, a, live = fake(6)

    def go(rows=64, cols=96, live=live, act=3, dy=dy, zc=zc, zs=zs, dz=dz, a=a):
        return m.lib.moe_activation_backward(rows, cols, live, act, dy, zc, zs, dz, a, None)

    off8 = ctypes.c_void_p(dy.value + 8)
    for kw in (dict(rows=-1), dict(rows=1 << 39), dict(cols=0), dict(cols=-32), dict(cols=48), dict(act=5), dict(dy=None),
               dict(zc=None), dict(zs=None), dict(dz=None), dict(dy=off8), dict(zc=off8),
               dict(dz=off8), dict(a=off8), dict(dz=dy), dict(a=dz), dict(a=zc), dict(dz=live)):
        assert go(**kw) == m.MOE_ERR_INVALID_ARG, kw
    assert go(rows=0) == m.MOE_OK


@pytest.mark.parametrize("op", [0, 1, 2])
def test_workspace_is_checked(op):
    """Wherever an operator splits a reduction, a missing, short or misaligned workspace is
    refused."""
    m = moe()
    p = m.GroupedProblem(R=4096 if op == 2 else 16, K=256, N=256)
    if op != 2:
        p = m.GroupedProblem(R=16, K=4096, N=4096)
    need = p.workspace_bytes(op)
    if need == 0:
        pytest.skip("no split at this shape")
    f = fake(8)
    name, args = {
        0: ("moe_grouped_linear", (f[0], None, None, f[1], None, 0, None, f[2], None, None)),
        1: ("moe_grouped_linear_dx", (f[0], None, f[1], 0, None, None, f[2], None)),
        2: ("moe_grouped_linear_dw", (f[0], None, f[1], None, 0, f[2], None)),
    }[op]
    assert call(m, name, p, *args, None, 0, None) == m.MOE_ERR_WORKSPACE
    assert call(m, name, p, *args, f[7], need - 1, None) == m.MOE_ERR_WORKSPACE
    assert call(m, name, p, *args, ctypes.c_void_p(f[7].value + 16), need, None) == \
        m.MOE_ERR_INVALID_ARG
    assert call(m, name, p, *args, f[0], need, None) == m.MOE_ERR_INVALID_ARG  # aliases x


def test_python_refusals():
    m = moe()
    p = m.GroupedProblem(R=4, K=64, N=64, E=2)
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.zeros(2, 64, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="on the GPU"):
        m.grouped_linear(p, x, w, torch.tensor([0, 2, 4], dtype=torch.int32))
    with pytest.raises(ValueError, match="2-D"):
        m.activation_backward(x[0], (None, None), "silu")
    with pytest.raises(ValueError, match="multiple of 32"):
        m.checkpoint_buffers(4, 40, device="cpu")
    with pytest.raises(ValueError, match="unknown activation"):
        m._act("gelu")


def test_activation_backward_size_limit():
    """rows * cols up to 2^39 is taken, one row more is refused; the stand-in pointers lie so far
    apart that only the size can be the reason."""
    m = moe()
    dy, zc, zs, dz = fake(4, base=1 << 45)
    far = [ctypes.c_void_p(p.value + (i << 43)) for i, p in enumerate((dy, zc, zs, dz))]
    for cols in (32, 4096):
        rows = (1 << 39) // cols + 1
        st = m.lib.moe_activation_backward(rows, cols, None, 3, *far, None, None)
        assert st == m.MOE_ERR_INVALID_ARG


def test_problem_can_be_copied_and_pickled():
    """As Problem can: a program's configuration goes to worker processes and into checkpoints."""
    m = moe()
    for p in (m.GroupedProblem(64, 128, 96, 4, 32), m.GroupedProblem(R=16, K=4096, N=4096)):
        need = [p.workspace_bytes(op) for op in range(3)]  # derived state is there
        for q in (pickle.loads(pickle.dumps(p)), copy.copy(p), copy.deepcopy(p)):
            assert q == p and hash(q) == hash(p) and q.T == p.T
            assert q.check() == m.MOE_OK
            assert [q.workspace_bytes(op) for op in range(3)] == need
            assert (q.c().R, q.c().T, q.c().K, q.c().N, q.c().E) == \
                (p.R, p.x_tokens, p.K, p.N, p.E)
            assert q._c is not p._c and q._ws_bytes is not p._ws_bytes
