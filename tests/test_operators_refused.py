"""What the dense operators' calls refuse, on the host: the C calls before
anything is launched, the Python calls by their checks."""
import ctypes
import math

import pytest
import torch

import sparse_gradient_reduction_amd as sg

import os
if not os.path.exists(sg.LIB_PATH):
    pytest.skip("libsparcml.so not built", allow_module_level=True)

A = ctypes.c_void_p(4096)      # never dereferenced
ODD = ctypes.c_void_p(4097)
HALF = ctypes.c_void_p(4098)   # a 16-bit element's border, not an fp32's
BAD, OK, WS = sg.ERR_INVALID_ARG, sg.OK, sg.ERR_WORKSPACE


def test_layer_norm_refuses():
    f = sg.lib().sparcml_layer_norm

    def call(type=1, rows=4, cols=8, x=A, xs=8, r=None, rs=0, w=A, b=A, eps=1e-5, y=A, tot=None, mean=A, rstd=A):
        return f(type, rows, cols, x, xs, r, rs, w, b, eps, y, tot, mean, rstd, None)

    for bad in (dict(type=3), dict(cols=0), dict(cols=1 << 31), dict(rows=1 << 40), dict(rows=1 << 38, cols=8),
                dict(eps=-1e-6), dict(eps=math.nan), dict(eps=math.inf), dict(x=None), dict(y=None), dict(mean=None),
                dict(rstd=None), dict(r=A), dict(tot=A), dict(x=ODD), dict(type=0, x=HALF), dict(type=0, y=HALF),
                dict(w=HALF), dict(b=HALF), dict(mean=HALF), dict(r=ODD, tot=A), dict(r=A, tot=ODD)):
        assert call(**bad) == BAD, bad
    assert call(rows=0, x=None, y=None, mean=None, rstd=None) == OK


def test_layer_norm_backward_refuses():
    L = sg.lib()
    need = L.sparcml_layer_norm_backward_workspace(2, 4, 8)
    assert need > 0
    assert L.sparcml_layer_norm_backward_workspace(0, 4, 8) == 0
    assert L.sparcml_layer_norm_backward_workspace(2, 1 << 40, 8) == 0
    assert L.sparcml_layer_norm_backward_workspace(65535, 1 << 26, 1 << 30) == 0

    def call(type=2, nodes=2, rows=4, cols=8, dy=A, x=A, r=None, w=A, mean=A, rstd=A, dx=A, dw=A, dws=8, db=A, dbs=8,
             ws=A, n=need):
        return L.sparcml_layer_norm_backward(type, nodes, rows, cols, dy, 8, x, 8, r, 8, w, mean, rstd, dx, dw, dws,
                                             db, dbs, ws, n, None)

    for bad in (dict(type=9), dict(nodes=0), dict(nodes=65536), dict(cols=0), dict(rows=1 << 39), dict(dy=None),
                dict(x=None), dict(dx=None), dict(mean=None), dict(rstd=None), dict(dy=ODD), dict(x=ODD), dict(dx=ODD),
                dict(r=ODD), dict(w=HALF), dict(dw=HALF), dict(db=HALF), dict(dws=7), dict(dbs=7)):
        assert call(**bad) == BAD, bad
    for bad in (dict(ws=None), dict(ws=ctypes.c_void_p(4096 + 128)), dict(n=need - 1)):
        assert call(**bad) == WS, bad


def test_momentum_refuses():
    f = sg.lib().sparcml_momentum_step

    def call(N=100, res=A, idx=A, cap=10, val=A, m=A, t=1, u=A):
        return f(N, res, idx, cap, val, m, 0.9, 1.0, 0, t, u, None)

    for bad in (dict(N=0), dict(N=1 << 32), dict(t=3), dict(res=None), dict(res=ctypes.c_void_p(4100)), dict(idx=None),
                dict(val=None), dict(val=HALF), dict(m=None), dict(m=HALF), dict(idx=HALF), dict(u=ODD),
                dict(t=0, u=HALF)):
        assert call(**bad) == BAD, bad


def _ms(ms):
    n = len(ms)
    return (n, (ctypes.c_uint64 * n)(*[m[0] for m in ms]), (ctypes.c_uint32 * n)(*[m[1] for m in ms]),
            (ctypes.c_uint32 * n)(*[m[2] for m in ms]))


def test_orthogonalize_refuses():
    L = sg.lib()
    good = [(0, 4, 8), (32, 8, 8)]
    need = L.sparcml_orthogonalize_workspace(96, *_ms(good))
    assert need > 0
    for ms, N in ((good, 95), ([(0, 4, 8), (31, 8, 8)], 96), ([(32, 8, 8), (0, 4, 8)], 96),
                  ([(0, 65537, 65537)], (1 << 40) - 1), ([(0, 1, (1 << 21) + 1)], 1 << 30), ([(97, 0, 0)], 96),
                  ([(0, 1 << 16, (1 << 16) + 1)], 1 << 39), ([(0, 1, 1)], 1 << 40),
                  ([(k << 21, 1, 1 << 21) for k in range(512)], 1 << 30)):
        assert L.sparcml_orthogonalize_workspace(N, *_ms(ms)) == 0, ms[:3]
        assert L.sparcml_orthogonalize(N, *_ms(ms), 5, 1, 1, 1, 0, 0, A, 0, A, A, 1 << 40, None) == BAD
    assert L.sparcml_orthogonalize_workspace(96, 2, None, None, None) == 0

    def call(steps=5, a=1.0, eps=1e-7, t=0, u=A, ot=0, o=A, ws=A, n=need):
        return L.sparcml_orthogonalize(96, *_ms(good), steps, a, 1.0, 1.0, eps, t, u, ot, o, ws, n, None)

    def step(lr=0.1, decay=0.0, w=A, wt=1):
        return L.sparcml_orthogonal_step(96, *_ms(good), 5, 1.0, 1.0, 1.0, 1e-7, 0, A, wt, w, lr, decay, A, need, None)

    for bad in (dict(steps=65), dict(a=math.nan), dict(a=math.inf), dict(eps=-1.0), dict(eps=math.nan), dict(t=3),
                dict(ot=3), dict(u=None), dict(o=None), dict(u=HALF), dict(ot=1, o=ODD)):
        assert call(**bad) == BAD, bad
    for bad in (dict(lr=math.nan), dict(lr=1e300), dict(lr=1.0, decay=math.inf), dict(w=None), dict(wt=0, w=HALF)):
        assert step(**bad) == BAD, bad
    for bad in (dict(ws=None), dict(ws=ctypes.c_void_p(4096 + 128)), dict(n=need - 1)):
        assert call(**bad) == WS, bad
    empty = _ms([])
    assert L.sparcml_orthogonalize(96, *empty, 5, 1, 1, 1, 0, 0, None, 0, None, None, 0, None) == OK


def test_workspace_grows_with_the_matrices():
    L = sg.lib()
    one = L.sparcml_orthogonalize_workspace(1 << 20, *_ms([(0, 100, 200)]))
    two = L.sparcml_orthogonalize_workspace(1 << 20, *_ms([(0, 100, 200), (30000, 100, 200)]))
    assert one < two < 2 * one + 4096 and sg.orthogonalize_workspace_bytes(1 << 20, [(0, 100, 200)]) == one


def test_python_checks():
    """No GPU tensor is needed to be refused: host tensors and wrong types are."""
    x = torch.zeros(4, 8)
    v = torch.zeros(8)
    with pytest.raises(TypeError):
        sg.layer_norm(x, v, v)
    with pytest.raises(TypeError):
        sg.layer_norm(torch.zeros(4, 8, dtype=torch.float64))
    with pytest.raises(TypeError):
        sg.layer_norm(torch.tensor(1.0))
    with pytest.raises(TypeError):
        sg.layer_norm_backward(x, x, v, torch.zeros(4), torch.zeros(4))
    with pytest.raises(TypeError):
        sg.momentum_step(sg.ReduceOutput(torch.zeros(16, dtype=torch.uint8), v, v, 8), v, 0.9)
    with pytest.raises(TypeError):
        sg.orthogonalize(v, [(0, 2, 4)])
    with pytest.raises(TypeError):
        sg.orthogonal_step(v, v, [(0, 2, 4)], lr=0.1)


@pytest.mark.parametrize("wrong", [(-1, 2, 4), (0, -2, 4), (0, 2, 1 << 32), (0, (1 << 32) + 2, 4)])
def test_matrices_out_of_range(wrong):
    """Numbers that a C integer would wrap are refused before the call."""
    with pytest.raises(ValueError):
        sg.orthogonalize_workspace_bytes(1 << 20, [wrong])


@pytest.mark.gpu
def test_python_checks_on_the_gpu(dev):
    x = torch.zeros(4, 8, device=dev)
    v = torch.zeros(8, device=dev)
    r = torch.zeros(4, device=dev)
    for wrong, kw in ((ValueError, dict(x=x.t())), (ValueError, dict(weight=r)), (TypeError, dict(bias=v.double())),
                      (TypeError, dict(residual=x.bfloat16())), (TypeError, dict(residual=x[:2])),
                      (TypeError, dict(y=x.half())), (ValueError, dict(mean=v)), (ValueError, dict(total=x)),
                      (ValueError, dict(x=torch.zeros(3, 4, 16, device=dev)[:, :3, :8].transpose(0, 1)))):
        with pytest.raises(wrong):
            sg.layer_norm(**{"x": x, **kw})
    with pytest.raises(sg.SparcmlError):
        sg.layer_norm(x, eps=-1.0)
    for wrong, kw in ((ValueError, dict(nodes=3)), (ValueError, dict(nodes=0)), (ValueError, dict(mean=v)),
                      (ValueError, dict(dweight=torch.zeros(2, 8, device=dev))), (TypeError, dict(dy=x[:2])),
                      (ValueError, dict(dbias=torch.zeros(1, 16, device=dev)[:, ::2])),
                      (TypeError, dict(dweight=torch.zeros(1, 8, device=dev).half()))):
        with pytest.raises(wrong):
            sg.layer_norm_backward(**{"dy": x, "x": x, "weight": v, "mean": r, "rstd": r, **kw})
    red = sg.ReduceOutput(torch.zeros(16, dtype=torch.uint8, device=dev), torch.zeros(1, dtype=torch.int32, device=dev), v, 8)
    with pytest.raises(ValueError):
        sg.momentum_step(red, r, 0.9)
    with pytest.raises(ValueError):
        sg.momentum_step(red, v, 0.9, update=r)
    with pytest.raises(TypeError):
        sg.momentum_step(red, v, 0.9, dtype=torch.int32)
    with pytest.raises(sg.SparcmlError):
        sg.orthogonalize(v, [(0, 3, 4)])
    with pytest.raises(ValueError):
        sg.orthogonalize(v, [(0, 2, 4)], out=r)
    with pytest.raises(ValueError):
        sg.orthogonal_step(r, v, [(0, 2, 4)], lr=0.1)
