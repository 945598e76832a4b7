"""Layer norm and its gradients against the formulas in 64 bits: types, odd
sizes, strides, rows that repeat, per-node gradients in the columns of the
[P, N] gradients, differences, graphs and streams."""
import pytest
import torch

import sparse_gradient_reduction_amd as sg
from tests.operator_util import (U, assert_within, half_step, layer_norm_backward_reference, layer_norm_reference)

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]


def _check_forward(x, residual, weight, bias, eps, got):
    y, mean, rstd, total, e_y, e_mean, e_rstd = layer_norm_reference(
        x.cpu(), None if residual is None else residual.cpu(), None if weight is None else weight.cpu(),
        None if bias is None else bias.cpu(), eps)
    t = x.dtype
    assert_within(got[1], mean, e_mean + U * mean.abs(), "mean")
    assert_within(got[2], rstd, e_rstd + U * rstd.abs(), "rstd")
    if total is not None:
        assert_within(got[3], total, half_step(t, total), "total")
    assert_within(got[0], y, e_y + half_step(t, y.abs() + e_y), "y")


SIZES = [(1, 1), (3, 2), (1, 7), (5, 16), (2, 63), (9, 64), (7, 65), (4, 255), (33, 256), (3, 1000), (5, 1537),
         (17, 1024), (2, 2048), (3, 4096), (2, 4097), (3, 8192), (2, 16384), (2, 16392), (1, 40001), (300, 24)]


@pytest.mark.parametrize("t", TYPES, ids=str)
@pytest.mark.parametrize("rows,cols", SIZES)
def test_forward(dev, rows, cols, t):
    g = torch.Generator(device=dev).manual_seed(rows * 31 + cols)
    x = (torch.randn(rows, cols, generator=g, device=dev) * 1.5 + 0.25).to(t)
    r = torch.randn(rows, cols, generator=g, device=dev).to(t)
    w = 1 + 0.1 * torch.randn(cols, generator=g, device=dev)
    b = 0.1 * torch.randn(cols, generator=g, device=dev)
    _check_forward(x, None, w, b, 1e-5, sg.layer_norm(x, w, b))
    _check_forward(x, r, w, b, 1e-5, sg.layer_norm(x, w, b, residual=r))
    _check_forward(x, r, None, None, 1e-3, sg.layer_norm(x, eps=1e-3, residual=r))
    _check_forward(x, None, w, None, 1e-5, sg.layer_norm(x, w))


@pytest.mark.parametrize("t", TYPES, ids=str)
@pytest.mark.parametrize("pad,shift", [(1, 0), (63, 0), (64, 0), (8, 8), (16, 3)])
def test_forward_of_slices(dev, t, pad, shift):
    """Rows that are slices of a wider buffer, aligned and not."""
    for rows, cols in ((37, 257), (16, 512), (5, 2048), (3, 5000)):
        wide = (torch.randn(rows, cols + pad + shift, device=dev) * 2 - 1).to(t)
        x = wide[:, shift: shift + cols]
        rw = torch.randn(rows, cols + pad, device=dev).to(t)
        w, b = torch.randn(cols, device=dev), torch.randn(cols + 1, device=dev)[1:].clone()
        _check_forward(x, None, w, b, 1e-5, sg.layer_norm(x, w, b))
        _check_forward(x, rw[:, :cols], w, b, 1e-5, sg.layer_norm(x, w, b, residual=rw[:, :cols]))


def test_forward_shapes(dev):
    """Leading dimensions, no rows, a row repeated, vectors off their 16-byte border."""
    x = torch.randn(2, 3, 4, 40, device=dev)
    y, mean, rstd = sg.layer_norm(x)
    assert y.shape == x.shape and mean.shape == rstd.shape == (2, 3, 4)
    _check_forward(x, None, None, None, 1e-5, (y, mean, rstd))
    _check_forward(x[:, :, 0], None, None, None, 1e-5, sg.layer_norm(x[:, :, 0]))
    one = torch.randn(1, 100, device=dev).expand(7, 100)
    _check_forward(one, None, None, None, 1e-5, sg.layer_norm(one))
    y, mean, rstd = sg.layer_norm(torch.empty(0, 32, device=dev))
    assert y.shape == (0, 32) and mean.shape == (0,)
    v = torch.randn(2, 4097, device=dev)[:, 1:]
    w, b = v[0].clone(), torch.randn(4100, device=dev)[3:4099]
    assert b.data_ptr() % 16
    _check_forward(v, None, w, b, 1e-5, sg.layer_norm(v, w, b))
    _check_forward(x[0, 0, 0], None, None, None, 1e-5, sg.layer_norm(x[0, 0, 0]))


@pytest.mark.parametrize("t", TYPES, ids=str)
def test_forward_values(dev, t):
    """A far mean, constant rows, an infinity or NaN in one row only."""
    x = torch.randn(6, 320, device=dev).to(t)
    x[1] = 3.0
    x[2] = (x[2].float() + 200).to(t)
    x[3] *= 1e-3
    _check_forward(x, None, None, None, 1e-5, sg.layer_norm(x))
    clean = sg.layer_norm(x)
    x[4, 7] = float("inf")
    x[5, 300] = float("nan")
    y, mean, rstd = sg.layer_norm(x)
    assert torch.equal(y[:4], clean[0][:4]) and torch.equal(mean[:4], clean[1][:4])
    assert torch.isnan(y[4:]).all() and torch.isnan(rstd[4:]).all()


def _backward_inputs(dev, nodes, rows, cols, t, seed):
    g = torch.Generator(device=dev).manual_seed(seed)
    x = (torch.randn(nodes, rows, cols, generator=g, device=dev) * 1.5 + 0.25).to(t)
    dy = torch.randn(nodes, rows, cols, generator=g, device=dev).to(t)
    dr = torch.randn(nodes, rows, cols, generator=g, device=dev).to(t)
    w = 1 + 0.1 * torch.randn(cols, generator=g, device=dev)
    _, mean, rstd = sg.layer_norm(x, w)
    return dy, x, w, mean, rstd, dr


def _check_backward(dy, x, w, mean, rstd, nodes, dr, got):
    dx, dw, db, e_dx, e_dw, e_db = layer_norm_backward_reference(
        dy.cpu(), x.cpu(), None if w is None else w.cpu(), mean.cpu(), rstd.cpu(), nodes,
        None if dr is None else dr.cpu())
    assert_within(got[0], dx, e_dx + half_step(x.dtype, dx.abs() + e_dx), "dx")
    assert_within(got[1], dw, e_dw, "dweight")
    assert_within(got[2], db, e_db, "dbias")


BACK = [(1, 1, 1), (2, 1, 3), (3, 5, 16), (1, 33, 63), (4, 16, 64), (2, 100, 65), (64, 3, 130), (5, 7, 256),
        (3, 41, 1000), (4, 16, 1024), (2, 9, 1537), (2, 300, 520), (8, 12, 4096), (1, 5, 8200), (1, 3, 16384),
        (1, 2, 33001), (1, 1500, 40), (2, 4096, 16)]


@pytest.mark.parametrize("t", TYPES, ids=str)
@pytest.mark.parametrize("nodes,rows,cols", BACK)
def test_backward(dev, nodes, rows, cols, t):
    dy, x, w, mean, rstd, dr = _backward_inputs(dev, nodes, rows, cols, t, cols * 7 + rows)
    _check_backward(dy, x, w, mean, rstd, nodes, None, sg.layer_norm_backward(dy, x, w, mean, rstd, nodes))
    _check_backward(dy, x, w, mean, rstd, nodes, dr,
                    sg.layer_norm_backward(dy, x, w, mean, rstd, nodes, dresidual=dr))
    _check_backward(dy, x, None, mean, rstd, nodes, None, sg.layer_norm_backward(dy, x, None, mean, rstd, nodes))


@pytest.mark.parametrize("t", TYPES, ids=str)
def test_backward_strides(dev, t):
    """Slices of wider rows, a gradient that is one row repeated, and no rows."""
    rows, cols = 50, 192
    wide = torch.randn(3, rows, cols + 13, device=dev).to(t)
    x, dy = wide[0, :, 5: 5 + cols], wide[1, :, :cols]
    _, mean, rstd = sg.layer_norm(x)
    _check_backward(dy, x, None, mean, rstd, 2, wide[2, :, 8: 8 + cols],
                    sg.layer_norm_backward(dy, x, None, mean, rstd, 2, dresidual=wide[2, :, 8: 8 + cols]))
    one = torch.randn(1, cols, device=dev).to(t).expand(rows, cols)
    _check_backward(one, x, None, mean, rstd, 5, None, sg.layer_norm_backward(one, x, None, mean, rstd, 5))
    e = torch.empty(0, 24, device=dev, dtype=t)
    none = torch.empty(0, device=dev)
    dx, dw, db = sg.layer_norm_backward(e, e, None, none, none, 3)
    assert dx.shape == (0, 24) and not dw.any() and not db.any() and dw.shape == (3, 24)


def test_backward_into_gradient_columns(dev):
    """dweight and dbias as columns of the [P, N] gradients; the other columns stay."""
    P, N, cols = 4, 1000, 96
    dy, x, w, mean, rstd, _ = _backward_inputs(dev, P, 30, cols, torch.bfloat16, 5)
    grad = torch.full((P, N), 7.0, device=dev)
    got = sg.layer_norm_backward(dy, x, w, mean, rstd, P, dweight=grad[:, 101:197], dbias=grad[:, 300:396])
    _check_backward(dy, x, w, mean, rstd, P, None, got)
    want = sg.layer_norm_backward(dy, x, w, mean, rstd, P)
    assert torch.equal(grad[:, 101:197], want[1]) and torch.equal(grad[:, 300:396], want[2])
    grad[:, 101:197] = 7
    grad[:, 300:396] = 7
    assert (grad == 7).all()


def test_backward_repeats_bit_for_bit(dev):
    dy, x, w, mean, rstd, dr = _backward_inputs(dev, 3, 700, 333, torch.float32, 6)
    a = sg.layer_norm_backward(dy, x, w, mean, rstd, 3, dresidual=dr)
    for _ in range(3):
        for u, v in zip(a, sg.layer_norm_backward(dy, x, w, mean, rstd, 3, dresidual=dr)):
            assert torch.equal(u, v)


def test_backward_against_differences(dev):
    """Directional derivatives of L = sum(c * y): (L(p + h d) - L(p - h d)) / 2h
    in 64 bits is the formula's to h^2 ~ 1e-8, and the kernel's to fp32."""
    rows, cols, h = 12, 48, 1e-4
    dy, x, w, mean, rstd, _ = _backward_inputs(dev, 1, rows, cols, torch.float32, 8)
    dx, dw, db = sg.layer_norm_backward(dy, x, w, mean, rstd)
    xc, wc, c = x.double().cpu()[0], w.double().cpu(), dy.double().cpu()[0]
    b = torch.zeros(cols, dtype=torch.float64)

    def loss(x_, w_, b_):
        m = x_.mean(-1, keepdim=True)
        v = (x_ - m).square().mean(-1, keepdim=True)
        return float((c * ((x_ - m) / (v + 1e-5).sqrt() * w_ + b_)).sum())

    g = torch.Generator().manual_seed(9)
    for got, at in ((dx[0], 0), (dw[0], 1), (db[0], 2)):
        base = [xc, wc, b]
        d = torch.randn(base[at].shape, generator=g, dtype=torch.float64)
        up, down = list(base), list(base)
        up[at], down[at] = base[at] + h * d, base[at] - h * d
        want = (loss(*up) - loss(*down)) / (2 * h)
        terms = (got.double().cpu() * d).abs().sum()
        assert abs(float((got.double().cpu() * d).sum()) - want) <= 1e-5 * float(terms) + 1e-6


def test_layer_norm_in_a_graph_and_on_a_stream(dev):
    """Captured with its own outputs and workspace; every replay follows new inputs. A side stream gives the same."""
    P, rows, cols = 2, 65, 1000
    t = torch.bfloat16
    dy, x, w, mean, rstd, dr = _backward_inputs(dev, P, rows, cols, t, 11)
    y, tot = torch.empty_like(x), torch.empty_like(x)
    dx, dw, db = torch.empty_like(x), torch.empty(P, cols, device=dev), torch.empty(P, cols, device=dev)
    ws = torch.empty(sg.layer_norm_backward_workspace_bytes(P, rows, cols), dtype=torch.uint8, device=dev)

    def step():
        sg.layer_norm(x, w, None, residual=dr, y=y, mean=mean, rstd=rstd, total=tot)
        sg.layer_norm_backward(dy, tot, w, mean, rstd, P, dx=dx, dweight=dw, dbias=db, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for k in range(3):
        x.copy_(torch.randn(P, rows, cols, device=dev).to(t))
        step()
        want = [v.clone() for v in (y, mean, rstd, tot, dx, dw, db)]
        for v in (y, mean, rstd, tot, dx, dw, db):
            v.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for u, v in zip(want, (y, mean, rstd, tot, dx, dw, db)):
            assert torch.equal(u, v), k
        (x.float() * 0.5).sum().item()
