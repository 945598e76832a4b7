"""Orthogonalised updates of a matrix with a NaN or an infinity, of every kind
of matrix: it becomes NaN whole, and its neighbours stay as they are. And how
large the iterates may get."""
import pytest
import torch

import sparse_gradient_reduction_amd as sg
from tests.operator_util import newton_schulz_tolerance

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("steps", [0, 1, 2, 5])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")], ids=str)
@pytest.mark.parametrize("rows,cols", [(1, 1), (7, 5), (20, 30), (30, 20), (64, 576), (100, 300), (300, 100), (257, 300)])
def test_matrix_becomes_nan(dev, rows, cols, value, steps):
    size = rows * cols
    where = [(k * size, rows, cols) for k in range(3)]
    u = torch.randn(3 * size, generator=torch.Generator().manual_seed(size)).to(dev)
    bad = u.clone()
    bad[size + size // 2] = value
    want = sg.orthogonalize(u, where, steps=steps)
    got = sg.orthogonalize(bad, where, steps=steps)
    assert torch.isnan(got[size: 2 * size]).all()
    assert torch.equal(got[:size], want[:size]) and torch.equal(got[2 * size:], want[2 * size:])
    weight = torch.ones(3 * size, device=dev)
    sg.orthogonal_step(weight, bad, where, lr=0.1, steps=steps)
    assert torch.isnan(weight[size: 2 * size]).all()
    assert not torch.isnan(weight[:size]).any() and not torch.isnan(weight[2 * size:]).any()


@pytest.mark.parametrize("rows,cols,a,steps", [(1, 1, 3.9, 2), (1, 9, 3.9, 2), (1, 1, 250.0, 1), (60, 90, 15.0, 2),
                                               (200, 300, 30.0, 2), (300, 200, 30.0, 2)])
def test_room_of_the_iterates(dev, rows, cols, a, steps):
    """X <- a X: right while rows of X have norms below 4 after all steps but
    the last, not finite after two more steps (a row of a random matrix of 200
    rows starts with a norm of about 200^-1/2)."""
    u = torch.randn(rows * cols, generator=torch.Generator().manual_seed(rows))
    co = (a, 0.0, 0.0)
    ref, tol = newton_schulz_tolerance(u.view(rows, cols), torch.float32, steps, coefficients=co)
    wide = ref if rows <= cols else ref.t()
    assert (wide / a).norm(dim=1).max() < 4 < wide.norm(dim=1).max()
    got = sg.orthogonalize(u.to(dev), [(0, rows, cols)], steps=steps, coefficients=co).double().cpu().view(rows, cols)
    assert float((got - ref).norm()) <= tol
    over = sg.orthogonalize(u.to(dev), [(0, rows, cols)], steps=steps + 2, coefficients=co)
    assert not torch.isfinite(over).any()
