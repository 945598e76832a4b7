"""Orthogonalised updates of a matrix with a NaN or an infinity, of every kind
of matrix: it becomes NaN whole, and its neighbours stay as they are."""
import pytest
import torch

import sparse_gradient_reduction_amd as sg

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
