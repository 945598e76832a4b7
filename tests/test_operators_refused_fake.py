"""What the dense operators' Python calls refuse of tensors on a GPU, on the
host: tensors without storage stand for the GPU's."""
import os

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import sparse_gradient_reduction_amd as sg

if not os.path.exists(sg.LIB_PATH):
    pytest.skip("libsparcml.so not built", allow_module_level=True)


@pytest.fixture
def fake():
    with FakeTensorMode():
        yield lambda *shape, t=torch.float32, device="cuda:0": torch.empty(shape, dtype=t, device=device)


@pytest.mark.parametrize("wrong", ["host", "fp32", "gaps"])
def test_workspaces(fake, wrong):
    """A workspace that is not bytes on a GPU never reaches a kernel."""
    ws = {"host": lambda: fake(1 << 20, t=torch.uint8, device="cpu"), "fp32": lambda: fake(1 << 20),
          "gaps": lambda: fake(1 << 20, 2, t=torch.uint8)[:, 0]}[wrong]()
    x, v, r = fake(4, 8), fake(8), fake(4)
    for call in (lambda: sg.layer_norm_backward(x, x, v, r, r, workspace=ws),
                 lambda: sg.orthogonalize(v, [(0, 2, 4)], workspace=ws),
                 lambda: sg.orthogonal_step(v, v, [(0, 2, 4)], lr=0.1, workspace=ws)):
        with pytest.raises(TypeError, match="workspace"):
            call()


def test_rows_past_a_c_integer(fake):
    """2^32 + 8 columns are not 8."""
    long, r = fake(4, (1 << 32) + 8, t=torch.bfloat16), fake(4)
    with pytest.raises(ValueError, match="2\\^31"):
        sg.layer_norm(long)
    with pytest.raises(ValueError, match="2\\^31"):
        sg.layer_norm_backward(long, long, None, r, r)


@pytest.mark.parametrize("nodes", [65536, (1 << 32) + 1])
def test_nodes_past_the_limit(fake, nodes):
    x, r = fake(nodes, 1, t=torch.bfloat16), fake(nodes)
    with pytest.raises(ValueError, match="nodes"):
        sg.layer_norm_backward(x, x, None, r, r, nodes=nodes)


@pytest.mark.parametrize("wrong", [dict(steps=1 << 32), dict(steps=-1), dict(steps=65), dict(coefficients=(1.0, 2.0)),
                                   dict(coefficients=(1.0, 2.0, 3.0, 4.0))], ids=str)
def test_steps_and_coefficients(fake, wrong):
    v = fake(8)
    with pytest.raises(ValueError):
        sg.orthogonalize(v, [(0, 2, 4)], **wrong)
    with pytest.raises(ValueError):
        sg.orthogonal_step(v, v, [(0, 2, 4)], lr=0.1, **wrong)


def test_workspace_sizes_of_numbers_that_wrap():
    for nodes, rows, cols in (((1 << 32) + 1, 4, 8), (1, (1 << 64) + 4, 8), (1, 4, (1 << 32) + 8), (-1, 4, 8), (1, -4, 8)):
        with pytest.raises(ValueError):
            sg.layer_norm_backward_workspace_bytes(nodes, rows, cols)
    for N, matrices in (((1 << 64) + 8, [(0, 2, 4)]), (-1, []), (8, [(1 << 64, 2, 4)])):
        with pytest.raises(ValueError):
            sg.orthogonalize_workspace_bytes(N, matrices)
