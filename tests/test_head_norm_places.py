"""Where head_norm_rotate takes a tensor's tokens to be: those of an empty one are nowhere."""
import pytest
import torch

import sparse_gradient_reduction_amd as sg

EMPTY = [torch.empty(5, 0, 4, 64), torch.empty(0, 5, 4, 64), torch.empty(2, 6, 4, 64)[:0, :3], torch.empty(2, 0, 3, 4, 64),
         torch.empty(0, 4, 64), torch.empty(3, 6, 4, 64)[:, 6:]]


@pytest.mark.parametrize("x", EMPTY, ids=lambda x: "x".join(map(str, x.shape)))
def test_no_tokens(x):
    assert sg._token_heads(x, "q")[3] == 64


def test_evenly_spaced():
    x = torch.empty(2, 6, 4, 64)
    assert sg._token_heads(x, "q")[1:] == (0, 256, 64) and sg._token_heads(x[:1, :3], "q")[1:] == (0, 256, 64)
    assert sg._token_heads(x[:, 2:3], "q")[1:] == (0, 6 * 256, 64) and sg._token_heads(x[0, 0], "q")[3] == 64
    with pytest.raises(ValueError):
        sg._token_heads(x[:, :3], "q")


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(5, 0), (0, 5), (2, 0, 3), (0,)])
def test_no_tokens_on_the_gpu(shape):
    q, k = torch.empty(*shape, 4, 64, device="cuda"), torch.empty(*shape, 2, 64, device="cuda")
    positions, frequencies = torch.empty(0, dtype=torch.int32, device="cuda"), sg.rotation_frequencies(64, device="cuda")
    y = sg.head_norm_rotate(q, k, positions=positions, frequencies=frequencies)
    assert y[0].shape == q.shape and y[1].shape == k.shape
    dq, dk, dqw, dkw = sg.head_norm_rotate_backward(q, k, q, k, positions=positions, frequencies=frequencies, nodes=2)
    assert dq.shape == q.shape and dk.shape == k.shape and bool((dqw == 0).all()) and bool((dkw == 0).all())
