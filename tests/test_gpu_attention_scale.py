"""Attention and its gradients at the smallest and largest scales that it takes."""
import math

import pytest
import torch

import sparse_gradient_reduction_amd as sg
from tests.test_gpu_attention import check_backward, check_forward, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("scale", [1e-30, 1e30])
def test_scores_of_ordinary_size(t, scale):
    """q and k make up for the scale."""
    q, k, v, dout = make(t, 1, 70, 90, 4, 2, 64, seed=41)
    by = math.sqrt(1 / scale / 8)
    q, k = (q.float() * by).to(t), (k.float() * by).to(t)
    gq, gk, gv, gd = (x.cuda() for x in (q, k, v, dout))
    out, lse = sg.attention(gq, gk, gv, causal=True, scale=scale)
    check_forward((out, lse), q, k, v, causal=True, scale=scale)
    got = sg.attention_backward(gd, gq, gk, gv, out, lse, causal=True, scale=scale)
    check_backward(got, dout, q, k, v, out, lse, causal=True, scale=scale)


@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("scale", [1e-30, 1e30])
def test_one_key(t, scale):
    """Its probability is 1 and ds is 0, with whole numbers exactly so; with fp16,
    dout and v are as large as their sums over a head allow."""
    gen = torch.Generator().manual_seed(42)
    q, k = torch.zeros(2, 33, 2, 64, dtype=t, device="cuda"), torch.ones(2, 1, 2, 64, dtype=t, device="cuda")
    v = (1024 * torch.randint(-7, 8, (2, 1, 2, 64), generator=gen)).to(t).cuda()
    dout = (1024 * torch.randint(-7, 8, (2, 33, 2, 64), generator=gen)).to(t).cuda()
    out, lse = sg.attention(q, k, v, scale=scale)
    assert torch.equal(out, v.expand_as(out)) and bool((lse == 0).all())
    dq, dk, dv = sg.attention_backward(dout, q, k, v, out, lse, scale=scale)
    assert bool((dq == 0).all()) and bool((dk == 0).all())
    assert torch.equal(dv, dout.double().sum(1, keepdim=True).to(t))
