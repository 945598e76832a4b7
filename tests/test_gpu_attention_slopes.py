"""Attention's gradients against the change of sum(out * dout) in 64 bits, along
directions in which a gradient that is 0, turned round or a quarter off fails for
every type."""
import math

import pytest
import torch

import sparse_gradient_reduction_amd as sg
from tests import attention_util as au
from tests.test_gpu_attention import make

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]
# queries, keys, heads, groups, D, causal, window
CASES = [(40, 60, 4, 2, 32, True, None), (33, 33, 2, 2, 64, False, 9), (70, 45, 3, 1, 80, True, None), (5, 1100, 2, 1, 128, False, None)]


def loss(q, k, v, dout, causal, window, scale):
    total = 0.0
    for _, h, g, _, _, see in au._each(q, k, None, causal, window):
        s = torch.where(see, scale * q[0, :, h] @ k[0, :, g].t(), -math.inf)
        some = see.any(1, keepdim=True)
        p = torch.where(see, torch.softmax(torch.where(some, s, 0.0), 1), 0.0)
        total += float((p @ v[0, :, g] * dout[0, :, h]).sum())
    return total


def shifts(q, k, v, dout, out, e_out, e_lse, way, causal, window, scale):
    """How far <dq, way> and <dk, way> may be off because out and lse are: a row's
    delta by |dout| e_out, its probabilities by e_lse of their value."""
    by_q = by_k = 0.0
    for _, h, g, _, _, see in au._each(q, k, None, causal, window):
        x, y, z, d = q[0, :, h], k[0, :, g], v[0, :, g], dout[0, :, h]
        s = torch.where(see, scale * x @ y.t(), -math.inf)
        p = torch.where(see, torch.exp(s - torch.where(see.any(1), torch.logsumexp(s, 1), 0.0)[:, None]), 0.0)
        e_delta, gap = (d.abs() * e_out[0, :, h]).sum(1), (d @ z.t() - (d * out[0, :, h]).sum(1, keepdim=True)).abs()
        e_p = p * gap * e_lse[0, h][:, None]
        if way.shape == q.shape:
            w = y @ way[0, :, h].t()  # [keys, queries]
            by_q += float(scale * ((p * w.t()).sum(1).abs() * e_delta).sum() + scale * (e_p * w.t().abs()).sum())
        if way.shape == k.shape:
            w = x @ way[0, :, g].t()  # [queries, keys]
            by_k += float(scale * ((p * w).sum(1).abs() * e_delta).sum() + scale * (e_p * w.abs()).sum())
    return by_q, by_k


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("case", CASES)
def test_slopes_along_the_gradients(t, case):
    """The directions are the 64-bit gradient's own, whole and of every third row,
    so that the slope is as large as it can be beside the gradients' roundings."""
    queries, keys, heads, groups, dim, causal, window = case
    scale = dim ** -0.5
    q, k, v, dout = make(t, 1, queries, keys, heads, groups, dim, seed=13)
    mask = {"causal": causal, "window": window, "scale": scale}
    gq, gk, gv, gd = (x.cuda() for x in (q, k, v, dout))
    out, lse = sg.attention(gq, gk, gv, **mask)
    got = sg.attention_backward(gd, gq, gk, gv, out, lse, **mask)
    compare([x.cpu() for x in got], q, k, v, dout, out.cpu(), lse.cpu(), causal, window, scale)


def compare(got, q, k, v, dout, out, lse, causal, window, scale):
    tols = au.backward(dout, q, k, v, out, lse, causal=causal, window=window, scale=scale)
    _, _, e_out, e_lse = au.forward(q, k, v, causal=causal, window=window, scale=scale)
    start, d64 = [x.double() for x in (q, k, v)], dout.double()
    for which, name in enumerate(("dq", "dk", "dv")):
        for part in (slice(None), slice(0, None, 3), slice(1, None, 3), slice(2, None, 3)):
            way = torch.zeros_like(start[which])
            way[:, part] = tols[which][0][:, part]
            if float(way.norm()) == 0:
                continue
            way /= way.norm()
            step = 1e-4
            ends = [loss(*[x + sign * step * way if i == which else x for i, x in enumerate(start)], d64, causal, window, scale)
                    for sign in (1, -1)]
            slope = (ends[0] - ends[1]) / (2 * step)
            mine = float((got[which].double() * way).sum())
            tol = float((tols[which][1] * way.abs()).sum()) + 1e-6 * (1 + abs(slope))
            if which < 2:
                tol += shifts(*start, d64, out.double(), e_out, e_lse.nan_to_num(0.0), way, causal, window, scale)[which]
            assert tol < slope / 4, (name, part, slope, tol)
            assert abs(mine - slope) <= tol, (name, part, mine, slope, tol)
