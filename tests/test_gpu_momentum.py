"""Momentum from a reduction's result against the formula in 64 bits: sparse
and dense results, the sizes around a tile, bad records, graphs."""
import numpy as np
import pytest
import torch

import sparse_gradient_reduction_amd as sg
from tests.operator_util import U, assert_within, half_step

pytestmark = pytest.mark.gpu


def _reduced(dev, N, idx, val, dense=False, cap=None, count=None):
    idx = np.asarray(idx, np.uint32)
    out_idx = torch.full((max(1, len(idx) if cap is None else cap),), -1, dtype=torch.int32, device=dev)
    out_val = torch.full((N,), float("nan"), device=dev)
    if dense:
        out_val.copy_(torch.as_tensor(val))
    else:
        out_idx[: len(idx)] = torch.from_numpy(idx.view(np.int32)).to(dev)
        out_val[: len(idx)] = torch.as_tensor(val).to(dev)
    res = torch.tensor([len(idx) if count is None else count, int(dense)], dtype=torch.int64).view(torch.uint8).to(dev)
    return sg.ReduceOutput(res, out_idx, out_val, N)


def _check(out, g, m0, m, u, mu, scale, nesterov):
    """g: the dense fp64 sum. mu and scale as fp32 holds them."""
    mu, scale = float(np.float32(mu)), float(np.float32(scale))
    s, p = scale * g, mu * m0.double().cpu()
    want = p + s
    e = U * (s.abs() + want.abs())          # the product, then one fused rounding
    assert_within(m, want, e, "momentum")
    if nesterov:
        want = s + mu * want
        e = abs(mu) * e + U * (s.abs() + want.abs()) + U * e
    assert_within(u, want, e + (half_step(u.dtype, want.abs() + e) if u.dtype != torch.float32 else 0 * e), "update")


CASES = [(1, 1.0), (1, 0.0), (2, 0.5), (63, 0.3), (255, 1.0), (4095, 0.24), (4096, 0.5), (4097, 0.01), (8193, 0.3),
         (100003, 0.001), (272474, 0.24), (1 << 20, 0.27), (1000003, 0.0), ((1 << 22) + 4099, 0.01), (1 << 22, 0.3)]


@pytest.mark.parametrize("nesterov", [False, True])
@pytest.mark.parametrize("t", [torch.float32, torch.bfloat16, torch.float16], ids=str)
@pytest.mark.parametrize("N,density", CASES)
def test_momentum(dev, N, density, t, nesterov):
    rng = np.random.default_rng(N)
    keep = np.flatnonzero(rng.random(N) < density)
    val = rng.standard_normal(len(keep)).astype(np.float32)
    m0 = torch.from_numpy(rng.standard_normal(N).astype(np.float32)).to(dev)
    g = torch.zeros(N, dtype=torch.float64)
    g[torch.from_numpy(keep)] = torch.from_numpy(val).double()
    for dense in (False, True):
        out = _reduced(dev, N, keep, g.float().to(dev) if dense else val, dense)
        m = m0.clone()
        u = sg.momentum_step(out, m, 0.95, scale=1 / 16, nesterov=nesterov, dtype=t)
        assert u.dtype == t
        _check(out, g, m0, m, u, 0.95, 1 / 16, nesterov)


@pytest.mark.parametrize("N", [3 * 4096 + 1001, (1 << 22) + 1001])
@pytest.mark.parametrize("where", ["first", "last", "cluster", "all in one tile", "every 4096th"])
def test_momentum_of_uneven_pairs(dev, where, N):
    keep = {"first": [0], "last": [N - 1], "cluster": list(range(5000, 5600)), "all in one tile": list(range(4096, 8192)),
            "every 4096th": list(range(0, N, 4096))}[where]
    val = torch.randn(len(keep))
    g = torch.zeros(N, dtype=torch.float64)
    g[keep] = val.double()
    m0 = torch.randn(N, device=dev)
    m = m0.clone()
    u = sg.momentum_step(_reduced(dev, N, keep, val), m, 0.9, nesterov=True)
    _check(None, g, m0, m, u, 0.9, 1.0, True)


@pytest.mark.parametrize("N", [5000, 1 << 22])
def test_momentum_on_slices(dev, N):
    """Arrays off their 16-byte borders."""
    N = N + 5
    keep = list(range(0, N, 3))
    val = torch.randn(len(keep))
    g = torch.zeros(N, dtype=torch.float64)
    g[keep] = val.double()
    for off in (1, 2, 3):
        red = _reduced(dev, N, keep, val)
        m0 = torch.randn(N + off, device=dev)[off:]
        m, u = torch.empty(N + off, device=dev)[off:], torch.empty(N + off, device=dev, dtype=torch.bfloat16)[off:]
        m.copy_(m0)
        sg.momentum_step(red, m, 0.9, update=u)
        _check(None, g, m0, m, u, 0.9, 1.0, False)
        v = torch.empty(N + off, device=dev)[off:]
        v.copy_(g)
        m.copy_(m0)
        dense = sg.ReduceOutput(_reduced(dev, N, keep, g.float().to(dev), True).result, red.out_idx, v, N)
        sg.momentum_step(dense, m, 0.9, update=u)
        _check(None, g, m0, m, u, 0.9, 1.0, False)


def test_momentum_keeps_to_its_arrays(dev):
    """A record that counts more pairs than the array holds is cut to it; positions past the end are passed over."""
    N = 9000
    keep = np.arange(0, 900, 9)
    val = torch.randn(len(keep))
    m0 = torch.randn(N, device=dev)
    guard = torch.full((N + 64,), 5.0, device=dev)
    m = guard[32: 32 + N]
    m.copy_(m0)
    idx = np.concatenate([keep[:-1], [N + 7]])
    sg.momentum_step(_reduced(dev, N, idx, val, count=1 << 40), m, 0.9)
    g = torch.zeros(N, dtype=torch.float64)
    g[torch.from_numpy(keep[:-1])] = val[:-1].double()
    _check(None, g, m0, m, m, 0.9, 1.0, False)
    assert (guard[:32] == 5).all() and (guard[32 + N:] == 5).all()


@pytest.mark.parametrize("delta", [0.5, 0.05])
def test_momentum_after_a_reduction_in_a_graph(dev, delta):
    """The reduction and the momentum captured together; whether the result is
    dense is read on the device at every replay."""
    P, N, k = 4, 60001, 3000
    rng = np.random.default_rng(3)
    off = [p * k for p in range(P + 1)]
    idx = torch.empty(P * k, dtype=torch.int32, device=dev)
    val = torch.empty(P * k, device=dev)
    T = sg.dense_threshold(delta, N)
    oi, ov = torch.zeros(max(1, min(N, T - 1)), dtype=torch.int32, device=dev), torch.zeros(N, device=dev)
    res = torch.zeros(16, dtype=torch.uint8, device=dev)
    ws = torch.empty(sg.sparse_reduce_workspace_bytes(P, N, P * k), dtype=torch.uint8, device=dev)
    m, u = torch.zeros(N, device=dev), torch.zeros(N, device=dev)

    def step():
        out = sg.sparse_reduce(off, idx, val, N, delta, out_idx=oi, out_val=ov, result=res, workspace=ws)
        sg.momentum_step(out, m, 0.9, scale=0.25, nesterov=True, update=u)
        return out

    def fill():
        i = np.concatenate([np.sort(rng.choice(N, k, replace=False)) for _ in range(P)]).astype(np.uint32)
        v = rng.standard_normal(P * k).astype(np.float32)
        idx.copy_(torch.from_numpy(i.view(np.int32)))
        val.copy_(torch.from_numpy(v))
        g = torch.zeros(N, dtype=torch.float64)
        g.index_add_(0, torch.from_numpy(i.astype(np.int64)), torch.from_numpy(v).double())
        return g

    fill()
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(3):
        g = fill()
        m0 = torch.randn(N, device=dev)
        m.copy_(m0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert out.read()[1] == (delta < 0.1)
        want = g.float().double()  # the reduction rounds its sums once
        _check(None, want, m0, m, u, 0.9, 0.25, True)
        (m * 2).sum().item()
