"""The norms of queries and keys with the rotation, and their gradients, against 64-bit forms."""
import math

import pytest
import torch

import sparse_gradient_reduction_amd as sg
from tests import attention_util as au
from tests.operator_util import assert_within

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]
# nodes, tokens of a node, heads, groups, D, rotated
SIZES = [(1, 1, 1, 1, 1, 0), (1, 1, 1, 1, 2, 2), (1, 3, 4, 2, 64, 64), (2, 5, 3, 1, 128, 128), (3, 7, 5, 2, 80, 40),
         (1, 9, 2, 2, 256, 256), (2, 33, 1, 3, 45, 22), (1, 130, 12, 4, 96, 32), (4, 2, 2, 1, 63, 0), (1, 11, 3, 3, 200, 6),
         (1, 6, 2, 2, 255, 254), (5, 300, 6, 2, 40, 40), (1, 4, 7, 1, 8, 8), (2, 3, 1, 1, 16, 4), (1, 5, 2, 1, 72, 12)]
EPS = 1e-6


def make(t, nodes, tokens, heads, groups, dim, rotated, seed=0, first=0):
    gen = torch.Generator().manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen)

    n = nodes * tokens
    q, k, dq, dk = (normal(n, h, dim).to(t) for h in (heads, groups, heads, groups))
    qw, kw = 1 + 0.3 * normal(dim), 1 + 0.3 * normal(dim)
    positions = (first + torch.randperm(n, generator=gen)).to(torch.int32)
    return q, k, dq, dk, qw, kw, positions, sg.rotation_frequencies(rotated) if rotated else None


def on(*xs):
    return [None if x is None else x.cuda() for x in xs]


def check(got, q, k, qw, kw, positions, frequencies, interleaved, eps=EPS):
    for y, x, w, name in zip(got, (q, k), (qw, kw), "qk"):
        ref, tol, _, _ = au.norm_rotate(x, w, positions, frequencies, eps, interleaved)
        assert_within(y, ref, tol, name)


def check_backward(got, dq, dk, q, k, qw, kw, positions, frequencies, interleaved, nodes, eps=EPS):
    for i, (dy, x, w, name) in enumerate(((dq, q, qw, "q"), (dk, k, kw, "k"))):
        dx, e_dx, dw, e_dw = au.norm_rotate_backward(dy, x, w, positions, frequencies, eps, interleaved, nodes)
        assert_within(got[i], dx, e_dx, "d" + name)
        assert_within(got[2 + i], dw, e_dw, "dweight " + name)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("size", SIZES)
def test_against_64_bits(t, interleaved, size):
    q, k, dq, dk, qw, kw, pos, fr = make(t, *size, seed=sum(size), first=100000 if size[1] % 2 else 0)
    gq, gk, gdq, gdk, gqw, gkw, gpos, gfr = on(q, k, dq, dk, qw, kw, pos, fr)
    check(sg.head_norm_rotate(gq, gk, gqw, gkw, gpos, gfr, eps=EPS, interleaved=interleaved), q, k, qw, kw, pos, fr, interleaved)
    got = sg.head_norm_rotate_backward(gdq, gdk, gq, gk, gqw, gkw, gpos, gfr, eps=EPS, interleaved=interleaved, nodes=size[0])
    check_backward(got, dq, dk, q, k, qw, kw, pos, fr, interleaved, size[0])


@pytest.mark.parametrize("t", TYPES)
def test_without_weights(t):
    q, k, dq, dk, _, _, pos, fr = make(t, 1, 20, 3, 2, 64, 32, seed=1)
    gq, gk, gdq, gdk, gpos, gfr = on(q, k, dq, dk, pos, fr)
    check(sg.head_norm_rotate(gq, gk, positions=gpos, frequencies=gfr), q, k, None, None, pos, fr, False)
    check_backward(sg.head_norm_rotate_backward(gdq, gdk, gq, gk, positions=gpos, frequencies=gfr), dq, dk, q, k, None,
                   None, pos, fr, False, 1)


@pytest.mark.parametrize("t", TYPES)
def test_views_of_one_projection(t):
    """q and k of a [batch, tokens, heads + 2 groups, D] projection, their gradients into one of the same shape,
    the weights' into columns of the nodes' gradients; what is not theirs is left as it was."""
    b, n, h, g, d = 2, 30, 4, 2, 64
    gen = torch.Generator().manual_seed(2)
    every, grads = (torch.randn(b, n, h + 2 * g, d, generator=gen).to(t) for _ in range(2))
    qw, kw = torch.rand(d, generator=gen), torch.rand(d, generator=gen)
    pos, fr = torch.arange(n, dtype=torch.int32).repeat(b), sg.rotation_frequencies(d)
    (q, k, _), (dq, dk, _) = every.split((h, g, g), 2), grads.split((h, g, g), 2)
    ge, gg = every.cuda(), grads.cuda()
    (gq, gk, gv), (gdq, gdk, _) = ge.split((h, g, g), 2), gg.split((h, g, g), 2)
    gqw, gkw, gpos, gfr = on(qw, kw, pos, fr)
    check([x.flatten(0, 1) for x in sg.head_norm_rotate(gq, gk, gqw, gkw, gpos, gfr)], q.flatten(0, 1), k.flatten(0, 1),
          qw, kw, pos, fr, False)
    flat = torch.full((b, 500), 7.0, device="cuda")
    wide = torch.full_like(ge, 7.0)
    parts = wide.split((h, g, g), 2)
    got = sg.head_norm_rotate_backward(gdq, gdk, gq, gk, gqw, gkw, gpos, gfr, nodes=b, q_out=parts[0], k_out=parts[1],
                                       dq_weight=flat[:, 3:3 + d], dk_weight=flat[:, 300:300 + d])
    check_backward([x.flatten(0, 1) for x in got[:2]] + list(got[2:]), dq.flatten(0, 1), dk.flatten(0, 1),
                   q.flatten(0, 1), k.flatten(0, 1), qw, kw, pos, fr, False, b)
    assert bool((parts[2] == 7).all())
    rest = torch.cat((flat[:, :3], flat[:, 3 + d:300], flat[:, 300 + d:]), 1)
    assert bool((rest == 7).all())


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("interleaved", [False, True])
def test_in_place(t, interleaved):
    q, k, dq, dk, qw, kw, pos, fr = make(t, 2, 40, 4, 2, 96, 48, seed=3)
    args = on(qw, kw, pos, fr)
    gq, gk, gdq, gdk = on(q, k, dq, dk)
    want = sg.head_norm_rotate_backward(gdq, gdk, gq, gk, *args, nodes=2, interleaved=interleaved)
    got = sg.head_norm_rotate_backward(gdq, gdk, gq, gk, *args, nodes=2, interleaved=interleaved, q_out=gdq, k_out=gdk)
    assert got[0] is gdq and all(torch.equal(x, y) for x, y in zip(want, got))
    want = sg.head_norm_rotate(gq, gk, *args, interleaved=interleaved)
    got = sg.head_norm_rotate(gq, gk, *args, interleaved=interleaved, q_out=gq, k_out=gk)
    assert got[0] is gq and all(torch.equal(x, y) for x, y in zip(want, got))


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("shift", [1, 5])
def test_off_16_byte_borders(t, shift):
    q, k, dq, dk, qw, kw, pos, fr = make(t, 1, 25, 3, 2, 64, 64, seed=4)
    def moved(x):
        flat = torch.empty(x.numel() + shift, dtype=t, device="cuda")
        flat[shift:] = x.flatten().cuda()
        return flat[shift:].view(x.shape)
    gq, gk, gdq, gdk = (moved(x) for x in (q, k, dq, dk))
    args = on(qw, kw, pos, fr)
    check(sg.head_norm_rotate(gq, gk, *args, q_out=moved(q), k_out=moved(k)), q, k, qw, kw, pos, fr, False)
    check_backward(sg.head_norm_rotate_backward(gdq, gdk, gq, gk, *args), dq, dk, q, k, qw, kw, pos, fr, False, 1)


@pytest.mark.parametrize("base", [10000.0, 500000.0])
def test_far_and_negative_positions(base):
    q, k, _, _, qw, kw, _, _ = make(torch.float32, 1, 12, 2, 1, 64, 64, seed=5)
    pos = torch.tensor([0, 1, -1, 131071, 1 << 20, 10 ** 7, 2 ** 31 - 1, -2 ** 31, 4095, -77777, 999983, 5], dtype=torch.int32)
    fr = sg.rotation_frequencies(64, base)
    check(sg.head_norm_rotate(*on(q, k, qw, kw, pos, fr)), q, k, qw, kw, pos, fr, False)


@pytest.mark.parametrize("t", TYPES)
def test_not_finite_head_touches_no_other(t):
    q, k, dq, dk, qw, kw, pos, fr = make(t, 1, 6, 3, 2, 64, 32, seed=6)
    args = on(qw, kw, pos, fr)
    clean = sg.head_norm_rotate(*on(q, k), *args)
    cleanb = sg.head_norm_rotate_backward(*on(dq, dk, q, k), *args)
    q[2, 1, 5], k[4, 0, 63], dq[3, 2, 40] = math.nan, math.inf, -math.inf
    got = sg.head_norm_rotate(*on(q, k), *args)
    gotb = sg.head_norm_rotate_backward(*on(dq, dk, q, k), *args)
    for a, b, spared in ((clean[0], got[0], [(2, 1)]), (clean[1], got[1], [(4, 0)]),
                         (cleanb[0], gotb[0], [(2, 1), (3, 2)]), (cleanb[1], gotb[1], [(4, 0)])):
        same = (a == b).all(-1)
        for at in spared:
            assert not bool(same[at])
            same[at] = True
        assert bool(same.all())


def test_no_tokens():
    q, k = torch.empty(0, 3, 64, device="cuda"), torch.empty(0, 2, 64, device="cuda")
    y = sg.head_norm_rotate(q, k)
    assert y[0].shape == q.shape
    dq, dk, dqw, dkw = sg.head_norm_rotate_backward(q, k, q, k, nodes=2)
    assert dqw.shape == (2, 64) and bool((dqw == 0).all()) and bool((dkw == 0).all())


def test_repeated_captured_and_on_another_stream():
    q, k, dq, dk, qw, kw, pos, fr = on(*make(torch.bfloat16, 2, 500, 8, 2, 128, 128, seed=7))
    q_out, k_out, dqo, dko = (torch.empty_like(x) for x in (q, k, q, k))
    dqw, dkw = torch.empty(2, 2, 128, device="cuda").unbind()
    ws = torch.empty(sg.head_norm_rotate_backward_workspace_bytes(2, 500, 128), dtype=torch.uint8, device="cuda")

    def step():
        sg.head_norm_rotate(q, k, qw, kw, pos, fr, q_out=q_out, k_out=k_out)
        sg.head_norm_rotate_backward(dq, dk, q, k, qw, kw, pos, fr, nodes=2, q_out=dqo, k_out=dko, dq_weight=dqw,
                                     dk_weight=dkw, workspace=ws)
        return [x.clone() for x in (q_out, k_out, dqo, dko, dqw, dkw)]

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for turn in range(3):
        q.copy_(torch.randn(q.shape, generator=torch.Generator().manual_seed(turn)))
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in held]
        assert all(torch.equal(x, y) for x, y in zip(step(), got))


def test_gradients_against_differences():
    """Along random directions, the change of sum(y * dy) in 64 bits."""
    q, k, dq, dk, qw, kw, pos, fr = make(torch.float32, 1, 6, 2, 1, 40, 20, seed=8)
    got = sg.head_norm_rotate_backward(*on(dq, dk, q, k, qw, kw, pos, fr))
    for x, dy, w, dx, dw in ((q, dq, qw, got[0], got[2]), (k, dk, kw, got[1], got[3])):
        def loss(v, u):
            y = v / (v.square().mean(-1, keepdim=True) + EPS).sqrt() * u
            return float((au.turn(y, torch.zeros_like(y), pos, fr, False, 1)[0] * dy.double()).sum())
        _, e_dx, _, e_dw = au.norm_rotate_backward(dy, x, w, pos, fr, EPS, False, 1)
        for base, grad, tol, call in ((x, dx, e_dx, lambda v: loss(v, w.double())), (w, dw[0], e_dw[0], lambda v: loss(x.double(), v))):
            way = torch.randn(base.shape, generator=torch.Generator().manual_seed(1), dtype=torch.float64)
            slope = (call(base.double() + 1e-5 * way) - call(base.double() - 1e-5 * way)) / 2e-5
            mine = float((grad.double().cpu() * way).sum())
            assert abs(mine - slope) <= float((tol * way.abs()).sum()) + 1e-6 * (1 + abs(slope))
