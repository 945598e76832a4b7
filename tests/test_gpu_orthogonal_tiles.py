"""Orthogonalised updates by tiles of every side, wide and tall, results and
weights of every type, against the steps in 64 bits on the GPU."""
import math

import pytest
import torch

import sparse_gradient_reduction_amd as sg
from tests.operator_util import COEFFICIENTS, U
from tests.orthogonal_tiles import TILES

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]


def _steps(g, noise=0.0, seed=0):
    """Five steps in fp64; with noise, every operand of every product is moved
    by up to that fraction of its value."""
    a, b, c = COEFFICIENTS
    gen = torch.Generator(device=g.device).manual_seed(seed)

    def off(v):
        return v * (1 + noise * (2 * torch.rand(v.shape, generator=gen, device=v.device, dtype=v.dtype) - 1)) if noise else v

    x = g.double()
    tall = x.shape[0] > x.shape[1]
    if tall:
        x = x.t().contiguous()
    x = x / (x.norm() + 1e-7)
    for _ in range(5):
        p = off(x) @ off(x).t().contiguous()
        q = b * p + c * (off(p) @ off(p))
        x = a * off(x) + off(q) @ off(x)
    return x.t().contiguous() if tall else x


def _reference(g):
    """The result, and how far one of fp32 may be: eight times what operands of 22 bits cost."""
    ref = _steps(g)
    far = max(float((_steps(g, 2.0 ** -22, k) - ref).norm()) for k in range(2))
    return ref, 8 * far + 8 * U * float(ref.norm())


@pytest.mark.parametrize("turn", [False, True], ids=["as is", "turned"])
@pytest.mark.parametrize("shape,count", [t[:2] for t in TILES], ids=str)
def test_tiles(dev, shape, count, turn):
    rows, cols = shape[::-1] if turn else shape
    size, gap = rows * cols, 3
    where = [(gap + k * size, rows, cols) for k in range(count)]
    gen = torch.Generator(device=dev).manual_seed(size)
    u = torch.randn(gap + count * size + gap, generator=gen, device=dev)
    w0 = 0.02 * torch.randn(u.shape, generator=gen, device=dev)
    lr, s = 0.5, 0.5 * math.sqrt(max(1.0, rows / cols))
    got, moved = {}, {}
    for t in TYPES:
        got[t] = sg.orthogonalize(u, where, out=torch.full(u.shape, 9.0, dtype=t, device=dev))
        moved[t] = sg.orthogonal_step(w0.to(t, copy=True), u, where, lr=lr, weight_decay=0.1)
        for flat, old in ((got[t], torch.full_like(got[t], 9.0)), (moved[t], w0.to(t))):
            assert torch.equal(flat[:gap], old[:gap]) and torch.equal(flat[-gap:], old[-gap:])
    for k in sorted({0, count // 2, count - 1}):
        here = slice(where[k][0], where[k][0] + size)
        ref, tol = _reference(u[here].view(rows, cols))
        ref = ref.view(-1)
        for t in TYPES:
            # 5% of the roundings' norm for those that fall otherwise beside the reference
            far = float((got[t][here].double() - ref).norm())
            room = tol + 1.05 * float((ref.to(t).double() - ref).norm())
            want = (1 - lr * 0.1) * w0.to(t)[here].double() - s * ref
            far_w = float((moved[t][here].double() - want).norm())
            room_w = s * tol + 1.05 * float((want.to(t).double() - want).norm()) + 8 * U * float(want.norm())
            print(f"{rows}x{cols} {k} {t}: off by {far:.3g} of {room:.3g}, weights {far_w:.3g} of {room_w:.3g}")
            assert far <= room and far_w <= room_w, (k, t, far, room, far_w, room_w)
