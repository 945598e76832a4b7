"""Orthogonalised updates against the Newton-Schulz steps in 64 bits: sides of
every kind, several matrices, types, the weights' step, values, graphs."""
import math

import pytest
import torch

import sparse_gradient_reduction_amd as sg
from tests.operator_util import U, half_step, newton_schulz, newton_schulz_tolerance

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]


def _update(shapes, seed, gap=0):
    """Flat update of matrices with a few directions that stand out, and where they lie."""
    g = torch.Generator().manual_seed(seed)
    parts, where, at = [], [], gap
    parts.append(torch.zeros(gap))
    for rows, cols in shapes:
        m = torch.randn(rows, cols, generator=g)
        for i in range(3):
            m += 4 / (i + 1) * torch.randn(rows, 1, generator=g) * torch.randn(1, cols, generator=g)
        parts += [1e-3 * m.view(-1), torch.zeros(gap)]
        where.append((at, rows, cols))
        at += rows * cols + gap
    return torch.cat(parts), where


def _check(got, update, where, t, **kw):
    got = got.double().cpu()
    for at, rows, cols in where:
        g = update[at: at + rows * cols].double().cpu().view(rows, cols)
        ref, tol = newton_schulz_tolerance(g, t, **kw)
        o = got[at: at + rows * cols].view(rows, cols)
        far = float((o - ref).norm())
        round_ = float(half_step(t, ref).norm()) if t != torch.float32 else 0.0
        print(f"{rows}x{cols} {t}: off by {far:.3g}, tolerance {tol + round_:.3g} of norm {float(ref.norm()):.3g}")
        assert far <= tol + round_, (rows, cols, far, tol, round_)


SHAPES = [(1, 1), (1, 7), (9, 1), (2, 2), (16, 27), (27, 16), (10, 64), (31, 33), (64, 64), (64, 576), (65, 63),
          (63, 65), (128, 128), (100, 333), (129, 127), (333, 100), (257, 771), (256, 1024), (1030, 200), (16, 3000),
          (500, 500)]


@pytest.mark.parametrize("t", TYPES, ids=str)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_one_matrix(dev, rows, cols, t):
    u, where = _update([(rows, cols)], rows * 1000 + cols)
    u = u.to(dev)
    _check(sg.orthogonalize(u, where, dtype=t), u, where, t)


BORDERS = [(32, 32), (33, 33), (32, 257), (32, 4096), (32, 4097), (17, 256), (16, 8), (48, 289), (64, 256), (64, 2048),
           (64, 2049), (63, 1000), (1, 300), (300, 1), (130, 4100)]


@pytest.mark.parametrize("turn", [False, True])
@pytest.mark.parametrize("rows,cols", BORDERS)
def test_borders_of_the_kinds(dev, rows, cols, turn):
    """Short sides around 16, 32 and 64, long ones around a workgroup's reach; wide and tall."""
    if turn:
        rows, cols = cols, rows
    u, where = _update([(rows, cols)] * 2, rows + 7 * cols)
    u = u.to(dev)
    _check(sg.orthogonalize(u, where), u, where, torch.float32)
    _check(sg.orthogonalize(u.bfloat16(), where), u.bfloat16(), where, torch.bfloat16)


def test_long_sums(dev):
    """fp32 results keep their accuracy over sums of thousands of terms, one
    side's and several matrices' together (tiles of 64 and of 128)."""
    for shapes in ([(100, 9000)], [(1300, 2100)], [(700, 900)] * 4):
        u, where = _update(shapes, len(shapes))
        u = u.to(dev)
        _check(sg.orthogonalize(u, where), u, where[:1], torch.float32)


@pytest.mark.parametrize("source", TYPES, ids=str)
@pytest.mark.parametrize("gap", [0, 1, 5])
def test_several_matrices(dev, source, gap):
    """Equal ones in a row, others between, gaps that stay as they were."""
    shapes = [(16, 27)] * 3 + [(40, 24)] + [(130, 70)] * 2 + [(70, 130), (16, 27), (3, 200)]
    u, where = _update(shapes, 4, gap)
    u = u.to(source).to(dev)
    _check(sg.orthogonalize(u, where, dtype=torch.float32), u, where, torch.float32)
    out = torch.full(u.shape, 9.0, device=dev)
    sg.orthogonalize(u, where, out=out)
    _check(out, u, where, torch.float32)
    for at, rows, cols in where:
        out[at: at + rows * cols] = 9
    assert (out == 9).all()


def test_many_groups(dev):
    """More different shapes than one set of launches holds."""
    shapes = [(k % 13 + 1, 3 * k + 2) for k in range(60)]
    u, where = _update(shapes, 5)
    u = u.to(dev)
    _check(sg.orthogonalize(u, where), u, where, torch.float32)


def test_no_matrices_and_empty_ones(dev):
    u = torch.randn(100, device=dev)
    assert not sg.orthogonalize(u, []).any()
    out = sg.orthogonalize(u, [(0, 0, 5), (0, 4, 8), (32, 7, 0), (40, 6, 10)])
    _check(out, u, [(0, 4, 8), (40, 6, 10)], torch.float32)
    assert not out[32:40].any()


@pytest.mark.parametrize("t", TYPES, ids=str)
@pytest.mark.parametrize("shape", [(48, 200), (200, 48), (150, 150)])
def test_step(dev, shape, t):
    """w = (1 - lr decay) w - lr s o in place, gaps untouched."""
    rows, cols = shape
    u, where = _update([shape, shape], 6, gap=3)
    w0 = (torch.randn(u.shape, generator=torch.Generator().manual_seed(7)) * 0.02).to(t)
    w = w0.to(dev)
    assert sg.orthogonal_step(w, u.to(dev), where, lr=0.5, weight_decay=0.1) is w
    s = 0.5 * math.sqrt(max(1.0, rows / cols))
    want = w0.double().clone()
    room = torch.zeros(())
    for at, r, c in where:
        here = slice(at, at + r * c)
        o, tol = newton_schulz_tolerance(u[here].double().view(r, c), t)
        want[here] = (1 - 0.5 * 0.1) * want[here] - s * o.reshape(-1)
        room = room + s * tol
    room = room + half_step(t, want).norm() + 8 * U * want.norm()
    assert float((w.double().cpu() - want).norm()) <= float(room)
    gaps = torch.ones(u.shape, dtype=torch.bool)
    for at, r, c in where:
        gaps[at: at + r * c] = False
    assert torch.equal(w.cpu()[gaps], w0[gaps])


@pytest.mark.parametrize("steps", [0, 1, 2, 3, 4, 6, 7, 12])
def test_steps_and_coefficients(dev, steps):
    for shape in ((40, 90), (130, 300), (520, 130)):
        u, where = _update([shape], 8)
        u = u.to(dev)
        for t in TYPES:
            got = sg.orthogonalize(u, where, steps=steps, coefficients=(1.875, -1.25, 0.375), eps=1e-3, dtype=t)
            _check(got, u, where, t, steps=steps, coefficients=(1.875, -1.25, 0.375), eps=1e-3)


def test_values(dev):
    """Zeros stay zeros; tiny and huge updates; NaN and infinity stay in their matrix."""
    shapes = [(20, 30)] * 5
    u, where = _update(shapes, 9)
    u[:600] = 0
    u[600:1200] *= 1e-18
    u[1200:1800] *= 1e18
    u = u.to(dev)
    out = sg.orthogonalize(u, where, eps=1e-30)
    assert not out[:600].any()
    for k in (1, 2, 3, 4):
        _check(out, u, [where[k]], torch.float32, eps=1e-30)
    v = u.clone()
    v[1800] = float("nan")
    v[2400] = float("inf")
    bad = sg.orthogonalize(v, where, eps=1e-30)
    assert torch.equal(bad[:1800], out[:1800])
    assert torch.isnan(bad[1800:3000]).any()


def test_result_is_nearly_orthogonal(dev):
    """The coefficients' five steps take singular values to 0.6 .. 1.25."""
    u = torch.randn(200 * 600, generator=torch.Generator().manual_seed(1)).to(dev)
    o = sg.orthogonalize(u, [(0, 200, 600)]).double().cpu().view(200, 600)
    s = torch.linalg.svdvals(o)
    assert 0.6 < s.min() and s.max() < 1.25


def test_repeats_bit_for_bit(dev):
    u, where = _update([(140, 300), (64, 64), (300, 140)], 10)
    u = u.to(dev)
    first = sg.orthogonalize(u, where)
    for _ in range(3):
        assert torch.equal(first, sg.orthogonalize(u, where))


def test_graph_and_stream(dev):
    """The step captured with its workspace; replays follow new updates. A side stream gives the same."""
    u, where = _update([(16, 27)] * 2 + [(150, 90), (64, 576)], 11)
    u = u.to(dev)
    w0 = torch.randn(u.shape, device=dev) * 0.02
    w = w0.clone()
    ws = torch.empty(sg.orthogonalize_workspace_bytes(u.numel(), where), dtype=torch.uint8, device=dev)

    def step():
        sg.orthogonal_step(w, u, where, lr=0.02, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        u.copy_(torch.randn_like(u))
        w.copy_(w0)
        step()
        want = w.clone()
        w.copy_(w0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(w, want)
        (w * 2).sum().item()
    with torch.cuda.stream(side):
        side.wait_stream(torch.cuda.current_stream())
        again = sg.orthogonal_step(w0.clone(), u, where, lr=0.02)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(again, want)


def test_plain_form_is_the_reference():
    """The reference itself: a 2 x 2 worked by hand. G = diag(3, 4): X0 =
    diag(.6, .8); one step of x -> a x + b x^3 + c x^5."""
    got = newton_schulz(torch.diag(torch.tensor([3.0, 4.0])), steps=1, coefficients=(2.0, -1.5, 0.5), eps=0.0)
    assert abs(float(got[0, 0]) - (2 * .6 - 1.5 * .6 ** 3 + .5 * .6 ** 5)) < 1e-14
    assert abs(float(got[1, 1]) - (2 * .8 - 1.5 * .8 ** 3 + .5 * .8 ** 5)) < 1e-14 and float(got[0, 1]) == 0
