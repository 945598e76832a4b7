"""Orthogonalised updates of every spectrum: noise without strong directions,
updates thinned as the Top-k and the reduction leave them, equal singular
values, ones that fall steeply, rows of very different size."""
import pytest
import torch

import sparse_gradient_reduction_amd as sg
from tests.operator_util import newton_schulz_tolerance

pytestmark = pytest.mark.gpu
TYPES = [torch.float32, torch.bfloat16, torch.float16]


def _noise(r, c, g):
    return torch.randn(r, c, generator=g)


def _thinned(keep):
    return lambda r, c, g: torch.randn(r, c, generator=g) * (torch.rand(r, c, generator=g) < keep)


def _flat(r, c, g):
    q = torch.linalg.qr(torch.randn(max(r, c), min(r, c), generator=g, dtype=torch.float64))[0].float()
    return q if r >= c else q.t()


def _falling(r, c, g):
    m = min(r, c)
    u = torch.linalg.qr(torch.randn(r, m, generator=g))[0]
    v = torch.linalg.qr(torch.randn(c, m, generator=g))[0]
    return (u / torch.arange(1, m + 1)) @ v.t()


def _low_rank(r, c, g):
    return torch.randn(r, 8, generator=g) @ torch.randn(8, c, generator=g) + 1e-3 * torch.randn(r, c, generator=g)


def _graded(r, c, g):
    return torch.randn(r, c, generator=g) * torch.exp(2 * torch.randn(r, 1, generator=g))


SPECTRA = {"noise": _noise, "thinned to 27%": _thinned(0.27), "thinned to 1%": _thinned(0.01),
           "thinned to 0.5%": _thinned(0.005), "flat": _flat, "falling": _falling, "low rank": _low_rank,
           "graded rows": _graded}


def _tolerance(g, t):
    """The reference, and how far (in norm) a result of type t may be: what
    operands of 22 bits cost, and for 16 bits the reference's own rounding to
    the type. That a result near the reference is rounded instead moves the
    norm of some 10^4 roundings or more by about 1%, so 5% are left for it."""
    ref, tol = newton_schulz_tolerance(g, torch.float32)
    return ref, tol + 1.05 * float((ref.to(t).double() - ref).norm())


@pytest.mark.parametrize("name", SPECTRA)
@pytest.mark.parametrize("rows,cols", [(48, 200), (100, 1000), (256, 256), (256, 512), (512, 200), (200, 1500)])
def test_spectra(dev, rows, cols, name):
    g = SPECTRA[name](rows, cols, torch.Generator().manual_seed(rows + cols)).contiguous()
    u = g.view(-1).to(dev)
    for t in TYPES:
        ref, tol = _tolerance(g, t)
        got = sg.orthogonalize(u, [(0, rows, cols)], dtype=t).double().cpu().view(rows, cols)
        far = float((got - ref).norm())
        print(f"{rows}x{cols} {name} {t}: off by {far:.3g}, tolerance {tol:.3g} of norm {float(ref.norm()):.3g}")
        assert far <= tol, (name, t, far, tol)


@pytest.mark.parametrize("name", ["noise", "thinned to 1%", "graded rows"])
@pytest.mark.parametrize("t", TYPES, ids=str)
@pytest.mark.parametrize("steps,coefficients", [(3, (3.4445, -4.7750, 2.0315)), (8, (3.4445, -4.7750, 2.0315)),
                                                (5, (1.875, -1.25, 0.375)), (9, (1.5, -0.5, 0.0))])
def test_other_steps(dev, steps, coefficients, t, name):
    """The accuracy does not hang on the number of steps or on what they do to the singular values."""
    rows, cols = 256, 300
    g = SPECTRA[name](rows, cols, torch.Generator().manual_seed(steps)).contiguous()
    ref, tol = newton_schulz_tolerance(g, torch.float32, steps, coefficients=coefficients)
    tol += 1.05 * float((ref.to(t).double() - ref).norm())
    got = sg.orthogonalize(g.view(-1).to(dev), [(0, rows, cols)], dtype=t, steps=steps, coefficients=coefficients)
    far = float((got.double().cpu().view(rows, cols) - ref).norm())
    print(f"{name} {t} {steps} steps: off by {far:.3g}, tolerance {tol:.3g}")
    assert far <= tol, (far, tol)
