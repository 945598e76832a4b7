"""Plain 64-bit forms of the dense operators and the error that fp32 sums and
one rounding to the type leave, for the GPU tests.

u = 2^-24 is fp32's rounding (half a step); a sum of n terms of which no
partial sum adds more than `adds` terms one by one is off by at most
adds * u * sum |terms|. An output of type t is rounded once more, by at most
finfo(t).eps / 2 of its value (or half the smallest subnormal)."""
import math

import torch

U = 2.0 ** -24


def half_step(t, ref):
    f = torch.finfo(t)
    return f.eps / 2 * ref.abs() + f.smallest_normal * f.eps / 2


def assert_within(got, ref, tol, what):
    got = got.detach().double().cpu()
    ref, tol = ref.double().cpu(), tol.double().cpu().expand_as(ref)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{what}: NaN in other places"
    fine = ~torch.isnan(ref)
    off = ((got - ref).abs() - tol)[fine]
    if off.numel() == 0:
        return
    at = int(off.argmax())
    assert off.max() <= 0, (f"{what}: {int((off > 0).sum())} of {off.numel()} outside, worst at {at}: "
                            f"{got[fine][at].item()!r} for {ref[fine][at].item()!r}, tolerance {tol[fine][at].item()!r}")


def adds(cols):
    """Additions one after the other in a sum over a row: at worst one wave,
    cols / 64 terms a lane, then a tree and its waves."""
    return math.ceil(cols / 64) + 16


def layer_norm_reference(x, residual, weight, bias, eps):
    """(y, mean, rstd, total) in fp64 of CPU tensors, and the tolerances of y
    (before its own rounding), mean and rstd."""
    t = x.dtype
    v = x.double()
    total = None
    if residual is not None:
        total = v + residual.double()
        v = (x.float() + residual.float()).to(t).double()
    n, k = x.shape[-1], adds(x.shape[-1])
    mean = v.mean(-1, keepdim=True)
    var = (v - mean).square().mean(-1, keepdim=True)
    rstd = 1 / (var + eps).sqrt()
    e_mean = k * U * v.abs().mean(-1, keepdim=True) + 2 * U * mean.abs()
    # the squares' sum about a mean that is e_mean off: relative roundings and e_mean^2
    r_rstd = 0.5 * ((k + 6) * U + (e_mean.square() + 2 * U * e_mean * (v - mean).abs().mean(-1, keepdim=True)) / (var + eps)) + 6 * U
    h = (v - mean) * rstd
    w = torch.ones(n, dtype=torch.float64) if weight is None else weight.double()
    b = torch.zeros(n, dtype=torch.float64) if bias is None else bias.double()
    y = h * w + b
    e_y = w.abs() * (rstd * e_mean * (1 + r_rstd) + h.abs() * (r_rstd + 4 * U)) + 2 * U * y.abs()
    return y, mean[..., 0], rstd[..., 0], total, e_y, e_mean[..., 0], (rstd * r_rstd)[..., 0]


def layer_norm_backward_reference(dy, x, weight, mean, rstd, nodes, dresidual):
    """(dx, dweight, dbias) in fp64 of CPU tensors, and their tolerances
    (dx's before its own rounding)."""
    cols = x.shape[-1]
    g0, r = dy.double(), rstd.double()[..., None]
    h = (x.double() - mean.double()[..., None]) * r
    e_h = 2 * U * h.abs()
    w = torch.ones(cols, dtype=torch.float64) if weight is None else weight.double()
    g = g0 * w
    k = adds(cols)
    s0, s1 = g.mean(-1, keepdim=True), (g * h).mean(-1, keepdim=True)
    e0 = (k + 3) * U * g.abs().mean(-1, keepdim=True)
    e1 = (k + 6) * U * (g * h).abs().mean(-1, keepdim=True)
    inner = g - s0 - h * s1
    dx = r * inner
    e_dx = r * (U * g.abs() + e0 + h.abs() * e1 + e_h * s1.abs() + 3 * U * (g.abs() + s0.abs() + (h * s1).abs())) + 2 * U * dx.abs()
    if dresidual is not None:
        dx = dx + dresidual.double()
        e_dx = e_dx + U * dx.abs()
    per = (nodes, x.numel() // cols // nodes, cols)
    dw, db = (g0 * h).reshape(per).sum(1), g0.reshape(per).sum(1)
    rows = per[1] + 16  # in any order
    e_dw = (rows + 4) * U * (g0 * h).abs().reshape(per).sum(1)
    e_db = rows * U * g0.abs().reshape(per).sum(1)
    return dx, dw, db, e_dx, e_dw, e_db


COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def newton_schulz(g, steps=5, coefficients=COEFFICIENTS, eps=1e-7, noise=None, seed=0):
    """The orthogonalised [rows, cols] fp64 matrix. noise[k] = (of the first
    product's operands, of the others') moves every operand of step k's
    products by up to that fraction of its value, in a random direction."""
    a, b, c = coefficients
    gen = torch.Generator().manual_seed(seed)

    def off(v, by):
        return v * (1 + by * (2 * torch.rand(v.shape, generator=gen, dtype=torch.float64) - 1)) if by else v

    x = g.double()
    tall = x.shape[0] > x.shape[1]
    if tall:
        x = x.t()
    x = x / (x.norm() + eps)
    for k in range(steps):
        n0, n1 = noise[k] if noise else (0, 0)
        p = off(x, n0) @ off(x, n0).t()
        q = b * p + c * (off(p, n1) @ off(p, n1))
        x = a * off(x, n1 and 2.0 ** -22) + off(q, n1) @ off(x, n1)
    return x.t() if tall else x


def newton_schulz_tolerance(g, t, steps=5, **kw):
    """How far (in norm) a result of type t may be before its own rounding:
    eight times what operands held to 22 bits cost, which is what two fp16 parts
    hold. A 16-bit result leaves room for products of single fp16 values (11
    bits, 2^-12 of a value) in the steps whose error the later ones wear off:
    all but the last two for fp16, for bf16 all but the last one and its
    Gram matrix."""
    s, o = 2.0 ** -22, 2.0 ** -12
    noise = [(s, s)] * steps
    if t == torch.float16:
        noise = [(o, o)] * max(0, steps - 2) + [(s, s)] * min(2, steps)
    if t == torch.bfloat16:
        noise = [(o, o)] * max(0, steps - 1) + [(o, s)] * min(1, steps)
    ref = newton_schulz(g, steps, **kw)
    far = max(float((newton_schulz(g, steps, noise=noise, seed=k, **kw) - ref).norm()) for k in range(2))
    return ref, 8 * far + 8 * U * float(ref.norm())
