"""64-bit forms of attention and of the norms of queries and keys, with the
error that fp32 sums and the documented roundings leave, for the GPU tests.

u = 2^-24 is fp32's rounding (half a step). A sum of n terms is off by at most
n u sum |terms| in any order. With 16-bit types the probabilities and ds are
rounded to the type before the second products: by at most e = finfo(t).eps / 2
of their value each (0 for fp32)."""
import math

import torch

from tests.operator_util import U, half_step


def sees(n, m, queries, keys, causal, window):
    """[queries, keys]: query i of n sees key j of m."""
    i, j = torch.arange(queries)[:, None], torch.arange(keys)
    ahead = j - (i + m - n)
    ok = (i < n) & (j < m)
    if causal:
        ok &= ahead <= 0
    if window is not None:
        ok &= ahead > -window
        if not causal:
            ok &= ahead < window
    return ok


def _rounding(t):
    return 0.0 if t == torch.float32 else torch.finfo(t).eps / 2


def _scores(q, k, see, scale):
    """(scores, -inf where not seen; how far fp32 may be from them), of fp64 [rows, D]."""
    s = scale * q @ k.t()
    # D products (rounded) and additions; scaling, the logarithms' base and what is taken off it
    e = scale * (q.shape[1] + 2) * U * (q.abs() @ k.abs().t()) + 4 * U * s.abs()
    return torch.where(see, s, -math.inf), e


def head_forward(q, k, v, see, scale, t):
    """(out, lse, tolerance of out before its own rounding, of lse) of one head."""
    s, e_s = _scores(q, k, see, scale)
    lse = torch.logsumexp(s, 1)
    some = see.any(1)
    shift = torch.where(some, lse, 0.0)[:, None]
    p = torch.where(see, torch.exp(s - shift), 0.0)
    out = p @ v
    keys = k.shape[0]
    # the exponential's argument is rounded, and that of every rescaling on the way (one to 32 keys at worst)
    top = torch.where(see, s, 0.0).abs().amax(1, keepdim=True) if keys else 0.0
    e_p = torch.where(see, e_s + 4 * U * (1 + top + (torch.where(see, s, 0.0) - shift).abs()), 0.0)
    slips = (keys / 32 + keys + 64) * U
    both = (p * e_p).sum(1, keepdim=True)
    e_out = (p * (e_p + _rounding(t))) @ v.abs() + (both + slips) * (p @ v.abs()) + 4 * U * out.abs()
    if t == torch.float16 and keys:  # its smallest steps, below a row's largest probability
        e_out = e_out + 2.0 ** -25 * v.abs().sum(0)
    e_lse = (both[:, 0] + slips) + 4 * U * torch.where(some, lse, 0.0).abs() + 4 * U
    return out, lse, e_out, e_lse


def head_backward(dout, q, k, v, out, lse, see, scale, t):
    """(dq, dk, dv, tolerance of each before its own rounding) of one head, from the given out and lse."""
    s, e_s = _scores(q, k, see, scale)
    some = see.any(1)
    shift = torch.where(some, lse, 0.0)[:, None]
    p = torch.where(see, torch.exp(s - shift), 0.0)
    gap = (torch.where(see, s, 0.0) - shift).abs()
    e_p = torch.where(see, e_s + 4 * U * (1 + shift.abs() + gap), 0.0)
    d, n, m = q.shape[1], q.shape[0], k.shape[0]
    delta = (dout * out).sum(1, keepdim=True)
    g = dout @ v.t() - delta
    e_g = (d + 2) * U * (dout.abs() @ v.abs().t() + (dout * out).abs().sum(1, keepdim=True)) + 2 * U * g.abs()
    ds = p * g
    e_ds = p * (e_p * g.abs() + (1 + e_p) * e_g) + (2 * U + _rounding(t)) * ds.abs()
    if t == torch.float16 and n and m:  # its smallest steps, below the largest ds there can be
        e_ds = e_ds + see * 2.0 ** -36 * dout.norm(dim=1).max() * v.norm(dim=1).max()
    dq, dk, dv = scale * ds @ k, scale * ds.t() @ q, p.t() @ dout
    e_dq = scale * (e_ds @ k.abs() + (m + 64) * U * ds.abs() @ k.abs()) + 3 * U * dq.abs()
    e_dk = scale * (e_ds.t() @ q.abs() + (n + 64) * U * ds.abs().t() @ q.abs()) + 3 * U * dk.abs()
    e_dv = (p * (e_p + _rounding(t))).t() @ dout.abs() + (n + 64) * U * p.t() @ dout.abs() + 3 * U * dv.abs()
    if t == torch.float16:
        e_dv = e_dv + 2.0 ** -38 * see.double().t() @ dout.abs()
    return dq, dk, dv, e_dq, e_dk, e_dv


def _each(q, k, lengths, causal, window):
    batch, queries, heads, _ = q.shape
    keys, groups = k.shape[1], k.shape[2]
    for b in range(batch):
        n, m = lengths[b] if lengths else (queries, keys)
        see = sees(n, m, queries, keys, causal, window)
        for h in range(heads):
            yield b, h, h * groups // heads, n, m, see[:n, :m]


def forward(q, k, v, causal=False, window=None, scale=None, lengths=None):
    """(out, lse) in fp64 of CPU tensors, and the tolerances of both (out's with its own rounding)."""
    t, scale = q.dtype, q.shape[-1] ** -0.5 if scale is None else scale
    out, e_out = torch.zeros(q.shape, dtype=torch.float64), torch.zeros(q.shape, dtype=torch.float64)
    lse = torch.full((q.shape[0], q.shape[2], q.shape[1]), -math.inf, dtype=torch.float64)
    e_lse = torch.zeros_like(lse)
    for b, h, g, n, m, see in _each(q, k, lengths, causal, window):
        o, l, e_o, e_l = head_forward(q[b, :n, h].double(), k[b, :m, g].double(), v[b, :m, g].double(), see, scale, t)
        out[b, :n, h], lse[b, h, :n], e_out[b, :n, h], e_lse[b, h, :n] = o, l, e_o, e_l
    return out, lse, e_out + half_step(t, out), e_lse


def backward(dout, q, k, v, out, lse, causal=False, window=None, scale=None, lengths=None):
    """[(gradient, tolerance with its own rounding)] of q, k and v."""
    t, scale = q.dtype, q.shape[-1] ** -0.5 if scale is None else scale
    got = [torch.zeros(x.shape, dtype=torch.float64) for x in (q, k, v, q, k, v)]
    for b, h, g, n, m, see in _each(q, k, lengths, causal, window):
        r = head_backward(dout[b, :n, h].double(), q[b, :n, h].double(), k[b, :m, g].double(), v[b, :m, g].double(),
                          out[b, :n, h].double(), lse[b, h, :n].double(), see, scale, t)
        for x, at, part in zip(got, ((b, slice(n), h), (b, slice(m), g), (b, slice(m), g)) * 2, r):
            x[at] += part
    return [(x, e + (q.shape[2] // k.shape[2]) * U * x.abs() + half_step(t, x)) for x, e in zip(got, got[3:])]


def norm_rotate(x, weight, positions, frequencies, eps, interleaved):
    """(y, tolerance with its own rounding, the parts that the gradients need) of [tokens, heads, D]."""
    t, v, d = x.dtype, x.double(), x.shape[-1]
    r = 1 / (v.square().mean(-1, keepdim=True) + eps).sqrt()
    w = torch.ones(d, dtype=torch.float64) if weight is None else weight.double()
    h = v * r
    e_h = (d / 2 + 8) * U * h.abs()  # the sum's additions, half of them relative to r
    y, e = turn(h * w, e_h * w.abs() + 2 * U * (h * w).abs(), positions, frequencies, interleaved, 1)
    return y, e + half_step(t, y), h, r


def turn(x, e, positions, frequencies, interleaved, sign):
    """x turned by sign * position * frequency, and the tolerance that e becomes:
    the angle's place in the turn is rounded to fp32 (2^-25 of half a turn, by
    pi), cosine and sine are off by 4 u, products and sum by 3 u."""
    n = 0 if frequencies is None else frequencies.numel()
    if n == 0:
        return x, e
    angle = sign * positions.double().view(-1, 1, 1) * frequencies.double()
    a = [x[..., 0:2 * n:2], x[..., 1:2 * n:2]] if interleaved else [x[..., :n], x[..., n:2 * n]]
    ea = [e[..., 0:2 * n:2], e[..., 1:2 * n:2]] if interleaved else [e[..., :n], e[..., n:2 * n]]
    off = math.pi * U + 8 * U + 2.0 ** -52 * angle.abs() * 4
    c, s = torch.cos(angle), torch.sin(angle)
    y = [a[0] * c - a[1] * s, a[1] * c + a[0] * s]
    ey = [ea[0] * c.abs() + ea[1] * s.abs(), ea[1] * c.abs() + ea[0] * s.abs()]
    ey = [v + off * (a[0].abs() + a[1].abs()) for v in ey]
    y, ey = ((torch.stack(v, -1).flatten(-2) if interleaved else torch.cat(v, -1)) for v in (y, ey))
    return torch.cat((y, x[..., 2 * n:]), -1), torch.cat((ey, e[..., 2 * n:]), -1)


def norm_rotate_backward(dy, x, weight, positions, frequencies, eps, interleaved, nodes):
    """(dx, its tolerance with its own rounding, dweight [nodes, D], its tolerance)."""
    t, d = x.dtype, x.shape[-1]
    _, _, h, r = norm_rotate(x, None, None, None, eps, False)
    e_h = (d / 2 + 8) * U * h.abs()
    g0 = dy.double()
    u, e_u = turn(g0, torch.zeros_like(g0), positions, frequencies, interleaved, -1)
    w = torch.ones(d, dtype=torch.float64) if weight is None else weight.double()
    g, e_g = u * w, (e_u + U * u.abs()) * w.abs()
    m = (g * h).mean(-1, keepdim=True)
    e_m = (e_g * h.abs() + g.abs() * e_h + (d + 3) * U * (g * h).abs()).mean(-1, keepdim=True)
    dx = r * (g - h * m)
    e_dx = r * (e_g + e_h * m.abs() + h.abs() * e_m + 3 * U * (g.abs() + (h * m).abs())) + (d / 2 + 8) * U * dx.abs()
    per = (nodes, -1, d)
    dw = (u * h).reshape(per).sum(1)
    rows = x.numel() // d // nodes + 16  # in any order
    e_dw = (e_u * h.abs() + u.abs() * e_h + rows * U * (u * h).abs()).reshape(per).sum(1)
    return dx, e_dx + half_step(t, dx), dw, e_dw
