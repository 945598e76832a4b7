"""A block's step made of these calls, for P nodes next to each other: layer
norm, a projection, the norms of queries and keys with the rotation, attention,
the projection back and the residual; and its gradients the same way back, the
weights' of every node into the nodes' rows, from which they are sent and
reduced. Against 64-bit automatic differentiation of the formulas.

The tolerances: a result is behind fewer than 2000 roundings of fp32 one after
the other (sums of 96 to 160 terms and what lies between them), each of which
moves it by 2^-24 of the largest value around it at most."""
import math

import pytest
import torch

import sparse_gradient_reduction_amd as sg

pytestmark = pytest.mark.gpu

P, S, WIDTH, H, G, D = 3, 53, 96, 4, 2, 32
NAMES = ("gain", "bias", "into", "q_weight", "k_weight", "back")
SHAPES = ((WIDTH,), (WIDTH,), (WIDTH, (H + 2 * G) * D), (D,), (D,), (H * D, WIDTH))
NEAR = 2000 * 2.0 ** -24


def start(seed=0):
    gen = torch.Generator().manual_seed(seed)
    x, dy = (torch.randn(P, S, WIDTH, generator=gen) for _ in range(2))
    flat = torch.randn(sum(math.prod(s) for s in SHAPES), generator=gen) * WIDTH ** -0.5
    parts, at = {}, 0
    for name, shape in zip(NAMES, SHAPES):
        parts[name] = slice(at, at + math.prod(shape))
        at += math.prod(shape)
    for name in ("gain", "q_weight", "k_weight"):
        flat[parts[name]] += 1
    return x, dy, flat, parts


def views(flat, parts):
    return {n: flat[parts[n]].view(s) for n, s in zip(NAMES, SHAPES)}


def definition(x, flat, parts, positions, frequencies):
    """y of one node's sequence, in 64 bits."""
    w = views(flat, parts)
    c = x - x.mean(-1, keepdim=True)
    y = c / (c.square().mean(-1, keepdim=True) + 1e-5).sqrt() * w["gain"] + w["bias"]
    q, k, v = (y @ w["into"]).view(S, H + 2 * G, D).split((H, G, G), 1)
    angle = positions.double()[:, None, None] * frequencies

    def norm(z, weight):
        z = z / (z.square().mean(-1, keepdim=True) + 1e-6).sqrt() * weight
        a, b = z.chunk(2, -1)
        return torch.cat((a * angle.cos() - b * angle.sin(), b * angle.cos() + a * angle.sin()), -1)

    q, k = norm(q, w["q_weight"]), norm(k, w["k_weight"]).repeat_interleave(H // G, 1)
    score = torch.einsum("ihd,jhd->hij", q, k) * D ** -0.5
    score = score.masked_fill(torch.ones(S, S, dtype=torch.bool).triu(1), -math.inf)
    out = torch.einsum("hij,jhd->ihd", score.softmax(-1), v.repeat_interleave(H // G, 1))
    return out.flatten(1) @ w["back"] + x


def step(x, dy, flat, parts, grad, positions, frequencies):
    """(y, dx), the weights' gradients of node p in grad[p]."""
    w = views(flat, parts)
    y, mean, rstd = sg.layer_norm(x, w["gain"], w["bias"])
    q0, k0, v = (y @ w["into"]).view(P, S, H + 2 * G, D).split((H, G, G), 2)
    q, k = sg.head_norm_rotate(q0, k0, w["q_weight"], w["k_weight"], positions, frequencies)
    out, lse = sg.attention(q, k, v, causal=True)
    result = out.flatten(2) @ w["back"] + x

    dout = dy @ w["back"].t()
    dheads = torch.empty(P, S, H + 2 * G, D, device=x.device)
    dq0, dk0, dv = dheads.split((H, G, G), 2)
    dq, dk, _ = sg.attention_backward(dout.view(P, S, H, D), q, k, v, out, lse, causal=True, dv=dv)
    sg.head_norm_rotate_backward(dq, dk, q0, k0, w["q_weight"], w["k_weight"], positions, frequencies, nodes=P,
                                 q_out=dq0, k_out=dk0, dq_weight=grad[:, parts["q_weight"]], dk_weight=grad[:, parts["k_weight"]])
    dheads = dheads.flatten(2)
    grad[:, parts["into"]] = (y.transpose(1, 2) @ dheads).flatten(1)
    grad[:, parts["back"]] = (out.flatten(2).transpose(1, 2) @ dy).flatten(1)
    dx, _, _ = sg.layer_norm_backward(dheads @ w["into"].t(), x, w["gain"], mean, rstd, nodes=P, dresidual=dy,
                                      dweight=grad[:, parts["gain"]], dbias=grad[:, parts["bias"]])
    return result, dx


def test_a_blocks_step():
    x, dy, flat, parts = start()
    positions, frequencies = torch.arange(S, dtype=torch.int32) + 1000, sg.rotation_frequencies(D)
    on = [t.cuda() for t in (x, dy, flat)]
    grad = torch.full((P, flat.numel()), math.nan, device="cuda")
    y, dx = step(*on, parts, grad, positions.repeat(P).cuda(), frequencies.cuda())
    assert bool(torch.isfinite(grad).all())

    def near(got, want, what):
        assert float((got.double().cpu() - want).abs().max()) <= NEAR * float(want.abs().max()), what

    for p in range(P):
        xp, w = x[p].double().requires_grad_(), flat.double().requires_grad_()
        want = definition(xp, w, parts, positions, frequencies)
        want.backward(dy[p].double())
        near(y[p], want.detach(), "y")
        near(dx[p], xp.grad, "dx")
        for name in NAMES:
            near(grad[p, parts[name]], w.grad[parts[name]], name)

    # and on to the exchange: what is sent and what stays make the gradients again
    k = flat.numel() // 10
    residual, whole = torch.zeros_like(grad), grad.clone()
    idx, val = sg.topk_ef(grad, residual, k)
    out = sg.sparse_reduce([p * k for p in range(P + 1)], idx.view(-1), val.view(-1), flat.numel(), delta=0.3)
    sent = torch.zeros_like(grad).scatter_(1, idx.long(), val)
    assert torch.equal(sent + residual, whole)
    momentum = torch.zeros(flat.numel(), device="cuda")
    update = sg.momentum_step(out, momentum, 0.9, scale=1 / P)
    assert torch.allclose(update.double(), sent.double().sum(0) / P, rtol=1e-6, atol=1e-7)


def test_a_blocks_step_captured():
    """The calls of a step in a graph, replayed on other inputs with eager work between the replays."""
    _, _, flat, parts = start()
    w = views(flat.cuda(), parts)
    pos, fr = (torch.arange(S, dtype=torch.int32).repeat(P) + 5).cuda(), sg.rotation_frequencies(D).cuda()
    x, dout, heads = torch.randn(P, S, WIDTH, device="cuda"), torch.randn(P, S, H, D, device="cuda"), torch.randn(P, S, H + 2 * G, D, device="cuda")
    grad = torch.empty(P, 2 * D, device="cuda")

    def calls():
        y, _, _ = sg.layer_norm(x, w["gain"], w["bias"])
        q0, k0, v = heads.split((H, G, G), 2)
        q, k = sg.head_norm_rotate(q0, k0, w["q_weight"], w["k_weight"], pos, fr)
        out, lse = sg.attention(q, k, v, causal=True)
        dq, dk, dv = sg.attention_backward(dout, q, k, v, out, lse, causal=True)
        dq0, dk0, _, _ = sg.head_norm_rotate_backward(dq, dk, q0, k0, w["q_weight"], w["k_weight"], pos, fr, nodes=P,
                                                      dq_weight=grad[:, :D], dk_weight=grad[:, D:])
        return y, out, lse, dq0, dk0, dv

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = calls()
    for turn in range(3):
        for t in (x, dout, heads):
            t.copy_(torch.randn(t.shape, generator=torch.Generator().manual_seed(turn)))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held] + [grad.clone()]
        want = list(calls()) + [grad]
        assert all(torch.equal(a, b) for a, b in zip(got, want))
