"""Attention and its gradients against 64-bit forms."""
import math

import pytest
import torch

import sparse_gradient_reduction_amd as sg
from tests import attention_util as au
from tests.operator_util import assert_within

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]
# batch, queries, keys, heads, groups, D, causal, window, lengths [(queries, keys)]
CASES = [
    (1, 1, 1, 1, 1, 1, False, None, None),
    (2, 1, 1, 2, 1, 64, True, None, None),
    (1, 1, 200, 3, 3, 128, True, None, None),
    (3, 7, 5, 4, 2, 33, False, None, None),
    (2, 64, 64, 4, 4, 64, True, None, None),
    (1, 65, 63, 2, 2, 128, True, None, None),        # the first queries see nothing
    (1, 128, 128, 2, 1, 128, False, None, None),
    (2, 129, 257, 6, 2, 80, True, 40, None),
    (1, 100, 300, 2, 2, 72, False, 17, None),
    (1, 300, 100, 3, 1, 40, True, 1, None),
    (5, 150, 150, 4, 2, 64, True, None, [(150, 150), (0, 0), (1, 1), (97, 97), (130, 130)]),
    (4, 90, 260, 2, 2, 128, False, None, [(90, 260), (90, 0), (0, 260), (33, 65)]),
    (3, 70, 70, 8, 1, 96, True, 30, [(70, 10), (10, 70), (64, 64)]),
    (1, 17, 1500, 2, 1, 64, False, None, None),
    (1, 1200, 33, 1, 1, 128, False, None, None),
    (1, 3, 4000, 6, 2, 48, True, None, None),        # few queries, few keys: the way is split
    (2, 60, 5000, 2, 1, 128, True, 1500, [(60, 5000), (60, 100)]),
    (2, 4000, 70, 4, 2, 80, False, None, [(4000, 70), (5, 1)]),
    (1, 9, 40, 130, 1, 16, True, None, None),        # a head's queries in more than one tile
    (2, 5, 70, 131, 1, 8, False, None, [(5, 70), (3, 66)]),
    (2, 200, 180, 15, 3, 64, True, None, None),
    (3, 2500, 2500, 1, 1, 32, True, 700, [(2500, 2500), (0, 0), (2000, 2000)]),
    (1, 515, 515, 2, 2, 127, True, None, None),
]


def make(t, batch, queries, keys, heads, groups, dim, seed=0, sharp=1.0):
    gen = torch.Generator().manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen)

    q, k, v = normal(batch, queries, heads, dim) * sharp, normal(batch, keys, groups, dim), normal(batch, keys, groups, dim)
    return [x.to(t) for x in (q, k, v, normal(batch, queries, heads, dim))]


def on_gpu(lengths):
    if lengths is None:
        return {}
    n, m = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in zip(*lengths))
    return {"q_lengths": n, "k_lengths": m}


def check_forward(got, q, k, v, lengths=None, **mask):
    out, lse, e_out, e_lse = au.forward(q, k, v, lengths=lengths, **mask)
    assert_within(got[0], out, e_out, "out")
    seen = lse != -math.inf
    assert torch.equal(got[1].cpu() == -math.inf, ~seen)
    assert_within(got[1].cpu()[seen], lse[seen], e_lse[seen], "lse")


def check_backward(got, dout, q, k, v, out, lse, lengths=None, **mask):
    for g, (ref, tol), name in zip(got, au.backward(dout, q, k, v, out.cpu(), lse.cpu(), lengths=lengths, **mask),
                                   ("dq", "dk", "dv")):
        assert_within(g, ref, tol, name)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("case", CASES)
def test_against_64_bits(t, case):
    batch, queries, keys, heads, groups, dim, causal, window, lengths = case
    q, k, v, dout = make(t, batch, queries, keys, heads, groups, dim, seed=queries * 7 + keys, sharp=1.5)
    mask = {"causal": causal, "window": window}
    gq, gk, gv, gd = (x.cuda() for x in (q, k, v, dout))
    out, lse = sg.attention(gq, gk, gv, **mask, **on_gpu(lengths))
    check_forward((out, lse), q, k, v, lengths, **mask)
    got = sg.attention_backward(gd, gq, gk, gv, out, lse, **mask, **on_gpu(lengths))
    check_backward(got, dout, q, k, v, out, lse, lengths, **mask)


@pytest.mark.parametrize("t", TYPES)
def test_views_of_one_projection(t):
    """Inputs and gradients that are parts of wider buffers; what lies between them is left as it was."""
    b, n, h, g, d = 2, 83, 4, 2, 64
    every = torch.randn(b, n, h + 2 * g, d + 8, generator=torch.Generator().manual_seed(3)).to(t)
    dout = torch.randn(b, n, h, d, generator=torch.Generator().manual_seed(4)).to(t)
    q, k, v = (x[..., :d] for x in every.split((h, g, g), 2))
    on = every.cuda()
    gq, gk, gv = (x[..., :d] for x in on.split((h, g, g), 2))
    wide = torch.full((b, n, h, d + 8), 7.0, dtype=t, device="cuda")
    out, lse = sg.attention(gq, gk, gv, causal=True, out=wide[..., :d])
    check_forward((out, lse), q, k, v, causal=True)
    assert bool((wide[..., d:] == 7).all())
    dwide = torch.full_like(on, 7.0)
    parts = [x[..., :d] for x in dwide.split((h, g, g), 2)]
    got = sg.attention_backward(dout.cuda(), gq, gk, gv, out, lse, causal=True, dq=parts[0], dk=parts[1], dv=parts[2])
    check_backward(got, dout, q, k, v, out, lse, causal=True)
    assert bool((dwide[..., d:] == 7).all())


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("shift", [1, 3])
def test_heads_off_16_byte_borders(t, shift):
    b, n, h, d = 1, 70, 3, 50
    q, k, v, dout = make(t, b, n, n, h, h, d, seed=5)
    def moved(x):
        flat = torch.empty(x.numel() + shift, dtype=t, device="cuda")
        flat[shift:] = x.flatten().cuda()
        return flat[shift:].view(x.shape)
    gq, gk, gv, gd = (moved(x) for x in (q, k, v, dout))
    out, lse = sg.attention(gq, gk, gv)
    check_forward((out, lse), q, k, v)
    check_backward(sg.attention_backward(gd, gq, gk, gv, moved(out.cpu()), lse), dout, q, k, v, out, lse)


@pytest.mark.parametrize("t", TYPES)
def test_heads_before_tokens(t):
    """[batch, heads, tokens, D] in memory, and one key and value head for all by a stride of 0."""
    b, n, h, d = 2, 75, 4, 64
    q, k, v, dout = make(t, b, n, n, h, 1, d, seed=6)
    turn = lambda x: x.transpose(1, 2).contiguous().cuda().transpose(1, 2)
    gq, gd = turn(q), turn(dout)
    gk, gv = k.cuda().expand(b, n, h, d), v.cuda().expand(b, n, h, d)
    out, lse = sg.attention(gq, gk, gv, causal=True)
    kk, vv = k.expand(b, n, h, d), v.expand(b, n, h, d)
    check_forward((out, lse), q, kk, vv, causal=True)
    check_backward(sg.attention_backward(gd, gq, gk, gv, turn(out.cpu()), lse, causal=True), dout, q, kk, vv, out, lse,
                   causal=True)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("dim", [64, 100])
def test_padding_may_hold_anything(t, dim):
    """NaN and infinities behind the lengths reach nothing; rows there become 0 and -inf."""
    lengths = [(50, 50), (0, 0), (77, 77), (1, 1)]
    q, k, v, dout = make(t, 4, 77, 77, 4, 2, dim, seed=7)
    for b, (n, m) in enumerate(lengths):
        for x, e in ((q, n), (k, m), (v, m), (dout, n)):
            x[b, e:] = torch.tensor([math.nan, math.inf, -math.inf, torch.finfo(t).min]).to(t)[torch.arange(dim) % 4]
    on = [x.cuda() for x in (q, k, v)]
    for mask in ({"causal": True}, {"causal": False, "window": 20}):
        out, lse = sg.attention(*on, **mask, **on_gpu(lengths))
        check_forward((out, lse), q, k, v, lengths, **mask)
        filled, flse = out.clone(), lse.clone()
        for b, (n, _) in enumerate(lengths):
            filled[b, n:], flse[b, :, n:] = math.nan, math.nan
        got = sg.attention_backward(dout.cuda(), *on, filled, flse, **mask, **on_gpu(lengths))
        check_backward(got, dout, q, k, v, out, lse, lengths, **mask)


def test_lengths_outside_are_brought_inside():
    q, k, v, dout = (x.cuda() for x in make(torch.bfloat16, 3, 40, 60, 2, 2, 64, seed=8))
    n = torch.tensor([-5, 41, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    m = torch.tensor([60, -2 ** 31, 61], dtype=torch.int32, device="cuda")
    inside = {"q_lengths": n.clamp(0, 40), "k_lengths": m.clamp(0, 60)}
    a, b = sg.attention(q, k, v, q_lengths=n, k_lengths=m), sg.attention(q, k, v, **inside)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    for x, y in zip(sg.attention_backward(dout, q, k, v, *a, q_lengths=n, k_lengths=m),
                    sg.attention_backward(dout, q, k, v, *b, **inside)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("size", [1e-4, 30.0])
def test_sizes_of_gradients_and_values(t, size):
    """Small and large gradients keep their relative error."""
    q, k, v, dout = make(t, 1, 200, 200, 2, 2, 64, seed=9)
    dout, v = (dout.float() * size).to(t), (v.float() * size).to(t)
    gq, gk, gv, gd = (x.cuda() for x in (q, k, v, dout))
    out, lse = sg.attention(gq, gk, gv, causal=True)
    check_forward((out, lse), q, k, v, causal=True)
    check_backward(sg.attention_backward(gd, gq, gk, gv, out, lse, causal=True), dout, q, k, v, out, lse, causal=True)


@pytest.mark.parametrize("t", TYPES)
def test_sharp_and_rising_scores(t):
    """Scores far apart, and ones that grow along the keys, so that every tile has a new maximum."""
    q, k, v, dout = make(t, 1, 130, 400, 2, 2, 64, seed=10, sharp=8.0)
    k = (k.float() + 0.02 * torch.arange(400).view(1, -1, 1, 1) * q.float()[:, :1].sign()).to(t)
    gq, gk, gv, gd = (x.cuda() for x in (q, k, v, dout))
    out, lse = sg.attention(gq, gk, gv, scale=0.3)
    check_forward((out, lse), q, k, v, scale=0.3)
    check_backward(sg.attention_backward(gd, gq, gk, gv, out, lse, scale=0.3), dout, q, k, v, out, lse, scale=0.3)


@pytest.mark.parametrize("t", TYPES)
def test_not_finite_sequence_touches_no_other(t):
    q, k, v, dout = make(t, 3, 70, 70, 2, 1, 64, seed=11)
    clean = [x.clone().cuda() for x in (q, k, v, dout)]
    out, lse = sg.attention(*clean[:3], causal=True)
    want = sg.attention_backward(clean[3], *clean[:3], out, lse, causal=True)
    for x, value in ((q, math.nan), (k, math.inf), (v, math.nan), (dout, math.inf)):
        x[1, 30] = value
    dirty = [x.cuda() for x in (q, k, v, dout)]
    out2, lse2 = sg.attention(*dirty[:3], causal=True)
    got = sg.attention_backward(dirty[3], *dirty[:3], out2, lse2, causal=True)
    for a, b in zip((out, *want), (out2, *got)):
        assert torch.equal(a[0], b[0]) and torch.equal(a[2], b[2])
    assert torch.equal(lse[0], lse2[0]) and torch.equal(lse[2], lse2[2])


@pytest.mark.parametrize("t", TYPES)
def test_no_queries_no_keys_no_sequences(t):
    for b, n, m in ((2, 0, 5), (2, 5, 0), (0, 5, 5), (1, 0, 0)):
        q, k, v, dout = (x.cuda() for x in make(t, b, n, m, 2, 1, 64))
        out, lse = sg.attention(q, k, v)
        assert out.shape == q.shape and bool((out == 0).all()) and bool((lse == -math.inf).all())
        for g, x in zip(sg.attention_backward(dout, q, k, v, out, lse), (q, k, v)):
            assert g.shape == x.shape and bool((g == 0).all())


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("case", [(2, 300, 300, 4, 2, 128, True), (1, 40, 5000, 2, 2, 64, False), (1, 5000, 40, 2, 2, 64, False)])
def test_repeated_calls_give_the_same_bits(t, case):
    b, n, m, h, g, d, causal = case
    q, k, v, dout = (x.cuda() for x in make(t, b, n, m, h, g, d, seed=12))
    first = None
    for turn in range(3):
        out, lse = sg.attention(q, k, v, causal=causal, workspace=torch.full(
            (max(1, sg.attention_workspace_bytes(q, k)),), 255 * (turn % 2), dtype=torch.uint8, device="cuda"))
        got = (out, lse, *sg.attention_backward(dout, q, k, v, out, lse, causal=causal, workspace=torch.full(
            (max(1, sg.attention_workspace_bytes(q, k, backward=True)),), 255 * (turn % 2), dtype=torch.uint8, device="cuda")))
        first = first or got
        assert all(torch.equal(x, y) for x, y in zip(first, got))


@pytest.mark.parametrize("t", TYPES)
def test_gradients_against_differences(t):
    """Along random directions: the change of sum(out * dout) in 64 bits, with the type's tolerance on the gradients."""
    q, k, v, dout = make(t, 1, 40, 60, 4, 2, 32, seed=13)
    gq, gk, gv, gd = (x.cuda() for x in (q, k, v, dout))
    out, lse = sg.attention(gq, gk, gv, causal=True)
    got = sg.attention_backward(gd, gq, gk, gv, out, lse, causal=True)
    tols = au.backward(dout, q, k, v, out.cpu(), lse.cpu(), causal=True)

    def loss(*qkv):
        total = 0.0
        for _, h, g, _, _, see in au._each(q, k, None, True, None):
            x, y, z = qkv[0][0, :, h], qkv[1][0, :, g], qkv[2][0, :, g]
            p = torch.softmax(torch.where(see, x @ y.t() * 32 ** -0.5, -math.inf), 1)
            total += float((p @ z * dout[0, :, h].double()).sum())
        return total

    start = [x.double() for x in (q, k, v)]
    # delta is taken from out as it is stored: off by half a step of it at most
    e_delta = (dout.double().abs() * (torch.finfo(t).eps / 2 * out.cpu().double().abs())).sum(-1)
    for which in range(3):
        direction = torch.randn(start[which].shape, generator=torch.Generator().manual_seed(which), dtype=torch.float64)
        step = 1e-5
        ends = [loss(*[x + sign * step * direction if i == which else x for i, x in enumerate(start)]) for sign in (1, -1)]
        slope = (ends[0] - ends[1]) / (2 * step)
        mine = float((got[which].double().cpu() * direction).sum())
        tol = float((tols[which][1] * direction.abs()).sum()) + 1e-6 * (1 + abs(slope))
        if which < 2:  # ds moves by p * e_delta, of which a row's p are 1 in all
            other = start[1 - which].abs().amax() * 32 ** -0.5
            tol += float(e_delta.sum() * other * direction.abs().amax() * 32)
        assert abs(mine - slope) <= tol, (which, mine, slope, tol)


def test_captured_and_replayed():
    q, k, v, dout = (x.cuda() for x in make(torch.bfloat16, 2, 100, 100, 4, 2, 64, seed=14))
    n = torch.tensor([100, 60], dtype=torch.int32, device="cuda")
    ws = torch.empty(max(1, sg.attention_workspace_bytes(q, k)), dtype=torch.uint8, device="cuda")
    wsb = torch.empty(max(1, sg.attention_workspace_bytes(q, k, backward=True)), dtype=torch.uint8, device="cuda")
    out, dq, dk, dv = (torch.empty_like(x) for x in (q, q, k, v))
    lse = torch.empty(2, 4, 100, device="cuda")

    def step():
        sg.attention(q, k, v, causal=True, q_lengths=n, k_lengths=n, out=out, lse=lse, workspace=ws)
        sg.attention_backward(dout, q, k, v, out, lse, causal=True, q_lengths=n, k_lengths=n, dq=dq, dk=dk, dv=dv,
                              workspace=wsb)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for turn in range(3):
        q.copy_(torch.randn(q.shape, generator=torch.Generator().manual_seed(turn)))
        n.copy_(torch.tensor([100 - 7 * turn, 50 + turn]))
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in (out, lse, dq, dk, dv)]
        o, l = sg.attention(q, k, v, causal=True, q_lengths=n, k_lengths=n)
        want = (o, l, *sg.attention_backward(dout, q, k, v, o, l, causal=True, q_lengths=n, k_lengths=n))
        assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_on_another_stream():
    q, k, v, dout = (x.cuda() for x in make(torch.float16, 1, 300, 300, 4, 4, 64, seed=15))
    out, lse = sg.attention(q, k, v)
    want = sg.attention_backward(dout, q, k, v, out, lse)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        o, l = sg.attention(q, k, v)
        got = sg.attention_backward(dout, q, k, v, o, l)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip((out, lse, *want), (o, l, *got)))


def test_places_past_32_bits():
    """Heads of a wide buffer: sequence 16 starts past element 2^32, tokens are 2^22 elements apart."""
    b, n, d = 16, 70, 64
    wide = torch.empty(b, n, 1 << 22, dtype=torch.bfloat16, device="cuda")
    q, k, v, dout = make(torch.bfloat16, b, n, n, 2, 1, d, seed=16)
    parts = []
    for x, at in ((q, 0), (k, 1000), (v, 1 << 21), (dout, 3 << 20)):
        part = wide[..., at:at + x.shape[2] * d].unflatten(-1, (-1, d))
        part.copy_(x)
        parts.append(part)
    out, lse = sg.attention(*parts[:3], causal=True)
    got = sg.attention_backward(parts[3], *parts[:3], out, lse, causal=True)
    plain = [x.cuda() for x in (q, k, v, dout)]
    want = sg.attention(*plain[:3], causal=True)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    for x, y in zip(got, sg.attention_backward(plain[3], *plain[:3], *want, causal=True)):
        assert torch.equal(x, y)
    last = [x[-1:] for x in (q, k, v, dout)]
    check_forward((out[-1:], lse[-1:]), *last[:3], causal=True)


def test_tokens_too_far_apart_for_one_tile():
    """64 tokens that lie 2^25 elements apart are past what a tile's loads reach without registers."""
    n, d = 66, 64
    wide = torch.empty(n, 1 << 25, dtype=torch.bfloat16, device="cuda")
    q, k, v, dout = make(torch.bfloat16, 1, n, n, 1, 1, d, seed=17)
    parts = []
    for x, at in ((q, 0), (k, 1024), (v, 1 << 24), (dout, 3 << 20)):
        part = wide[:, at:at + d].view(1, n, 1, d)
        part.copy_(x)
        parts.append(part)
    out, lse = sg.attention(*parts[:3])
    check_forward((out, lse), q, k, v)
    check_backward(sg.attention_backward(parts[3], *parts[:3], out, lse), dout, q, k, v, out, lse)


def test_two_calls_side_by_side():
    """Calls on two streams, each with a workspace, that split their ways."""
    a, b = (make(torch.bfloat16, 1, 20, 6000, 4, 4, 64, seed=s) for s in (18, 19))
    a, b = [x.cuda() for x in a], [x.cuda() for x in b]
    want = []
    for q, k, v, dout in (a, b):
        out, lse = sg.attention(q, k, v)
        want.append((out, lse, *sg.attention_backward(dout, q, k, v, out, lse)))
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [None, None]
    for turn in range(3):
        for i, (q, k, v, dout) in enumerate((a, b)):
            with torch.cuda.stream(streams[i]):
                out, lse = sg.attention(q, k, v)
                got[i] = (out, lse, *sg.attention_backward(dout, q, k, v, out, lse))
        torch.cuda.synchronize()
        for x, y in zip(want, got):
            assert all(torch.equal(u, w) for u, w in zip(x, y))
