"""Keys within a sequence's length that a window leaves to no query: their values
reach no result, and their gradients are 0."""
import math

import pytest
import torch

import sparse_gradient_reduction_amd as sg
from tests.attention_util import sees
from tests.test_gpu_attention import check_backward, check_forward, make, on_gpu

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]
# batch, queries, keys, heads, groups, D, causal, window, lengths: the first keys
# that are seen lie inside a wave's 32 (141, 3441 and 42, 81, 201, 17)
CASES = [
    (1, 60, 300, 2, 1, 64, True, 100, None),
    (1, 60, 300, 3, 3, 50, False, 100, None),
    (2, 60, 5000, 2, 1, 128, True, 1500, [(60, 5000), (60, 1601)]),
    (3, 40, 260, 4, 2, 96, True, 20, [(40, 140), (0, 77), (7, 227)]),
    (1, 1, 48, 1, 1, 33, True, 31, None),
]
ODD = {"nan": [math.nan], "infinite": [math.inf, -math.inf], "huge": [3e4, -6e4]}


def unseen_keys(batch, queries, keys, causal, window, lengths):
    """[batch, keys]: no query sees the key."""
    each = lengths or [(queries, keys)] * batch
    return torch.stack([~sees(n, m, queries, keys, causal, window).any(0) for n, m in each])


def both(q, k, v, dout, lengths, mask):
    on = [x.cuda() for x in (q, k, v)]
    out, lse = sg.attention(*on, **mask, **on_gpu(lengths))
    return (out, lse, *sg.attention_backward(dout.cuda(), *on, out, lse, **mask, **on_gpu(lengths)))


@pytest.mark.parametrize("t,odd,which", [(t, odd, which) for t in TYPES for odd in ("nan", "infinite") for which in "kv"
                                         if (t, odd, which) != (torch.float16, "infinite", "v")])  # that one: below
@pytest.mark.parametrize("case", CASES)
def test_gradients_of_unseen_keys_are_zero(t, odd, which, case):
    batch, queries, keys, heads, groups, dim, causal, window, lengths = case
    mask = {"causal": causal, "window": window}
    q, k, v, dout = make(t, batch, queries, keys, heads, groups, dim, seed=21)
    unseen = unseen_keys(batch, queries, keys, causal, window, lengths)
    assert bool(unseen.any())
    k[unseen], v[unseen] = 0, 0
    want = both(q, k, v, dout, lengths, mask)
    check_forward(want[:2], q, k, v, lengths, **mask)
    check_backward(want[2:], dout, q, k, v, *want[:2], lengths, **mask)
    dk, dv = k.clone(), v.clone()
    {"k": dk, "v": dv}[which][unseen] = torch.tensor(ODD[odd]).to(t)[torch.arange(dim) % len(ODD[odd])]
    got = both(q, dk, dv, dout, lengths, mask)
    for x, y, name in zip(got, want, ("out", "lse", "dq", "dk", "dv")):
        assert torch.equal(x, y), name
    assert bool((got[3].cpu()[unseen] == 0).all()) and bool((got[4].cpu()[unseen] == 0).all())


@pytest.mark.parametrize("odd", ["infinite", "huge"])
@pytest.mark.parametrize("case", CASES)
def test_unseen_values_do_not_size_fp16_gradients(odd, case):
    """fp16 holds ds by the largest values that some query sees."""
    batch, queries, keys, heads, groups, dim, causal, window, lengths = case
    mask = {"causal": causal, "window": window}
    q, k, v, dout = make(torch.float16, batch, queries, keys, heads, groups, dim, seed=22)
    dout = (dout.float() * 100).half()
    unseen = unseen_keys(batch, queries, keys, causal, window, lengths)
    v[unseen] = 0
    want = both(q, k, v, dout, lengths, mask)
    check_backward(want[2:], dout, q, k, v, *want[:2], lengths, **mask)
    dirty = v.clone()
    dirty[unseen] = torch.tensor(ODD[odd]).half()[torch.arange(dim) % len(ODD[odd])]
    got = both(q, k, dirty, dout, lengths, mask)
    for x, y, name in zip(got, want, ("out", "lse", "dq", "dk", "dv")):
        assert torch.equal(x, y), name
