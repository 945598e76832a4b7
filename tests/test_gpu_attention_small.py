"""fp16 attention whose results are made of small probabilities, or of gradients
of unequal size: fp16 has few binary digits below 1."""
import math

import pytest
import torch

import sparse_gradient_reduction_amd as sg
from tests import attention_util as au
from tests.operator_util import assert_within, half_step
from tests.test_gpu_attention import check_forward, make

pytestmark = pytest.mark.gpu

BOOST = 13  # the probabilities that the products take are held 2^13 times as large: fp16's smallest step is then 2^-37


def check_small(got, q, k, v, **mask):
    """As check_forward, with fp16's smallest steps (half of one: 2^-25) lowered by the boost."""
    out, lse, e_out, e_lse = au.forward(q, k, v, **mask)
    less = (2.0 ** -25 - 2.0 ** -(25 + BOOST)) * v.double().abs().sum(1)  # [batch, groups, D]
    e_out = e_out - less.repeat_interleave(q.shape[2] // k.shape[2], 1)[:, None]
    assert bool((e_out > 0).all())
    assert_within(got[0], out, e_out, "out")
    assert_within(got[1], lse, e_lse, "lse")


def one_large(queries, keys, heads, dim, at):
    """Scores 0 but for key `at`, which is 10 to 18 above (by query) and whose value is 0."""
    q, k = torch.zeros(1, queries, heads, dim), torch.zeros(1, keys, 1, dim)
    q[..., 0] = torch.linspace(10, 18, queries).view(1, -1, 1)
    k[:, at, :, 0] = 1
    v = 1000 * (0.5 + torch.rand(1, keys, 1, dim, generator=torch.Generator().manual_seed(keys)))
    v[:, at] = 0
    return q.half(), k.half(), v.half()


@pytest.mark.parametrize("at", ["first", "middle", "last"])
@pytest.mark.parametrize("keys,heads", [(1000, 1), (4096, 1), (16384, 2), (16384, 1)])
@pytest.mark.parametrize("dim", [64, 50])
def test_one_key_takes_most_of_a_row(at, keys, heads, dim):
    """1000 keys are walked over in one part, more of them in several; the weak keys make the result."""
    q, k, v = one_large(33, keys, heads, dim, {"first": 0, "middle": keys // 2 + 5, "last": keys - 1}[at])
    got = sg.attention(q.cuda(), k.cuda(), v.cuda(), scale=1.0)
    check_small(got, q, k, v, scale=1.0)


def test_one_key_takes_most_of_a_row_in_many_workgroups():
    """4096 keys and 260 heads: enough workgroups for one part each."""
    q, k, v = one_large(33, 4096, 1, 64, 0)
    heads = lambda x: x.cuda().expand(-1, -1, 260, -1)
    out, lse = sg.attention(heads(q), heads(k), heads(v), scale=1.0)
    assert torch.equal(out, out[:, :, :1].expand_as(out)) and torch.equal(lse, lse[:, :1].expand_as(lse))
    check_small((out[:, :, :1], lse[:, :1]), q, k, v, scale=1.0)


@pytest.mark.parametrize("rise", [0.5, 1.9, 2.1, 7.9, 8.1])
def test_rising_scores_stay_in_range(rise):
    """From one tile of 64 keys to the next all scores rise by 2^rise: the largest
    probabilities there are before the running maximum is moved on."""
    keys = 64 * 12
    q, k = torch.zeros(1, 40, 2, 32), torch.zeros(1, keys, 1, 32)
    q[..., 0] = 1
    k[..., 0] = (rise * math.log(2.0) * (torch.arange(keys) // 64)).view(1, -1, 1)
    v = torch.randn(1, keys, 1, 32, generator=torch.Generator().manual_seed(1)) * 10
    q, k, v = q.half(), k.half(), v.half()
    got = sg.attention(q.cuda(), k.cuda(), v.cuda(), scale=1.0)
    assert bool(torch.isfinite(got[0]).all())
    check_small(got, q, k, v, scale=1.0)


@pytest.mark.parametrize("sharp", [0.3, 1.5, 6.0])
def test_random_scores(sharp):
    q, k, v, _ = make(torch.float16, 2, 130, 500, 4, 2, 80, seed=31, sharp=sharp)
    got = sg.attention(q.cuda(), k.cuda(), v.cuda())
    check_forward(got, q, k, v)
    check_small(got, q, k, v)


@pytest.mark.parametrize("keys", [1, 64, 1024, 16384])
def test_equal_scores_have_an_exact_sum(keys):
    """Scores of 0 over 2^n keys: lse is the logarithm of 2^n, rounded as fp32's is (and 0 for one key)."""
    q, k = torch.zeros(1, 3, 1, 64, dtype=torch.float16, device="cuda"), torch.ones(1, keys, 1, 64, dtype=torch.float16, device="cuda")
    out, lse = sg.attention(q, k, k)
    _, lse32 = sg.attention(q.float(), k.float(), k.float())
    assert bool((out == 1).all()) and torch.equal(lse, lse32)
    assert abs(float(lse[0, 0, 0]) - math.log(keys)) <= 4 * 2.0 ** -24 * math.log(keys)


def assert_rounded(got, ref, tol, name):
    """assert_within, with values from 65520 on (half a step past fp16's largest, 65504) rounded to infinity."""
    got, limit = got.double().cpu(), 65520
    past, may_be = ref.abs() - tol >= limit, (ref.abs() + tol >= limit) & (got.abs() == math.inf)
    assert torch.equal(got[past], math.inf * ref[past].sign())
    assert torch.equal(got[may_be].sign(), ref[may_be].sign())
    rest = ~(past | may_be)
    assert_within(got[rest], ref[rest], tol[rest], name)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("keys", [200, 3000])
def test_gradients_of_rows_of_unequal_size(causal, keys):
    """A row's dq has the digits that its own dout leaves, whatever other rows'
    are; the queries' dout falls from 2^12 to 2^-12. With the ds of a row below
    2^15 and its steps 2^-25 at worst (half of fp16's smallest), dq is off by
    2^-36 |dout| max |v| a key, |dout| that row's own."""
    n, d, scale = 90, 64, 0.125
    q, k, v, dout = make(torch.float16, 1, n, keys, 2, 1, d, seed=32)
    v = (v.float() * 500).half()
    dout = (dout.float() * 2.0 ** torch.linspace(12, -12, n).view(1, -1, 1, 1)).half()
    gq, gk, gv, gd = (x.cuda() for x in (q, k, v, dout))
    out, lse = sg.attention(gq, gk, gv, causal=causal, scale=scale)
    got = sg.attention_backward(gd, gq, gk, gv, out, lse, causal=causal, scale=scale)
    for x, (ref, tol), name in zip(got, au.backward(dout, q, k, v, out.cpu(), lse.cpu(), causal=causal, scale=scale), ("dq", "dk", "dv")):
        assert_rounded(x, ref, tol, name)
    for h in range(2):
        x = [y.double() for y in (dout[0, :, h], q[0, :, h], k[0, :, 0], v[0, :, 0], out[0, :, h].cpu(), lse[0, h].cpu())]
        see = au.sees(n, keys, n, keys, causal, None)
        r = au.head_backward(*x, see, scale, torch.float16)
        own = x[0].norm(dim=1, keepdim=True)
        spare = 2.0 ** -36 * (own.max() - own) * x[3].norm(dim=1).max()  # of the other rows' size
        tol = r[3] - scale * (see * spare) @ x[2].abs() + half_step(torch.float16, r[0])
        assert bool((tol > 0).all())
        assert_rounded(got[0][0, :, h], r[0], tol, "dq")
