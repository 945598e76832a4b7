"""Attention and its gradients where ways are split and joined: few and many
parts of every width of heads, with loads that go to LDS directly and through
registers."""
import pytest
import torch

import sparse_gradient_reduction_amd as sg
from tests.test_gpu_attention import check_backward, check_forward, make, on_gpu

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]
# for tiles of 32, 64, 96 and 128 columns; 27, 50, 77 and 121 are not whole 16 bytes
DIMS = [32, 27, 64, 50, 96, 80, 77, 128, 121]


def run(t, batch, queries, keys, heads, groups, dim, seed, lengths=None, **mask):
    q, k, v, dout = make(t, batch, queries, keys, heads, groups, dim, seed=seed)
    gq, gk, gv, gd = (x.cuda() for x in (q, k, v, dout))
    out, lse = sg.attention(gq, gk, gv, **mask, **on_gpu(lengths))
    check_forward((out, lse), q, k, v, lengths, **mask)
    got = sg.attention_backward(gd, gq, gk, gv, out, lse, **mask, **on_gpu(lengths))
    check_backward(got, dout, q, k, v, out, lse, lengths, **mask)
    return sg.attention_workspace_bytes(gq, gk), sg.attention_workspace_bytes(gq, gk, backward=True)


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("keys", [1100, 2600])
def test_keys_in_parts(t, dim, keys):
    """1100 keys are 4 parts of 16-bit types, 2600 are 10; fp32 has more."""
    forward, _ = run(t, 2, 5, keys, 2, 1, dim, dim + keys, [(5, keys), (3, keys - 71)], causal=True)
    assert forward > 0


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("queries", [1100, 2600])
def test_queries_in_parts(t, dim, queries):
    """The same with the parts of the queries that dk and dv are summed over."""
    _, backward = run(t, 1, queries, 40, 2, 2, dim, dim + queries, [(queries - 100, 37)], causal=False)
    sums = 2 * queries * 2 * 4  # the rows' lse and delta, and fp16's norms
    assert backward > sums + 256 + 2 * 2 * 64 * 4


@pytest.mark.parametrize("t", TYPES)
@pytest.mark.parametrize("dim", [32, 80, 96, 128])
def test_windows_in_parts(t, dim):
    """Parts of which a row sees few, or none."""
    run(t, 1, 200, 4000, 1, 1, dim, dim, None, causal=True, window=1300)
