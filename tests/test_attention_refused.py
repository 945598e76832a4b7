"""What attention and the norms of queries and keys refuse, on the host: the C
calls before anything is launched, the Python calls by their checks (tensors
without storage stand for the GPU's)."""
import ctypes
import math
import os

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import sparse_gradient_reduction_amd as sg

if not os.path.exists(sg.LIB_PATH):
    pytest.skip("libsparcml.so not built", allow_module_level=True)

A, ODD, HALF = 4096, 4097, 4098  # never dereferenced
BAD, OK, WS = sg.ERR_INVALID_ARG, sg.OK, sg.ERR_WORKSPACE
u32, u64, f32 = ctypes.c_uint32, ctypes.c_uint64, ctypes.c_float


class Heads(ctypes.Structure):
    _fields_ = [("data", u64), ("batch", u64), ("token", u64), ("head", u64)]


class Attention(ctypes.Structure):
    _fields_ = ([(n, u32) for n in "type batch queries keys heads groups dim before after".split()] + [("scale", f32)]
                + [(n, u64) for n in ("q_lengths", "k_lengths")] + [(n, Heads) for n in "q k v out".split()]
                + [("lse", u64)] + [(n, Heads) for n in "dout dq dk dv".split()])


class HeadNorm(ctypes.Structure):
    _fields_ = ([(n, u32) for n in "type nodes heads groups dim rotated interleaved".split()] + [("eps", f32), ("tokens", u64)]
                + [(n, Heads) for n in "q k q_out k_out".split()]
                + [(n, u64) for n in "q_weight k_weight positions frequencies".split()] + [(n, Heads) for n in ("dq", "dk")]
                + [(n, u64) for n in "dq_weight dk_weight dq_stride dk_stride".split()])


def attention_args(**change):
    h = Heads(A, 4 * 2 * 64, 2 * 64, 64)
    values = dict(type=1, batch=2, queries=4, keys=4, heads=2, groups=2, dim=64, before=0xFFFFFFFF, after=0, scale=0.125,
                  q=h, k=h, v=h, out=h, lse=A, dout=h, dq=h, dk=h, dv=h)
    values.update(change)
    return Attention(**values)


def norm_args(**change):
    h = Heads(A, 0, 2 * 64, 64)
    values = dict(type=1, nodes=1, heads=2, groups=2, dim=64, rotated=64, eps=1e-6, tokens=4, q=h, k=h, q_out=h, k_out=h,
                  q_weight=A, k_weight=A, positions=A, frequencies=A, dq=h, dk=h, dq_weight=A, dk_weight=A, dq_stride=64,
                  dk_stride=64)
    values.update(change)
    return HeadNorm(**values)


def test_the_binding_packs_what_the_header_declares():
    assert sg._ATTENTION_ARGS.size == ctypes.sizeof(Attention)
    assert sg._HEAD_NORM_ARGS.size == ctypes.sizeof(HeadNorm)


ATTENTION_BAD = [dict(type=3), dict(batch=65536), dict(queries=1 << 29), dict(keys=1 << 29), dict(heads=0), dict(heads=65536),
                 dict(groups=0), dict(groups=3), dict(dim=0), dict(dim=129), dict(scale=0.0), dict(scale=-1.0),
                 dict(scale=1e-31), dict(scale=math.nan), dict(scale=math.inf), dict(q_lengths=HALF), dict(k_lengths=HALF),
                 dict(q=Heads(0, 0, 0, 0)), dict(k=Heads(0, 0, 0, 0)), dict(v=Heads(ODD, 0, 0, 0)), dict(out=Heads(0, 0, 0, 0)),
                 dict(lse=0), dict(lse=HALF), dict(q=Heads(A, 1 << 40, 0, 0)), dict(k=Heads(A, 0, 1 << 40, 0)),
                 dict(v=Heads(A, 0, 0, 1 << 40)), dict(type=0, q=Heads(HALF, 0, 0, 0)),
                 dict(batch=65535, heads=256, groups=256, queries=1 << 20)]


@pytest.mark.parametrize("bad", ATTENTION_BAD, ids=lambda b: ",".join(b))
def test_attention(bad):
    L, a = sg.lib(), attention_args(**bad)
    assert L.sparcml_attention(ctypes.addressof(a), A, 1 << 40, None) == BAD
    assert L.sparcml_attention_backward(ctypes.addressof(a), A, 1 << 40, None) == BAD


def test_attention_backward_arrays():
    L = sg.lib()
    for name in ("dout", "dq", "dk", "dv"):
        for h in (Heads(0, 0, 0, 0), Heads(ODD, 0, 0, 0), Heads(A, 0, 1 << 40, 0)):
            a = attention_args(**{name: h})
            assert L.sparcml_attention_backward(ctypes.addressof(a), A, 1 << 40, None) == BAD, name


def test_attention_nothing_to_do_and_workspaces():
    L, none = sg.lib(), Heads(0, 0, 0, 0)
    assert L.sparcml_attention(None, None, 0, None) == BAD and L.sparcml_attention_backward(None, None, 0, None) == BAD
    assert L.sparcml_attention_workspace(None) == 0 and L.sparcml_attention_backward_workspace(None) == 0
    empty = attention_args(batch=0, q=none, k=none, v=none, out=none, lse=0, dout=none, dq=none, dk=none, dv=none)
    assert L.sparcml_attention(ctypes.addressof(empty), None, 0, None) == OK
    assert L.sparcml_attention_backward(ctypes.addressof(empty), None, 0, None) == OK
    for bad in (dict(type=3), dict(groups=3), dict(dim=129)):
        a = attention_args(**bad)
        assert L.sparcml_attention_workspace(ctypes.addressof(a)) == 0
    long = attention_args(queries=1, keys=100000)
    need = L.sparcml_attention_workspace(ctypes.addressof(long))
    assert need > 0
    for ws, n in ((None, need), (A + 128, need), (A, need - 1)):
        assert L.sparcml_attention(ctypes.addressof(long), ws, n, None) == WS
    # what is enough without a mask is enough with any
    for before, after in ((0xFFFFFFFF, 0), (99, 99), (5000, 0), (0, 0)):
        a = attention_args(queries=1, keys=100000, before=before, after=after)
        assert L.sparcml_attention_workspace(ctypes.addressof(a)) <= need
        b = attention_args(queries=1, keys=100000, before=before, after=0xFFFFFFFF)
        assert L.sparcml_attention_backward_workspace(ctypes.addressof(a)) <= L.sparcml_attention_backward_workspace(ctypes.addressof(b))
    a = attention_args()
    need = L.sparcml_attention_backward_workspace(ctypes.addressof(a))
    for ws, n in ((None, need), (A + 128, need), (A, need - 1)):
        assert L.sparcml_attention_backward(ctypes.addressof(a), ws, n, None) == WS


NORM_BAD = [dict(type=3), dict(nodes=0), dict(nodes=65536), dict(heads=0), dict(heads=65536), dict(groups=0),
            dict(groups=65536), dict(dim=0), dict(dim=257), dict(rotated=66), dict(rotated=3), dict(eps=-1.0),
            dict(eps=math.nan), dict(eps=math.inf), dict(tokens=1 << 31), dict(q=Heads(0, 0, 0, 0)), dict(k=Heads(ODD, 0, 0, 0)),
            dict(q_out=Heads(0, 0, 0, 0)), dict(k_out=Heads(A, 0, 1 << 40, 0)), dict(q=Heads(A, 0, 0, 1 << 40)),
            dict(q_weight=HALF), dict(k_weight=HALF), dict(positions=0), dict(positions=HALF), dict(frequencies=0),
            dict(frequencies=4100), dict(type=0, q=Heads(HALF, 0, 0, 0))]


@pytest.mark.parametrize("bad", NORM_BAD, ids=lambda b: ",".join(b))
def test_head_norm_rotate(bad):
    L, a = sg.lib(), norm_args(**bad)
    assert L.sparcml_head_norm_rotate(ctypes.addressof(a), None) == BAD
    assert L.sparcml_head_norm_rotate_backward(ctypes.addressof(a), A, 1 << 40, None) == BAD


def test_head_norm_rotate_gradients_and_workspace():
    L = sg.lib()
    assert L.sparcml_head_norm_rotate(None, None) == BAD and L.sparcml_head_norm_rotate_backward(None, A, 1 << 40, None) == BAD
    nodes = norm_args(nodes=2)
    assert L.sparcml_head_norm_rotate(ctypes.addressof(nodes), None) == BAD  # a node's part is the gradients' matter
    for bad in (dict(dq=Heads(0, 0, 0, 0)), dict(dk=Heads(ODD, 0, 0, 0)), dict(dq_weight=HALF), dict(dk_weight=HALF),
                dict(dq_stride=63), dict(dk_stride=0)):
        a = norm_args(**bad)
        assert L.sparcml_head_norm_rotate_backward(ctypes.addressof(a), A, 1 << 40, None) == BAD, bad
    need = L.sparcml_head_norm_rotate_backward_workspace(2, 4, 64)
    assert need > 0
    for nodes_, tokens, dim in ((0, 4, 64), (65536, 4, 64), (2, 1 << 30, 64), (2, 4, 0), (2, 4, 257)):
        assert L.sparcml_head_norm_rotate_backward_workspace(nodes_, tokens, dim) == 0
    for ws, n in ((None, need), (A + 128, need), (A, need - 1)):
        assert L.sparcml_head_norm_rotate_backward(ctypes.addressof(nodes), ws, n, None) == WS
    none = Heads(0, 0, 0, 0)
    empty = norm_args(tokens=0, q=none, k=none, q_out=none, k_out=none, positions=0, frequencies=0)
    assert L.sparcml_head_norm_rotate(ctypes.addressof(empty), None) == OK


@pytest.fixture
def fake():
    with FakeTensorMode():
        yield lambda *shape, t=torch.bfloat16, device="cuda:0": torch.empty(shape, dtype=t, device=device)


def test_attention_tensors(fake):
    q, k, lse = fake(2, 5, 4, 64), fake(2, 7, 2, 64), fake(2, 4, 5, t=torch.float32)
    i32 = torch.int32
    for error, call in (
            (TypeError, lambda: sg.attention(q[0], k, k)), (TypeError, lambda: sg.attention(q, k, fake(2, 7, 2, 64, t=torch.float16))),
            (TypeError, lambda: sg.attention(fake(2, 5, 4, 64, device="cpu"), k, k)),
            (TypeError, lambda: sg.attention(q, fake(2, 7, 2, 64, device="cpu"), k)),
            (TypeError, lambda: sg.attention(q, k, fake(2, 7, 2, 64, device="cuda:1"))),
            (TypeError, lambda: sg.attention(q.to(torch.float64), k.to(torch.float64), k.to(torch.float64))),
            (ValueError, lambda: sg.attention(q, fake(3, 7, 2, 64), fake(3, 7, 2, 64))),
            (ValueError, lambda: sg.attention(q, k, fake(2, 6, 2, 64))),
            (ValueError, lambda: sg.attention(q, fake(2, 7, 2, 32), fake(2, 7, 2, 32))),
            (ValueError, lambda: sg.attention(q, fake(2, 7, 3, 64), fake(2, 7, 3, 64))),
            (ValueError, lambda: sg.attention(q, fake(2, 7, 0, 64), fake(2, 7, 0, 64))),
            (ValueError, lambda: sg.attention(fake(2, 5, 4, 129), fake(2, 7, 2, 129), fake(2, 7, 2, 129))),
            (ValueError, lambda: sg.attention(fake(2, 5, 4, 128)[..., ::2], k, k)),
            (ValueError, lambda: sg.attention(q, k, k, window=0)), (ValueError, lambda: sg.attention(q, k, k, scale=0.0)),
            (ValueError, lambda: sg.attention(q, k, k, scale=math.nan)), (ValueError, lambda: sg.attention(q, k, k, scale=math.inf)),
            (TypeError, lambda: sg.attention(q, k, k, q_lengths=fake(2, t=torch.int64))),
            (ValueError, lambda: sg.attention(q, k, k, k_lengths=fake(3, t=i32))),
            (ValueError, lambda: sg.attention(q, k, k, k_lengths=fake(2, t=i32, device="cuda:1"))),
            (ValueError, lambda: sg.attention(q, k, k, out=fake(2, 5, 4, 32))),
            (TypeError, lambda: sg.attention(q, k, k, out=fake(2, 5, 4, 64, t=torch.float32))),
            (ValueError, lambda: sg.attention(q, k, k, out=fake(2, 5, 1, 64).expand(2, 5, 4, 64))),
            (ValueError, lambda: sg.attention(q, k, k, lse=fake(2, 5, 4, t=torch.float32))),
            (ValueError, lambda: sg.attention(fake(1, (1 << 29), 1, 8), fake(1, 7, 1, 8), fake(1, 7, 1, 8))),
            (ValueError, lambda: sg.attention(fake(65536, 1, 1, 8), fake(65536, 1, 1, 8), fake(65536, 1, 1, 8))),
            (TypeError, lambda: sg.attention(fake(1, 1, 1, 8), fake(1, 100000, 1, 8), fake(1, 100000, 1, 8), workspace=fake(1 << 24))),
            (TypeError, lambda: sg.attention_backward(fake(2, 5, 4, 64, t=torch.float32), q, k, k, q, lse)),
            (ValueError, lambda: sg.attention_backward(fake(2, 5, 2, 64), q, k, k, q, lse)),
            (ValueError, lambda: sg.attention_backward(q, q, k, k, q, fake(2, 5, 4, t=torch.float32))),
            (TypeError, lambda: sg.attention_backward(q, q, k, k, q, fake(2, 4, 5))),
            (ValueError, lambda: sg.attention_backward(q, q, k, k, q, lse, dk=fake(2, 1, 2, 64).expand(2, 7, 2, 64))),
            (TypeError, lambda: sg.attention_backward(q, q, k, k, q, lse, workspace=fake(64)))):
        with pytest.raises(error):
            call()


def test_head_norm_rotate_tensors(fake):
    q, k, w, f = fake(6, 4, 64), fake(6, 2, 64), fake(64, t=torch.float32), fake(32, t=torch.float64)
    pos = fake(6, t=torch.int32)
    n, b = sg.head_norm_rotate, sg.head_norm_rotate_backward
    for error, call in (
            (TypeError, lambda: n(fake(64), k)), (TypeError, lambda: n(fake(6, 4, 64, device="cpu"), k)),
            (TypeError, lambda: n(q, fake(6, 2, 64, t=torch.float16))), (ValueError, lambda: n(q, fake(5, 2, 64))),
            (ValueError, lambda: n(q, fake(6, 2, 32))), (ValueError, lambda: n(fake(6, 4, 257), fake(6, 2, 257))),
            (ValueError, lambda: n(q, fake(6, 0, 64))), (ValueError, lambda: n(fake(6, 4, 128)[..., ::2], k)),
            (TypeError, lambda: n(q.to(torch.float64), k.to(torch.float64))),
            (TypeError, lambda: n(q, k, fake(64))), (ValueError, lambda: n(q, k, fake(63, t=torch.float32))),
            (ValueError, lambda: n(q, k, w, fake(64, t=torch.float32, device="cuda:1"))),
            (TypeError, lambda: n(q, k, w, w, None, f)), (TypeError, lambda: n(q, k, w, w, fake(6, t=torch.int64), f)),
            (ValueError, lambda: n(q, k, w, w, fake(5, t=torch.int32), f)), (TypeError, lambda: n(q, k, w, w, pos, w)),
            (ValueError, lambda: n(q, k, w, w, pos, fake(33, t=torch.float64))),
            (ValueError, lambda: n(q, k, q_out=fake(6, 1, 64).expand(6, 4, 64))), (ValueError, lambda: n(q, k, k_out=q)),
            (ValueError, lambda: n(fake(2, 6, 4, 64)[:, :3], k.view(2, 3, 2, 64))),
            (ValueError, lambda: b(q, k, q, k, nodes=4)), (ValueError, lambda: b(q, k, q, k, nodes=0)),
            (ValueError, lambda: b(k, k, q, k)), (TypeError, lambda: b(q, fake(6, 2, 64, t=torch.float32), q, k)),
            (ValueError, lambda: b(q, k, q, k, nodes=2, dq_weight=fake(1, 64, t=torch.float32))),
            (ValueError, lambda: b(q, k, q, k, nodes=2, dk_weight=fake(1, 64, t=torch.float32).expand(2, 64))),
            (TypeError, lambda: b(q, k, q, k, workspace=fake(64)))):
        with pytest.raises(error):
            call()
    with pytest.raises(ValueError):
        sg.rotation_frequencies(7)
    for nodes, tokens, cols in (((1 << 32) + 1, 4, 8), (1, (1 << 64) + 4, 8), (1, 4, (1 << 32) + 8), (-1, 4, 8)):
        with pytest.raises(ValueError):
            sg.head_norm_rotate_backward_workspace_bytes(nodes, tokens, cols)


def test_frequencies():
    f = sg.rotation_frequencies(8, 10000.0)
    assert f.dtype == torch.float64
    assert torch.allclose(f, torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64), rtol=1e-15)
    assert sg.rotation_frequencies(0).numel() == 0
