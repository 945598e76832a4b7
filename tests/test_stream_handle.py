"""The stream handle that every call takes: torch's own short way to it, and
the public one where a torch lacks it."""
import types

import pytest
import torch

import sparse_gradient_reduction_amd as sg


def test_public_way(monkeypatch):
    asked = []

    def current(device):
        asked.append(device)
        return types.SimpleNamespace(cuda_stream=1234)

    monkeypatch.setattr(sg, "_raw_stream", None)
    monkeypatch.setattr(torch.cuda, "current_stream", current)
    device = torch.device("cuda", 3)
    assert sg._stream(device) == 1234 and asked == [device]


@pytest.mark.gpu
def test_both_ways_agree(dev, monkeypatch):
    device = torch.zeros(1, device=dev).device
    side = torch.cuda.Stream()
    for stream in (torch.cuda.default_stream(), side):
        with torch.cuda.stream(stream):
            short = sg._stream(device)
            with monkeypatch.context() as m:
                m.setattr(sg, "_raw_stream", None)
                assert sg._stream(device) == short == stream.cuda_stream
