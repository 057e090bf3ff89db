"""The stream that the binding's calls go to."""

import types

import pytest
import torch


def test_without_torch_s_short_way_the_public_one_is_asked(monkeypatch):
    from mixture_experts_layer_pft_gb300 import binding as B

    monkeypatch.setattr(torch.cuda, "current_stream", lambda: types.SimpleNamespace(cuda_stream=4242))
    for name in ("_raw_stream", "_raw_device"):
        with monkeypatch.context() as m:
            m.setattr(B, name, None)
            assert B._stream() == 4242


@pytest.mark.gpu
def test_both_ways_name_the_current_stream(monkeypatch):
    from mixture_experts_layer_pft_gb300 import binding as B

    torch.zeros(1, device="cuda")
    side = torch.cuda.Stream()
    for stream in (torch.cuda.current_stream(), side):
        with torch.cuda.stream(stream):
            assert B._stream() == stream.cuda_stream
            with monkeypatch.context() as m:
                m.setattr(B, "_raw_stream", None)
                assert B._stream() == stream.cuda_stream
