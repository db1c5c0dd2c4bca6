"""The binding's current stream, with and without torch's short way to it (CPU)."""
import importlib.util
import types

import torch


def test_current_stream_without_the_short_way(monkeypatch):
    from sparse_attention_fp4_gb300 import build
    build.build()
    from sparse_attention_fp4_gb300 import fp4idx
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev: types.SimpleNamespace(cuda_stream=1000 + dev))
    spec = importlib.util.spec_from_file_location("fp4idx_without", fp4idx.__file__)
    other = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(other)
    monkeypatch.setattr(other, "_current_device", lambda: 3)
    assert other._here(None) == (3, 1003)
    assert other._here(types.SimpleNamespace(cuda_stream=77)) == (3, 77)
