"""The binding under a torch that lacks the private names it prefers for their lower host time."""
import importlib.util
import os

import torch

import w4a4_gemm_quantize_b200 as nv


def test_streams_and_devices_without_torchs_private_names(monkeypatch):
    monkeypatch.delattr(torch._C, "_cuda_getDevice", raising=False)
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    asked = []

    class Stream:
        cuda_stream = 1234

    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: asked.append(device) or Stream())
    path = os.path.join(os.path.dirname(nv.__file__), "__init__.py")
    spec = importlib.util.spec_from_file_location("binding_without_private_names", path)
    binding = importlib.util.module_from_spec(spec)
    monkeypatch.setitem(__import__("sys").modules, spec.name, binding)
    spec.loader.exec_module(binding)
    assert binding._stream(None) == 1234 and asked == [3]
    assert binding._stream(Stream()) == 1234 and binding._stream(7) == 7
    assert binding._current_device() == 3 and binding._current_stream(2) == 1234 and asked[-1] == 2
