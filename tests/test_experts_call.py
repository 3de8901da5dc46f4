"""A call finds its stream and the current device through torch's public names where the quicker ones are missing (no GPU)."""
import contextlib
import importlib.util
import types

import pytest
import torch

from combine_moe_get_amd import experts


@pytest.mark.parametrize("missing", [(), ("_cuda_getCurrentRawStream",), ("_cuda_getDevice",),
                                     ("_cuda_getCurrentRawStream", "_cuda_getDevice")])
@pytest.mark.parametrize("current", [0, 1])
def test_stream_and_device(missing, current, monkeypatch):
    handles = {0: 70, 1: 71}
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", handles.get, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: current, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: types.SimpleNamespace(cuda_stream=handles[d]))
    entered = []
    monkeypatch.setattr(torch.cuda, "device", lambda d: entered.append(d) or contextlib.nullcontext())
    for name in missing:
        monkeypatch.delattr(torch._C, name)
    spec = importlib.util.spec_from_file_location("combine_moe_get_amd.experts_again", experts.__file__)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    seen = []
    device = torch.device("cuda", 1)
    call = module.ExpertsCall(lambda *a: seen.append(a) or 0, ["x", None], "call", (), "result", device)
    assert call() == "result" and seen == [("x", 71)]
    assert entered == ([] if current == 1 else [device])
    assert call(types.SimpleNamespace(device=device, cuda_stream=9)) == "result" and seen[1] == ("x", 9)
