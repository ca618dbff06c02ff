"""CPU check: whether a call is being captured is asked of the layer's device,
not of the one that happens to be current."""
from __future__ import annotations

import contextlib

import torch

from dense_gemm_18_amd import MoeLayer, binding


def test_capture_is_asked_of_the_layers_device(monkeypatch):
    current = [0]

    @contextlib.contextmanager
    def on(device):
        before, current[0] = current[0], torch.device(device).index
        yield
        current[0] = before

    made = []

    def zeros(n, dtype, device):
        made.append((n, device.index))
        return torch.empty(16, dtype=torch.uint8)

    layer = MoeLayer.__new__(MoeLayer)
    layer.device, layer.topk, layer._workspaces = torch.device("cuda", 1), 2, {}
    layer._weights = binding.moe_nt_weights(None, None, None, None, None, None, None, 8, 256, 64,
                                            0, 0)
    layer._ws_bytes = binding.moe_nt_ws_size(64, layer._weights, 2)
    monkeypatch.setattr(torch.cuda, "device", on)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    # device 1 captures, device 0, the current one, does not
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: current[0] == 1)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 100 + i, raising=False)
    monkeypatch.setattr(torch, "zeros", zeros)
    ws, need, handle = layer._workspace(4, None)
    assert handle == 101 and current == [0]
    assert not layer._workspaces, "a captured call took the layer's own workspace"
    assert need == binding.moe_nt_ws_size(4, layer._weights, 2) and made == [(need, 1)]
    # and the other way round: an eager call while the current device captures
    layer.device = torch.device("cuda", 0)
    current[0] = 1
    ws, need, handle = layer._workspace(4, None)
    assert handle == 100 and list(layer._workspaces) == [100] and need == layer._ws_bytes
