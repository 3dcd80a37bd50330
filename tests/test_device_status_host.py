"""device_status reads the word behind the work of the workspace's own device,
whichever device is current (on the host, with the library and streams faked)."""
import types

import pytest
import torch

import muon_newton_schulz_05_b200 as mb


@pytest.mark.parametrize("device", [torch.device("cuda", 0), torch.device("cuda", 1)])
def test_the_stream_is_the_workspaces_devices(monkeypatch, device):
    calls = []
    current = torch.device("cuda", 0)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: types.SimpleNamespace(
        cuda_stream=100 + torch.device(d if d is not None else current).index))
    monkeypatch.setattr(mb, "_lib", types.SimpleNamespace(muon_device_status=lambda *a: calls.append(a) or 8))
    ws = types.SimpleNamespace(device=device, is_contiguous=lambda: True, data_ptr=lambda: 4096, numel=lambda: 8192,
                               element_size=lambda: 1)
    assert mb.device_status(ws, clear=True) == 8
    assert mb.device_status(ws, stream=7) == 8
    assert calls == [(4096, 8192, 100 + device.index, 1), (4096, 8192, 7, 0)]
