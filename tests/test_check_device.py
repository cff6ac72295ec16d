"""check() waits for the stream of the workspace's device, not of the current
one (fakes of the device calls; no GPU needed)."""
import contextlib

import torch

from w4_weight_only_b200 import api


class Workspace:
    device, is_cuda = torch.device("cuda", 1), True

    def data_ptr(self):
        return 0x1000

    def numel(self):
        return 256


def test_check_waits_on_the_workspaces_device(monkeypatch):
    current, calls = [0], []

    @contextlib.contextmanager
    def device(dev):
        keep, current[0] = current[0], torch.device(dev).index
        yield
        current[0] = keep

    stream = lambda i: 1000 + i
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current[0])
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_stream",
                        lambda: type("S", (), {"cuda_stream": stream(current[0])}))
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", stream, raising=False)
    value = lambda x: getattr(x, "value", x)
    monkeypatch.setattr(api, "call", lambda name, *a: calls.append((name, current[0], value(a[-1]))))
    ws = Workspace()
    api.check(ws)
    assert calls == [("w4a_check", 1, 1001)] and current == [0]
    ws.device = torch.device("cuda", 0)
    api.check(ws)
    assert calls[1] == ("w4a_check", 0, 1000)
