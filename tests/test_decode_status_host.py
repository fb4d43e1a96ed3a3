"""check_decode_status on the CPU: which device's record it asks for."""
from __future__ import annotations

import pytest
import torch

import blackwell_tensor_core_fp16_gb300 as g
from blackwell_tensor_core_fp16_gb300 import decode
from test_decode_host import built_library  # noqa: F401


class Stream:
    def __init__(self, device, handle):
        self.device, self.cuda_stream = torch.device(device), handle


@pytest.mark.parametrize("stream,device,handle", [
    (Stream("cuda:1", 0), 1, 0), (Stream("cuda:2", 0x1230), 2, 0x1230), (0x4560, None, 0x4560)],
    ids=["default stream", "stream", "handle"])
def test_the_streams_device_is_asked(stream, device, handle, monkeypatch):
    current, asked = [None], []

    class Device:
        def __init__(self, x):
            self.x = torch.device(x).index

        def __enter__(self):
            current.append(self.x)

        def __exit__(self, *a):
            current.pop()

    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(decode, "decode_check_status",
                        lambda h: (asked.append((current[-1], h)), (0, 2))[1])
    with pytest.raises(g.GemmError, match="cache slot"):
        g.check_decode_status(stream)
    assert asked == [(device, handle)] and current == [None]
