"""In which order MxLinear launches, and on which stream, and DeviceLayer's streams: CPU tests with
stand-ins for the streams and the calls."""
import types

import pytest
import torch

import moegen
import quantized_expert_ffn_router_amd as q


class Stream:
    def __init__(self, name, log):
        self.name, self.log, self.cuda_stream = name, log, id(self)

    def wait_stream(self, other):
        if other is not self:
            self.log.append(f"{self.name} waits for {other.name}")

    def synchronize(self):
        self.log.append(f"host waits for {self.name}")


@pytest.fixture
def log(monkeypatch):
    """What happens, in order; tensors stay on the CPU, where nothing is launched."""
    out = []
    current = Stream("current", out)
    call = lambda name: lambda *a: out.append(f"{name} on {(a[-1] or current).name}")  # noqa: E731
    monkeypatch.setattr(q, "_launches_on", lambda device, stream: True)
    monkeypatch.setattr(q, "moe_mx_quant", call("quant"))
    monkeypatch.setattr(q, "moe_mx_pack", call("pack"))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: current)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: Stream("default", out))
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: Stream(f"stream {handle}", out))
    return types.SimpleNamespace(out=out, current=current)


@pytest.mark.parametrize("codes", [False, True])
def test_another_stream_waits_for_the_current_one(log, codes):
    """The weights may still be written there, and the allocator's memory still be read."""
    weight = torch.zeros(16, 64, dtype=torch.uint8) if codes else torch.zeros(16, 128, dtype=torch.bfloat16)
    q.MxLinear(weight, torch.zeros(16, 4, dtype=torch.uint8) if codes else None, stream=Stream("side", log.out))
    quant = [] if codes else ["quant on side"]
    assert log.out == ["side waits for current", *quant, "pack on side", "host waits for side"]


def test_without_a_stream_it_is_the_current_one(log):
    q.MxLinear(torch.zeros(16, 128, dtype=torch.bfloat16))
    assert log.out == ["quant on current", "pack on current", "host waits for current"]


@pytest.mark.parametrize("handle,name", [(4096, "stream 4096"), (0, "default")])
def test_raw_handles(log, handle, name):
    """As every call takes them; 0 is the device's default stream."""
    q.MxLinear(torch.zeros(16, 128, dtype=torch.bfloat16), stream=handle)
    assert log.out == [f"{name} waits for current", f"quant on {name}", f"pack on {name}", f"host waits for {name}"]


@pytest.mark.parametrize("handle,name", [(4096, "stream 4096"), (0, "default"), (None, "current")])
def test_raw_handles_of_a_layer(log, monkeypatch, handle, name):
    monkeypatch.setattr(q, "moe_pack_experts", lambda *a: log.out.append(a[-1]))
    w = moegen.make_layer(moegen.Workload("streams", E=4, k=2, H=128, I=128, T=1))
    q.DeviceLayer(w, device="cpu", stream=handle)
    assert log.out == [handle, f"host waits for {name}"]


def test_a_stream_of_another_gpu():
    """Its kernels would run there, on memory that may not be reachable from it."""
    here = torch.device("cuda:0")
    stream = lambda index: types.SimpleNamespace(cuda_stream=1, device=torch.device("cuda", index))  # noqa: E731
    assert q._launches_on(here, stream(0)) and q._launches_on(here, 4096)
    assert not q._launches_on(here, stream(1)) and not q._launches_on(torch.device("cpu"), stream(0))
