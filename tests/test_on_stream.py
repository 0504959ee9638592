"""When a pipeline object switches to its own stream or device, on the CPU with a fake of the CUDA runtime's
current device and stream."""
import pytest

torch = pytest.importorskip("torch")
pytest.importorskip("moe_expert_routing_top_gb300._native")
from moe_expert_routing_top_gb300 import pipeline  # noqa: E402


class _Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


def _object(device, stream):
    o = pipeline._OnStream()
    o.device, o.stream = torch.device(device), stream
    return o


@pytest.mark.parametrize("device,stream,current,handle,want", [
    ("cpu", _Stream(7), 0, 9, False),
    ("cuda:0", _Stream(7), 0, 7, False), ("cuda:0", 7, 0, 7, False), ("cuda:0", _Stream(7), 0, 9, True), ("cuda:0", 7, 0, 9, True),
    ("cuda:1", _Stream(7), 0, 7, True),              # the same handle, but another device is the current one
    ("cuda:1", 0, 0, 0, True), ("cuda:1", _Stream(7), 1, 7, False),
    ("cuda", _Stream(7), 3, 7, False), ("cuda", _Stream(7), 3, 9, True)])
def test_elsewhere(monkeypatch, device, stream, current, handle, want):
    asked = []
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current)
    monkeypatch.setattr(pipeline.nat, "current_handle", lambda index=None: asked.append(index) or handle)
    o = _object(device, stream)
    assert o._elsewhere() is want
    assert all(i == o.device.index for i in asked)
    if not want:
        assert o._on_stream() is pipeline._AS_IT_IS


def test_results_are_recorded_elsewhere_alone(monkeypatch):
    seen = []
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda self, s: seen.append((self.data_ptr(), s)))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: ("current", device))
    o, t = _object("cuda:1", _Stream(7)), torch.zeros(3)
    for there in (False, True):
        monkeypatch.setattr(pipeline._OnStream, "_elsewhere", lambda self: there)
        assert o._results(t) == (t,)
    assert seen == [(t.data_ptr(), ("current", torch.device("cuda:1")))]
    for cls in (pipeline.RoutingStats, pipeline.ExpertLayer):
        assert issubclass(cls, pipeline._OnStream) and "_elsewhere" not in vars(cls)
