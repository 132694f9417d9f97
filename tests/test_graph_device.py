"""DecodeGraph of a pool whose device is not the current one, with torch's CUDA
module replaced by a record of what it is asked for (no second GPU is needed)."""
import contextlib
import types

import pytest


class FakeCuda:
    """The parts of torch.cuda that DecodeGraph uses: a current device and, on
    each device, a current stream (None: its default one)."""

    def __init__(self):
        self.at, self.streams, self.captured, self.replayed = 0, {0: None, 1: None}, [], []

    @contextlib.contextmanager
    def device(self, d):
        before, self.at = self.at, d.index
        yield
        self.at = before

    def Stream(self):
        return types.SimpleNamespace(device=self.at, wait_stream=lambda s: None)

    def current_stream(self):
        return types.SimpleNamespace(device=self.at, wait_stream=lambda s: None)

    @contextlib.contextmanager
    def stream(self, s):
        before, self.streams[s.device] = self.streams[s.device], s
        yield
        self.streams[s.device] = before

    def CUDAGraph(self):
        return types.SimpleNamespace(replay=lambda: self.replayed.append(self.at))

    @contextlib.contextmanager
    def graph(self, g):
        with self.stream(types.SimpleNamespace(device=self.at, capturing=True)):
            yield


@pytest.mark.parametrize("index", [0, 1])
def test_the_graph_is_captured_on_the_pools_device(monkeypatch, index):
    torch = pytest.importorskip("torch")
    import prefix_shared_decode_gb300 as P
    cuda = FakeCuda()
    for name in ("device", "Stream", "current_stream", "stream", "CUDAGraph", "graph"):
        monkeypatch.setattr(torch.cuda, name, getattr(cuda, name))
    seen = []

    def call(pool, sched, q, **kw):             # a call runs on its pool's device's current stream
        s = cuda.streams[pool._device.index]
        seen.append("default" if s is None else "captured" if getattr(s, "capturing", False) else "side")

    monkeypatch.setattr(P, "decode_attention", call)
    pool = types.SimpleNamespace(_device=torch.device("cuda", index))
    sched = types.SimpleNamespace(_key=lambda: 1, workspace=lambda: "ws")
    g = P.DecodeGraph(pool, sched, [(0, "q", "out"), (1, "q", "out")])
    assert seen == ["side", "side", "captured", "captured"]
    g.replay()
    assert cuda.replayed == [index] and cuda.at == 0 and len(seen) == 4
