"""The first calls of several threads at once: torch's functions are looked up
once for all operators, and no thread may meet half of that.  No CUDA call is
made."""
import threading

import pytest

torch = pytest.importorskip("torch")

import entropy_bounded_softmax_gb300 as cs

NAMES = ("_cuda_getDevice", "_cuda_getCurrentRawStream")


class Slow:
    """torch._C whose first look at `name` waits until it is let go."""

    def __init__(self, name):
        self.name, self.first = name, threading.Lock()
        self.reached, self.go = threading.Event(), threading.Event()

    def __getattr__(self, name):
        if name == self.name and self.first.acquire(blocking=False):
            self.reached.set()
            assert self.go.wait(60)
        return {"_cuda_getDevice": lambda: 0,
                "_cuda_getCurrentRawStream": lambda index: 100 + index}[name]


@pytest.mark.parametrize("held", NAMES)
@pytest.mark.parametrize("call", ["device", "stream"])
def test_a_thread_in_the_middle_of_the_look_up(monkeypatch, held, call):
    slow = Slow(held)
    monkeypatch.setattr(cs, "_raw_stream", None)
    monkeypatch.setattr(cs, "_current_device", None)
    monkeypatch.setattr(torch, "_C", slow)
    failed = []

    def work(device):
        try:
            assert cs._on_device(device) is cs._STAY
            assert cs._stream_handle(device) == 100
        except BaseException as e:
            failed.append(e)

    first = threading.Thread(target=work, args=(torch.device("cuda", 0),))
    first.start()
    assert slow.reached.wait(60)
    try:
        device = torch.device("cuda", 0) if call == "device" else \
            torch.device("cuda")
        if call == "device":
            assert cs._on_device(device) is cs._STAY
        else:
            assert cs._stream_handle(device) == 100
    finally:
        slow.go.set()
        first.join(60)
    assert not failed and not first.is_alive()
    assert cs._raw_stream(3) == 103 and cs._current_device() == 0
