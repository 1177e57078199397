"""A Workspace's buffers and captured graphs, with a stand-in for torch that has two
devices: what is asked is the stream of the buffer's own device."""
import contextlib
import types

import pytest

import bit_nf4_quantized_07_amd as q


class Buffer:
    is_cuda = True

    def __init__(self, n, device):
        self.n, self.device = n, types.SimpleNamespace(type="cuda", index=device)

    def numel(self):
        return self.n

    def record_stream(self, stream):
        pass


@pytest.fixture
def torch_of_two(monkeypatch):
    """`captured`: the devices whose current stream is being captured."""
    state = types.SimpleNamespace(current=0, captured=set())

    @contextlib.contextmanager
    def device(d):
        before, state.current = state.current, d.index
        yield
        state.current = before

    cuda = types.SimpleNamespace(current_device=lambda: state.current, device=device,
                                 is_current_stream_capturing=lambda: state.current in state.captured)
    stand_in = types.SimpleNamespace(cuda=cuda, uint8=None,
                                     empty=lambda n, dtype, device: Buffer(n, device))
    monkeypatch.setattr(q, "_torch", lambda: stand_in)
    return state


@pytest.mark.parametrize("current", [0, 1])
def test_a_captured_buffer_is_kept(torch_of_two, current):
    state, ws = torch_of_two, q.Workspace(1)
    state.current = current
    first, _ = ws.get(10)
    assert ws._captured == []
    state.captured = {1}
    assert ws.get(10)[0] is first
    state.captured = set()
    assert ws.get(20)[0] is not first and ws._captured == [first]
    assert state.current == current


def test_another_device_s_capture_keeps_nothing(torch_of_two):
    state, ws = torch_of_two, q.Workspace(1)
    state.captured = {0}
    ws.get(10)
    assert ws._captured == []
