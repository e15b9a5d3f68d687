"""Host side of the operators' own workspaces: which stream's memory they are.

No GPU is needed: torch's streams and its allocator are stood in for, and the
stand-in notes which stream was current when a block was asked for.
"""

import contextlib

import pytest

import fsdp_layout_aware_gb300 as tide


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle

    def __eq__(self, other):
        return isinstance(other, Stream) and self.cuda_stream == other.cuda_stream


class External(Stream):
    def __init__(self, handle, device=None):
        assert handle > 1, "torch makes a stream of its own of a null handle"
        super().__init__(handle)


class Block:
    def __init__(self, nbytes, stream):
        self.nbytes, self.stream = nbytes, stream

    def data_ptr(self):
        return 1 << 20

    def record_stream(self, stream):
        pass


class Cuda:
    Stream, ExternalStream = Stream, External

    def __init__(self):
        self.current = Stream(77)

    def default_stream(self, device=None):
        return Stream(0)

    @contextlib.contextmanager
    def stream(self, s):
        before, self.current = self.current, s
        try:
            yield
        finally:
            self.current = before


class Torch:
    uint8 = "uint8"

    def __init__(self):
        self.cuda = Cuda()

    def empty(self, n, dtype=None, device=None):
        return Block(n, self.cuda.current)


class Handle:
    """Any object that has a stream's handle."""

    def __init__(self, handle):
        self.cuda_stream = handle


@pytest.mark.parametrize("stream,runs_on", [(None, 77), (Stream(5), 5), (Handle(6), 6), (7, 7), (0, 0), (1, 0), (Stream(0), 0)])
def test_a_workspace_is_memory_of_the_stream_that_the_call_runs_on(monkeypatch, stream, runs_on):
    tide.tide_linear  # loads the operators
    from fsdp_layout_aware_gb300 import ops
    fake = Torch()
    monkeypatch.setattr(ops, "torch", fake)
    ws, address, nbytes = ops._workspace(None, 4096, stream, 0)
    assert (ws.nbytes, address, nbytes) == (4096, 1 << 20, 4096)
    assert ws.stream == Stream(runs_on)
    assert fake.cuda.current == Stream(77)


def test_no_workspace_is_taken_where_none_is_needed(monkeypatch):
    tide.tide_linear
    from fsdp_layout_aware_gb300 import ops
    monkeypatch.setattr(ops, "torch", Torch())
    assert ops._workspace(None, 0, Stream(5), 0) == (None, None, 0)
