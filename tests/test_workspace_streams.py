"""Where a call that is given no workspace takes one from: the allocator's pool of the stream that the call
runs on.  A block of another stream's pool may still be in use there (the allocator hands a block out again
as soon as its tensor is dropped, in the order of the pool's stream only).  On the host, with stand-ins for
torch and the library; the same on a GPU in test_gpu_workspace_streams.py."""

import contextlib

import pytest

from speculative_decoding_verify_attn_gb300 import serving

MAIN, SIDE = 0x1000, 0x2000


class FakeStream:
    def __init__(self, handle):
        self.cuda_stream = handle


class FakeTensor:
    def __init__(self, torch, nbytes):
        self.torch, self.nbytes, self.pool, self.recorded = torch, nbytes, torch.current, []
        torch.made.append(self)

    def data_ptr(self):
        return 0x700000000000

    def get_device(self):
        return 0

    def is_contiguous(self):
        return True

    def numel(self):
        return self.nbytes

    def element_size(self):
        return 1

    def record_stream(self, stream):
        self.recorded.append(stream.cuda_stream)


class FakeTorch:
    """The parts of torch that the bindings' calls use, with the current stream as plain state."""

    uint8 = "uint8"

    def __init__(self):
        self.current, self.made = MAIN, []
        outer = self

        class C:
            _cuda_getDevice = staticmethod(lambda: 0)
            _cuda_getCurrentRawStream = staticmethod(lambda index: outer.current)

        class Cuda:
            Stream = FakeStream
            ExternalStream = FakeStream

            @staticmethod
            def current_stream():
                return FakeStream(outer.current)

            @staticmethod
            @contextlib.contextmanager
            def stream(s):
                before, outer.current = outer.current, s.cuda_stream
                yield
                outer.current = before

        self._C, self.cuda = C, Cuda

    def empty(self, n, dtype=None, device=None):
        return FakeTensor(self, n)


class FakeLib:
    def __init__(self):
        self.handles = []

    def spec_paged_attn_workspace(self, ref):
        return 4096

    def spec_paged_attn(self, ref, handle):
        self.handles.append(handle)
        return 0


@pytest.fixture
def fakes(monkeypatch):
    torch, lib = FakeTorch(), FakeLib()
    monkeypatch.setattr(serving, "_torch", torch)
    monkeypatch.setattr(serving, "_lib", lib)
    monkeypatch.setattr(serving, "_sizes", {})
    return torch, lib


@pytest.mark.parametrize("stream", [FakeStream(SIDE), SIDE])
def test_serving_workspace_comes_from_the_launching_stream(fakes, stream):
    torch, lib = fakes
    serving._call("spec_paged_attn", serving.SpecPagedArgs(), ("sizes",), 0, None, stream)
    assert lib.handles == [SIDE] and [x.pool for x in torch.made] == [SIDE]
    assert torch.current == MAIN


@pytest.mark.parametrize("stream", [None, FakeStream(MAIN), MAIN])
def test_serving_workspace_of_the_current_stream(fakes, stream):
    torch, lib = fakes
    serving._call("spec_paged_attn", serving.SpecPagedArgs(), ("sizes",), 0, None, stream)
    assert lib.handles == [MAIN] and [x.pool for x in torch.made] == [MAIN]


def test_serving_callers_workspace_is_kept_for_the_launching_stream(fakes):
    torch, lib = fakes
    mine = FakeTensor(torch, 8192)
    serving._call("spec_paged_attn", serving.SpecPagedArgs(), ("sizes",), 0, mine, FakeStream(SIDE))
    assert lib.handles == [SIDE] and torch.made == [mine] and mine.recorded == [SIDE]
