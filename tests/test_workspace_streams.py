"""Where a call that is given no workspace takes one from: the allocator's pool of the stream that the call
runs on.  A block of another stream's pool may still be in use there (the allocator hands a block out again
as soon as its tensor is dropped, in the order of the pool's stream only).  On the host, with stand-ins for
torch and the library; the same on a GPU in test_gpu_workspace_streams.py."""

import contextlib

import pytest
import torch as real

from speculative_decoding_verify_attn_gb300 import binding, serving

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

    uint8, float32, bfloat16 = "uint8", real.float32, real.bfloat16

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


class FakeRoundLib:
    """Every *_workspace function says 4096, every call notes its stream."""

    def __init__(self):
        self.handles = []

    def __getattr__(self, name):
        if name.endswith("_workspace"):
            return lambda ref: 4096
        return lambda ref, handle: self.handles.append(handle) or 0


def round_call(name, stream):
    z, i32 = real.zeros, real.int32
    ints = z(2, dtype=i32)
    if name == "spec_verify_attn":
        return binding.spec_verify_attn(z(2, 3, 4, 8), z(2, 2, 16, 8), z(2, 2, 16, 8), ints, z(2, 3, 4, 8), stream=stream)
    if name == "spec_draft_window_attn":
        return binding.spec_draft_window_attn(z(2, 4, 8), z(2, 2, 16, 8), z(2, 2, 16, 8), ints, z(2, 4, 8), stream=stream)
    if name == "spec_sample":
        return binding.spec_sample(binding.SPEC_SAMPLE_CHAIN_GREEDY, z(2, 3, 10), z((2, 3), dtype=i32), ints,
                                   draft_tokens=z((2, 2), dtype=i32), stream=stream)
    if name == "spec_lmhead_sample":
        return binding.spec_lmhead_sample(binding.SPEC_SAMPLE_CHAIN_GREEDY, z(2, 3, 8), z(10, 8), z((2, 3), dtype=i32),
                                          ints, draft_tokens=z((2, 2), dtype=i32), stream=stream)
    return binding.spec_commit(binding.SPEC_COMMIT_CHAIN, ints, ints, 3, stream=stream)


@pytest.mark.parametrize("stream,handle", [(FakeStream(SIDE), SIDE), (SIDE, SIDE), (FakeStream(MAIN), MAIN), (None, MAIN)])
@pytest.mark.parametrize("name", ["spec_verify_attn", "spec_draft_window_attn", "spec_sample", "spec_lmhead_sample",
                                  "spec_commit"])
def test_round_workspace_comes_from_the_launching_stream(monkeypatch, name, stream, handle):
    torch, lib = FakeTorch(), FakeRoundLib()
    monkeypatch.setattr(binding, "_torch", lambda: torch)
    monkeypatch.setattr(binding, "_check_cuda", lambda *ts: None)
    monkeypatch.setattr(binding, "lib", lambda: lib)
    round_call(name, stream)
    assert lib.handles == [handle] and [x.pool for x in torch.made] == [handle]
    assert torch.current == MAIN
