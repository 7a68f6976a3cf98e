"""Calls without a workspace where torch has its allocator's raw blocks (test_workspace_streams.py has the calls where it has
not): the block comes from the launching stream's pool, with the size that the library asks for, and goes back behind the
launch, also when the call fails.  On the host, with stand-ins for torch and the library."""

import pytest

from speculative_decoding_verify_attn_gb300 import cache, serving

from .test_workspace_streams import MAIN, SIDE, FakeStream, FakeTensor, FakeTorch

BLOCK = 0x7100000000
NEED = 4096

ARGS = {
    "spec_paged_attn": serving.SpecPagedArgs, "spec_prefill_attn": serving.SpecPrefillArgs,
    "spec_token_logprobs": serving.SpecLogprobArgs, "spec_rotary": cache.SpecRotaryArgs,
    "spec_kv8_append": cache.SpecKv8AppendArgs, "spec_paged_attn8": cache.SpecPaged8Args,
    "spec_page_fork": cache.SpecPageForkArgs, "spec_page_compact": cache.SpecPageCompactArgs,
}


class RawTorch(FakeTorch):
    def __init__(self, events, fails=False):
        super().__init__()

        def alloc(size, handle):
            events.append(("alloc", size, handle))
            if fails:
                raise RuntimeError("out of memory")
            return BLOCK

        self._C._cuda_cudaCachingAllocator_raw_alloc = staticmethod(alloc)
        self._C._cuda_cudaCachingAllocator_raw_delete = staticmethod(lambda block: events.append(("delete", block)))


class Lib:
    """Notes every call with what its workspace is."""

    def __init__(self, events, result):
        self.events, self.result = events, result

    def __getattr__(self, name):
        if name.endswith("_workspace"):
            return lambda ref: NEED

        def call(ref, handle):
            self.events.append((name, handle, ref._obj.workspace, ref._obj.workspace_bytes))
            if isinstance(self.result, Exception):
                raise self.result
            return self.result

        return call


@pytest.fixture
def setup(monkeypatch):
    def make(result=0, fails=False):
        events = []
        torch = RawTorch(events, fails)
        monkeypatch.setattr(serving, "_torch", torch)
        monkeypatch.setattr(serving, "_lib", Lib(events, result))
        monkeypatch.setattr(serving, "_sizes", {})
        return torch, events
    return make


@pytest.mark.parametrize("stream,handle", [(None, MAIN), (FakeStream(MAIN), MAIN), (FakeStream(SIDE), SIDE), (SIDE, SIDE), (MAIN, MAIN)])
@pytest.mark.parametrize("name", ARGS)
def test_the_block_is_the_launching_streams(setup, name, stream, handle):
    torch, events = setup()
    for _ in range(2):  # the second call finds the size of the first
        serving._call(name, ARGS[name](), ("sizes",), 0, None, stream)
    once = [("alloc", NEED, handle), (name, handle, BLOCK, NEED), ("delete", BLOCK)]
    assert events == 2 * once and torch.made == [] and torch.current == MAIN


@pytest.mark.parametrize("result,error", [(-1, serving.SpecError), (-4, serving.SpecError), (OSError("lost"), OSError)])
def test_the_block_goes_back_after_a_failure(setup, result, error):
    _, events = setup(result)
    with pytest.raises(error):
        serving._call("spec_rotary", cache.SpecRotaryArgs(), ("sizes",), 0, None, SIDE)
    assert [e[0] for e in events] == ["alloc", "spec_rotary", "delete"] and events[-1] == ("delete", BLOCK)


def test_without_memory_nothing_is_launched(setup):
    _, events = setup(fails=True)
    with pytest.raises(RuntimeError, match="out of memory"):
        serving._call("spec_rotary", cache.SpecRotaryArgs(), ("sizes",), 0, None, None)
    assert events == [("alloc", NEED, MAIN)]


@pytest.mark.parametrize("stream,recorded", [(FakeStream(SIDE), [SIDE]), (None, [])])
def test_a_callers_workspace_is_used_as_it_is(setup, stream, recorded):
    torch, events = setup()
    mine = FakeTensor(torch, 2 * NEED)
    serving._call("spec_rotary", cache.SpecRotaryArgs(), ("sizes",), 0, mine, stream)
    assert events == [("spec_rotary", SIDE if recorded else MAIN, mine.data_ptr(), 2 * NEED)] and mine.recorded == recorded
