"""What spec_page_fork has to notice about the pages that rows hold, whether a row goes on from itself, from another or
ends: nothing is changed, and the status says why."""

import numpy as np
import pytest

from .test_gpu_pages import Beams

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    import speculative_decoding_verify_attn_gb300 as sv
    sv.lib()
    return sv


@pytest.mark.parametrize("grow", [0, 5])
@pytest.mark.parametrize("entry", [-1, 10 ** 6])
@pytest.mark.parametrize("row,col", [(0, 0), (2, 1), (5, 1)])
def test_fork_checks_the_pages_of_rows_that_stay(sv, row, col, entry, grow):
    """A kept entry that is no page, though nothing is written to it or given back: the step of rows that go on."""
    b = Beams(6, 16, 100, 50, 3, 5, drop=0.0, spread=False)
    b.kv_len[:], b.held[:], b.grow[:] = 40, 3, grow
    b.table[:, :3] = np.arange(18).reshape(6, 3)
    b.refs[:] = np.arange(b.pages) < 18
    b.table[row, col] = entry
    for in_place in (True, False):
        got, before, after, status = b.run(sv, in_place)
        assert status == sv.SPEC_STATUS_BAD_PAGE
        for a, ref in zip(got, (b.table, b.held, b.kv_len, b.refs)):
            assert np.array_equal(a, ref)
        assert all(np.array_equal(x, y) for x, y in zip(before, after))


@pytest.mark.parametrize("count", [0, -1])
@pytest.mark.parametrize("parent", [[0, 1, 2, 3], [0, 2, 2, 3], [0, -1, 2, 3]])
@pytest.mark.parametrize("col", [0, 2, 3])
def test_fork_reports_held_pages_that_count_as_free(sv, col, parent, count):
    """A page of a row that nobody is counted to hold would go out as another row's new page."""
    b = Beams(4, 16, 100, 50, 3, 5, drop=0.0)
    b.parent = np.array(parent, np.int32)
    b.kv_len[:], b.held[:], b.grow[:] = 40, 4, 20
    b.table[:, :4] = np.arange(16).reshape(4, 4)
    b.refs[:] = np.arange(b.pages) < 16
    b.refs[4 + col] = count  # row 1's
    for in_place in (True, False):
        got, before, after, status = b.run(sv, in_place)
        assert status == sv.SPEC_STATUS_BAD_PAGE
        for a, ref in zip(got, (b.table, b.held, b.kv_len, b.refs)):
            assert np.array_equal(a, ref)
        assert all(np.array_equal(x, y) for x, y in zip(before, after))
