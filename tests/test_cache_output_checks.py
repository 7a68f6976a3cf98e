"""Outputs of spec_paged_attn8 whose rows overlap are refused on the host, before any launch."""

import ctypes

import pytest

from .test_cache_abi import L, paged8  # noqa: F401


@pytest.mark.parametrize("kw", [
    dict(o_stride_t=0), dict(o_stride_t=64), dict(o_stride_h=0), dict(o_stride_h=127), dict(o_stride_t=127, o_stride_h=1280),
    dict(o_dtype=0, o_stride_h=64)])
def test_outputs_that_overlap(L, kw):  # noqa: F811
    assert L.spec_paged_attn8(ctypes.byref(paged8(**kw)), None) == -1


@pytest.mark.parametrize("kw", [
    dict(), dict(o_stride_t=128, o_stride_h=1280), dict(o_stride_t=1031, o_stride_h=129),
    dict(T=1, o_stride_t=0), dict(Hq=1, Hkv=1, o_stride_h=0)])
def test_outputs_that_do_not(L, kw):  # noqa: F811
    """The next thing that is looked at is the workspace, which is missing."""
    assert L.spec_paged_attn8(ctypes.byref(paged8(**kw, workspace=None)), None) == -3
