"""What the serving binding makes of its tensors, on the host: the argument structs are filled without a GPU."""

import ctypes

import pytest
import torch

from speculative_decoding_verify_attn_gb300 import build
from speculative_decoding_verify_attn_gb300 import serving as s

from .test_serve_abi import paged as paged_struct
from .test_serve_abi import prefill as prefill_struct

I32 = torch.int32


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def odd(*shape, dtype=torch.bfloat16):
    """A tensor whose dimensions of one element have strides that no vector access could use."""
    strides, at = [], 1
    for n in reversed(shape):
        strides.insert(0, at if n > 1 or not strides else 3 * at + 1)
        at *= n
    strides[-1] = 1
    return torch.empty_strided(shape, strides, dtype=dtype)


def aligned(args, names, dtype):
    per = 16 // dtype.itemsize
    return [x for x in names if getattr(args, x) % per or getattr(args, x) < 1]


PAGED = ["q_stride_t", "q_stride_h", "kv_stride_p", "kv_stride_h", "kv_stride_t", "new_stride_t", "new_stride_h"]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,Hq,Hkv,pages,page", [(1, 4, 2, 3, 16), (1, 1, 1, 1, 1), (5, 1, 1, 3, 16), (5, 4, 2, 1, 16),
                                                 (1, 32, 1, 8, 1)])
def test_strides_of_single_elements_do_not_matter(T, Hq, Hkv, pages, page, dtype):
    q, o = odd(T, Hq, 64, dtype=dtype), odd(T, Hq, 64, dtype=torch.float32)
    k, v = odd(pages, Hkv, page, 64, dtype=dtype), torch.empty(pages, Hkv, page, 64, dtype=dtype)
    kn, vn = odd(T, Hkv, 64, dtype=dtype), torch.empty(T, Hkv, 64, dtype=dtype)
    table, start, lens = torch.zeros((1, 4), dtype=I32), torch.zeros(2, dtype=I32), torch.zeros(1, dtype=I32)
    a = s.paged_attn_args(q, k, v, table, start, lens, o, max_q=T, k_new=kn, v_new=vn)
    assert aligned(a, PAGED, dtype) == []
    # the others are as they were
    assert T == 1 or a.q_stride_t == q.stride(0)
    assert page == 1 or a.kv_stride_t == k.stride(2)
    assert pages == 1 or a.kv_stride_p == k.stride(0)
    a = s.prefill_attn_args(q, odd(T, Hkv, 64, dtype=dtype), torch.empty(T, Hkv, 64, dtype=dtype), start, o)
    assert aligned(a, ["q_stride_t", "q_stride_h", "kv_stride_t", "kv_stride_h"], dtype) == []


def test_unequal_strides_are_still_refused():
    z = torch.zeros
    ok = dict(q=z(4, 4, 64), k_pages=z(3, 2, 16, 64), v_pages=z(3, 2, 16, 64), page_table=z((1, 2), dtype=I32),
              q_start=z(2, dtype=I32), kv_len=z(1, dtype=I32), o=z(4, 4, 64), max_q=4)
    with pytest.raises(ValueError):
        s.paged_attn_args(**dict(ok, v_pages=z(3, 16, 2, 64).transpose(1, 2)))
    with pytest.raises(ValueError):
        s.paged_attn_args(**dict(ok, k_new=z(4, 2, 64), v_new=z(4, 3, 64)[:, :2]))
    with pytest.raises(ValueError):
        s.prefill_attn_args(ok["q"], z(4, 2, 64), z(4, 3, 64)[:, :2], ok["q_start"], ok["o"])
    with pytest.raises(ValueError):
        s.paged_attn_args(**dict(ok, q=z(4, 64, 4).transpose(1, 2)))


def paged(**kw):
    z = torch.zeros
    return dict(dict(q=z(4, 4, 64), k_pages=z(3, 2, 16, 64), v_pages=z(3, 2, 16, 64), page_table=z((1, 2), dtype=I32),
                     q_start=z(2, dtype=I32), kv_len=z(1, dtype=I32), o=z(4, 4, 64), max_q=4), **kw)


@pytest.mark.parametrize("value,kept", [(3, 3), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31, 2 ** 31 - 1), (2 ** 32, 2 ** 31 - 1),
                                        (2 ** 32 + 1, 2 ** 31 - 1), (2 ** 63 - 1, 2 ** 31 - 1), (2 ** 70 + 5, 2 ** 31 - 1),
                                        (-1, -1), (-2 ** 31 - 1, -1), (-2 ** 32 + 5, -1)])
def test_numbers_past_32_bits(value, kept):
    """A window or a bound on the chunk lengths past 32 bits is more than any sequence has, a negative one stays
    negative (and is refused by the call)."""
    a = s.paged_attn_args(**paged(window=value, max_q=value))
    assert (a.window, a.max_q) == (kept, kept)
    z = torch.zeros
    assert s.prefill_attn_args(z(4, 2, 64), z(4, 2, 64), z(4, 2, 64), z(2, dtype=I32), z(4, 2, 64),
                               window=value).window == kept


def test_numbers_that_are_not_whole():
    for bad in (2.0, "3", None):
        for name in ("window", "max_q"):
            with pytest.raises(TypeError):
                s.paged_attn_args(**paged(**{name: bad}))
        with pytest.raises(TypeError):
            s.spec_paged_attn_workspace(*(paged()[x] for x in ("q", "k_pages", "page_table", "o")), max_q=bad)


def test_sizes_past_32_bits_stay_too_large():
    """Rows and vocabularies past 32 bits keep a size that the call refuses (shapes without memory)."""
    big = 2 ** 32 + 5
    logits = torch.empty(1, device="meta").expand(big, 3)
    for x, K in ((logits, 2), (logits.T, 2), (logits[:2], big)):
        with pytest.raises(s.SpecError):
            s.spec_token_logprobs_workspace(x, K)
    q = torch.empty(1, device="meta", dtype=torch.bfloat16).expand(big, 4, 64)
    kp = torch.empty(1, device="meta", dtype=torch.bfloat16).expand(big, 2, 16, 64)
    table = torch.empty(1, device="meta", dtype=I32).expand(big, 3)
    with pytest.raises(s.SpecError):
        s.spec_paged_attn_workspace(q, kp, table[:1], q, max_q=4)
    with pytest.raises(s.SpecError):
        s.spec_paged_attn_workspace(q[:4], kp, table, q, max_q=4)
    with pytest.raises(s.SpecError):
        s.spec_prefill_attn_workspace(q, q[:, :2], torch.zeros(2, dtype=I32), q)


def test_scales_that_32_bits_cannot_hold():
    """0 stands for 1 / sqrt(D), so a scale that rounds to it is refused and not replaced."""
    z = torch.zeros
    for bad in (1e-50, -1e-50, 1e-46):
        with pytest.raises(ValueError):
            s.paged_attn_args(**paged(scale=bad))
        with pytest.raises(ValueError):
            s.prefill_attn_args(z(4, 2, 64), z(4, 2, 64), z(4, 2, 64), z(2, dtype=I32), z(4, 2, 64), scale=bad)
    for good in (0, 0.0, 1e-40, 0.125, 2):
        assert s.paged_attn_args(**paged(scale=good)).scale == pytest.approx(good, rel=1e-4)


@pytest.mark.parametrize("scale", [3e38, 2.4e38])
def test_scales_whose_binary_exponent_factor_is_infinite(scale):
    """scale log2(e) multiplies every score in fp32.  (Refused before any launch.)"""
    L = s._serve_lib()
    assert L.spec_paged_attn(ctypes.byref(paged_struct(scale=scale)), None) == -1
    assert L.spec_prefill_attn(ctypes.byref(prefill_struct(scale=scale)), None) == -1
