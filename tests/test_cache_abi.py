"""CPU checks of the cache operators' C ABI and binding: struct layouts, workspace sizes and the host's refusals,
each of which returns before any launch."""

import ctypes

import pytest
import torch

FAKE = 0x7f0000000000  # never dereferenced: validation fails before any launch
I32 = torch.int32


@pytest.fixture(scope="module")
def L():
    from speculative_decoding_verify_attn_gb300 import build, cache
    build.build()
    return cache._cache_lib()


def rotary(**kw):
    from speculative_decoding_verify_attn_gb300 import SpecRotaryArgs
    d = dict(T=10, Hq=8, Hkv=2, D=128, rot=64, layout=0, dtype=1, inverse=0, B=2, amplitude=1.0,
             q=FAKE, q_stride_t=1024, q_stride_h=128, k=FAKE + 4096, k_stride_t=256, k_stride_h=128,
             q_out=FAKE + 8192, qo_stride_t=1024, qo_stride_h=128, k_out=FAKE + 16384, ko_stride_t=256, ko_stride_h=128,
             steps=FAKE, q_start=FAKE, kv_len=FAKE, workspace=FAKE, workspace_bytes=256)
    d.update(kw)
    return SpecRotaryArgs(**d)


def cache8(**kw):
    d = dict(B=2, Hkv=2, D=128, T=10, page_size=16, num_pages=64, table_cols=20, block=8, k_new=FAKE, v_new=FAKE,
             new_stride_t=256, new_stride_h=128, k_pages=FAKE, v_pages=FAKE + (1 << 20), kv_stride_p=4096, kv_stride_h=2048,
             kv_stride_t=128, k_exp=FAKE + 1, v_exp=FAKE + 3, exp_stride_p=4, exp_stride_h=2, page_table=FAKE,
             table_stride=20, q_start=FAKE, kv_len=FAKE, workspace=FAKE, workspace_bytes=1 << 40)
    d.update(kw)
    return d


def append(**kw):
    from speculative_decoding_verify_attn_gb300 import SpecKv8AppendArgs
    return SpecKv8AppendArgs(**cache8(**{**dict(src_dtype=1), **kw}))


def paged8(**kw):
    from speculative_decoding_verify_attn_gb300 import SpecPaged8Args
    return SpecPaged8Args(**cache8(**{**dict(Hq=8, max_q=5, q_dtype=1, o_dtype=1, window=0, scale=0.0, q=FAKE,
                                             q_stride_t=1024, q_stride_h=128, o=FAKE, o_stride_t=1024, o_stride_h=128), **kw}))


def arrays(*items):
    from speculative_decoding_verify_attn_gb300 import SpecPageArray
    return (SpecPageArray * len(items))(*[SpecPageArray(*x) for x in items])


def fork(items=((FAKE, 4096, 4096),), **kw):
    from speculative_decoding_verify_attn_gb300 import SpecPageForkArgs
    a = arrays(*items)
    d = dict(B=3, table_cols=20, page_size=16, num_pages=64, num_arrays=len(items), page_table=FAKE, table_stride=20,
             held=FAKE, kv_len=FAKE, refs=FAKE, parent=FAKE, grow=FAKE, table_out=FAKE, table_out_stride=20, held_out=FAKE,
             kv_len_out=FAKE, refs_out=FAKE, arrays=ctypes.cast(a, ctypes.c_void_p), workspace=FAKE, workspace_bytes=1 << 40)
    d.update(kw)
    s = SpecPageForkArgs(**d)
    s.keep = a
    return s


def compact(items=((FAKE, 4096, 4096),), **kw):
    from speculative_decoding_verify_attn_gb300 import SpecPageCompactArgs
    a = arrays(*items)
    d = dict(B=3, table_cols=20, num_pages=64, num_arrays=len(items), page_table=FAKE, table_stride=20, held=FAKE, refs=FAKE,
             table_out=FAKE, table_out_stride=20, refs_out=FAKE, moved=FAKE, num_live=FAKE,
             arrays=ctypes.cast(a, ctypes.c_void_p), workspace=FAKE, workspace_bytes=1 << 40)
    d.update(kw)
    s = SpecPageCompactArgs(**d)
    s.keep = a
    return s


def test_struct_sizes(L):
    from speculative_decoding_verify_attn_gb300 import cache
    for i, cls in enumerate(cache._STRUCTS):
        assert L.spec_cache_struct_size(i) == ctypes.sizeof(cls)
    assert L.spec_cache_struct_size(6) == 0 and L.spec_cache_struct_size(-1) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), -1), (dict(T=(1 << 22) + 1), -2), (dict(Hq=0, Hkv=0), -1), (dict(Hq=-1), -1), (dict(Hkv=4097), -1),
    (dict(D=0), -1), (dict(D=60, rot=30), -2), (dict(D=2048), -2), (dict(rot=0), -1), (dict(rot=63), -1), (dict(rot=130), -1),
    (dict(layout=2), -1), (dict(dtype=3), -1), (dict(inverse=2), -1), (dict(B=0), -1), (dict(B=4097), -1),
    (dict(amplitude=-1.0), -1), (dict(amplitude=float("inf")), -1), (dict(amplitude=float("nan")), -1), (dict(q=None), -1),
    (dict(q=FAKE + 8), -1), (dict(q_stride_t=1028), -1), (dict(k_out=None), -1), (dict(ko_stride_h=-8), -1),
    (dict(q_out=FAKE, qo_stride_t=2048), -1), (dict(k_out=FAKE + 4096, ko_stride_h=0), -1), (dict(steps=None), -1),
    (dict(steps=FAKE + 4), -1), (dict(q_start=None), -1), (dict(kv_len=FAKE + 2), -1), (dict(positions=FAKE + 1), -1),
    (dict(workspace=None), -3), (dict(workspace_bytes=255), -3), (dict(workspace=FAKE + 64), -3),
])
def test_rotary_refusals(L, kw, status):
    assert L.spec_rotary(ctypes.byref(rotary(**kw)), None) == status


@pytest.mark.parametrize("kw", [
    dict(q_out=FAKE, q_stride_t=0, qo_stride_t=0), dict(qo_stride_t=64), dict(qo_stride_h=0), dict(ko_stride_t=0),
    dict(ko_stride_h=120), dict(q_out=FAKE + 256, k_out=FAKE + 256), dict(q_out=FAKE + 4096, k=FAKE + 4096),
])
def test_rotary_outputs_that_overlap(L, kw):
    assert L.spec_rotary(ctypes.byref(rotary(**kw)), None) == -1


@pytest.mark.parametrize("kw", [
    dict(v_pages=FAKE, k_pages=FAKE), dict(k_exp=FAKE, v_exp=FAKE), dict(kv_stride_p=0), dict(kv_stride_h=0),
    dict(kv_stride_t=64), dict(exp_stride_p=0), dict(exp_stride_h=0),
])
def test_caches_that_overlap_are_not_written(L, kw):
    assert L.spec_kv8_append(ctypes.byref(append(**kw)), None) == -1
    assert L.spec_paged_attn8(ctypes.byref(paged8(**kw)), None) == -1


CACHE = [
    (dict(B=0), -1), (dict(B=4097), -1), (dict(Hkv=0), -1), (dict(D=96), -2), (dict(T=-1), -1), (dict(T=(1 << 22) + 1), -2),
    (dict(page_size=0), -1), (dict(page_size=65537), -1), (dict(num_pages=0), -1), (dict(table_cols=0), -1),
    (dict(table_cols=1 << 28), -1), (dict(table_stride=-1), -1), (dict(block=0), -1), (dict(block=3), -1), (dict(block=32), -1),
    (dict(k_new=FAKE + 8), -1), (dict(new_stride_t=260), -1), (dict(k_pages=None), -1), (dict(v_pages=FAKE + 8), -1),
    (dict(kv_stride_t=136), -1), (dict(kv_stride_p=-16), -1), (dict(k_exp=None), -1), (dict(v_exp=None), -1),
    (dict(exp_stride_p=-1), -1), (dict(page_table=None), -1), (dict(q_start=FAKE + 2), -1), (dict(kv_len=None), -1),
    (dict(workspace=None), -3), (dict(workspace=FAKE + 16), -3), (dict(workspace_bytes=128), -3),
]


@pytest.mark.parametrize("kw,status", CACHE + [(dict(src_dtype=2), -1), (dict(k_new=None), -1), (dict(v_new=None), -1)])
def test_append_refusals(L, kw, status):
    assert L.spec_kv8_append(ctypes.byref(append(**kw)), None) == status


@pytest.mark.parametrize("kw,status", CACHE + [
    (dict(Hq=7), -1), (dict(Hq=66), -2), (dict(max_q=0), -1), (dict(window=-1), -1), (dict(q_dtype=0), -2),
    (dict(q_dtype=7), -1), (dict(o_dtype=2), -1), (dict(scale=-1.0), -1), (dict(scale=float("nan")), -1),
    (dict(scale=3e38), -1), (dict(k_new=None), -1), (dict(v_new=None), -1), (dict(q=None), -1), (dict(q_stride_h=4), -1),
    (dict(o=None), -1), (dict(o=FAKE + 1), -1), (dict(o_dtype=0, o=FAKE + 2), -1), (dict(o_stride_t=-1), -1),
    (dict(workspace_bytes=512), -3),
])
def test_paged8_refusals(L, kw, status):
    assert L.spec_paged_attn8(ctypes.byref(paged8(**kw)), None) == status


TABLES = [
    (dict(B=0), -1), (dict(B=4097), -1), (dict(table_cols=0), -1), (dict(B=4096, table_cols=(1 << 14) + 1), -1),
    (dict(num_pages=0), -1), (dict(num_pages=(1 << 24) + 1), -1), (dict(num_arrays=-1), -1), (dict(num_arrays=4097), -1),
    (dict(arrays=None), -1), (dict(items=((None, 64, 64),)), -1), (dict(items=((FAKE, 32, 64),)), -1),
    (dict(items=((FAKE, 64, 0),)), -1), (dict(page_table=None), -1), (dict(table_out=FAKE + 2), -1),
    (dict(table_stride=-1), -1), (dict(table_out_stride=19), -1), (dict(table_stride=40), -1), (dict(held=None), -1),
    (dict(refs=None), -1), (dict(refs_out=FAKE + 1), -1), (dict(workspace=None), -3), (dict(workspace_bytes=512), -3),
]


@pytest.mark.parametrize("kw,status", TABLES + [
    (dict(page_size=0), -1), (dict(page_size=65537), -1), (dict(table_cols=1 << 20, page_size=2048), -1), (dict(kv_len=None), -1),
    (dict(parent=None), -1), (dict(grow=FAKE + 3), -1), (dict(held_out=None), -1), (dict(kv_len_out=None), -1)])
def test_fork_refusals(L, kw, status):
    assert L.spec_page_fork(ctypes.byref(fork(**kw)), None) == status


@pytest.mark.parametrize("kw,status", TABLES + [(dict(moved=FAKE + 2), -1), (dict(num_live=FAKE + 2), -1)])
def test_compact_refusals(L, kw, status):
    assert L.spec_page_compact(ctypes.byref(compact(**kw)), None) == status


def test_empty_calls_launch_nothing(L):
    assert L.spec_rotary(ctypes.byref(rotary(T=0, q=None, workspace=None)), None) == 0
    assert L.spec_kv8_append(ctypes.byref(append(T=0, k_new=None, workspace=None)), None) == 0
    assert L.spec_paged_attn8(ctypes.byref(paged8(T=0, q=None, workspace=None)), None) == 0
    for name in ("spec_rotary", "spec_kv8_append", "spec_paged_attn8", "spec_page_fork", "spec_page_compact"):
        assert getattr(L, name)(None, None) == -1 and getattr(L, name + "_workspace")(None) == 0


def test_workspace_sizes(L):
    assert L.spec_rotary_workspace(ctypes.byref(rotary())) == L.spec_kv8_append_workspace(ctypes.byref(append())) == 256
    assert L.spec_paged_attn8_workspace(ctypes.byref(paged8(D=96))) == 0
    assert L.spec_paged_attn8_workspace(ctypes.byref(paged8(T=100000, max_q=3000))) > L.spec_paged_attn8_workspace(
        ctypes.byref(paged8(T=100, max_q=100)))
    assert L.spec_page_fork_workspace(ctypes.byref(fork(B=100, table_cols=1000, num_pages=5000))) >= 4 * (100000 + 4 * 5000)
    assert L.spec_page_compact_workspace(ctypes.byref(compact(num_pages=5000))) >= 4 * 4 * 5000


# ------------------------------------------------------------------------------ the binding, on the host
def z(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def tensors(T=4, Hq=4, Hkv=2, D=64, pages=3, size=16, blocks=2, B=1, cols=2):
    e4 = torch.float8_e4m3fn
    return dict(q=z(T, Hq, D), k_pages=z(pages, Hkv, size, D, dtype=e4), v_pages=z(pages, Hkv, size, D, dtype=e4),
                k_exp=z(pages, Hkv, blocks, dtype=torch.uint8), v_exp=z(pages, Hkv, blocks, dtype=torch.uint8),
                page_table=z(B, cols, dtype=I32), q_start=z(B + 1, dtype=I32), kv_len=z(B, dtype=I32), o=z(T, Hq, D), max_q=T)


def test_paged8_arguments():
    from speculative_decoding_verify_attn_gb300 import cache
    ok = tensors()
    a = cache.paged_attn8_args(**ok)
    assert (a.B, a.Hq, a.Hkv, a.D, a.T, a.page_size, a.num_pages, a.table_cols, a.block) == (1, 4, 2, 64, 4, 16, 3, 2, 8)
    assert (a.kv_stride_p, a.kv_stride_h, a.kv_stride_t, a.exp_stride_p, a.exp_stride_h) == (2048, 1024, 64, 4, 2)
    assert a.k_new is None and a.o_stride_t == 256
    nhd = z(3, 16, 2, 64, dtype=torch.float8_e4m3fn).permute(0, 2, 1, 3)
    a = cache.paged_attn8_args(**{**ok, "k_pages": nhd, "v_pages": nhd})
    assert (a.kv_stride_h, a.kv_stride_t) == (64, 128)
    for bad, err in ((dict(k_pages=z(3, 2, 16, 64)), TypeError), (dict(v_pages=z(3, 2, 16, 32, dtype=torch.float8_e4m3fn)), ValueError),
                     (dict(k_exp=z(3, 2, 2)), TypeError), (dict(k_exp=z(3, 2, 3, dtype=torch.uint8), v_exp=z(3, 2, 3, dtype=torch.uint8)), ValueError),
                     (dict(v_exp=z(3, 2, 4, dtype=torch.uint8)), ValueError), (dict(q_start=z(3, dtype=I32)), ValueError),
                     (dict(page_table=z(1, 2, dtype=torch.int64)), ValueError), (dict(o=z(4, 2, 64)), ValueError),
                     (dict(k_new=z(4, 2, 64)), ValueError), (dict(k_new=z(4, 1, 64), v_new=z(4, 1, 64)), ValueError),
                     (dict(k_new=z(4, 2, 64, dtype=torch.float32), v_new=z(4, 2, 64, dtype=torch.float32)), TypeError),
                     (dict(scale=1e-60), ValueError), (dict(q=z(4, 4, 64, dtype=torch.float16)), TypeError)):
        with pytest.raises(err):
            cache.paged_attn8_args(**{**ok, **bad})


def test_append_arguments():
    from speculative_decoding_verify_attn_gb300 import cache
    t = tensors(T=1, Hkv=1, pages=1, size=1, blocks=1)
    ok = {k: t[k] for k in ("k_pages", "v_pages", "k_exp", "v_exp", "page_table", "q_start", "kv_len")}
    a = cache.kv8_append_args(z(1, 1, 64, dtype=torch.float32), z(1, 1, 64, dtype=torch.float32), **ok)
    assert (a.src_dtype, a.block, a.new_stride_t, a.kv_stride_p) == (0, 1, 64, 64)
    with pytest.raises(ValueError):
        cache.kv8_append_args(z(1, 2, 64), z(1, 2, 64), **ok)
    with pytest.raises(TypeError):
        cache.kv8_append_args(z(1, 1, 64), z(1, 1, 64, dtype=torch.float32), **ok)


def test_rotary_arguments():
    from speculative_decoding_verify_attn_gb300 import cache
    steps = z(16, dtype=torch.int64)
    q, k = z(5, 4, 64), z(5, 2, 64)
    a = cache.rotary_args(q, k, steps, positions=z(5, dtype=I32))
    assert (a.T, a.Hq, a.Hkv, a.D, a.rot, a.dtype) == (5, 4, 2, 64, 32, 1) and a.q == a.q_out and a.ko_stride_t == 128
    a = cache.rotary_args(None, k, steps, q_start=z(3, dtype=I32), kv_len=z(2, dtype=I32), k_out=z(5, 2, 64), inverse=True)
    assert (a.Hq, a.Hkv, a.B, a.inverse) == (0, 2, 2, 1) and a.q is None and a.k != a.k_out
    for args, kw in (((None, None, steps), dict(positions=z(5, dtype=I32))), ((q, k, steps), {}),
                     ((q, k, steps), dict(positions=z(4, dtype=I32))), ((q, k, steps), dict(positions=z(5, dtype=torch.int64))),
                     ((q, k, steps), dict(positions=z(5, dtype=I32), kv_len=z(2, dtype=I32))),
                     ((q, z(4, 2, 64), steps), dict(positions=z(5, dtype=I32))),
                     ((q, z(5, 2, 64, dtype=torch.float32), steps), dict(positions=z(5, dtype=I32))),
                     ((q, k, z(16, dtype=torch.float32)), dict(positions=z(5, dtype=I32))),
                     ((q, k, steps), dict(positions=z(5, dtype=I32), q_out=z(5, 4, 32))),
                     ((q, None, steps), dict(positions=z(5, dtype=I32), k_out=k)),
                     ((q, k, steps), dict(positions=z(5, dtype=I32), amplitude=0.0)),
                     ((q, k, steps), dict(q_start=z(3, dtype=I32), kv_len=z(3, dtype=I32)))):
        with pytest.raises(ValueError):
            cache.rotary_args(*args, **kw)


def test_page_arguments():
    from speculative_decoding_verify_attn_gb300 import cache
    i = lambda *s: z(*s, dtype=I32)  # noqa: E731
    ok = dict(page_table=i(2, 5), held=i(2), kv_len=i(2), refs=i(7), parent=i(2), page_size=16)
    both = z(7, 16, 2, 2, 64)  # K and V of a page side by side
    a = cache.page_fork_args(**ok, grow=i(2), caches=[both, z(7, 3, dtype=torch.uint8), z(7, 2, 16, 64).permute(0, 2, 1, 3)])
    assert [tuple(a.keep[3 * i + 1:3 * i + 3]) for i in range(3)] == [(8192, 8192), (3, 3), (4096, 4096)]
    assert a.keep[0] == both.data_ptr() and ctypes.sizeof(cache.SpecPageArray) == 3 * a.keep.itemsize
    assert a.num_arrays == 3 and a.table_out == a.page_table and a.refs_out == a.refs and a.table_out_stride == 5
    a = cache.page_fork_args(**ok, caches=[z(14, 8)[::2]])
    assert (*a.keep[1:3], a.grow) == (32, 16, None)
    for bad in (dict(caches=[both[:, :, 0]]), dict(caches=[z(6, 4)]), dict(caches=[z(7, 0)]), dict(caches=[z(7, 4).expand(7, 4)[:, :1].expand(7, 4)]),
                dict(held=i(3)), dict(refs=z(7)), dict(grow=i(1)), dict(table_out=i(2, 6)), dict(page_table=z(2, 5)),
                dict(parent=z(2, dtype=torch.int64))):
        with pytest.raises(ValueError):
            cache.page_fork_args(**{**ok, **bad})
    a = cache.page_compact_args(i(2, 5), i(2), i(7), moved=i(7))
    assert a.num_arrays == 0 and a.num_live is None
    for bad in (dict(moved=i(6)), dict(num_live=i(2)), dict(refs_out=i(8))):
        with pytest.raises(ValueError):
            cache.page_compact_args(i(2, 5), i(2), i(7), **bad)


def test_host_tensors_are_refused():
    import speculative_decoding_verify_attn_gb300 as sv
    i = lambda *s: z(*s, dtype=I32)  # noqa: E731
    t = tensors()
    with pytest.raises(ValueError, match="CUDA"):
        sv.spec_paged_attn8(**t)
    with pytest.raises(ValueError, match="CUDA"):
        sv.spec_rotary(z(4, 2, 64), None, z(8, dtype=torch.int64), positions=i(4))
    with pytest.raises(ValueError, match="CUDA"):
        sv.spec_kv8_append(z(4, 2, 64), z(4, 2, 64), *[t[k] for k in ("k_pages", "v_pages", "k_exp", "v_exp", "page_table", "q_start", "kv_len")])
    with pytest.raises(ValueError, match="CUDA"):
        sv.spec_page_fork(i(2, 5), i(2), i(2), i(7), i(2), page_size=16)
    with pytest.raises(ValueError, match="CUDA"):
        sv.spec_page_compact(i(2, 5), i(2), i(7))


def test_dependent_grids_wait_before_they_leave():
    """As test_dependent_launches.py, for kernels that may also be a call's first: what comes before the wait is
    nothing that could leave; the append, which needs nothing of the kernel before it, waits where it ends."""
    from .test_dependent_launches import kernels, source
    seen = set()
    for name in ("kv8_append.cu", "paged8_mma.cu", "chunk8_tc.cu", "pages.cu"):
        for kernel, body in kernels(source(name)).items():
            if kernel in ("page_fork", "page_compact"):  # never launched as dependents
                continue
            seen.add(kernel)
            if kernel == "kv8_append":
                assert "return;" not in body and body.rstrip().endswith("pdl_wait();")
                continue
            before, wait, _ = body.partition("pdl_wait();")
            assert wait and "return" not in before, kernel
    assert seen == {"kv8_append", "paged8_mma", "chunk8_attn_tc", "page_copy"}
