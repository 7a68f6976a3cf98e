"""CPU checks of the serving operators' C ABI: struct layouts, workspace sizes and the host's refusals,
each of which returns before any launch."""

import ctypes

import pytest

FAKE = 0x7f0000000000  # never dereferenced: validation fails before any launch


@pytest.fixture(scope="module")
def L():
    from speculative_decoding_verify_attn_gb300 import build, serving
    build.build()
    return serving._serve_lib()


def paged(**kw):
    from speculative_decoding_verify_attn_gb300.serving import SpecPagedArgs
    B, Hq, Hkv, D, T, page, pages = 2, 8, 2, 128, 10, 16, 64
    d = dict(B=B, Hq=Hq, Hkv=Hkv, D=D, T=T, max_q=5, q_dtype=1, kv_dtype=1, o_dtype=1, page_size=page,
             num_pages=pages, table_cols=20, window=0, scale=0.0, q=FAKE, q_stride_t=Hq * D, q_stride_h=D,
             k_pages=FAKE, v_pages=FAKE + (1 << 30), kv_stride_p=Hkv * page * D, kv_stride_h=page * D, kv_stride_t=D,
             page_table=FAKE, table_stride=20, q_start=FAKE, kv_len=FAKE, o=FAKE, o_stride_t=Hq * D, o_stride_h=D,
             workspace=FAKE, workspace_bytes=1 << 40)
    d.update(kw)
    return SpecPagedArgs(**d)


def prefill(**kw):
    from speculative_decoding_verify_attn_gb300.serving import SpecPrefillArgs
    Hq, Hkv, D, T = 8, 2, 64, 100
    d = dict(B=3, Hq=Hq, Hkv=Hkv, D=D, T=T, window=0, q_dtype=1, kv_dtype=1, o_dtype=0, scale=0.0, q=FAKE,
             q_stride_t=Hq * D, q_stride_h=D, k=FAKE, v=FAKE, kv_stride_t=Hkv * D, kv_stride_h=D, seq_start=FAKE,
             o=FAKE, o_stride_t=Hq * D, o_stride_h=D, workspace=FAKE, workspace_bytes=1 << 40)
    d.update(kw)
    return SpecPrefillArgs(**d)


def logp(**kw):
    from speculative_decoding_verify_attn_gb300.serving import SpecLogprobArgs
    d = dict(N=7, V=1001, K=4, dtype=1, logits=FAKE, logits_stride=1001, tokens=FAKE, logprobs=FAKE, entropy=FAKE,
             top_ids=FAKE, top_logprobs=FAKE, workspace=FAKE, workspace_bytes=1 << 40)
    d.update(kw)
    return SpecLogprobArgs(**d)


def test_struct_sizes(L):
    from speculative_decoding_verify_attn_gb300 import serving as s
    for i, cls in enumerate((s.SpecPagedArgs, s.SpecPrefillArgs, s.SpecLogprobArgs)):
        assert L.spec_serve_struct_size(i) == ctypes.sizeof(cls)
    assert L.spec_serve_struct_size(3) == 0 and L.spec_serve_struct_size(-1) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(D=96), -2), (dict(Hq=7), -1), (dict(Hq=0), -1), (dict(Hkv=0), -1), (dict(B=0), -1), (dict(B=4097), -1),
    (dict(T=-1), -1), (dict(T=(1 << 22) + 1, max_q=5), -2), (dict(max_q=0), -1), (dict(max_q=-1), -1),
    (dict(Hq=66, Hkv=2), -2), (dict(q_dtype=0), -2), (dict(kv_dtype=5, q_dtype=5), -1), (dict(o_dtype=2), -1),
    (dict(page_size=0), -1), (dict(page_size=65537), -1), (dict(num_pages=0), -1), (dict(table_cols=0), -1),
    (dict(table_cols=1 << 28, page_size=16), -1), (dict(table_cols=(1 << 26) + 1, page_size=16), -1), (dict(table_stride=-1), -1), (dict(window=-1), -1),
    (dict(scale=float("nan")), -1), (dict(scale=-1.0), -1), (dict(q=None), -1), (dict(q=FAKE + 8), -1),
    (dict(q_stride_t=1028), -1), (dict(k_pages=None), -1), (dict(v_pages=FAKE + 4), -1), (dict(kv_stride_t=132), -1),
    (dict(kv_stride_p=-8), -1), (dict(k_new=FAKE), -1), (dict(v_new=FAKE), -1),
    (dict(k_new=FAKE, v_new=FAKE + 2, new_stride_t=256, new_stride_h=128), -1),
    (dict(k_new=FAKE, v_new=FAKE, new_stride_t=260, new_stride_h=128), -1), (dict(page_table=None), -1),
    (dict(q_start=FAKE + 2), -1), (dict(kv_len=None), -1), (dict(o=None), -1), (dict(o=FAKE + 1), -1),
    (dict(o_stride_h=-1), -1), (dict(workspace=None), -3), (dict(workspace=FAKE + 16), -3),
    (dict(workspace_bytes=512), -3),
])
def test_paged_refusals(L, kw, status):
    assert L.spec_paged_attn(ctypes.byref(paged(**kw)), None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(D=32), -2), (dict(Hq=9), -1), (dict(B=0), -1), (dict(window=-3), -1), (dict(scale=float("inf")), -1),
    (dict(q=None), -1), (dict(k=FAKE + 2), -1), (dict(v=None), -1), (dict(kv_stride_h=68), -1),
    (dict(seq_start=None), -1), (dict(o=FAKE + 2), -1), (dict(q_dtype=0), -2), (dict(workspace_bytes=1000), -3),
])
def test_prefill_refusals(L, kw, status):
    assert L.spec_prefill_attn(ctypes.byref(prefill(**kw)), None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), -1), (dict(V=0), -1), (dict(V=(1 << 24) + 1), -1), (dict(K=-1), -1), (dict(K=33), -2),
    (dict(V=3, logits_stride=3), -1), (dict(dtype=2), -1), (dict(logits=None), -1), (dict(logits=FAKE + 1), -1),
    (dict(logits_stride=1000), -1), (dict(tokens=None), -1), (dict(logprobs=None), -1), (dict(top_ids=None), -1),
    (dict(top_logprobs=None), -1), (dict(K=0), -1), (dict(entropy=FAKE + 2), -1), (dict(workspace=None), -3),
    (dict(K=0, top_ids=None, top_logprobs=None, tokens=None, logprobs=None, entropy=None), -1),
])
def test_logprobs_refusals(L, kw, status):
    assert L.spec_token_logprobs(ctypes.byref(logp(**kw)), None) == status


def test_empty_calls_launch_nothing(L):
    assert L.spec_paged_attn(ctypes.byref(paged(T=0, max_q=1, q=None, o=None, workspace=None)), None) == 0
    assert L.spec_prefill_attn(ctypes.byref(prefill(T=0, q=None, o=None, workspace=None)), None) == 0
    assert L.spec_token_logprobs(ctypes.byref(logp(N=0, logits=None, workspace=None)), None) == 0
    assert L.spec_paged_attn(None, None) == -1 and L.spec_paged_attn_workspace(None) == 0


def test_workspace_sizes(L):
    assert L.spec_paged_attn_workspace(ctypes.byref(paged(D=96))) == 0
    assert L.spec_paged_attn_workspace(ctypes.byref(paged(T=0, max_q=1))) > 0
    assert L.spec_prefill_attn_workspace(ctypes.byref(prefill(T=100000))) > L.spec_prefill_attn_workspace(
        ctypes.byref(prefill(T=1)))
    assert L.spec_token_logprobs_workspace(ctypes.byref(logp(N=2, V=128256, K=20))) > 256


def test_binding_refuses_host_tensors():
    import torch
    import speculative_decoding_verify_attn_gb300 as sv
    z = torch.zeros
    with pytest.raises(ValueError, match="CUDA"):
        sv.spec_token_logprobs(z(2, 8), z(2, dtype=torch.int32), z(2))
    with pytest.raises(ValueError, match="CUDA"):
        sv.spec_prefill_attn(z(4, 2, 64), z(4, 1, 64), z(4, 1, 64), z(2, dtype=torch.int32), z(4, 2, 64))
    with pytest.raises(ValueError, match="CUDA"):
        sv.spec_paged_attn(z(4, 2, 64), z(3, 1, 16, 64), z(3, 1, 16, 64), z((1, 2), dtype=torch.int32),
                           z(2, dtype=torch.int32), z(1, dtype=torch.int32), z(4, 2, 64), max_q=4)


def test_binding_argument_checks():
    """The argument structs are filled on the host, so shapes and types are checked without a GPU."""
    import torch
    from speculative_decoding_verify_attn_gb300 import serving as s
    z, i32 = torch.zeros, torch.int32
    ok = dict(q=z(4, 4, 64), k_pages=z(3, 2, 16, 64), v_pages=z(3, 2, 16, 64), page_table=z((1, 2), dtype=i32),
              q_start=z(2, dtype=i32), kv_len=z(1, dtype=i32), o=z(4, 4, 64), max_q=4)
    a = s.paged_attn_args(**ok)
    assert (a.B, a.Hq, a.Hkv, a.D, a.T, a.page_size, a.num_pages, a.table_cols) == (1, 4, 2, 64, 4, 16, 3, 2)
    assert (a.kv_stride_p, a.kv_stride_h, a.kv_stride_t) == (2048, 1024, 64)
    nhd = z(3, 16, 2, 64).permute(0, 2, 1, 3)
    a = s.paged_attn_args(**dict(ok, k_pages=nhd, v_pages=nhd))
    assert (a.kv_stride_h, a.kv_stride_t) == (64, 128)
    for bad, err in ((dict(kv_len=z(1, dtype=torch.int64)), ValueError), (dict(q_start=z(3, dtype=i32)), ValueError),
                     (dict(o=z(4, 2, 64)), ValueError), (dict(v_pages=z(3, 2, 16, 32)), ValueError),
                     (dict(k_new=z(4, 2, 64)), ValueError), (dict(k_new=z(4, 1, 64), v_new=z(4, 1, 64)), ValueError),
                     (dict(q=z(4, 4, 64).half()), TypeError)):
        with pytest.raises(err):
            s.paged_attn_args(**dict(ok, **bad))
    with pytest.raises(ValueError):
        s.token_logprobs_args(z(2, 8), z(2, dtype=torch.int64), z(2))
    with pytest.raises(ValueError):
        s.token_logprobs_args(z(2, 8), None, z(2))
    with pytest.raises(ValueError):
        s.prefill_attn_args(z(4, 2, 64), z(3, 1, 64), z(3, 1, 64), z(2, dtype=i32), z(4, 2, 64))
