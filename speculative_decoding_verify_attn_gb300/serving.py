"""ctypes binding of the serving operators (include/spec_serve.h): attention of new-token chunks over a
paged KV cache, attention over packed prompts, and token log probabilities.

Same names as the C ABI and the same manner as ``binding``: every function checks its tensors,
marshals them into the argument struct and calls the library on the current stream of the tensors'
device (or on ``stream``, which the caller orders behind whatever wrote the tensors).  There is no
fallback.
"""

from __future__ import annotations

import ctypes
import operator
from ctypes import POINTER, Structure, byref, c_float, c_int, c_int32, c_int64, c_size_t, c_void_p

from .binding import SPEC_BF16, SPEC_ERR_INVALID_ARG, SPEC_F32, SPEC_OK, SpecError, lib

SPEC_STATUS_BAD_RANGE = 16
SPEC_STATUS_BAD_PAGE = 32


class SpecPagedArgs(Structure):
    _fields_ = [
        ("B", c_int32), ("Hq", c_int32), ("Hkv", c_int32), ("D", c_int32), ("T", c_int32), ("max_q", c_int32),
        ("q_dtype", c_int32), ("kv_dtype", c_int32), ("o_dtype", c_int32),
        ("page_size", c_int32), ("num_pages", c_int32), ("table_cols", c_int32),
        ("window", c_int32), ("scale", c_float),
        ("q", c_void_p), ("q_stride_t", c_int64), ("q_stride_h", c_int64),
        ("k_pages", c_void_p), ("v_pages", c_void_p),
        ("kv_stride_p", c_int64), ("kv_stride_h", c_int64), ("kv_stride_t", c_int64),
        ("page_table", c_void_p), ("table_stride", c_int64), ("q_start", c_void_p), ("kv_len", c_void_p),
        ("k_new", c_void_p), ("v_new", c_void_p), ("new_stride_t", c_int64), ("new_stride_h", c_int64),
        ("o", c_void_p), ("o_stride_t", c_int64), ("o_stride_h", c_int64),
        ("workspace", c_void_p), ("workspace_bytes", c_size_t),
    ]


class SpecPrefillArgs(Structure):
    _fields_ = [
        ("B", c_int32), ("Hq", c_int32), ("Hkv", c_int32), ("D", c_int32), ("T", c_int32), ("window", c_int32),
        ("q_dtype", c_int32), ("kv_dtype", c_int32), ("o_dtype", c_int32), ("scale", c_float),
        ("q", c_void_p), ("q_stride_t", c_int64), ("q_stride_h", c_int64),
        ("k", c_void_p), ("v", c_void_p), ("kv_stride_t", c_int64), ("kv_stride_h", c_int64),
        ("seq_start", c_void_p),
        ("o", c_void_p), ("o_stride_t", c_int64), ("o_stride_h", c_int64),
        ("workspace", c_void_p), ("workspace_bytes", c_size_t),
    ]


class SpecLogprobArgs(Structure):
    _fields_ = [
        ("N", c_int32), ("V", c_int32), ("K", c_int32), ("dtype", c_int32),
        ("logits", c_void_p), ("logits_stride", c_int64), ("tokens", c_void_p),
        ("logprobs", c_void_p), ("entropy", c_void_p), ("top_ids", c_void_p), ("top_logprobs", c_void_p),
        ("workspace", c_void_p), ("workspace_bytes", c_size_t),
    ]


_lib = None


def _serve_lib():
    """The loaded library with this header's prototypes set (once)."""
    global _lib
    if _lib is None:
        L = lib()
        for name, cls in (("spec_paged_attn", SpecPagedArgs), ("spec_prefill_attn", SpecPrefillArgs),
                          ("spec_token_logprobs", SpecLogprobArgs)):
            fn, ws = getattr(L, name), getattr(L, name + "_workspace")
            fn.argtypes, fn.restype = [POINTER(cls), c_void_p], c_int
            ws.argtypes, ws.restype = [POINTER(cls)], c_size_t
        L.spec_serve_struct_size.argtypes, L.spec_serve_struct_size.restype = [c_int], c_size_t
        for i, cls in enumerate((SpecPagedArgs, SpecPrefillArgs, SpecLogprobArgs)):
            if L.spec_serve_struct_size(i) != ctypes.sizeof(cls):
                raise RuntimeError(f"ABI mismatch for {cls.__name__}: library {L.spec_serve_struct_size(i)} bytes, "
                                   f"binding {ctypes.sizeof(cls)}")
        _lib = L
    return _lib


# ---------------------------------------------------------------------------- helpers
# A decode step's kernel is done in a few microseconds, so what happens here per call is kept short:
# torch's objects are looked up once, sizes and strides are read once per tensor.
_torch = _i32 = _f32 = None
_codes = {}


def _t():
    """torch, imported on first use."""
    global _torch, _i32, _f32
    if _torch is None:
        import torch
        _torch, _i32, _f32 = torch, torch.int32, torch.float32
        _codes[torch.bfloat16], _codes[torch.float32] = SPEC_BF16, SPEC_F32
    return _torch


def _dtype_code(t) -> int:
    _torch or _t()
    code = _codes.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return code


def _check(tensors) -> int:
    """The index of the one CUDA device all tensors (None: not given) are on."""
    index = tensors[0].get_device()
    for t in tensors:
        if t is not None and (t.get_device() != index or index < 0):
            raise ValueError("all tensors must be CUDA tensors on one device (host buffers: copy them there first): "
                             + ", ".join(str(x.device) for x in tensors if x is not None))
    return index


def _rows(name, t):
    """The strides of a tensor whose innermost dimension has to be contiguous."""
    st = t.stride()
    if st[-1] != 1 and t.shape[-1] > 1:
        raise ValueError(f"{name}: innermost dimension must be contiguous")
    return st


def _equal(a, b) -> bool:
    """Whether two tensors of one shape step alike: dimensions of one element are never stepped over."""
    return all(x == y or n == 1 for n, x, y in zip(a.shape, a.stride(), b.stride()))


_TOP = 2 ** 31 - 1


def _whole(x) -> int:
    """A caller's whole number for a 32-bit field: what lies past 32 bits stays as large (or below zero) as the
    field can say, which for a window or a bound on lengths is the same."""
    x = operator.index(x)
    return x if -1 <= x <= _TOP else _TOP if x > 0 else -1


def _scale(x) -> float:
    """A caller's scale; one that is 0 in 32 bits would be taken for the default."""
    if x and c_float(x).value == 0:
        raise ValueError(f"scale {x} is 0 in 32 bits")
    return x


def _size(n) -> int:
    """A tensor's size for a 32-bit field; the largest value is above every limit of the calls."""
    return n if n <= _TOP else _TOP


def _vector(name, t, n, dtype):
    """Checks a contiguous vector of n elements."""
    if t.dtype is not dtype or t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} vector of {n}, got {t.dtype} {tuple(t.shape)}")


def _handle(stream) -> int:
    """A stream as its raw handle."""
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


_sizes = {}


def _call(name, args, sizes, index, workspace, stream):
    """Sizes the workspace, fills it in and makes the call on the tensors' device.  `sizes` is what the
    workspace's size depends on: the library is asked once for each."""
    torch = _torch or _t()
    if index != torch._C._cuda_getDevice():
        with torch.cuda.device(index):
            return _call(name, args, sizes, index, workspace, stream)
    L = _lib or _serve_lib()
    ref = byref(args)
    need = _sizes.get(sizes)
    if need is None:
        need = getattr(L, name + "_workspace")(ref)
        if need == 0:
            # the call itself says why the sizes are refused
            raise SpecError(getattr(L, name)(ref, None) or SPEC_ERR_INVALID_ARG, name)
        if len(_sizes) > 4096:
            _sizes.clear()
        _sizes[sizes] = need
    handle = torch._C._cuda_getCurrentRawStream(index)
    other = None  # a stream other than the current one
    if stream is not None:
        own = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(_handle(stream))
        if own.cuda_stream != handle:
            other, handle = own, own.cuda_stream
    if workspace is None:
        if other is None:
            workspace = torch.empty(need, dtype=torch.uint8, device="cuda")
        else:
            # from the launching stream's pool: a block of the current stream's may still be in use there
            with torch.cuda.stream(other):
                workspace = torch.empty(need, dtype=torch.uint8, device="cuda")
        given = need
    else:
        if workspace.get_device() != index or not workspace.is_contiguous():
            raise ValueError(f"workspace must be contiguous and on cuda:{index}")
        given = workspace.numel() * workspace.element_size()
        if given < need:
            raise ValueError(f"workspace too small: need {need} bytes")
        if other is not None:
            # its memory is not handed out again before the other stream has passed this call
            workspace.record_stream(other)
    args.workspace = workspace.data_ptr()
    args.workspace_bytes = given
    st = getattr(L, name)(ref, handle)
    if st != SPEC_OK:
        raise SpecError(st, name)


def _workspace_bytes(name, args) -> int:
    need = getattr(_serve_lib(), name + "_workspace")(byref(args))
    if need == 0:
        raise SpecError(SPEC_ERR_INVALID_ARG, name + "_workspace")
    return need


# ---------------------------------------------------------------------------- paged attention
def paged_attn_args(q, k_pages, v_pages, page_table, q_start, kv_len, o, *, max_q, k_new=None, v_new=None,
                    window: int = 0, scale: float = 0.0) -> SpecPagedArgs:
    """Fill SpecPagedArgs from tensors (no workspace yet)."""
    _torch or _t()
    q_shape, shape = q.shape, k_pages.shape
    T, Hq, D = q_shape
    pages, Hkv, page_size, D2 = shape
    B, cols = page_table.shape
    qs, ks, os_, ts = _rows("q", q), _rows("k_pages", k_pages), _rows("o", o), _rows("page_table", page_table)
    if D2 != D or v_pages.shape != shape or not (v_pages.stride() == ks or _equal(v_pages, k_pages)):
        raise ValueError("k_pages and v_pages must be [pages, Hkv, page_size, D] with q's D and equal strides")
    if v_pages.dtype is not k_pages.dtype:
        raise TypeError("k_pages and v_pages must share a dtype")
    if o.shape != q_shape:
        raise ValueError("o must have q's shape")
    if page_table.dtype is not _i32:
        raise ValueError(f"page_table must be int32, got {page_table.dtype}")
    _vector("q_start", q_start, B + 1, _i32)
    _vector("kv_len", kv_len, B, _i32)
    kn = vn = None
    ns = (0, 0)
    if k_new is not None or v_new is not None:
        if k_new is None or v_new is None:
            raise ValueError("k_new and v_new go together")
        ns = _rows("k_new", k_new)
        if k_new.shape != (T, Hkv, D) or v_new.shape != k_new.shape or not (
                v_new.stride() == ns or _equal(v_new, k_new)):
            raise ValueError("k_new, v_new must be [T, Hkv, D] with equal strides")
        if k_new.dtype is not k_pages.dtype or v_new.dtype is not k_pages.dtype:
            raise TypeError("k_new, v_new must have the cache's dtype")
        kn, vn = k_new.data_ptr(), v_new.data_ptr()
    if max_q.__class__ is not int or not 0 <= max_q <= _TOP:
        max_q = _whole(max_q)
    if window.__class__ is not int or not 0 <= window <= _TOP:
        window = _whole(window)
    if B > _TOP or T > _TOP or page_size > _TOP or pages > _TOP or cols > _TOP:
        raise ValueError("sizes past 32 bits")
    # the stride of a dimension of one element may be anything: D stands in its place
    return SpecPagedArgs(
        B, Hq, Hkv, D, T, max_q, _dtype_code(q), _dtype_code(k_pages), _dtype_code(o), page_size, pages, cols,
        window, _scale(scale) if scale else 0.0, q.data_ptr(), qs[0] if T > 1 else D, qs[1] if Hq > 1 else D,
        k_pages.data_ptr(), v_pages.data_ptr(), ks[0] if pages > 1 else D, ks[1] if Hkv > 1 else D,
        ks[2] if page_size > 1 else D, page_table.data_ptr(), ts[0], q_start.data_ptr(), kv_len.data_ptr(), kn, vn,
        ns[0] if T > 1 else D, ns[1] if Hkv > 1 else D, o.data_ptr(), os_[0], os_[1], None, 0)


def spec_paged_attn_workspace(q, k_pages, page_table, o, *, max_q) -> int:
    """Bytes of workspace spec_paged_attn needs for tensors of these shapes."""
    T, Hq, D = q.shape
    a = SpecPagedArgs(B=_size(page_table.shape[0]), Hq=Hq, Hkv=k_pages.shape[1], D=D, T=_size(T), max_q=_whole(max_q),
                      q_dtype=_dtype_code(q), kv_dtype=_dtype_code(k_pages), o_dtype=_dtype_code(o))
    return _workspace_bytes("spec_paged_attn", a)


def spec_paged_attn(q, k_pages, v_pages, page_table, q_start, kv_len, o, *, max_q, k_new=None, v_new=None,
                    window: int = 0, scale: float = 0.0, workspace=None, stream=None):
    """Attention of a ragged batch of new-token chunks over a paged cache.

    q, o [T, Hq, D]; k_pages, v_pages [pages, Hkv, page_size, D] (any strides, so a permuted view of
    another page layout serves too); page_table [B, cols] int32; q_start [B + 1] int32, the rows of
    sequence b being q_start[b] .. q_start[b + 1] - 1; kv_len [B] int32, the new tokens included.
    max_q: an upper bound on the chunk lengths.  With k_new, v_new [T, Hkv, D] the call also writes
    them into the new tokens' slots.  window > 0: rows see the last `window` tokens only.  Writes o
    and returns it."""
    index = _check((q, k_pages, v_pages, page_table, q_start, kv_len, o, k_new, v_new))
    a = paged_attn_args(q, k_pages, v_pages, page_table, q_start, kv_len, o, max_q=max_q, k_new=k_new, v_new=v_new,
                        window=window, scale=scale)
    _call("spec_paged_attn", a, (a.B, a.Hq, a.Hkv, a.D, a.T, a.max_q, a.kv_dtype, "paged"), index, workspace, stream)
    return o


# ---------------------------------------------------------------------------- packed prompts
def prefill_attn_args(q, k, v, seq_start, o, *, window: int = 0, scale: float = 0.0) -> SpecPrefillArgs:
    """Fill SpecPrefillArgs from tensors (no workspace yet)."""
    _torch or _t()
    T, Hq, D = q.shape
    qs, ks, os_ = _rows("q", q), _rows("k", k), _rows("o", o)
    if k.dim() != 3 or k.shape[0] != T or k.shape[2] != D or v.shape != k.shape or not (
            v.stride() == ks or _equal(v, k)):
        raise ValueError("k, v must be [T, Hkv, D] with equal strides")
    if v.dtype is not k.dtype:
        raise TypeError("k and v must share a dtype")
    if o.shape != q.shape:
        raise ValueError("o must have q's shape")
    B = seq_start.shape[0] - 1
    _vector("seq_start", seq_start, B + 1, _i32)
    Hkv = k.shape[1]
    if B > _TOP or T > _TOP:
        raise ValueError("sizes past 32 bits")
    # the stride of a dimension of one element may be anything: D stands in its place
    return SpecPrefillArgs(
        B, Hq, Hkv, D, T, _whole(window), _dtype_code(q), _dtype_code(k), _dtype_code(o),
        _scale(scale) if scale else 0.0, q.data_ptr(), qs[0] if T > 1 else D, qs[1] if Hq > 1 else D, k.data_ptr(),
        v.data_ptr(), ks[0] if T > 1 else D, ks[1] if Hkv > 1 else D, seq_start.data_ptr(), o.data_ptr(), os_[0],
        os_[1], None, 0)


def spec_prefill_attn_workspace(q, k, seq_start, o) -> int:
    """Bytes of workspace spec_prefill_attn needs for tensors of these shapes."""
    T, Hq, D = q.shape
    a = SpecPrefillArgs(B=_size(seq_start.shape[0] - 1), Hq=Hq, Hkv=k.shape[1], D=D, T=_size(T), q_dtype=_dtype_code(q),
                        kv_dtype=_dtype_code(k), o_dtype=_dtype_code(o))
    return _workspace_bytes("spec_prefill_attn", a)


def spec_prefill_attn(q, k, v, seq_start, o, *, window: int = 0, scale: float = 0.0, workspace=None, stream=None):
    """Causal attention over whole prompts packed one after the other.

    q, o [T, Hq, D]; k, v [T, Hkv, D]; seq_start [B + 1] int32, sequence b being rows seq_start[b] ..
    seq_start[b + 1] - 1.  window > 0: rows see the last `window` tokens only.  Writes o and returns
    it."""
    index = _check((q, k, v, seq_start, o))
    a = prefill_attn_args(q, k, v, seq_start, o, window=window, scale=scale)
    _call("spec_prefill_attn", a, (a.B, a.Hq, a.Hkv, a.D, a.T, a.kv_dtype, "prefill"), index, workspace, stream)
    return o


# ---------------------------------------------------------------------------- log probabilities
def token_logprobs_args(logits, tokens, logprobs, *, entropy=None, top_ids=None, top_logprobs=None) -> SpecLogprobArgs:
    """Fill SpecLogprobArgs from tensors (no workspace yet)."""
    _torch or _t()
    N, V = logits.shape
    K = 0
    lp = ent = tok = ids = top = None
    if tokens is not None or logprobs is not None:
        if tokens is None or logprobs is None:
            raise ValueError("tokens and logprobs go together")
        _vector("tokens", tokens, N, _i32)
        _vector("logprobs", logprobs, N, _f32)
        tok, lp = tokens.data_ptr(), logprobs.data_ptr()
    if entropy is not None:
        _vector("entropy", entropy, N, _f32)
        ent = entropy.data_ptr()
    if top_ids is not None or top_logprobs is not None:
        if top_ids is None or top_logprobs is None:
            raise ValueError("top_ids and top_logprobs go together")
        K = top_ids.shape[1]
        for name, x, dtype in (("top_ids", top_ids, _i32), ("top_logprobs", top_logprobs, _f32)):
            if x.dtype is not dtype or x.shape != (N, K) or not x.is_contiguous():
                raise ValueError(f"{name} must be contiguous {dtype} of shape {(N, K)}")
        if K:
            ids, top = top_ids.data_ptr(), top_logprobs.data_ptr()
    if N > _TOP or V > _TOP or K > _TOP:
        raise ValueError("sizes past 32 bits")
    # the stride of a single row may be anything
    return SpecLogprobArgs(N, V, K, _dtype_code(logits), logits.data_ptr(), _rows("logits", logits)[0] if N > 1 else V,
                           tok, lp, ent, ids, top, None, 0)


def spec_token_logprobs_workspace(logits, K: int = 0) -> int:
    """Bytes of workspace spec_token_logprobs needs for these logits and K alternatives."""
    return _workspace_bytes("spec_token_logprobs", SpecLogprobArgs(N=_size(logits.shape[0]), V=_size(logits.shape[1]),
                                                                   K=_whole(K), dtype=_dtype_code(logits)))


def spec_token_logprobs(logits, tokens, logprobs, *, entropy=None, top_ids=None, top_logprobs=None, workspace=None,
                        stream=None):
    """Log probabilities of given tokens, with the rows' entropies and top alternatives.

    logits [N, V] fp32 or bf16; tokens [N] int32 and logprobs [N] fp32 (both or neither); entropy [N]
    fp32; top_ids [N, K] int32 and top_logprobs [N, K] fp32 (K <= 32, descending, lower ids first
    among equals).  Outputs not wanted are None.  Writes them and returns logprobs."""
    index = _check((logits, tokens, logprobs, entropy, top_ids, top_logprobs))
    a = token_logprobs_args(logits, tokens, logprobs, entropy=entropy, top_ids=top_ids, top_logprobs=top_logprobs)
    _call("spec_token_logprobs", a, (a.N, a.V, a.K, "logprobs"), index, workspace, stream)
    return logprobs
