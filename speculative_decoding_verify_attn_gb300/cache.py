"""ctypes binding of the operators around a paged KV cache (include/spec_cache.h): rotary positions, K/V
written into a cache held in 8 bits and attention over it, pages forked and compacted.

Same names as the C ABI and the same manner as ``serving``: every function checks its tensors, marshals
them into the argument struct and calls the library on the current stream of the tensors' device (or on
``stream``, which the caller orders behind whatever wrote the tensors).  There is no fallback.
"""

from __future__ import annotations

import ctypes
from array import array
from ctypes import POINTER, Structure, byref, c_double, c_float, c_int, c_int32, c_int64, c_size_t, c_void_p

from . import serving as _s
from .binding import SPEC_OK, SpecError
from .serving import _TOP, _call, _check, _dtype_code, _equal, _rows, _scale, _serve_lib, _size, _t, _vector, _whole, _workspace_bytes

SPEC_STATUS_NO_PAGE = 64

SPEC_ROTARY_HALF = 0
SPEC_ROTARY_PAIRS = 1

SPEC_ROTARY_PLAIN = 0
SPEC_ROTARY_LINEAR = 1
SPEC_ROTARY_NTK = 2
SPEC_ROTARY_BANDS = 3
SPEC_ROTARY_YARN = 4


class SpecRotaryArgs(Structure):
    _fields_ = [
        ("T", c_int32), ("Hq", c_int32), ("Hkv", c_int32), ("D", c_int32), ("rot", c_int32),
        ("layout", c_int32), ("dtype", c_int32), ("inverse", c_int32), ("B", c_int32), ("amplitude", c_float),
        ("q", c_void_p), ("q_stride_t", c_int64), ("q_stride_h", c_int64),
        ("k", c_void_p), ("k_stride_t", c_int64), ("k_stride_h", c_int64),
        ("q_out", c_void_p), ("qo_stride_t", c_int64), ("qo_stride_h", c_int64),
        ("k_out", c_void_p), ("ko_stride_t", c_int64), ("ko_stride_h", c_int64),
        ("steps", c_void_p), ("positions", c_void_p), ("q_start", c_void_p), ("kv_len", c_void_p),
        ("workspace", c_void_p), ("workspace_bytes", c_size_t),
    ]


class SpecKv8AppendArgs(Structure):
    _fields_ = [
        ("B", c_int32), ("Hkv", c_int32), ("D", c_int32), ("T", c_int32), ("src_dtype", c_int32),
        ("page_size", c_int32), ("num_pages", c_int32), ("table_cols", c_int32), ("block", c_int32),
        ("reserved0", c_int32),
        ("k_new", c_void_p), ("v_new", c_void_p), ("new_stride_t", c_int64), ("new_stride_h", c_int64),
        ("k_pages", c_void_p), ("v_pages", c_void_p),
        ("kv_stride_p", c_int64), ("kv_stride_h", c_int64), ("kv_stride_t", c_int64),
        ("k_exp", c_void_p), ("v_exp", c_void_p), ("exp_stride_p", c_int64), ("exp_stride_h", c_int64),
        ("page_table", c_void_p), ("table_stride", c_int64), ("q_start", c_void_p), ("kv_len", c_void_p),
        ("workspace", c_void_p), ("workspace_bytes", c_size_t),
    ]


class SpecPaged8Args(Structure):
    _fields_ = [
        ("B", c_int32), ("Hq", c_int32), ("Hkv", c_int32), ("D", c_int32), ("T", c_int32), ("max_q", c_int32),
        ("q_dtype", c_int32), ("o_dtype", c_int32),
        ("page_size", c_int32), ("num_pages", c_int32), ("table_cols", c_int32),
        ("window", c_int32), ("block", c_int32), ("scale", c_float),
        ("q", c_void_p), ("q_stride_t", c_int64), ("q_stride_h", c_int64),
        ("k_pages", c_void_p), ("v_pages", c_void_p),
        ("kv_stride_p", c_int64), ("kv_stride_h", c_int64), ("kv_stride_t", c_int64),
        ("k_exp", c_void_p), ("v_exp", c_void_p), ("exp_stride_p", c_int64), ("exp_stride_h", c_int64),
        ("page_table", c_void_p), ("table_stride", c_int64), ("q_start", c_void_p), ("kv_len", c_void_p),
        ("k_new", c_void_p), ("v_new", c_void_p), ("new_stride_t", c_int64), ("new_stride_h", c_int64),
        ("o", c_void_p), ("o_stride_t", c_int64), ("o_stride_h", c_int64),
        ("workspace", c_void_p), ("workspace_bytes", c_size_t),
    ]


class SpecPageArray(Structure):
    _fields_ = [("base", c_void_p), ("stride_bytes", c_int64), ("page_bytes", c_int64)]


class SpecPageForkArgs(Structure):
    _fields_ = [
        ("B", c_int32), ("table_cols", c_int32), ("page_size", c_int32), ("num_pages", c_int32),
        ("num_arrays", c_int32), ("reserved0", c_int32),
        ("page_table", c_void_p), ("table_stride", c_int64), ("held", c_void_p), ("kv_len", c_void_p),
        ("refs", c_void_p), ("parent", c_void_p), ("grow", c_void_p),
        ("table_out", c_void_p), ("table_out_stride", c_int64), ("held_out", c_void_p), ("kv_len_out", c_void_p),
        ("refs_out", c_void_p), ("arrays", c_void_p),
        ("workspace", c_void_p), ("workspace_bytes", c_size_t),
    ]


class SpecPageCompactArgs(Structure):
    _fields_ = [
        ("B", c_int32), ("table_cols", c_int32), ("num_pages", c_int32), ("num_arrays", c_int32),
        ("page_table", c_void_p), ("table_stride", c_int64), ("held", c_void_p), ("refs", c_void_p),
        ("table_out", c_void_p), ("table_out_stride", c_int64), ("refs_out", c_void_p), ("moved", c_void_p),
        ("num_live", c_void_p), ("arrays", c_void_p),
        ("workspace", c_void_p), ("workspace_bytes", c_size_t),
    ]


_STRUCTS = (SpecRotaryArgs, SpecKv8AppendArgs, SpecPaged8Args, SpecPageForkArgs, SpecPageCompactArgs, SpecPageArray)
_lib = None


def _cache_lib():
    """The loaded library with this header's prototypes set (once)."""
    global _lib
    if _lib is None:
        L = _serve_lib()
        for name, cls in (("spec_rotary", SpecRotaryArgs), ("spec_kv8_append", SpecKv8AppendArgs),
                          ("spec_paged_attn8", SpecPaged8Args), ("spec_page_fork", SpecPageForkArgs),
                          ("spec_page_compact", SpecPageCompactArgs)):
            fn, ws = getattr(L, name), getattr(L, name + "_workspace")
            fn.argtypes, fn.restype = [POINTER(cls), c_void_p], c_int
            ws.argtypes, ws.restype = [POINTER(cls)], c_size_t
        L.spec_rotary_steps.argtypes = [c_int32, c_int32] + [c_double] * 5 + [c_void_p, POINTER(c_float)]
        L.spec_rotary_steps.restype = c_int
        L.spec_cache_struct_size.argtypes, L.spec_cache_struct_size.restype = [c_int], c_size_t
        for i, cls in enumerate(_STRUCTS):
            if L.spec_cache_struct_size(i) != ctypes.sizeof(cls):
                raise RuntimeError(f"ABI mismatch for {cls.__name__}: library {L.spec_cache_struct_size(i)} bytes, "
                                   f"binding {ctypes.sizeof(cls)}")
        _lib = L
    return _lib


def _run(name, args, sizes, index, workspace, stream):
    _lib or _cache_lib()
    _call(name, args, sizes, index, workspace, stream)


def _need(name, args) -> int:
    _lib or _cache_lib()
    return _workspace_bytes(name, args)


def _ints(name, t, n):
    _vector(name, t, n, _s._i32)


# ---------------------------------------------------------------------------- rotary positions
def spec_rotary_steps(rot: int, base: float = 10000.0, *, kind: int = SPEC_ROTARY_PLAIN, factor: float = 1.0,
                      length: float = 0.0, low: float = 1.0, high: float = 32.0, device="cuda"):
    """Turns per position of the rot / 2 pairs, in units of 2^-64, as an int64 tensor on `device`, and the
    amplitude that goes with them.

    kind: SPEC_ROTARY_PLAIN, _LINEAR (positions divided by factor), _NTK (a larger base), _BANDS (only long
    wavelengths are stretched; low and high are those of the bands) or _YARN (a ramp between the pairs that
    make `high` and `low` turns over `length` positions, and an amplitude); length is the context of the
    training."""
    torch = _t()
    rot = _whole(rot)
    steps = torch.empty(max(rot, 0) // 2, dtype=torch.int64)
    amplitude = c_float()
    st = _cache_lib().spec_rotary_steps(rot, _whole(kind), base, factor, length, low, high, steps.data_ptr() or None,
                                        byref(amplitude))
    if st != SPEC_OK:
        raise SpecError(st, "spec_rotary_steps")
    return steps.to(device), amplitude.value


_NONE = (0, None, 0, 0, None, 0, 0)


def _heads(name, x, out, T, D, dtype):
    """Heads of q or k, its pointer and strides and its output's."""
    if x is None:
        if out is not None:
            raise ValueError(f"{name}_out without {name}")
        return _NONE
    shape = x.shape
    if len(shape) != 3 or shape[0] != T or shape[2] != D or x.dtype is not dtype:
        raise ValueError(f"{name} must be [{T}, heads, {D}] of {dtype}")
    H, st = shape[1], _rows(name, x)
    # the stride of a dimension of one element may be anything: D stands in its place
    ptr, s0, s1 = x.data_ptr(), st[0] if T > 1 else D, st[1] if H > 1 else D
    if out is None or out is x:
        return H, ptr, s0, s1, ptr, s0, s1
    if out.shape != shape or out.dtype is not dtype:
        raise ValueError(f"{name}_out must be like {name}")
    st = _rows(name + "_out", out)
    return H, ptr, s0, s1, out.data_ptr(), st[0] if T > 1 else D, st[1] if H > 1 else D


def rotary_args(q, k, steps, *, positions=None, q_start=None, kv_len=None, q_out=None, k_out=None,
                layout: int = SPEC_ROTARY_HALF, amplitude: float = 1.0, inverse: bool = False) -> SpecRotaryArgs:
    """Fill SpecRotaryArgs from tensors (no workspace yet)."""
    torch = _t()
    x = q if q is not None else k
    if x is None:
        raise ValueError("neither q nor k")
    T, _, D = x.shape
    dtype = x.dtype
    Hq, q_ptr, q0, q1, qo_ptr, qo0, qo1 = _heads("q", q, q_out, T, D, dtype)
    Hkv, k_ptr, k0, k1, ko_ptr, ko0, ko1 = _heads("k", k, k_out, T, D, dtype)
    if steps.dim() != 1 or steps.dtype is not torch.int64 or not steps.is_contiguous():
        raise ValueError("steps must be a contiguous int64 vector")
    B = 0
    ps = st = kl = None
    if positions is not None:
        if q_start is not None or kv_len is not None:
            raise ValueError("positions, or q_start and kv_len, not both")
        _ints("positions", positions, T)
        ps = positions.data_ptr()
    else:
        if q_start is None or kv_len is None:
            raise ValueError("positions, or q_start and kv_len")
        B = kv_len.shape[0]
        _ints("q_start", q_start, B + 1)
        _ints("kv_len", kv_len, B)
        st, kl = q_start.data_ptr(), kv_len.data_ptr()
    amplitude = float(amplitude)
    if not c_float(amplitude).value > 0:  # the struct's 0 stands for 1
        raise ValueError(f"amplitude must be above 0, got {amplitude}")
    rot = 2 * steps.shape[0]
    if T > _TOP or D > _TOP or B > _TOP or rot > _TOP:
        raise ValueError("sizes past 32 bits")
    return SpecRotaryArgs(T, Hq, Hkv, D, rot, _whole(layout), _dtype_code(x), 1 if inverse else 0, B, amplitude, q_ptr, q0, q1,
                          k_ptr, k0, k1, qo_ptr, qo0, qo1, ko_ptr, ko0, ko1, steps.data_ptr(), ps, st, kl, None, 0)


def spec_rotary_workspace(q, k, steps) -> int:
    """Bytes of workspace spec_rotary needs for tensors of these shapes."""
    x = q if q is not None else k
    return _need("spec_rotary", SpecRotaryArgs(T=_size(x.shape[0]), Hq=q.shape[1] if q is not None else 0,
                                               Hkv=k.shape[1] if k is not None else 0, D=_size(x.shape[2]),
                                               rot=_size(2 * steps.shape[0]), dtype=_dtype_code(x)))


def spec_rotary(q, k, steps, *, positions=None, q_start=None, kv_len=None, q_out=None, k_out=None,
                layout: int = SPEC_ROTARY_HALF, amplitude: float = 1.0, inverse: bool = False, workspace=None,
                stream=None):
    """Turns the new tokens' queries and keys to their positions.

    q [T, Hq, D], k [T, Hkv, D] (either may be None); steps [rot / 2] int64 from spec_rotary_steps: the first
    rot values of each head are turned, in halves (SPEC_ROTARY_HALF) or in pairs (SPEC_ROTARY_PAIRS).
    positions [T] int32, or q_start [B + 1] and kv_len [B] as in spec_paged_attn (rows of no sequence are left
    as they were).  q_out, k_out: outputs, None for in place.  inverse turns back, which is also what gradients
    take.  Returns (q_out, k_out)."""
    index = _check((steps, q, k, positions, q_start, kv_len, q_out, k_out))
    a = rotary_args(q, k, steps, positions=positions, q_start=q_start, kv_len=kv_len, q_out=q_out, k_out=k_out,
                    layout=layout, amplitude=amplitude, inverse=inverse)
    _run("spec_rotary", a, (a.T, a.Hq, a.Hkv, a.D, a.rot, a.layout, a.dtype, "rotary"), index, workspace, stream)
    return q if q_out is None else q_out, k if k_out is None else k_out


# ---------------------------------------------------------------------------- the cache in 8 bits
_e4m3 = _u8 = None


def _types():
    global _e4m3, _u8
    torch = _t()
    _e4m3, _u8 = torch.float8_e4m3fn, torch.uint8


def _cache8(k_pages, v_pages, k_exp, v_exp, page_table, q_start, kv_len, D):
    """Checks the cache and the tables; (B, Hkv, page_size, pages, cols, block, pointers and strides)."""
    _e4m3 or _types()
    shape, ks = k_pages.shape, k_pages.stride()
    if k_pages.dtype is not _e4m3 or v_pages.dtype is not _e4m3 or len(shape) != 4:
        raise TypeError("k_pages, v_pages must be [pages, Hkv, page_size, D] of float8_e4m3fn")
    pages, Hkv, page_size, D2 = shape
    if D2 != D or v_pages.shape != shape or not (v_pages.stride() == ks or _equal(v_pages, k_pages)):
        raise ValueError("k_pages and v_pages must be [pages, Hkv, page_size, D] with equal strides")
    if ks[3] != 1:
        _rows("k_pages", k_pages)
    if k_exp.dtype is not _u8 or v_exp.dtype is not _u8:
        raise TypeError("k_exp, v_exp must be uint8")
    eshape, es = k_exp.shape, k_exp.stride()
    blocks = eshape[-1]
    if eshape != (pages, Hkv, blocks) or v_exp.shape != eshape or not (v_exp.stride() == es or _equal(v_exp, k_exp)):
        raise ValueError("k_exp and v_exp must be [pages, Hkv, blocks] with equal strides")
    if es[2] != 1:
        _rows("k_exp", k_exp)
    if blocks < 1 or page_size % blocks:
        raise ValueError(f"{blocks} blocks do not divide a page of {page_size} tokens")
    B, cols = page_table.shape
    ts = page_table.stride()
    if ts[1] != 1:
        _rows("page_table", page_table)
    if page_table.dtype is not _s._i32:
        raise ValueError(f"page_table must be int32, got {page_table.dtype}")
    _vector("q_start", q_start, B + 1, _s._i32)
    _vector("kv_len", kv_len, B, _s._i32)
    if B > _TOP or page_size > _TOP or pages > _TOP or cols > _TOP:
        raise ValueError("sizes past 32 bits")
    # the stride of a dimension of one element may be anything: D (or 1) stands in its place
    layout = (k_pages.data_ptr(), v_pages.data_ptr(), ks[0] if pages > 1 else D, ks[1] if Hkv > 1 else D,
              ks[2] if page_size > 1 else D, k_exp.data_ptr(), v_exp.data_ptr(), es[0] if pages > 1 else 1,
              es[1] if Hkv > 1 else 1, page_table.data_ptr(), ts[0], q_start.data_ptr(), kv_len.data_ptr())
    return B, Hkv, page_size, pages, cols, page_size // blocks, layout


def _new_rows(k_new, v_new, T, Hkv, D):
    """Pointers and strides of the new rows."""
    shape, ns = k_new.shape, k_new.stride()
    if shape != (T, Hkv, D) or v_new.shape != shape or not (v_new.stride() == ns or _equal(v_new, k_new)):
        raise ValueError("k_new, v_new must be [T, Hkv, D] with equal strides")
    if v_new.dtype is not k_new.dtype:
        raise TypeError("k_new and v_new must share a dtype")
    if ns[2] != 1:
        _rows("k_new", k_new)
    return k_new.data_ptr(), v_new.data_ptr(), ns[0] if T > 1 else D, ns[1] if Hkv > 1 else D


def kv8_append_args(k_new, v_new, k_pages, v_pages, k_exp, v_exp, page_table, q_start, kv_len) -> SpecKv8AppendArgs:
    """Fill SpecKv8AppendArgs from tensors (no workspace yet)."""
    _t()
    T, _, D = k_new.shape
    B, Hkv, page_size, pages, cols, block, layout = _cache8(k_pages, v_pages, k_exp, v_exp, page_table, q_start, kv_len, D)
    new = _new_rows(k_new, v_new, T, Hkv, D)
    return SpecKv8AppendArgs(B, Hkv, _size(D), _size(T), _dtype_code(k_new), page_size, pages, cols, block, 0, *new, *layout,
                             None, 0)


def spec_kv8_append_workspace(k_new, page_table) -> int:
    """Bytes of workspace spec_kv8_append needs for tensors of these shapes."""
    T, Hkv, D = k_new.shape
    return _need("spec_kv8_append", SpecKv8AppendArgs(B=_size(page_table.shape[0]), Hkv=Hkv, D=D, T=_size(T),
                                                      src_dtype=_dtype_code(k_new)))


def spec_kv8_append(k_new, v_new, k_pages, v_pages, k_exp, v_exp, page_table, q_start, kv_len, *, workspace=None,
                    stream=None):
    """Writes new tokens' K/V into a paged cache in 8 bits.

    k_new, v_new [T, Hkv, D] bf16 or fp32; k_pages, v_pages [pages, Hkv, page_size, D] float8_e4m3fn; k_exp,
    v_exp [pages, Hkv, page_size / block] uint8, the scale of a block being 2^(byte - 127); page_table [B,
    cols], q_start [B + 1] and kv_len [B] (new tokens included) as in spec_paged_attn.  A block's scale is
    the least power of two that brings its values within 448; one that grows brings the block's earlier
    tokens along."""
    index = _check((k_new, v_new, k_pages, v_pages, k_exp, v_exp, page_table, q_start, kv_len))
    a = kv8_append_args(k_new, v_new, k_pages, v_pages, k_exp, v_exp, page_table, q_start, kv_len)
    _run("spec_kv8_append", a, (a.B, a.Hkv, a.D, a.T, a.src_dtype, "kv8"), index, workspace, stream)


def paged_attn8_args(q, k_pages, v_pages, k_exp, v_exp, page_table, q_start, kv_len, o, *, max_q, k_new=None, v_new=None,
                     window: int = 0, scale: float = 0.0) -> SpecPaged8Args:
    """Fill SpecPaged8Args from tensors (no workspace yet)."""
    q_shape = q.shape
    T, Hq, D = q_shape
    B, Hkv, page_size, pages, cols, block, layout = _cache8(k_pages, v_pages, k_exp, v_exp, page_table, q_start, kv_len, D)
    qs, os_ = _rows("q", q), _rows("o", o)
    if o.shape != q_shape:
        raise ValueError("o must have q's shape")
    new = (None, None, 0, 0)
    if k_new is not None or v_new is not None:
        if k_new is None or v_new is None:
            raise ValueError("k_new and v_new go together")
        if k_new.dtype is not q.dtype:
            raise TypeError("k_new, v_new must have q's dtype")
        new = _new_rows(k_new, v_new, T, Hkv, D)
    if T > _TOP:
        raise ValueError("sizes past 32 bits")
    if max_q.__class__ is not int or not 0 <= max_q <= _TOP:
        max_q = _whole(max_q)
    if window.__class__ is not int or not 0 <= window <= _TOP:
        window = _whole(window)
    return SpecPaged8Args(
        B, Hq, Hkv, D, T, max_q, _dtype_code(q), _dtype_code(o), page_size, pages, cols, window, block,
        _scale(scale) if scale else 0.0, q.data_ptr(), qs[0] if T > 1 else D, qs[1] if Hq > 1 else D, *layout, *new,
        o.data_ptr(), os_[0], os_[1], None, 0)


def spec_paged_attn8_workspace(q, k_pages, page_table, o, *, max_q) -> int:
    """Bytes of workspace spec_paged_attn8 needs for tensors of these shapes."""
    T, Hq, D = q.shape
    return _need("spec_paged_attn8", SpecPaged8Args(B=_size(page_table.shape[0]), Hq=Hq, Hkv=k_pages.shape[1], D=D,
                                                    T=_size(T), max_q=_whole(max_q), q_dtype=_dtype_code(q),
                                                    o_dtype=_dtype_code(o)))


def spec_paged_attn8(q, k_pages, v_pages, k_exp, v_exp, page_table, q_start, kv_len, o, *, max_q, k_new=None, v_new=None,
                     window: int = 0, scale: float = 0.0, workspace=None, stream=None):
    """Attention of a ragged batch of new-token chunks over a paged cache in 8 bits.

    As spec_paged_attn, with the cache of spec_kv8_append; q (and k_new, v_new) bf16.  With k_new, v_new the
    call first appends them as spec_kv8_append does, and sees them as the cache holds them.  Writes o and
    returns it."""
    index = _check((q, k_pages, v_pages, k_exp, v_exp, page_table, q_start, kv_len, o, k_new, v_new))
    a = paged_attn8_args(q, k_pages, v_pages, k_exp, v_exp, page_table, q_start, kv_len, o, max_q=max_q, k_new=k_new,
                         v_new=v_new, window=window, scale=scale)
    _run("spec_paged_attn8", a, (a.B, a.Hq, a.Hkv, a.D, a.T, a.max_q, a.q_dtype, "paged8"), index, workspace, stream)
    return o


# ---------------------------------------------------------------------------- pages
def _page_arrays(caches, pages):
    """The caches [pages, ...] as the library takes them.  A page has to be one run of bytes, in any order of
    its dimensions."""
    words = array("q")  # SpecPageArray is three of them
    for t in caches:
        shape = t.shape
        if not shape or shape[0] != pages:
            raise ValueError(f"a cache must be [pages, ...] with {pages} pages, got {tuple(shape)}")
        run = stride = t.nbytes // pages if pages else 0
        if run < 1:
            raise ValueError("a cache's pages are empty")
        if not t.is_contiguous():
            st, n = t.stride(), 1
            for s, m in sorted(zip(st[1:], shape[1:])):
                if m != 1:
                    if s != n:
                        raise ValueError("a page of a cache must be one run of memory (pass the buffer that holds its parts)")
                    n *= m
            if pages > 1:
                stride = st[0] * t.element_size()
        words.extend((t.data_ptr(), stride, run))
    return words


def _table_out(page_table, out):
    shape = page_table.shape
    B, cols = shape
    if out is None:
        out = page_table
    elif out.shape != shape:
        raise ValueError("page_table and table_out must have one shape")
    if page_table.dtype is not _s._i32 or out.dtype is not _s._i32:
        raise ValueError("page_table and table_out must be int32")
    ts, os_ = _rows("page_table", page_table), _rows("table_out", out)
    if B > _TOP or cols > _TOP:
        raise ValueError("sizes past 32 bits")
    return B, cols, out, ts[0] if B > 1 else cols, os_[0] if B > 1 else cols


def _state(n, named):
    """Checks int32 vectors of n elements, None among them for those not given."""
    i32, shape = _s._i32, (n,)
    for name, t in named:
        if t is not None and (t.dtype is not i32 or t.shape != shape or not t.is_contiguous()):
            _vector(name, t, n, i32)


def page_fork_args(page_table, held, kv_len, refs, parent, *, page_size, grow=None, caches=(), table_out=None, held_out=None,
                   len_out=None, refs_out=None):
    """Fill SpecPageForkArgs from tensors (no workspace yet); the arrays live as long as what is returned."""
    _t()
    B, cols, table_out, ts, os_ = _table_out(page_table, table_out)
    pages = refs.shape[0]
    if held_out is None:
        held_out = held
    if len_out is None:
        len_out = kv_len
    if refs_out is None:
        refs_out = refs
    _state(B, (("held", held), ("kv_len", kv_len), ("parent", parent), ("grow", grow), ("held_out", held_out), ("len_out", len_out)))
    _state(pages, (("refs", refs), ("refs_out", refs_out)))
    if pages > _TOP or len(caches) > _TOP:
        raise ValueError("sizes past 32 bits")
    arrays = _page_arrays(caches, pages)
    a = SpecPageForkArgs(
        B, cols, _whole(page_size), pages, len(caches), 0, page_table.data_ptr(), ts, held.data_ptr(), kv_len.data_ptr(),
        refs.data_ptr(), parent.data_ptr(), None if grow is None else grow.data_ptr(), table_out.data_ptr(), os_,
        held_out.data_ptr(), len_out.data_ptr(), refs_out.data_ptr(), arrays.buffer_info()[0] or None, None, 0)
    a.keep = arrays
    return a


def spec_page_fork_workspace(page_table, refs) -> int:
    """Bytes of workspace spec_page_fork needs for tensors of these shapes."""
    B, cols = page_table.shape
    return _need("spec_page_fork", SpecPageForkArgs(B=_size(B), table_cols=_size(cols), page_size=1, num_pages=_size(refs.shape[0])))


def spec_page_fork(page_table, held, kv_len, refs, parent, *, page_size, grow=None, caches=(), table_out=None, held_out=None,
                   len_out=None, refs_out=None, workspace=None, stream=None):
    """One step of sequences that share pages: row b goes on from row parent[b] with room for grow[b] tokens.

    page_table [B, cols], held [B] (pages of each row), kv_len [B], refs [pages] (holders of each page, free
    where it is not above 0), parent [B] (-1: the row becomes empty) and grow [B] (None: 0), all int32.
    caches: tensors [pages, ...] (K and V of every layer, block exponents) in which pages that are held by
    others too are copied before the new tokens are written into them.  The state is changed in place, or
    written to table_out, held_out, len_out and refs_out; the new lengths include grow, as spec_paged_attn's
    do.  With bad data or too few free pages nothing is changed and the status word says why.  Returns
    (table, held, lengths, refs)."""
    index = _check((page_table, held, kv_len, refs, parent, grow, table_out, held_out, len_out, refs_out, *caches))
    a = page_fork_args(page_table, held, kv_len, refs, parent, page_size=page_size, grow=grow, caches=caches,
                       table_out=table_out, held_out=held_out, len_out=len_out, refs_out=refs_out)
    _run("spec_page_fork", a, (a.B, a.table_cols, a.page_size, a.num_pages, "fork"), index, workspace, stream)
    return (page_table if table_out is None else table_out, held if held_out is None else held_out,
            kv_len if len_out is None else len_out, refs if refs_out is None else refs_out)


def page_compact_args(page_table, held, refs, *, caches=(), table_out=None, refs_out=None, moved=None, num_live=None):
    """Fill SpecPageCompactArgs from tensors (no workspace yet); the arrays live as long as what is returned."""
    _t()
    B, cols, table_out, ts, os_ = _table_out(page_table, table_out)
    pages = refs.shape[0]
    if refs_out is None:
        refs_out = refs
    _state(B, (("held", held),))
    _state(pages, (("refs", refs), ("refs_out", refs_out), ("moved", moved)))
    _state(1, (("num_live", num_live),))
    if pages > _TOP or len(caches) > _TOP:
        raise ValueError("sizes past 32 bits")
    arrays = _page_arrays(caches, pages)
    a = SpecPageCompactArgs(
        B, cols, pages, len(caches), page_table.data_ptr(), ts, held.data_ptr(), refs.data_ptr(), table_out.data_ptr(), os_,
        refs_out.data_ptr(), None if moved is None else moved.data_ptr(), None if num_live is None else num_live.data_ptr(),
        arrays.buffer_info()[0] or None, None, 0)
    a.keep = arrays
    return a


def spec_page_compact_workspace(page_table, refs) -> int:
    """Bytes of workspace spec_page_compact needs for tensors of these shapes."""
    B, cols = page_table.shape
    return _need("spec_page_compact", SpecPageCompactArgs(B=_size(B), table_cols=_size(cols), num_pages=_size(refs.shape[0])))


def spec_page_compact(page_table, held, refs, *, caches=(), table_out=None, refs_out=None, moved=None, num_live=None,
                      workspace=None, stream=None):
    """Moves the pages in use to the lowest ids, in all caches, and the tables and holders with them.

    page_table [B, cols], held [B], refs [pages] int32 as in spec_page_fork; caches: tensors [pages, ...].
    Changed in place, or written to table_out and refs_out.  moved [pages] gets each page's new id (-1: free),
    num_live [1] the number of pages in use; both optional.  Returns (table, refs)."""
    index = _check((page_table, held, refs, table_out, refs_out, moved, num_live, *caches))
    a = page_compact_args(page_table, held, refs, caches=caches, table_out=table_out, refs_out=refs_out, moved=moved,
                          num_live=num_live)
    _run("spec_page_compact", a, (a.B, a.table_cols, a.num_pages, "compact"), index, workspace, stream)
    return page_table if table_out is None else table_out, refs if refs_out is None else refs_out
