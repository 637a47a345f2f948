"""In-place partial rotary position embedding (RoPE) on MI355X (gfx950).

A thin ctypes binding over ``librope_partial.so``, whose C ABI is declared in
``include/rope_partial.h``. Every step of the operation runs in the library's
HIP kernels; this module only marshals torch tensors (device pointers, shapes,
strides, the current HIP stream) into the C calls and turns status codes into
exceptions. There is no CPU fallback: without the built library every call
raises.

The operation follows "CANN ops-transformer 算子详解：inplace_partial_rotary_mul
原地部分旋转位置编码" (sections 功能与计算公式, 函数原型与参数说明, 约束说明,
自动微分说明) and, for the rotate_half pairing, "ANE实战RoPE位置编码在MIL中的纯
ANE实现" (section 先搞懂RoPE).
"""
from __future__ import annotations

import ctypes
import functools
import operator
import os

__all__ = [
    "rope_partial_fwd_inplace", "rope_partial_bwd_inplace", "rope_status_string", "inplace_partial_rotary_mul",
    "rope_partial_fwd_inplace_multi", "rope_partial_bwd_inplace_multi", "MULTI_MAX", "rope_partial_check",
    "rope_partial_launch_info", "rope_partial_fwd_out", "rope_partial_bwd_out", "partial_rotary_mul",
    "rope_partial_fwd_inplace_pos", "rope_partial_bwd_inplace_pos", "rope_inv_freq",
    "rope_partial_fwd_out_pos", "rope_partial_bwd_out_pos", "partial_rotary_mul_pos",
    "inplace_partial_rotary_mul_pos", "rope_partial_fwd_inplace_pos_multi", "rope_partial_bwd_inplace_pos_multi",
    "rope_partial_fwd_inplace_axes", "rope_partial_bwd_inplace_axes", "rope_partial_fwd_out_axes",
    "rope_partial_bwd_out_axes", "rope_partial_fwd_inplace_axes_multi", "rope_partial_bwd_inplace_axes_multi",
    "inplace_partial_rotary_mul_axes", "partial_rotary_mul_axes", "rope_pair_axes", "rope_axes_inv_freq", "AXES_MAX",
    "RopeCache", "rope_cache", "rope_cache_write", "rope_cache_read", "rope_cache_reserve", "RESERVE_MAX",
    "rope_cache_attention", "rope_cache_attention_workspace", "rope_qk_norm_fwd", "rope_qk_norm_bwd",
    "rope_qk_norm_workspace", "qk_norm_rotary", "CACHE_FORMATS", "rope_proj_fwd",
    "rope_proj_lora_fwd", "rope_proj_lora_workspace", "LORA_RANK_MAX", "RopeError", "library", "LIB_PATH", "ROPE_OK", "ROPE_ERR_NULLPTR", "ROPE_ERR_INVALID",
    "ROPE_ERR_UNSUPPORTED", "ROPE_ERR_RUNTIME", "MODES", "DTYPE_CODES",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_lib", "librope_partial.so")

ROPE_OK, ROPE_ERR_NULLPTR, ROPE_ERR_INVALID, ROPE_ERR_UNSUPPORTED, ROPE_ERR_RUNTIME = range(5)
MODES = {"rotate_half": 0, "interleave": 1}
DTYPE_CODES = {"f32": 0, "f16": 1, "bf16": 2}
MULTI_MAX = 4
AXES_MAX = 4
LORA_RANK_MAX = 128
RESERVE_MAX = 16384
CACHE_FORMATS = {"f32": 0, "f16": 1, "bf16": 2, "e4m3": 3, "int8": 4, "int4": 5}

_I64x4 = ctypes.c_int64 * 4
_I64x3 = ctypes.c_int64 * 3
_I64x2 = ctypes.c_int64 * 2
_ENTRY_ARGTYPES = [
    ctypes.c_void_p, ctypes.POINTER(ctypes.c_int64), ctypes.c_int,
    ctypes.c_void_p, ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(ctypes.c_int64),
    ctypes.c_void_p, ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(ctypes.c_int64),
    ctypes.c_int, ctypes.c_int64, ctypes.POINTER(ctypes.c_int64),
    ctypes.c_void_p,
]


class RopeError(RuntimeError):
    """A non-OK status from the library; ``status`` holds the code."""

    def __init__(self, status: int, detail: str):
        self.status = status
        super().__init__(f"{rope_status_string(status)}: {detail}" if detail else rope_status_string(status))


class RopeRows(ctypes.Structure):
    """The C ABI's rope_rows_t."""
    _fields_ = [("data", ctypes.c_void_p), ("N", ctypes.c_int64), ("D", ctypes.c_int64),
                ("strides", ctypes.c_int64 * 3)]


class RopeCacheStruct(ctypes.Structure):
    """The C ABI's rope_cache_t."""
    _fields_ = [("data", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("format", ctypes.c_int32),
                ("pages", ctypes.c_int64), ("page_size", ctypes.c_int64), ("heads", ctypes.c_int64),
                ("dim", ctypes.c_int64), ("group", ctypes.c_int64), ("strides", ctypes.c_int64 * 3),
                ("scale_strides", ctypes.c_int64 * 3)]


class _StructPointer:
    """Argument type of a pointer to one of the structures above: the structure
    itself, an array of 64-bit numbers of the same layout (which is quicker to
    make), or None."""

    @classmethod
    def from_param(cls, v):
        return ctypes.byref(v) if isinstance(v, ctypes.Structure) else v


_RowsWords = ctypes.c_int64 * 6
_CacheWords = ctypes.c_int64 * 14      # the 32-bit format with its padding as one number


class RopeLora(ctypes.Structure):
    """The C ABI's rope_lora_t."""
    _fields_ = [("a", ctypes.c_void_p), ("b", ctypes.c_void_p), ("adapters", ctypes.c_void_p),
                ("scales", ctypes.c_void_p), ("count", ctypes.c_int64), ("rank", ctypes.c_int64)]


_lib = None


def library() -> ctypes.CDLL:
    """The loaded HIP library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with `python -m transformer_positional_encoding_amd.build` "
                "(or __graft_entry__.build()); there is no fallback path")
        L = ctypes.CDLL(LIB_PATH)
        for name in ("rope_partial_fwd_inplace", "rope_partial_bwd_inplace"):
            f = getattr(L, name)
            f.restype = ctypes.c_int
            f.argtypes = _ENTRY_ARGTYPES
        for name in ("rope_partial_fwd_out", "rope_partial_bwd_out"):
            f = getattr(L, name)
            f.restype = ctypes.c_int
            f.argtypes = [ctypes.c_void_p] + _ENTRY_ARGTYPES
        pos_args = [ctypes.c_void_p, ctypes.POINTER(ctypes.c_int64), ctypes.c_int, ctypes.c_void_p,
                    ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(ctypes.c_int64), ctypes.c_void_p,
                    ctypes.c_int, ctypes.c_int64, ctypes.POINTER(ctypes.c_int64)]
        for name in ("rope_partial_fwd_inplace_pos", "rope_partial_bwd_inplace_pos"):
            f = getattr(L, name)
            f.restype = ctypes.c_int
            f.argtypes = pos_args + [ctypes.c_void_p]
        for name in ("rope_partial_fwd_out_pos", "rope_partial_bwd_out_pos"):
            f = getattr(L, name)
            f.restype = ctypes.c_int
            f.argtypes = [ctypes.c_void_p] + pos_args + [ctypes.c_void_p]
        for name in ("rope_partial_fwd_inplace_pos_multi", "rope_partial_bwd_inplace_pos_multi"):
            f = getattr(L, name)
            f.restype = ctypes.c_int
            f.argtypes = [ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p] + pos_args[2:] + [ctypes.c_void_p]
        axes_args = pos_args[:7] + [ctypes.c_void_p] + pos_args[7:]   # the pairs' axes after the frequencies
        for name in ("rope_partial_fwd_inplace_axes", "rope_partial_bwd_inplace_axes"):
            f = getattr(L, name)
            f.restype = ctypes.c_int
            f.argtypes = axes_args + [ctypes.c_void_p]
        for name in ("rope_partial_fwd_out_axes", "rope_partial_bwd_out_axes"):
            f = getattr(L, name)
            f.restype = ctypes.c_int
            f.argtypes = [ctypes.c_void_p] + axes_args + [ctypes.c_void_p]
        for name in ("rope_partial_fwd_inplace_axes_multi", "rope_partial_bwd_inplace_axes_multi"):
            f = getattr(L, name)
            f.restype = ctypes.c_int
            f.argtypes = [ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p] + axes_args[2:] + [ctypes.c_void_p]
        L.rope_partial_launch_info_axes.restype = ctypes.c_int
        L.rope_partial_launch_info_axes.argtypes = axes_args + [ctypes.POINTER(ctypes.c_int64)]
        L.rope_partial_launch_info_pos.restype = ctypes.c_int
        L.rope_partial_launch_info_pos.argtypes = pos_args + [ctypes.POINTER(ctypes.c_int64)]
        for name in ("rope_partial_fwd_inplace_multi", "rope_partial_bwd_inplace_multi"):
            f = getattr(L, name)
            f.restype = ctypes.c_int
            f.argtypes = [ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p] + _ENTRY_ARGTYPES[2:]
        i64p, vp = ctypes.POINTER(ctypes.c_int64), ctypes.c_void_p
        turn = [vp, i64p, i64p, vp, vp, ctypes.c_int, ctypes.c_int64, i64p]   # positions to partial_slice
        rows = cache = _StructPointer
        L.rope_cache_write.restype = ctypes.c_int
        L.rope_cache_write.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int, rows, rows, rows, cache, cache, vp,
                                       i64p] + turn + [ctypes.c_int32, vp]
        L.rope_cache_read.restype = ctypes.c_int
        L.rope_cache_read.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int, rows, cache, vp, ctypes.c_int64,
                                      ctypes.c_int64, vp, vp] + turn + [vp]
        L.rope_cache_reserve.restype = ctypes.c_int
        L.rope_cache_reserve.argtypes = [ctypes.c_int64, ctypes.c_int64, vp, ctypes.c_int64, ctypes.c_int64, vp, vp, vp,
                                         ctypes.c_int64, vp, ctypes.c_int64, vp, vp, vp, vp]
        L.rope_cache_attention.restype = ctypes.c_int
        L.rope_cache_attention.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int, rows, rows, cache, cache, vp,
                                           ctypes.c_int64, ctypes.c_int64, vp, vp, ctypes.c_double, ctypes.c_int32, vp,
                                           ctypes.c_int64, vp]
        L.rope_cache_attention_workspace.restype = ctypes.c_int64
        L.rope_cache_attention_workspace.argtypes = [ctypes.c_int64] * 5
        weights = [vp, vp, ctypes.c_int, ctypes.c_double]
        L.rope_qk_norm_fwd.restype = ctypes.c_int
        L.rope_qk_norm_fwd.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int] + [rows] * 4 + weights + turn + [vp]
        L.rope_qk_norm_bwd.restype = ctypes.c_int
        L.rope_qk_norm_bwd.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int, rows, rows, vp, vp] + [rows] * 4 + \
            weights + turn + [vp, ctypes.c_int64, vp]
        L.rope_qk_norm_workspace.restype = ctypes.c_int64
        L.rope_qk_norm_workspace.argtypes = [ctypes.c_int64]
        L.rope_partial_check.restype = ctypes.c_int
        L.rope_partial_check.argtypes = _ENTRY_ARGTYPES[:-1]
        L.rope_partial_launch_info.restype = ctypes.c_int
        L.rope_partial_launch_info.argtypes = _ENTRY_ARGTYPES[:-1] + [ctypes.POINTER(ctypes.c_int64)]
        L.rope_proj_fwd.restype = ctypes.c_int
        L.rope_proj_fwd.argtypes = [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int,
                                    ctypes.POINTER(ctypes.c_int64), ctypes.c_int64] + _ENTRY_ARGTYPES[3:]
        L.rope_proj_lora_fwd.restype = ctypes.c_int
        L.rope_proj_lora_fwd.argtypes = L.rope_proj_fwd.argtypes[:7] + [ctypes.POINTER(RopeLora)] + \
            _ENTRY_ARGTYPES[3:-1] + [vp, ctypes.c_int64, vp]
        L.rope_proj_lora_launch_info.restype = ctypes.c_int
        L.rope_proj_lora_launch_info.argtypes = [ctypes.c_int, ctypes.c_int, i64p, ctypes.c_int64, ctypes.c_int64,
                                                 ctypes.c_int64] + _ENTRY_ARGTYPES[3:-1] + [i64p]
        L.rope_proj_lora_workspace.restype = ctypes.c_int64
        L.rope_proj_lora_workspace.argtypes = [i64p, ctypes.c_int64, ctypes.c_int64]
        L.rope_proj_launch_info.restype = ctypes.c_int
        L.rope_proj_launch_info.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.POINTER(ctypes.c_int64),
                                            ctypes.c_int64] + _ENTRY_ARGTYPES[3:-1] + [ctypes.POINTER(ctypes.c_int64)]
        L.rope_status_string.restype = ctypes.c_char_p
        L.rope_status_string.argtypes = [ctypes.c_int]
        L.rope_last_error.restype = ctypes.c_char_p
        L.rope_last_error.argtypes = []
        _lib = L
    return _lib


def rope_status_string(status: int) -> str:
    return library().rope_status_string(int(status)).decode()


def _arr4(v):
    if v is None:
        return None
    if len(v) != 4:
        raise ValueError(f"expected 4 values, got {len(v)}")
    try:
        return _I64x4(*v)                       # tuples of ints (torch sizes and strides)
    except TypeError:
        return _I64x4(*[int(t) for t in v])     # other integer types


@functools.lru_cache(maxsize=None)
def _words_entry(name):
    """A cache entry point whose structures are given as arrays of words, which
    ctypes passes on without a conversion in Python."""
    L = library()
    f = getattr(L, name)
    types = [ctypes.c_void_p if t is _StructPointer else t for t in f.argtypes]
    return ctypes.CFUNCTYPE(f.restype, *types)((name, L))


@functools.lru_cache(maxsize=64)
def _i32_array(values: tuple):
    """A tuple of ints as a C int32 array (the same array for the same
    values: a program's pairs keep their axes from call to call)."""
    return (ctypes.c_int32 * max(1, len(values)))(*values)


def raw_call(direction: str, x_ptr, x_shape, dtype: int, r1_ptr, r1_shape, r1_strides,
             r2_ptr, r2_shape, r2_strides, table_dtype: int, mode: int, partial_slice,
             stream=None) -> int:
    """Call an entry point with plain integers and sequences (None = NULL);
    returns the status code without raising."""
    fn = library().rope_partial_fwd_inplace if direction == "fwd" else library().rope_partial_bwd_inplace
    sl = None if partial_slice is None else _I64x2(int(partial_slice[0]), int(partial_slice[1]))
    a1, s1 = _arr4(r1_shape), _arr4(r1_strides)
    # r2 usually has r1's geometry: the same arrays then serve both
    a2 = a1 if r2_shape == r1_shape else _arr4(r2_shape)
    s2 = s1 if r2_strides == r1_strides else _arr4(r2_strides)
    return fn(x_ptr, _arr4(x_shape), int(dtype), r1_ptr, a1, s1, r2_ptr, a2, s2, int(table_dtype), int(mode), sl,
              stream)


def raw_out_call(direction: str, y_ptr, x_ptr, x_shape, dtype: int, r1_ptr, r1_shape, r1_strides,
                 r2_ptr, r2_shape, r2_strides, table_dtype: int, mode: int, partial_slice,
                 stream=None) -> int:
    """Call rope_partial_{fwd,bwd}_out with plain integers and sequences
    (None = NULL); returns the status code without raising."""
    fn = library().rope_partial_fwd_out if direction == "fwd" else library().rope_partial_bwd_out
    sl = None if partial_slice is None else _I64x2(int(partial_slice[0]), int(partial_slice[1]))
    a1, s1 = _arr4(r1_shape), _arr4(r1_strides)
    a2 = a1 if r2_shape == r1_shape else _arr4(r2_shape)
    s2 = s1 if r2_strides == r1_strides else _arr4(r2_strides)
    return fn(y_ptr, x_ptr, _arr4(x_shape), int(dtype), r1_ptr, a1, s1, r2_ptr, a2, s2, int(table_dtype), int(mode),
              sl, stream)


def raw_pos_call(direction: str, x_ptr, x_shape, dtype: int, pos_ptr, pos_shape, pos_strides, inv_freq_ptr,
                 table_dtype: int, mode: int, partial_slice, stream=None) -> int:
    """Call rope_partial_{fwd,bwd}_inplace_pos with plain integers and
    sequences (None = NULL); returns the status code without raising."""
    L = library()
    fn = L.rope_partial_fwd_inplace_pos if direction == "fwd" else L.rope_partial_bwd_inplace_pos
    sl = None if partial_slice is None else _I64x2(int(partial_slice[0]), int(partial_slice[1]))
    ps = None if pos_shape is None else _I64x2(int(pos_shape[0]), int(pos_shape[1]))
    pt = None if pos_strides is None else _I64x2(int(pos_strides[0]), int(pos_strides[1]))
    return fn(x_ptr, _arr4(x_shape), int(dtype), pos_ptr, ps, pt, inv_freq_ptr, int(table_dtype), int(mode), sl,
              stream)


def raw_out_pos_call(direction: str, y_ptr, x_ptr, x_shape, dtype: int, pos_ptr, pos_shape, pos_strides,
                     inv_freq_ptr, table_dtype: int, mode: int, partial_slice, stream=None) -> int:
    """Call rope_partial_{fwd,bwd}_out_pos with plain integers and sequences
    (None = NULL); returns the status code without raising."""
    L = library()
    fn = L.rope_partial_fwd_out_pos if direction == "fwd" else L.rope_partial_bwd_out_pos
    sl = None if partial_slice is None else _I64x2(int(partial_slice[0]), int(partial_slice[1]))
    ps = None if pos_shape is None else _I64x2(int(pos_shape[0]), int(pos_shape[1]))
    pt = None if pos_strides is None else _I64x2(int(pos_strides[0]), int(pos_strides[1]))
    return fn(y_ptr, x_ptr, _arr4(x_shape), int(dtype), pos_ptr, ps, pt, inv_freq_ptr, int(table_dtype),
              int(mode), sl, stream)


def _axes_source(pos_shape, pos_strides, pair_axes):
    """The C arrays of a positions shape and strides of three values and of
    the pairs' axes (None = NULL)."""
    ps = None if pos_shape is None else _I64x3(*pos_shape)
    pt = None if pos_strides is None else _I64x3(*pos_strides)
    return ps, pt, None if pair_axes is None else _i32_array(tuple(pair_axes))


def raw_axes_call(direction: str, x_ptr, x_shape, dtype: int, pos_ptr, pos_shape, pos_strides, inv_freq_ptr,
                  pair_axes, table_dtype: int, mode: int, partial_slice, stream=None, y_ptr=None,
                  out: bool = False) -> int:
    """rope_partial_{fwd,bwd}_inplace_axes, or with out=True the _out_axes
    form into y_ptr, with plain integers and sequences (None = NULL); returns
    the status code without raising."""
    L = library()
    ps, pt, pa = _axes_source(pos_shape, pos_strides, pair_axes)
    sl = None if partial_slice is None else _I64x2(int(partial_slice[0]), int(partial_slice[1]))
    rest = (x_ptr, _arr4(x_shape), int(dtype), pos_ptr, ps, pt, inv_freq_ptr, pa, int(table_dtype), int(mode), sl,
            stream)
    if out:
        return (L.rope_partial_fwd_out_axes if direction == "fwd" else L.rope_partial_bwd_out_axes)(y_ptr, *rest)
    return (L.rope_partial_fwd_inplace_axes if direction == "fwd" else L.rope_partial_bwd_inplace_axes)(*rest)


def raw_axes_multi_call(direction: str, x_ptrs, x_shapes, dtype: int, pos_ptr, pos_shape, pos_strides, inv_freq_ptr,
                        pair_axes, table_dtype: int, mode: int, partial_slice, stream=None, count=None) -> int:
    """Call an _axes_multi entry point with plain integers and sequences
    (None = NULL); returns the status code without raising."""
    L = library()
    fn = L.rope_partial_fwd_inplace_axes_multi if direction == "fwd" else L.rope_partial_bwd_inplace_axes_multi
    n = len(x_ptrs) if x_ptrs is not None else 0
    count = n if count is None else count
    ptrs = None if x_ptrs is None else (ctypes.c_void_p * max(n, 1))(*x_ptrs)
    flat = [] if x_shapes is None else [int(v) for sh in x_shapes for v in sh]
    shapes = None if x_shapes is None else (ctypes.c_int64 * max(len(flat), 4))(*flat)
    ps, pt, pa = _axes_source(pos_shape, pos_strides, pair_axes)
    sl = None if partial_slice is None else _I64x2(int(partial_slice[0]), int(partial_slice[1]))
    return fn(int(count), ptrs, shapes, int(dtype), pos_ptr, ps, pt, inv_freq_ptr, pa, int(table_dtype), int(mode),
              sl, stream)


def raw_check(x_ptr, x_shape, dtype: int, r1_ptr, r1_shape, r1_strides, r2_ptr, r2_shape, r2_strides,
              table_dtype: int, mode: int, partial_slice) -> int:
    """rope_partial_check with plain integers and sequences (None = NULL):
    the status the entry points would return, with nothing launched."""
    sl = None if partial_slice is None else _I64x2(int(partial_slice[0]), int(partial_slice[1]))
    return library().rope_partial_check(x_ptr, _arr4(x_shape), int(dtype), r1_ptr, _arr4(r1_shape),
                                        _arr4(r1_strides), r2_ptr, _arr4(r2_shape), _arr4(r2_strides),
                                        int(table_dtype), int(mode), sl)


LAUNCH_INFO_LEN = 8
KERNELS = {0: "none", 1: "vector", 2: "scalar", 3: "rows"}


def raw_launch_info(x_ptr, x_shape, dtype: int, r1_ptr, r1_shape, r1_strides, r2_ptr, r2_shape, r2_strides,
                    table_dtype: int, mode: int, partial_slice, info_out: bool = True):
    """rope_partial_launch_info with plain integers and sequences (None =
    NULL): (status, plan dict or None). The plan names the kernel and the
    launch shape; nothing is launched. info_out=False passes a NULL info."""
    sl = None if partial_slice is None else _I64x2(int(partial_slice[0]), int(partial_slice[1]))
    info = (ctypes.c_int64 * LAUNCH_INFO_LEN)() if info_out else None
    st = library().rope_partial_launch_info(x_ptr, _arr4(x_shape), int(dtype), r1_ptr, _arr4(r1_shape),
                                            _arr4(r1_strides), r2_ptr, _arr4(r2_shape), _arr4(r2_strides),
                                            int(table_dtype), int(mode), sl, info)
    if st != ROPE_OK or info is None:
        return st, None
    v = list(info)
    if v[0] == 3:
        return st, {"kernel": "rows", "blocks": v[1], "threads": v[2], "rows_per_block": v[4],
                    "threads_per_row": v[7]}
    return st, {"kernel": KERNELS.get(v[0], v[0]), "blocks": v[1], "threads": v[2], "heads_per_thread": v[3],
                "head_lanes": v[4], "tiles_per_block": v[5], "xcd_run": v[6], "row_vectors": v[7]}


def raw_launch_info_pos(x_ptr, x_shape, dtype: int, pos_ptr, pos_shape, pos_strides, inv_freq_ptr,
                        table_dtype: int, mode: int, partial_slice, info_out: bool = True):
    """rope_partial_launch_info_pos with plain integers and sequences (None =
    NULL): (status, plan dict or None); nothing is launched."""
    sl = None if partial_slice is None else _I64x2(int(partial_slice[0]), int(partial_slice[1]))
    ps = None if pos_shape is None else _I64x2(int(pos_shape[0]), int(pos_shape[1]))
    pt = None if pos_strides is None else _I64x2(int(pos_strides[0]), int(pos_strides[1]))
    info = (ctypes.c_int64 * LAUNCH_INFO_LEN)() if info_out else None
    st = library().rope_partial_launch_info_pos(x_ptr, _arr4(x_shape), int(dtype), pos_ptr, ps, pt, inv_freq_ptr,
                                                int(table_dtype), int(mode), sl, info)
    if st != ROPE_OK or info is None:
        return st, None
    v = list(info)
    if v[0] == 3:
        return st, {"kernel": "rows", "blocks": v[1], "threads": v[2], "rows_per_block": v[4],
                    "threads_per_row": v[7]}
    return st, {"kernel": KERNELS.get(v[0], v[0]), "blocks": v[1], "threads": v[2], "heads_per_thread": v[3],
                "head_lanes": v[4], "positions_per_block": v[5], "head_chunks": v[6], "row_vectors": v[7]}


def raw_launch_info_axes(x_ptr, x_shape, dtype: int, pos_ptr, pos_shape, pos_strides, inv_freq_ptr, pair_axes,
                         table_dtype: int, mode: int, partial_slice):
    """rope_partial_launch_info_axes with plain integers and sequences (None =
    NULL): (status, the kernel's name or None); nothing is launched."""
    ps, pt, pa = _axes_source(pos_shape, pos_strides, pair_axes)
    sl = None if partial_slice is None else _I64x2(int(partial_slice[0]), int(partial_slice[1]))
    info = (ctypes.c_int64 * LAUNCH_INFO_LEN)()
    st = library().rope_partial_launch_info_axes(x_ptr, _arr4(x_shape), int(dtype), pos_ptr, ps, pt, inv_freq_ptr, pa,
                                                 int(table_dtype), int(mode), sl, info)
    return st, KERNELS.get(info[0], info[0]) if st == ROPE_OK else None


def raw_multi_call(direction: str, x_ptrs, x_shapes, dtype: int, r1_ptr, r1_shape, r1_strides,
                   r2_ptr, r2_shape, r2_strides, table_dtype: int, mode: int, partial_slice,
                   stream=None, count=None) -> int:
    """Call a _multi entry point with plain integers and sequences (None =
    NULL); returns the status code without raising."""
    L = library()
    fn = L.rope_partial_fwd_inplace_multi if direction == "fwd" else L.rope_partial_bwd_inplace_multi
    n = len(x_ptrs) if x_ptrs is not None else 0
    count = n if count is None else count
    ptrs = None if x_ptrs is None else (ctypes.c_void_p * max(n, 1))(*x_ptrs)
    flat = [] if x_shapes is None else [int(v) for sh in x_shapes for v in sh]
    shapes = None if x_shapes is None else (ctypes.c_int64 * max(len(flat), 4))(*flat)
    sl = None if partial_slice is None else _I64x2(int(partial_slice[0]), int(partial_slice[1]))
    return fn(int(count), ptrs, shapes, int(dtype), r1_ptr, _arr4(r1_shape), _arr4(r1_strides),
              r2_ptr, _arr4(r2_shape), _arr4(r2_strides), int(table_dtype), int(mode), sl, stream)


def raw_pos_multi_call(direction: str, x_ptrs, x_shapes, dtype: int, pos_ptr, pos_shape, pos_strides,
                       inv_freq_ptr, table_dtype: int, mode: int, partial_slice, stream=None, count=None) -> int:
    """Call a _pos_multi entry point with plain integers and sequences
    (None = NULL); returns the status code without raising."""
    L = library()
    fn = L.rope_partial_fwd_inplace_pos_multi if direction == "fwd" else L.rope_partial_bwd_inplace_pos_multi
    n = len(x_ptrs) if x_ptrs is not None else 0
    count = n if count is None else count
    ptrs = None if x_ptrs is None else (ctypes.c_void_p * max(n, 1))(*x_ptrs)
    flat = [] if x_shapes is None else [int(v) for sh in x_shapes for v in sh]
    shapes = None if x_shapes is None else (ctypes.c_int64 * max(len(flat), 4))(*flat)
    sl = None if partial_slice is None else _I64x2(int(partial_slice[0]), int(partial_slice[1]))
    ps = None if pos_shape is None else _I64x2(int(pos_shape[0]), int(pos_shape[1]))
    pt = None if pos_strides is None else _I64x2(int(pos_strides[0]), int(pos_strides[1]))
    return fn(int(count), ptrs, shapes, int(dtype), pos_ptr, ps, pt, inv_freq_ptr, int(table_dtype), int(mode), sl,
              stream)


def raw_proj_call(y_ptr, y_dtype: int, x_ptr, w_ptr, dtype: int, y_shape, K: int, r1_ptr, r1_shape, r1_strides,
                  r2_ptr, r2_shape, r2_strides, table_dtype: int, mode: int, partial_slice, stream=None) -> int:
    """rope_proj_fwd with plain integers and sequences (None = NULL); returns
    the status code without raising."""
    sl = None if partial_slice is None else _I64x2(*partial_slice)
    return library().rope_proj_fwd(y_ptr, y_dtype, x_ptr, w_ptr, dtype, _arr4(y_shape), int(K),
                                   r1_ptr, _arr4(r1_shape), _arr4(r1_strides), r2_ptr, _arr4(r2_shape),
                                   _arr4(r2_strides), table_dtype, mode, sl, stream)


PROJ_KERNELS = {0: "none", 4: "heads", 5: "square", 6: "few", 7: "general"}
PROJ_EPILOGUES = {0: "general", 1: "vector", 2: "vector_partner"}


def raw_proj_launch_info(y_dtype: int, dtype: int, y_shape, K: int, r1_ptr, r1_shape, r1_strides, r2_ptr, r2_shape,
                         r2_strides, table_dtype: int, mode: int, partial_slice, info_out: bool = True):
    """rope_proj_launch_info with plain integers and sequences (None =
    NULL): (status, plan dict or None). The plan names the projection kernel,
    its tile and (square tiles) its epilogue; nothing is launched."""
    sl = None if partial_slice is None else _I64x2(*partial_slice)
    info = (ctypes.c_int64 * LAUNCH_INFO_LEN)() if info_out else None
    st = library().rope_proj_launch_info(int(y_dtype), int(dtype), _arr4(y_shape), int(K), r1_ptr, _arr4(r1_shape),
                                         _arr4(r1_strides), r2_ptr, _arr4(r2_shape), _arr4(r2_strides),
                                         int(table_dtype), int(mode), sl, info)
    if st != ROPE_OK or info is None:
        return st, None
    v = list(info)
    return st, {"kernel": PROJ_KERNELS.get(v[0], v[0]), "blocks": v[1], "threads": v[2], "tile_tokens": v[3],
                "tile_lanes": v[4], "epilogue": PROJ_EPILOGUES.get(v[5], v[5]) if v[0] == 5 else None,
                "tables_in_lds": bool(v[6])}


def raw_proj_lora_launch_info(y_dtype: int, dtype: int, y_shape, K: int, count: int, rank: int, r1_ptr, r1_shape,
                              r1_strides, r2_ptr, r2_shape, r2_strides, table_dtype: int, mode: int, partial_slice):
    """rope_proj_lora_launch_info with plain integers and sequences (None =
    NULL): (status, plan dict or None), as raw_proj_launch_info; "sorted": the
    tokens are sorted by adapter first."""
    sl = None if partial_slice is None else _I64x2(*partial_slice)
    v = (ctypes.c_int64 * LAUNCH_INFO_LEN)()
    st = library().rope_proj_lora_launch_info(int(y_dtype), int(dtype), _arr4(y_shape), int(K), int(count), int(rank),
                                              r1_ptr, _arr4(r1_shape), _arr4(r1_strides), r2_ptr, _arr4(r2_shape),
                                              _arr4(r2_strides), int(table_dtype), int(mode), sl, v)
    if st != ROPE_OK:
        return st, None
    return st, {"kernel": PROJ_KERNELS.get(v[0], v[0]), "blocks": v[1], "threads": v[2], "tile_tokens": v[3],
                "tile_lanes": v[4], "epilogue": PROJ_EPILOGUES.get(v[5], v[5]) if v[0] == 5 else None,
                "tables_in_lds": bool(v[6]), "sorted": bool(v[7])}


def last_error() -> str:
    return library().rope_last_error().decode()


_DTYPE_OF_TORCH = {}


def _dtype_code(t) -> int:
    if not _DTYPE_OF_TORCH:
        import torch
        _DTYPE_OF_TORCH.update({torch.float32: 0, torch.float16: 1, torch.bfloat16: 2})
    code = _DTYPE_OF_TORCH.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {t.dtype}; expected float32, float16 or bfloat16")
    return code


def _call(direction: str, x, r1, r2, mode, partial_slice, stream) -> None:
    import torch
    if isinstance(mode, str):
        if mode not in MODES:
            raise ValueError(f"rotary_mode must be one of {sorted(MODES)}")
        mode = MODES[mode]
    for name, t in (("x", x), ("r1", r1), ("r2", r2)):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.dim() != 4:
            raise ValueError(f"{name} must be 4-D (B,S,N,D layout), got {t.dim()}-D")
    if x.numel() and not x.is_cuda:
        raise ValueError("x must be a GPU tensor")
    if not x.is_contiguous():
        raise ValueError("x must be contiguous (BSND); non-contiguous tensors are not supported")
    dev = x.device
    for name, t in (("r1", r1), ("r2", r2)):
        if t.numel() and x.numel() and t.device != dev:
            raise ValueError(f"{name} must be on {dev}")
    if stream is None:
        handle = torch.cuda.current_stream(dev).cuda_stream if x.is_cuda else None
    else:
        handle = getattr(stream, "cuda_stream", stream)
    # the launch goes to the current device: switch only when x lives elsewhere
    switch = x.is_cuda and dev.index != torch.cuda.current_device()
    with torch.cuda.device(dev) if switch else _nullcontext():
        st = raw_call(direction, x.data_ptr() or None, tuple(x.shape), _dtype_code(x),
                      r1.data_ptr() or None, tuple(r1.shape), tuple(r1.stride()),
                      r2.data_ptr() or None, tuple(r2.shape), tuple(r2.stride()),
                      _dtype_code(r1) if r1.dtype == r2.dtype else -1, mode, partial_slice, handle)
    if st != ROPE_OK:
        raise RopeError(st, last_error())


def _call_out(direction: str, y, x, r1, r2, mode, partial_slice, stream) -> None:
    import torch
    if isinstance(mode, str):
        if mode not in MODES:
            raise ValueError(f"rotary_mode must be one of {sorted(MODES)}")
        mode = MODES[mode]
    for name, t in (("out", y), ("x", x), ("r1", r1), ("r2", r2)):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.dim() != 4:
            raise ValueError(f"{name} must be 4-D (B,S,N,D layout), got {t.dim()}-D")
    if y.shape != x.shape or y.dtype != x.dtype:
        raise ValueError(f"out must match x in shape and dtype: {tuple(y.shape)} {y.dtype} vs "
                         f"{tuple(x.shape)} {x.dtype}")
    if not (x.is_contiguous() and y.is_contiguous()):
        raise ValueError("x and out must be contiguous (BSND)")
    if x.numel() and not (x.is_cuda and y.is_cuda and y.device == x.device):
        raise ValueError("x and out must be GPU tensors on one device")
    dev = x.device
    for name, t in (("r1", r1), ("r2", r2)):
        if t.numel() and x.numel() and t.device != dev:
            raise ValueError(f"{name} must be on {dev}")
    if stream is None:
        handle = torch.cuda.current_stream(dev).cuda_stream if x.is_cuda else None
    else:
        handle = getattr(stream, "cuda_stream", stream)
    switch = x.is_cuda and dev.index != torch.cuda.current_device()
    with torch.cuda.device(dev) if switch else _nullcontext():
        st = raw_out_call(direction, y.data_ptr() or None, x.data_ptr() or None, tuple(x.shape), _dtype_code(x),
                          r1.data_ptr() or None, tuple(r1.shape), tuple(r1.stride()),
                          r2.data_ptr() or None, tuple(r2.shape), tuple(r2.stride()),
                          _dtype_code(r1) if r1.dtype == r2.dtype else -1, mode, partial_slice, handle)
    if st != ROPE_OK:
        raise RopeError(st, last_error())


def _call_multi(direction: str, xs, r1, r2, mode, partial_slice, stream) -> None:
    import torch
    xs = list(xs)
    if len(xs) > MULTI_MAX:
        raise ValueError(f"at most {MULTI_MAX} tensors per call")
    if not xs:
        return
    if isinstance(mode, str):
        if mode not in MODES:
            raise ValueError(f"rotary_mode must be one of {sorted(MODES)}")
        mode = MODES[mode]
    for name, t in [(f"xs[{i}]", x) for i, x in enumerate(xs)] + [("r1", r1), ("r2", r2)]:
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.dim() != 4:
            raise ValueError(f"{name} must be 4-D (B,S,N,D layout), got {t.dim()}-D")
    dtypes = {x.dtype for x in xs}
    if len(dtypes) != 1:
        raise TypeError("all tensors of one call must share a dtype")
    devs = {x.device for x in xs if x.numel()}
    if len(devs) > 1:
        raise ValueError("all tensors of one call must be on one device")
    for i, x in enumerate(xs):
        if x.numel() and not x.is_cuda:
            raise ValueError(f"xs[{i}] must be a GPU tensor")
        if not x.is_contiguous():
            raise ValueError(f"xs[{i}] must be contiguous (BSND)")
    dev = next(iter(devs)) if devs else None
    if stream is None:
        handle = torch.cuda.current_stream(dev).cuda_stream if dev is not None else None
    else:
        handle = getattr(stream, "cuda_stream", stream)
    with torch.cuda.device(dev) if dev is not None else _nullcontext():
        st = raw_multi_call(direction, [x.data_ptr() or None for x in xs], [tuple(x.shape) for x in xs],
                            _dtype_code(xs[0]), r1.data_ptr() or None, tuple(r1.shape), tuple(r1.stride()),
                            r2.data_ptr() or None, tuple(r2.shape), tuple(r2.stride()),
                            _dtype_code(r1) if r1.dtype == r2.dtype else -1, mode, partial_slice, handle)
    if st != ROPE_OK:
        raise RopeError(st, last_error())


class _nullcontext:
    def __enter__(self):
        return None

    def __exit__(self, *exc):
        return False


_NOTHING = _nullcontext()


def _on_device(t, stream):
    """(stream handle, context) of a launch on t's device: torch's current
    stream there unless one is given, and that device made current when it is
    not. A CPU tensor (an empty call) has neither."""
    import torch
    if not t.is_cuda:
        return None, _NOTHING
    index = t.device.index
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(index)
    else:
        handle = getattr(stream, "cuda_stream", stream)
    return handle, _NOTHING if index == torch._C._cuda_getDevice() else torch.cuda.device(index)


def rope_partial_check(x, r1, r2, rotary_mode="interleave", partial_slice=None) -> None:
    """Run the entry points' argument checks on tensors (on any device:
    nothing is launched or read); raises RopeError on the first failure."""
    if isinstance(rotary_mode, str):
        if rotary_mode not in MODES:
            raise ValueError(f"rotary_mode must be one of {sorted(MODES)}")
        rotary_mode = MODES[rotary_mode]
    st = raw_check(x.data_ptr() or None, tuple(x.shape), _dtype_code(x), r1.data_ptr() or None, tuple(r1.shape),
                   tuple(r1.stride()), r2.data_ptr() or None, tuple(r2.shape), tuple(r2.stride()),
                   _dtype_code(r1) if r1.dtype == r2.dtype else -1, rotary_mode, partial_slice)
    if st != ROPE_OK:
        raise RopeError(st, last_error())


def rope_partial_launch_info(x, r1, r2, rotary_mode="interleave", partial_slice=None) -> dict:
    """The kernel and launch shape a call with these tensors would use
    (nothing is launched or read); raises RopeError like the entry points."""
    if isinstance(rotary_mode, str):
        if rotary_mode not in MODES:
            raise ValueError(f"rotary_mode must be one of {sorted(MODES)}")
        rotary_mode = MODES[rotary_mode]
    st, plan = raw_launch_info(x.data_ptr() or None, tuple(x.shape), _dtype_code(x), r1.data_ptr() or None,
                               tuple(r1.shape), tuple(r1.stride()), r2.data_ptr() or None, tuple(r2.shape),
                               tuple(r2.stride()), _dtype_code(r1) if r1.dtype == r2.dtype else -1,
                               rotary_mode, partial_slice)
    if st != ROPE_OK:
        raise RopeError(st, last_error())
    return plan


def rope_partial_fwd_inplace(x, r1, r2, rotary_mode="interleave", partial_slice=None, stream=None) -> None:
    """Rotate ``x[..., start:end)`` in place (forward).

    x: contiguous (B,S,N,D) GPU tensor, float32/float16/bfloat16.
    r1, r2: cos and sin tables, 4-D, last dim ``end-start``, other dims 1 or
    equal to x's (any strides, e.g. from ``expand``); one dtype for both,
    which may differ from x's (e.g. bf16 x with fp32 tables).
    rotary_mode: "interleave" (pairs 2i, 2i+1), "rotate_half" (i, i+L/2), or
    an int rotary coefficient c (even, dividing L): the slice in c parts,
    lane k of part 2g paired with lane k of part 2g+1 (2: rotate_half; L:
    interleave).
    partial_slice: (start, end) or None for the empty slice [0, 0).
    stream: a torch stream or raw hipStream_t; default torch's current stream.

    The rope_partial_* calls are not recorded by autograd
    (:func:`inplace_partial_rotary_mul` is).
    """
    _call("fwd", x, r1, r2, rotary_mode, partial_slice, stream)


def rope_partial_bwd_inplace(dx, r1, r2, rotary_mode="interleave", partial_slice=None, stream=None) -> None:
    """Backward of :func:`rope_partial_fwd_inplace`: ``dx`` (the incoming
    gradient) is replaced in place by the gradient with respect to x."""
    _call("bwd", dx, r1, r2, rotary_mode, partial_slice, stream)


def rope_partial_fwd_out(out, x, r1, r2, rotary_mode="interleave", partial_slice=None, stream=None) -> None:
    """Out-of-place forward: ``out`` receives ``x`` with ``x[..., start:end)``
    rotated and every other lane copied; ``x`` is left unchanged. ``out``
    must be a contiguous tensor of x's shape and dtype that does not overlap
    x (``out is x`` is the in-place call). Arguments as in
    :func:`rope_partial_fwd_inplace`."""
    _call_out("fwd", out, x, r1, r2, rotary_mode, partial_slice, stream)


def rope_partial_bwd_out(dx, dy, r1, r2, rotary_mode="interleave", partial_slice=None, stream=None) -> None:
    """Out-of-place backward: ``dx`` receives the gradient with respect to x
    for the incoming gradient ``dy``, which is left unchanged."""
    _call_out("bwd", dx, dy, r1, r2, rotary_mode, partial_slice, stream)


def rope_inv_freq(L: int, base: float = 10000.0, device=None):
    """The frequencies base^(-2i/L), i < L/2, of the page's recipe, as the
    float64 tensor the _pos entry points take (computed in double on the
    host)."""
    import torch
    i = torch.arange(L // 2, dtype=torch.float64)
    return torch.pow(torch.tensor(float(base), dtype=torch.float64), -2.0 * i / L).to(device)


def _check_pair_axes(positions, pair_axes, partial_slice):
    """The pairs' axes as a tuple, one for each pair of the slice, and the
    three-dimensional positions they count on."""
    import torch
    if not isinstance(positions, torch.Tensor) or positions.dim() != 3 or positions.dtype != torch.int64:
        raise ValueError("positions must be a 3-D int64 tensor (A, B or 1, S)")
    pair_axes = pair_axes if type(pair_axes) is tuple else tuple(int(a) for a in pair_axes)
    L = 0 if partial_slice is None else int(partial_slice[1]) - int(partial_slice[0])
    if L > 0 and len(pair_axes) != L // 2:
        raise ValueError(f"pair_axes must hold (end - start) / 2 = {L // 2} axes, got {len(pair_axes)}")
    return pair_axes


def _call_pos(direction, x, positions, inv_freq, mode, partial_slice, table_dtype, stream, pair_axes=None, y=None):
    """The position entry points: in place on x, or (y given) out of place
    from x into y; with pair_axes, those with several axes."""
    import torch
    if isinstance(mode, str):
        if mode not in MODES:
            raise ValueError(f"rotary_mode must be one of {sorted(MODES)}")
        mode = MODES[mode]
    for name, t in (("x", x), ("positions", positions), ("inv_freq", inv_freq)) + ((("out", y),) if y is not None
                                                                                   else ()):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
    if x.dim() != 4:
        raise ValueError(f"x must be 4-D (B,S,N,D layout), got {x.dim()}-D")
    if pair_axes is not None:
        pair_axes = _check_pair_axes(positions, pair_axes, partial_slice)
    elif positions.dim() != 2 or positions.dtype != torch.int64:
        raise ValueError("positions must be a 2-D int64 tensor (B or 1, S)")
    if inv_freq.dtype != torch.float64 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise ValueError("inv_freq must be a contiguous 1-D float64 tensor")
    if not x.is_contiguous():
        raise ValueError("x must be contiguous (BSND); non-contiguous tensors are not supported")
    if y is not None:
        if y.shape != x.shape or y.dtype != x.dtype:
            raise ValueError(f"out must match x in shape and dtype: {tuple(y.shape)} {y.dtype} vs "
                             f"{tuple(x.shape)} {x.dtype}")
        if not y.is_contiguous():
            raise ValueError("out must be contiguous (BSND)")
        if x.numel() and not (x.is_cuda and y.is_cuda and y.device == x.device):
            raise ValueError("x and out must be GPU tensors on one device")
    sl = (0, 0) if partial_slice is None else (int(partial_slice[0]), int(partial_slice[1]))
    if x.numel() and sl[1] > sl[0]:
        if inv_freq.numel() != (sl[1] - sl[0]) // 2:
            raise ValueError(f"inv_freq must hold (end - start) / 2 = {(sl[1] - sl[0]) // 2} frequencies")
        if not x.is_cuda:
            raise ValueError("x must be a GPU tensor")
        for name, t in (("positions", positions), ("inv_freq", inv_freq)):
            if t.device != x.device:
                raise ValueError(f"{name} must be on {x.device}")
    if table_dtype is None:
        tdt = _dtype_code(x)
    else:
        tdt = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}.get(table_dtype, DTYPE_CODES.get(table_dtype))
        if tdt is None:
            raise TypeError(f"unsupported table dtype {table_dtype}")
    handle, current = _on_device(x, stream)
    with current:
        if pair_axes is not None:
            st = raw_axes_call(direction, x.data_ptr() or None, tuple(x.shape), _dtype_code(x),
                               positions.data_ptr() or None, tuple(positions.shape), tuple(positions.stride()),
                               inv_freq.data_ptr() or None, pair_axes, tdt, mode, partial_slice, handle,
                               None if y is None else y.data_ptr() or None, y is not None)
        elif y is None:
            st = raw_pos_call(direction, x.data_ptr() or None, tuple(x.shape), _dtype_code(x),
                              positions.data_ptr() or None, tuple(positions.shape), tuple(positions.stride()),
                              inv_freq.data_ptr() or None, tdt, mode, partial_slice, handle)
        else:
            st = raw_out_pos_call(direction, y.data_ptr() or None, x.data_ptr() or None, tuple(x.shape),
                                  _dtype_code(x), positions.data_ptr() or None, tuple(positions.shape),
                                  tuple(positions.stride()), inv_freq.data_ptr() or None, tdt, mode,
                                  partial_slice, handle)
    if st != ROPE_OK:
        raise RopeError(st, last_error())


def rope_partial_fwd_inplace_pos(x, positions, inv_freq, rotary_mode="interleave", partial_slice=None,
                                 table_dtype=None, stream=None) -> None:
    """Rotate ``x[..., start:end)`` in place with cos/sin computed in the
    kernel from positions: θ = positions[b, s] * inv_freq[i] (double), cos
    and sin in double precision rounded once to ``table_dtype`` (default:
    x's dtype) -- the values a table of that type built from the same angles
    would hold.

    positions: int64 GPU tensor (B or 1, S), any strides.
    inv_freq: contiguous float64 GPU tensor of (end - start) / 2 frequencies
    (``rope_inv_freq(L, base)`` gives base^(-2i/L)).
    """
    _call_pos("fwd", x, positions, inv_freq, rotary_mode, partial_slice, table_dtype, stream)


def rope_partial_bwd_inplace_pos(dx, positions, inv_freq, rotary_mode="interleave", partial_slice=None,
                                 table_dtype=None, stream=None) -> None:
    """Backward of :func:`rope_partial_fwd_inplace_pos`, in place on the
    incoming gradient."""
    _call_pos("bwd", dx, positions, inv_freq, rotary_mode, partial_slice, table_dtype, stream)


def rope_partial_fwd_out_pos(out, x, positions, inv_freq, rotary_mode="interleave", partial_slice=None,
                             table_dtype=None, stream=None) -> None:
    """Out-of-place :func:`rope_partial_fwd_inplace_pos`: ``out`` receives x
    with its slice rotated; x is left unchanged."""
    _call_pos("fwd", x, positions, inv_freq, rotary_mode, partial_slice, table_dtype, stream, y=out)


def rope_partial_bwd_out_pos(dx, dy, positions, inv_freq, rotary_mode="interleave", partial_slice=None,
                             table_dtype=None, stream=None) -> None:
    """Out-of-place backward of the position form: ``dx`` receives the
    gradient with respect to x for the incoming gradient ``dy``, which is
    left unchanged."""
    _call_pos("bwd", dy, positions, inv_freq, rotary_mode, partial_slice, table_dtype, stream, y=dx)


def rope_pair_axes(sections, dealt: bool = False) -> tuple:
    """The axis of each pair for axes that take ``sections[k]`` pairs each:
    in blocks, all of axis 0's pairs first (``sections=(16, 24, 24)`` gives
    axis 0 to pairs 0 to 15), or ``dealt``: to the axes in turn, 0, 1, 2, 0,
    1, 2, ..., an axis that has its pairs being passed over."""
    left = [int(n) for n in sections]
    if not 1 <= len(left) <= AXES_MAX or min(left) < 0:
        raise ValueError(f"sections must hold 1 to {AXES_MAX} counts of pairs")
    if not dealt:
        return tuple(a for a, n in enumerate(left) for _ in range(n))
    got = []
    while any(left):
        for a, n in enumerate(left):
            if n:
                left[a] -= 1
                got.append(a)
    return tuple(got)


def rope_axes_inv_freq(pair_axes, base: float = 10000.0, device=None):
    """Frequencies for axes that count their own pairs: base^(-j/n) for the
    j-th of the n pairs that an axis has in ``pair_axes``, as the float64
    tensor the _axes entry points take (computed in double on the host).
    Where the frequencies run over all pairs, use :func:`rope_inv_freq`."""
    import torch
    pair_axes = tuple(pair_axes)
    seen, share = {}, []
    for a in pair_axes:
        share.append(seen.get(a, 0) / pair_axes.count(a))
        seen[a] = seen.get(a, 0) + 1
    return torch.pow(torch.tensor(float(base), dtype=torch.float64),
                     -torch.tensor(share, dtype=torch.float64)).to(device)


def rope_partial_fwd_inplace_axes(x, positions, inv_freq, pair_axes, rotary_mode="interleave", partial_slice=None,
                                  table_dtype=None, stream=None) -> None:
    """:func:`rope_partial_fwd_inplace_pos` with positions on several axes
    (time, height and width of images and video): pair i of the slice turns by
    positions[pair_axes[i], b, s] * inv_freq[i].

    positions: int64 GPU tensor (A, B or 1, S), 1 to AXES_MAX axes, any
    strides.
    pair_axes: the axis of each of the (end - start) / 2 pairs, in [0, A)
    (``rope_pair_axes`` gives the usual orders). It stays on the host: a
    captured graph keeps the axes it was captured with.
    inv_freq: as there (``rope_axes_inv_freq`` where each axis counts its own
    pairs).
    """
    _call_pos("fwd", x, positions, inv_freq, rotary_mode, partial_slice, table_dtype, stream, pair_axes=pair_axes)


def rope_partial_bwd_inplace_axes(dx, positions, inv_freq, pair_axes, rotary_mode="interleave", partial_slice=None,
                                  table_dtype=None, stream=None) -> None:
    """Backward of :func:`rope_partial_fwd_inplace_axes`, in place on the
    incoming gradient."""
    _call_pos("bwd", dx, positions, inv_freq, rotary_mode, partial_slice, table_dtype, stream, pair_axes=pair_axes)


def rope_partial_fwd_out_axes(out, x, positions, inv_freq, pair_axes, rotary_mode="interleave", partial_slice=None,
                              table_dtype=None, stream=None) -> None:
    """Out-of-place :func:`rope_partial_fwd_inplace_axes`: ``out`` receives x
    with its slice rotated; x is left unchanged."""
    _call_pos("fwd", x, positions, inv_freq, rotary_mode, partial_slice, table_dtype, stream, y=out,
              pair_axes=pair_axes)


def rope_partial_bwd_out_axes(dx, dy, positions, inv_freq, pair_axes, rotary_mode="interleave", partial_slice=None,
                              table_dtype=None, stream=None) -> None:
    """Out-of-place backward with several axes: ``dx`` receives the gradient
    with respect to x for the incoming gradient ``dy``, which is left
    unchanged."""
    _call_pos("bwd", dy, positions, inv_freq, rotary_mode, partial_slice, table_dtype, stream, y=dx,
              pair_axes=pair_axes)


def rope_partial_fwd_inplace_multi(xs, r1, r2, rotary_mode="interleave", partial_slice=None, stream=None) -> None:
    """Forward on up to MULTI_MAX tensors that share r1/r2 (e.g. Q and K), in
    one kernel launch when they take the same kernel; same result as calling
    :func:`rope_partial_fwd_inplace` on each in order."""
    _call_multi("fwd", xs, r1, r2, rotary_mode, partial_slice, stream)


def rope_partial_bwd_inplace_multi(dxs, r1, r2, rotary_mode="interleave", partial_slice=None, stream=None) -> None:
    """Backward counterpart of :func:`rope_partial_fwd_inplace_multi`."""
    _call_multi("bwd", dxs, r1, r2, rotary_mode, partial_slice, stream)


# ---------------------------------------------------------------------------
# Autograd op over the C ABI ("CANN ops-transformer 算子详解：
# inplace_partial_rotary_mul 原地部分旋转位置编码", section 自动微分说明 and the
# training-mode example of section 调用说明): the forward rotates x in place
# and marks it dirty; the backward is the rotation in the other direction of
# the incoming gradient; what cos and sin come from receives no gradient.
# ---------------------------------------------------------------------------

_OTHER = {"fwd": "bwd", "bwd": "fwd"}
_TORCH = None


def _autograd():
    """torch's test of enabled gradients, its forward mode, what moves the
    version counters of tensors written in place unseen by autograd (so that a
    backward which needs an old value raises), and whether any of some tensors
    (or None) requires a gradient."""
    global _TORCH
    if _TORCH is None:
        import torch
        _TORCH = (torch.is_grad_enabled, torch.autograd.forward_ad, torch._C._increment_version,
                  torch._C._any_requires_grad)
    return _TORCH


def _differentiated(x):
    """Whether autograd follows x: it needs a gradient, or has a tangent."""
    enabled, fw, _, _ = _TORCH or _autograd()
    return x.requires_grad and enabled() or fw._current_level >= 0 and fw.unpack_dual(x).tangent is not None


def _refuse_differentiated(call, names, tensors):
    """A call that gives no gradient takes no tensor that needs one. names: of
    the first tensors; the rest belong to caches."""
    enabled, fw, _, any_requires_grad = _TORCH or _autograd()
    if fw._current_level < 0 and not (enabled() and any_requires_grad(*tensors)):
        return
    for i, t in enumerate(tensors):
        if t is not None and _differentiated(t):
            name = names[i] if i < len(names) else "the cache"
            raise RuntimeError(f"{call}: {name} needs a gradient, which this call does not give; call it under "
                               "torch.no_grad() or with a detached tensor")


def _rotated_new(rotate, direction, x, a, b, how):
    """A new contiguous tensor holding x with its slice rotated. x is never
    modified (as an incoming gradient, autograd may hand it to other
    consumers): a contiguous one is read by the out-of-place kernel (one pass),
    any other layout (e.g. the stride-0 gradient of an expand) is first made
    into a private contiguous copy, which is then rotated in place."""
    import torch
    if x.is_contiguous():
        y = torch.empty_like(x, memory_format=torch.contiguous_format)
        rotate(direction, x, a, b, *how, y)
        return y
    y = x.contiguous()
    rotate(direction, y, a, b, *how)
    return y


def _rotation_functions():
    """The autograd functions of a rotation, in place and out of place. Their
    arguments: rotate(direction, x, a, b, *how[, y]), the direction, x, the two
    tensors that cos and sin come from, and what else rotate takes. The
    rotation is linear in x, so its backward is the rotation in the other
    direction and its tangent the tangent's rotation, both recorded in their
    turn where something follows them."""
    import torch

    def save(ctx, rotate, direction, a, b, how):
        ctx.save_for_backward(a, b)
        if torch.autograd.forward_ad._current_level >= 0:
            ctx.save_for_forward(a, b)
        ctx.call = rotate, direction, how

    def backward(ctx, grad):
        rotate, direction, how = ctx.call
        a, b = ctx.saved_tensors
        turn = _autograd_out if _differentiated(grad) else _rotated_new
        return None, None, turn(rotate, _OTHER[direction], grad, a, b, how), None, None, None

    def tangent(ctx, t):
        rotate, direction, how = ctx.call
        a, b = ctx.saved_tensors
        return _autograd_out(rotate, direction, t, a, b, how)

    class InplaceRotationFn(torch.autograd.Function):
        @staticmethod
        def forward(ctx, rotate, direction, x, a, b, how):
            rotate(direction, x, a, b, *how)
            ctx.mark_dirty(x)
            save(ctx, rotate, direction, a, b, how)
            return x

        @staticmethod
        def jvp(ctx, _rotate, _direction, t, *_):
            # the tangent of a value changed in place has to change in place
            return t.copy_(tangent(ctx, t))

    class RotationFn(torch.autograd.Function):
        @staticmethod
        def forward(ctx, rotate, direction, x, a, b, how):
            y = _rotated_new(rotate, direction, x, a, b, how)
            save(ctx, rotate, direction, a, b, how)
            return y

        @staticmethod
        def jvp(ctx, _rotate, _direction, t, *_):
            return tangent(ctx, t)

    InplaceRotationFn.backward = RotationFn.backward = staticmethod(backward)
    return InplaceRotationFn, RotationFn


_ROTATION_FNS = None


def _rotation_fn(inplace):
    global _ROTATION_FNS
    if _ROTATION_FNS is None:
        _ROTATION_FNS = _rotation_functions()
    return _ROTATION_FNS[0 if inplace else 1]


def _autograd_inplace(name, rotate, x, a, b, how):
    if not _differentiated(x):
        rotate("fwd", x, a, b, *how)
        _TORCH[2]((x,))
        return
    if x.is_leaf and x.requires_grad and _TORCH[0]():
        raise RuntimeError(f"{name}: x is a leaf tensor that requires grad; "
                           "rotate a non-leaf copy of it (e.g. y = x * 1.0)")
    _rotation_fn(True).apply(rotate, "fwd", x, a, b, how)


def _autograd_out(rotate, direction, x, a, b, how):
    if _differentiated(x):
        return _rotation_fn(False).apply(rotate, direction, x, a, b, how)
    return _rotated_new(rotate, direction, x, a, b, how)


def _rotate_tables(direction, x, r1, r2, mode, partial_slice, y=None):
    """x rotated by tables in place, or into y."""
    if y is None:
        _call(direction, x, r1, r2, mode, partial_slice, None)
    else:
        _call_out(direction, y, x, r1, r2, mode, partial_slice, None)


def _tables_how(rotary_mode, partial_slice):
    return rotary_mode, None if partial_slice is None else (int(partial_slice[0]), int(partial_slice[1]))


def inplace_partial_rotary_mul(x, r1, r2, rotary_mode="interleave", partial_slice=None) -> None:
    """In-place partial RoPE that records itself for autograd when x needs a
    gradient, and calls the forward entry point directly otherwise.

    x must not be a leaf tensor that requires grad: in-place changes to such
    a tensor are illegal in autograd, so rotate a non-leaf copy (y = x * 1.0),
    as the training example on the page does. r1 and r2 never get gradients,
    nor are tangents of theirs followed. Differentiable any number of times
    and in forward mode.
    """
    _autograd_inplace("inplace_partial_rotary_mul", _rotate_tables, x, r1, r2, _tables_how(rotary_mode, partial_slice))


def partial_rotary_mul(x, r1, r2, rotary_mode="interleave", partial_slice=None):
    """Out-of-place partial RoPE: returns a new contiguous tensor holding x
    with ``x[..., start:end)`` rotated; x is not modified. Records itself for
    autograd (the backward is the out-of-place backward entry point) and
    works on leaf tensors too, so a training step needs no ``x * 1.0`` copy
    before the in-place op. Differentiable any number of times and in forward
    mode. r1 and r2 never get gradients, nor are tangents of theirs followed."""
    return _autograd_out(_rotate_tables, "fwd", x, r1, r2, _tables_how(rotary_mode, partial_slice))


# ---------------------------------------------------------------- autograd, cos/sin from positions

def _pos_how(rotary_mode, partial_slice, table_dtype, pair_axes=None):
    sl = None if partial_slice is None else (int(partial_slice[0]), int(partial_slice[1]))
    return rotary_mode, sl, table_dtype, None, pair_axes


def inplace_partial_rotary_mul_pos(x, positions, inv_freq, rotary_mode="interleave", partial_slice=None,
                                   table_dtype=None) -> None:
    """:func:`inplace_partial_rotary_mul` with cos and sin computed in the
    kernel from positions (see :func:`rope_partial_fwd_inplace_pos`).
    positions and inv_freq never get gradients; x must not be a leaf tensor
    that requires grad. Differentiable any number of times and in forward
    mode."""
    _autograd_inplace("inplace_partial_rotary_mul_pos", _call_pos, x, positions, inv_freq,
                      _pos_how(rotary_mode, partial_slice, table_dtype))


def partial_rotary_mul_pos(x, positions, inv_freq, rotary_mode="interleave", partial_slice=None,
                           table_dtype=None):
    """:func:`partial_rotary_mul` with cos and sin computed in the kernel from
    positions: returns a new tensor, x is not modified, and the backward is
    the out-of-place position backward, differentiable in its turn, as is the
    tangent in forward mode. positions and inv_freq never get gradients, nor
    are tangents of theirs followed."""
    return _autograd_out(_call_pos, "fwd", x, positions, inv_freq, _pos_how(rotary_mode, partial_slice, table_dtype))


def inplace_partial_rotary_mul_axes(x, positions, inv_freq, pair_axes, rotary_mode="interleave", partial_slice=None,
                                    table_dtype=None) -> None:
    """:func:`inplace_partial_rotary_mul_pos` with positions on several axes
    (see :func:`rope_partial_fwd_inplace_axes`)."""
    _autograd_inplace("inplace_partial_rotary_mul_axes", _call_pos, x, positions, inv_freq,
                      _pos_how(rotary_mode, partial_slice, table_dtype, tuple(pair_axes)))


def partial_rotary_mul_axes(x, positions, inv_freq, pair_axes, rotary_mode="interleave", partial_slice=None,
                            table_dtype=None):
    """:func:`partial_rotary_mul_pos` with positions on several axes (see
    :func:`rope_partial_fwd_inplace_axes`)."""
    return _autograd_out(_call_pos, "fwd", x, positions, inv_freq,
                         _pos_how(rotary_mode, partial_slice, table_dtype, tuple(pair_axes)))


def _call_pos_multi(direction, xs, positions, inv_freq, mode, partial_slice, table_dtype, stream, pair_axes=None):
    import torch
    xs = list(xs)
    if len(xs) > MULTI_MAX:
        raise ValueError(f"at most {MULTI_MAX} tensors per call")
    if not xs:
        return
    if isinstance(mode, str):
        if mode not in MODES:
            raise ValueError(f"rotary_mode must be one of {sorted(MODES)}")
        mode = MODES[mode]
    for i, x in enumerate(xs):
        if not isinstance(x, torch.Tensor) or x.dim() != 4:
            raise ValueError(f"xs[{i}] must be a 4-D torch.Tensor (B,S,N,D layout)")
        if not x.is_contiguous():
            raise ValueError(f"xs[{i}] must be contiguous (BSND)")
        if x.numel() and not x.is_cuda:
            raise ValueError(f"xs[{i}] must be a GPU tensor")
    if len({x.dtype for x in xs}) != 1:
        raise TypeError("all tensors of one call must share a dtype")
    devs = {x.device for x in xs if x.numel()}
    if len(devs) > 1:
        raise ValueError("all tensors of one call must be on one device")
    if pair_axes is not None:
        pair_axes = _check_pair_axes(positions, pair_axes, partial_slice)
    elif positions.dim() != 2 or positions.dtype != torch.int64:
        raise ValueError("positions must be a 2-D int64 tensor (B or 1, S)")
    if inv_freq.dtype != torch.float64 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise ValueError("inv_freq must be a contiguous 1-D float64 tensor")
    dev = next(iter(devs)) if devs else None
    sl = (0, 0) if partial_slice is None else (int(partial_slice[0]), int(partial_slice[1]))
    if dev is not None and sl[1] > sl[0]:
        if inv_freq.numel() != (sl[1] - sl[0]) // 2:
            raise ValueError(f"inv_freq must hold (end - start) / 2 = {(sl[1] - sl[0]) // 2} frequencies")
        for name, t in (("positions", positions), ("inv_freq", inv_freq)):
            if t.device != dev:
                raise ValueError(f"{name} must be on {dev}")
    if table_dtype is None:
        tdt = _dtype_code(xs[0])
    else:
        tdt = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}.get(table_dtype, DTYPE_CODES.get(table_dtype))
        if tdt is None:
            raise TypeError(f"unsupported table dtype {table_dtype}")
    if dev is not None:
        handle, current = _on_device(next(x for x in xs if x.numel()), stream)
    else:
        handle, current = getattr(stream, "cuda_stream", stream), _NOTHING
    with current:
        ptrs, shapes = [x.data_ptr() or None for x in xs], [tuple(x.shape) for x in xs]
        where = (positions.data_ptr() or None, tuple(positions.shape), tuple(positions.stride()),
                 inv_freq.data_ptr() or None)
        if pair_axes is not None:
            st = raw_axes_multi_call(direction, ptrs, shapes, _dtype_code(xs[0]), *where, pair_axes, tdt, mode,
                                     partial_slice, handle)
        else:
            st = raw_pos_multi_call(direction, ptrs, shapes, _dtype_code(xs[0]), *where, tdt, mode, partial_slice,
                                    handle)
    if st != ROPE_OK:
        raise RopeError(st, last_error())


def rope_partial_fwd_inplace_pos_multi(xs, positions, inv_freq, rotary_mode="interleave", partial_slice=None,
                                       table_dtype=None, stream=None) -> None:
    """:func:`rope_partial_fwd_inplace_pos` on up to 4 tensors sharing the
    positions (e.g. Q and K of one layer), in one launch when they share B,
    S and D: each pair's cos and sin is then evaluated once per position."""
    _call_pos_multi("fwd", xs, positions, inv_freq, rotary_mode, partial_slice, table_dtype, stream)


def rope_partial_bwd_inplace_pos_multi(xs, positions, inv_freq, rotary_mode="interleave", partial_slice=None,
                                       table_dtype=None, stream=None) -> None:
    """Backward of :func:`rope_partial_fwd_inplace_pos_multi`."""
    _call_pos_multi("bwd", xs, positions, inv_freq, rotary_mode, partial_slice, table_dtype, stream)


def rope_partial_fwd_inplace_axes_multi(xs, positions, inv_freq, pair_axes, rotary_mode="interleave",
                                        partial_slice=None, table_dtype=None, stream=None) -> None:
    """:func:`rope_partial_fwd_inplace_axes` on up to 4 tensors sharing the
    positions (e.g. Q and K of one layer), in one launch when they share B,
    S and D: each pair's cos and sin is then evaluated once per position."""
    _call_pos_multi("fwd", xs, positions, inv_freq, rotary_mode, partial_slice, table_dtype, stream, pair_axes)


def rope_partial_bwd_inplace_axes_multi(xs, positions, inv_freq, pair_axes, rotary_mode="interleave",
                                        partial_slice=None, table_dtype=None, stream=None) -> None:
    """Backward of :func:`rope_partial_fwd_inplace_axes_multi`."""
    _call_pos_multi("bwd", xs, positions, inv_freq, rotary_mode, partial_slice, table_dtype, stream, pair_axes)


# ------------------------------------------------------------------- paged, quantised cache

_CACHE_FORMAT_OF = {}


def _cache_format(dtype):
    if not _CACHE_FORMAT_OF:
        import torch
        _CACHE_FORMAT_OF.update({torch.float32: 0, torch.float16: 1, torch.bfloat16: 2, torch.float8_e4m3fn: 3,
                                 torch.int8: 4, torch.uint8: 5})
    return _CACHE_FORMAT_OF.get(dtype)


class RopeCache:
    """A paged cache of keys or values, over tensors that the caller owns:
    slot t is ``data[t // page_size, t % page_size]``.

    data: (pages, page_size, heads, dim) of float32, float16 or bfloat16 (no
    scales), float8_e4m3fn, or int8; or (pages, page_size, heads, dim // 2) of
    uint8, two 4-bit codes a byte. Any strides (for example one half of a
    (pages, 2, page_size, heads, dim) tensor), the lanes of a row consecutive.
    scales: (pages, page_size, heads, dim // group) of float32 for the
    quantised formats: lane j of a row stands for code[j] * scale[j // group].
    The object stays with these tensors: for others, make another.
    """

    __slots__ = ("_data", "_scales", "_device", "_words", "_tensors")

    def _stays(self, value=None):
        raise AttributeError("a RopeCache stays with the tensors it was made of: make another")

    data = property(operator.attrgetter("_data"), _stays, _stays)
    scales = property(operator.attrgetter("_scales"), _stays, _stays)
    device = property(operator.attrgetter("_device"), _stays, _stays)

    def __init__(self, data, scales=None):
        import torch
        if not isinstance(data, torch.Tensor) or data.dim() != 4:
            raise ValueError("data must be a 4-D torch.Tensor (pages, page_size, heads, dim)")
        fmt = _cache_format(data.dtype)
        if fmt is None:
            raise TypeError(f"unsupported cache type {data.dtype}")
        pages, size, heads, dim = data.shape
        s0, s1, s2, s3 = data.stride()
        if s3 != 1 and dim > 1:
            raise ValueError("data: the lanes of a row must be consecutive")
        self._data, self._scales, self._device = data, scales, data.device
        self._tensors = (data,) if scales is None else (data, scales)
        if fmt < 3:
            if scales is not None:
                raise ValueError(f"a {data.dtype} cache has no scales")
            es = data.element_size()
            self._words = _CacheWords(data.data_ptr(), 0, fmt, pages, size, heads, dim, dim, s0 * es, s1 * es, s2 * es)
            return
        if fmt == 5:
            dim *= 2
        if not isinstance(scales, torch.Tensor) or scales.dtype != torch.float32:
            raise TypeError("a quantised cache needs float32 scales")
        if scales.dim() != 4 or scales.device != data.device:
            raise ValueError("scales must be (pages, page_size, heads, dim // group), on data's device")
        p, z, h, groups = scales.shape
        if p != pages or z != size or h != heads:
            raise ValueError("scales must be (pages, page_size, heads, dim // group), on data's device")
        c0, c1, c2, c3 = scales.stride()
        if dim and (groups < 1 or dim % groups):
            raise ValueError(f"{groups} scales do not divide {dim} lanes")
        if groups > 1 and c3 != 1:
            raise ValueError("scales: the scales of a row must be consecutive")
        self._words = _CacheWords(data.data_ptr(), scales.data_ptr(), fmt, pages, size, heads, dim,
                                  dim // groups if groups else 0, s0, s1, s2, c0, c1, c2)

    @property
    def group(self) -> int:
        """Lanes per scale."""
        return self._words[7]

    @property
    def struct(self) -> RopeCacheStruct:
        """The C ABI's description of the cache."""
        return RopeCacheStruct.from_buffer(self._words)


def rope_cache(pages: int, page_size: int, heads: int, dim: int, format: str = "e4m3", group: int | None = None,
               device=None) -> RopeCache:
    """A new zeroed cache of a CACHE_FORMATS format, ``group`` lanes per scale
    (default: a row)."""
    import torch
    types = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn,
             "int8": torch.int8, "int4": torch.uint8}
    if format not in types:
        raise ValueError(f"format must be one of {sorted(types)}")
    device = "cuda" if device is None else device
    data = torch.zeros(pages, page_size, heads, dim // 2 if format == "int4" else dim, dtype=types[format],
                       device=device)
    if CACHE_FORMATS[format] < 3:
        return RopeCache(data)
    group = dim if group is None else group
    if group < 1 or dim % group:
        raise ValueError(f"group {group} does not divide {dim} lanes")
    return RopeCache(data, torch.zeros(pages, page_size, heads, dim // group, device=device))


def _rows(name, t):
    """A (B, S, N, D) tensor as the C ABI's rows."""
    _, _, n, d = t.shape
    sb, ss, sn, sd = t.stride()
    if sd != 1 and d > 1:
        raise ValueError(f"{name}: the lanes of a row must be consecutive")
    return _RowsWords(t.data_ptr(), n, d, sb, ss, sn)


def _rows_beside(name, t, B, S, dtype, dev):
    """The rows of q or v beside those of k."""
    import torch
    if not isinstance(t, torch.Tensor) or t.dim() != 4:
        raise ValueError(f"{name} must be a 4-D torch.Tensor (B, S, heads, dim)")
    if t.dtype != dtype:
        raise TypeError("q, k and v must share a dtype")
    b, s, n, d = t.shape
    if b != B or s != S:
        raise ValueError(f"{name} must have k's tokens")
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev}")
    if not t.is_cuda and t.numel():
        raise ValueError(f"{name} must be a GPU tensor")
    sb, ss, sn, sd = t.stride()
    if sd != 1 and d > 1:
        raise ValueError(f"{name}: the lanes of a row must be consecutive")
    return _RowsWords(t.data_ptr(), n, d, sb, ss, sn)


def _turn_args(positions, inv_freq, pair_axes, rotary_mode, partial_slice, table_dtype, dtype_code, device):
    """The C arguments from positions to partial_slice of a cache call, and
    the tensors that have to be on `device`."""
    import torch
    mode = rotary_mode
    if isinstance(mode, str):
        mode = MODES.get(mode)
        if mode is None:
            raise ValueError(f"rotary_mode must be one of {sorted(MODES)}")
    if table_dtype is None:
        tdt = dtype_code
    else:
        tdt = _DTYPE_OF_TORCH.get(table_dtype, DTYPE_CODES.get(table_dtype))
        if tdt is None:
            raise TypeError(f"unsupported table dtype {table_dtype}")
    if positions is None or partial_slice is None:
        return (None, None, None, None, None, tdt, mode, None)
    start, end = int(partial_slice[0]), int(partial_slice[1])
    if not (isinstance(positions, torch.Tensor) and isinstance(inv_freq, torch.Tensor)):
        raise TypeError("positions and inv_freq must be torch.Tensors")
    if positions.device != device or inv_freq.device != device:
        raise ValueError(f"positions and inv_freq must be on {device}")
    shape, st = positions.shape, positions.stride()
    if positions.dtype != torch.int64 or len(st) not in (2, 3):
        raise ValueError("positions must be an int64 tensor (B or 1, S), or (A, B or 1, S) with pair_axes")
    if len(st) == 2:
        if pair_axes is not None:
            raise ValueError("pair_axes goes with positions (A, B or 1, S)")
        shape, st = (1, *shape), (0, *st)
    else:
        if pair_axes is None:
            raise ValueError("positions on several axes need pair_axes")
        pair_axes = _check_pair_axes(positions, pair_axes, partial_slice)
    if inv_freq.dtype != torch.float64 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise ValueError("inv_freq must be a contiguous 1-D float64 tensor")
    if end > start and inv_freq.numel() != (end - start) // 2:
        raise ValueError(f"inv_freq must hold (end - start) / 2 = {(end - start) // 2} frequencies")
    return (positions.data_ptr() or None, _I64x3(*shape), _I64x3(*st), inv_freq.data_ptr() or None,
            None if pair_axes is None else _i32_array(pair_axes), tdt, mode, _I64x2(start, end))


def rope_cache_write(k, v, k_cache, v_cache, slots, positions=None, inv_freq=None, rotary_mode="interleave",
                     partial_slice=None, q=None, pair_axes=None, table_dtype=None, rotate_k: bool = True,
                     stream=None) -> None:
    """Rotate ``k[..., start:end)`` from positions and write it, with ``v``, to
    its slots of paged caches, quantised; rotate ``q`` in place beside it. One
    launch (two when v's format is not k's).

    k: (B, S, heads, dim) GPU tensor, float32/float16/bfloat16, any strides
    with consecutive lanes (a slice of a fused projection's output); v: the
    same of v_cache's heads and dim, or None with v_cache None; q: (B, S, any,
    dim) or None.
    k_cache, v_cache: :class:`RopeCache` of a quantised format or of k's type.
    slots: int64 (B, S), the slot each token goes to (page * page_size +
    offset); a negative one, or one past the cache, writes nothing. Slots of
    one call must differ.
    positions: int64 (B or 1, S), or (A, B or 1, S) with ``pair_axes`` (see
    :func:`rope_partial_fwd_inplace_axes`), or None: nothing is rotated.
    rotate_k=False stores k unrotated (q is still rotated), for a
    :func:`rope_cache_read` that rotates.

    The rotation is fp32 and k is not rounded before it is quantised: for
    each group of lanes scale = largest finite magnitude / Q (448 for e4m3,
    127, 7), code = k / scale rounded once to the nearest, ties to even.

    No gradient passes through the call: it refuses q, k, v and caches that
    need one (while gradients are enabled). Their changes in place are seen by
    a backward that needs the old values."""
    import torch
    if not isinstance(k, torch.Tensor) or k.dim() != 4:
        raise ValueError("k must be a 4-D torch.Tensor (B, S, heads, dim)")
    if k.numel() and not k.is_cuda:
        raise ValueError("k must be a GPU tensor")
    code, dev = _dtype_code(k), k.device
    B, S, n, d = k.shape
    sb, ss, sn, sd = k.stride()
    if sd != 1 and d > 1:
        raise ValueError("k: the lanes of a row must be consecutive")
    rows_v = None if v is None else _rows_beside("v", v, B, S, k.dtype, dev)
    rows_q = None if q is None else _rows_beside("q", q, B, S, k.dtype, dev)
    if (v is None) != (v_cache is None):
        raise ValueError("v and v_cache go together")
    if not isinstance(k_cache, RopeCache) or not (v_cache is None or isinstance(v_cache, RopeCache)):
        raise TypeError("k_cache and v_cache must be RopeCache objects")
    if k_cache._device != dev or (v_cache is not None and v_cache._device != dev):
        raise ValueError(f"k_cache and v_cache must be on {dev}")
    if not isinstance(slots, torch.Tensor) or slots.dtype != torch.int64 or slots.dim() != 2 or \
            slots.size(0) != B or slots.size(1) != S:
        raise ValueError("slots must be an int64 tensor (B, S)")
    if slots.device != dev:
        raise ValueError(f"slots must be on {dev}")
    written = k_cache._tensors if v_cache is None else k_cache._tensors + v_cache._tensors
    _refuse_differentiated("rope_cache_write", "kvq", (k, v, q) + written)
    turn = _turn_args(positions, inv_freq, pair_axes, rotary_mode, partial_slice, table_dtype, code, dev)
    handle, current = _on_device(k, stream)
    with current:
        st = _words_entry("rope_cache_write")(
            B, S, code, rows_q, _RowsWords(k.data_ptr(), n, d, sb, ss, sn), rows_v, k_cache._words,
            None if v_cache is None else v_cache._words, slots.data_ptr() or None,
            _I64x2(*slots.stride()), *turn, 1 if rotate_k else 0, handle)
    if st != ROPE_OK:
        raise RopeError(st, last_error())
    _TORCH[2](written if q is None else written + (q,))


def rope_cache_read(out, cache, block_table, lengths, starts=None, positions=None, inv_freq=None,
                    rotary_mode="interleave", partial_slice=None, pair_axes=None, table_dtype=None,
                    stream=None) -> None:
    """Read cached tokens back: ``out[b, s]`` becomes token ``starts[b] + s`` of
    sequence b for s < lengths[b], its codes times their scales; with
    positions its slice ``[start, end)`` is rotated on the way (keys stored
    unrotated, or moved to other positions). Every other row of out keeps its
    bytes: the padding behind a sequence, tokens past the block table, pages
    outside the cache.

    out: (B, S, heads, dim) GPU tensor, float32/float16/bfloat16, any strides
    with consecutive lanes.
    block_table: int32 (B, columns), token t of sequence b lies in page
    block_table[b, t // page_size].
    lengths: int32 (B); starts: int32 (B), 0 when None.
    positions, inv_freq, pair_axes: as in :func:`rope_cache_write`, for out's
    rows.

    No gradient passes through the call: out and a cache that need one are
    refused (while gradients are enabled)."""
    import torch
    if not isinstance(out, torch.Tensor) or out.dim() != 4:
        raise ValueError("out must be a 4-D torch.Tensor (B, S, heads, dim)")
    code, dev = _dtype_code(out), out.device
    if out.numel() and not out.is_cuda:
        raise ValueError("out must be a GPU tensor")
    if not isinstance(cache, RopeCache):
        raise TypeError("cache must be a RopeCache")
    if cache._device != dev:
        raise ValueError(f"cache must be on {dev}")
    B, S = out.shape[:2]
    if not isinstance(block_table, torch.Tensor) or block_table.dtype != torch.int32 or block_table.dim() != 2 or \
            block_table.shape[0] != B:
        raise ValueError("block_table must be an int32 tensor (B, columns)")
    if block_table.shape[1] > 1 and block_table.stride(1) != 1:
        raise ValueError("block_table: the pages of a sequence must be consecutive")
    for name, t in (("lengths", lengths), ("starts", starts)):
        if t is None and name == "starts":
            continue
        if not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or t.shape != (B,) or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous int32 tensor (B)")
        if t.device != dev:
            raise ValueError(f"{name} must be on {dev}")
    if block_table.device != dev:
        raise ValueError(f"block_table must be on {dev}")
    _refuse_differentiated("rope_cache_read", ("out",), (out,) + cache._tensors)
    turn = _turn_args(positions, inv_freq, pair_axes, rotary_mode, partial_slice, table_dtype, code, dev)
    handle, current = _on_device(out, stream)
    with current:
        st = _words_entry("rope_cache_read")(
            B, S, code, _rows("out", out), cache._words, block_table.data_ptr() or None, block_table.shape[1],
            block_table.stride(0), lengths.data_ptr() or None, None if starts is None else starts.data_ptr() or None,
            *turn, handle)
    if st != ROPE_OK:
        raise RopeError(st, last_error())
    _TORCH[2]((out,))


def _array(name, t, tensor, dtype, shape, dev):
    """The address of a contiguous tensor of a call's bookkeeping."""
    if not isinstance(t, tensor) or t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {str(dtype).split('.')[-1]} tensor {shape}")
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev}")
    return t.data_ptr() or None


def rope_cache_reserve(block_table, lengths, counts, free_pages, free_count, page_size: int, tokens: int | None = None,
                       slots=None, positions=None, granted=None, stream=None):
    """A step's bookkeeping of a paged cache, on the GPU: sequence b grows by
    ``counts[b]`` tokens, taking pages from the end of the list of free ones as
    it needs them, or where that is negative drops as many, its pages going
    back to the list (-lengths[b] or less ends it). Pages are given back before
    any are taken, both in the order of the sequences; a sequence is refused,
    and nothing of it changes, when the list is too short for the pages that it
    and those before it need, or its row of the table is.

    block_table: int32 (B, columns), lengths: int32 (B), free_pages: int32
    (capacity), free_count: int32 (1); all changed in place. counts: int32 (B).
    tokens: columns of slots and positions, the most that a sequence may grow
    (default: those of slots or positions, or 1).

    Returns (slots, positions, granted), allocated when None: the int64 (B,
    tokens) slots (-1 past a sequence's new tokens) and positions that
    :func:`rope_cache_write` takes, and int32 (B) what was added to each
    length: 0 for a refused sequence, the count for
    :func:`rope_cache_attention`. At most RESERVE_MAX sequences; no two of the
    tensors may overlap."""
    import torch
    if not isinstance(block_table, torch.Tensor) or block_table.dtype != torch.int32 or block_table.dim() != 2:
        raise ValueError("block_table must be an int32 tensor (B, columns)")
    B, cols = block_table.shape
    dev = block_table.device
    if cols > 1 and block_table.stride(1) != 1:
        raise ValueError("block_table: the pages of a sequence must be consecutive")
    if B and not block_table.is_cuda:
        raise ValueError("block_table must be a GPU tensor")
    if not isinstance(free_pages, torch.Tensor) or free_pages.dim() != 1:
        raise ValueError("free_pages must be a contiguous int32 tensor (capacity)")
    if tokens is None:
        given = slots if slots is not None else positions
        tokens = given.shape[1] if given is not None and given.dim() == 2 else 1
    T, i32, i64 = torch.Tensor, torch.int32, torch.int64
    capacity = free_pages.shape[0]
    at = (_array("lengths", lengths, T, i32, (B,), dev), _array("counts", counts, T, i32, (B,), dev),
          _array("free_pages", free_pages, T, i32, (capacity,), dev), capacity,
          _array("free_count", free_count, T, i32, (1,), dev))
    if slots is None or positions is None or granted is None:
        with _allocating_on(stream, dev) if stream is not None and block_table.is_cuda else _NOTHING:
            slots = torch.empty(B, tokens, dtype=i64, device=dev) if slots is None else slots
            positions = torch.empty(B, tokens, dtype=i64, device=dev) if positions is None else positions
            granted = torch.empty(B, dtype=i32, device=dev) if granted is None else granted
    outs = (_array("slots", slots, T, i64, (B, tokens), dev), _array("positions", positions, T, i64, (B, tokens), dev),
            _array("granted", granted, T, i32, (B,), dev))
    handle, current = _on_device(block_table, stream)
    with current:
        st = _words_entry("rope_cache_reserve")(B, tokens, block_table.data_ptr() or None, cols, block_table.stride(0), *at,
                                                page_size, *outs, handle)
    if st != ROPE_OK:
        raise RopeError(st, last_error())
    (_TORCH or _autograd())[2]((block_table, lengths, free_pages, free_count, slots, positions, granted))
    return slots, positions, granted


def rope_cache_attention_workspace(B: int, S: int, q_heads: int, heads: int, v_dim: int) -> int:
    """Bytes of workspace that :func:`rope_cache_attention` needs for queries
    (B, S, q_heads, any) over caches of ``heads`` heads, however many tokens
    are cached."""
    return library().rope_cache_attention_workspace(B, S, q_heads, heads, v_dim)


def rope_cache_attention(q, k_cache, v_cache, block_table, lengths, counts=None, causal: bool = True,
                         scale: float | None = None, out=None, workspace=None, stream=None):
    """Attention of a step's new tokens over a paged cache held in 4 bits:
    sequence b has ``lengths[b]`` cached tokens, of which the last
    ``counts[b]`` are new, and ``q[b, s]`` for s < counts[b] are their queries
    (each sees the tokens up to its own; without ``causal``, all). The heads of
    q share the caches' heads in groups.

    q: (B, S, heads, dim) GPU tensor, float32/float16/bfloat16, any strides
    with consecutive lanes, heads a multiple of the caches'.
    k_cache, v_cache: :class:`RopeCache` of 4 bits, filled by
    :func:`rope_cache_write`.
    block_table: int32 (B, columns); lengths: int32 (B); counts: int32 (B) or
    None: S.
    scale: of the products with k, positive; dim ** -0.5 when None.
    workspace: a contiguous GPU tensor of at least
    ``rope_cache_attention_workspace(B, S, heads, cache heads, v's dim)``
    bytes, 16-byte aligned, that no other call uses meanwhile; None allocates
    one.

    Returns ``out``, (B, S, heads, v's dim) of q's type (allocated when None,
    then zero past each sequence's count; a given one keeps its bytes there). A
    query that sees no token gives zeros. Long sequences are summed in parts,
    whose size follows from the lengths of the whole batch. No gradient passes through the call:
    tensors that need one are refused (while gradients are enabled)."""
    import torch
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise ValueError("q must be a 4-D torch.Tensor (B, S, heads, dim)")
    code, dev = _dtype_code(q), q.device
    if q.numel() and not q.is_cuda:
        raise ValueError("q must be a GPU tensor")
    if not isinstance(k_cache, RopeCache) or not isinstance(v_cache, RopeCache):
        raise TypeError("k_cache and v_cache must be RopeCache objects")
    if k_cache._device != dev or v_cache._device != dev:
        raise ValueError(f"k_cache and v_cache must be on {dev}")
    B, S, heads, dim = q.shape
    if not isinstance(block_table, torch.Tensor) or block_table.dtype != torch.int32 or block_table.dim() != 2 or \
            block_table.shape[0] != B:
        raise ValueError("block_table must be an int32 tensor (B, columns)")
    cols = block_table.shape[1]
    if cols > 1 and block_table.stride(1) != 1:
        raise ValueError("block_table: the pages of a sequence must be consecutive")
    if block_table.device != dev:
        raise ValueError(f"block_table must be on {dev}")
    at_lengths = _array("lengths", lengths, torch.Tensor, torch.int32, (B,), dev)
    at_counts = None if counts is None else _array("counts", counts, torch.Tensor, torch.int32, (B,), dev)
    _refuse_differentiated("rope_cache_attention", ("q", "out"), (q, out) + k_cache._tensors + v_cache._tensors)
    kv_heads, v_dim = k_cache._words[5], v_cache._words[6]
    given = out is not None
    if given:
        if not isinstance(out, torch.Tensor) or out.shape != (B, S, heads, v_dim):
            raise ValueError(f"out must be a {(B, S, heads, v_dim)} tensor")
        if out.dtype != q.dtype or out.device != dev:
            raise ValueError(f"out must be {q.dtype} on {dev}")
    if out is None or workspace is None:
        with _allocating_on(stream, dev) if stream is not None and q.is_cuda else _NOTHING:
            if out is None:
                make = torch.empty if counts is None else torch.zeros
                out = make(B, S, heads, v_dim, dtype=q.dtype, device=dev)
            if workspace is None:
                need = rope_cache_attention_workspace(B, S, heads, kv_heads, v_dim)
                workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    if not isinstance(workspace, torch.Tensor) or not workspace.is_contiguous() or workspace.device != dev:
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    handle, current = _on_device(q, stream)
    with current:
        st = _words_entry("rope_cache_attention")(
            B, S, code, _rows("out", out), _rows("q", q), k_cache._words, v_cache._words, block_table.data_ptr() or None,
            cols, block_table.stride(0), at_lengths, at_counts, dim ** -0.5 if scale is None and dim else scale or 0.0,
            1 if causal else 0, workspace.data_ptr() or None, workspace.nbytes, handle)
    if st != ROPE_OK:
        raise RopeError(st, last_error())
    if given:
        _TORCH[2]((out,))
    return out


# ------------------------------------------------- norms of query and key heads with their rotation

def _norm_weights(q, k, q_weight, k_weight):
    """(pointer, pointer, type) of the weights of a norm's heads."""
    import torch
    types = set()
    ptrs = []
    for name, w, x in (("q_weight", q_weight, q), ("k_weight", k_weight, k)):
        if w is None:
            ptrs.append(None)
            continue
        if x is None:
            raise ValueError("k_weight goes with k")
        if not isinstance(w, torch.Tensor) or w.dim() != 1 or w.shape[0] != x.shape[3] or not w.is_contiguous():
            raise ValueError(f"{name} must be a contiguous tensor ({x.shape[3]})")
        if w.device != x.device:
            raise ValueError(f"{name} must be on {x.device}")
        types.add(_dtype_code(w))
        ptrs.append(w.data_ptr() or None)
    if len(types) > 1:
        raise TypeError("q_weight and k_weight must share a dtype")
    return (*ptrs, types.pop() if types else 0)


def _norm_rows(name, t, like):
    """Rows beside those of q or k: the same shape, type and device."""
    import torch
    if not isinstance(t, torch.Tensor) or t.shape != like.shape or t.dtype != like.dtype or t.device != like.device:
        raise ValueError(f"{name} must be a {tuple(like.shape)} {like.dtype} tensor on {like.device}")
    return _rows(name, t)


def _new_rows(like):
    """A new contiguous tensor of the same shape, and its rows."""
    b, s, n, d = like.shape
    t = like.new_empty(like.shape)
    return t, _RowsWords(t.data_ptr(), n, d, s * n * d, n * d, d)


def _norm_args(q, k, names=("q", "k")):
    import torch
    for name, t in zip(names, (q, k)):
        if t is None and name != names[0]:
            continue
        if not isinstance(t, torch.Tensor) or t.dim() != 4:
            raise ValueError(f"{name} must be a 4-D torch.Tensor (B, S, heads, dim)")
        if t.numel() and not t.is_cuda:
            raise ValueError(f"{name} must be a GPU tensor")
    if k is not None and (k.dtype != q.dtype or k.device != q.device or k.shape[:2] != q.shape[:2]):
        raise ValueError("k must have q's tokens, type and device")


def rope_qk_norm_fwd(q, k, q_weight=None, k_weight=None, positions=None, inv_freq=None, rotary_mode="interleave",
                     partial_slice=None, eps: float = 1e-6, q_out=None, k_out=None, pair_axes=None, table_dtype=None,
                     stream=None):
    """RMS norms of the heads of q and k, and their rotation, in one pass: each
    row x of the last dimension becomes ``x / sqrt(mean(x^2) + eps) * weight``
    with its slice ``[start, end)`` rotated from positions, in fp32, rounded
    once.

    q, k: (B, S, heads, dim) GPU tensors of one type, any strides with
    consecutive lanes (slices of a fused projection's output); k may be None.
    q_weight, k_weight: (dim) tensors of one of the three types, or None: ones.
    positions, inv_freq, rotary_mode, partial_slice, pair_axes, table_dtype: as
    in :func:`rope_cache_write`; positions None: nothing is rotated.
    q_out, k_out: where the results go: tensors of q's and k's shapes, which
    may be q and k themselves (in place); new contiguous ones when None.

    Returns (q_out, k_out). No gradient passes through the call: tensors that
    need one are refused (while gradients are enabled; :func:`qk_norm_rotary`
    gives them)."""
    import torch
    _norm_args(q, k)
    ptrs = _norm_weights(q, k, q_weight, k_weight)
    _refuse_differentiated("rope_qk_norm_fwd", ("q", "k", "q_weight", "k_weight", "q_out", "k_out"),
                           (q, k, q_weight, k_weight, q_out, k_out))
    given = q_out is not None or k_out is not None
    if k is None and k_out is not None:
        raise ValueError("k_out goes with k")
    code = _dtype_code(q)
    rows_q = _rows("q", q)
    rows_k = None if k is None else _rows("k", k)
    turn = _turn_args(positions, inv_freq, pair_axes, rotary_mode, partial_slice, table_dtype, code, q.device)
    written = () if not given else tuple(t for t in (q_out, k_out) if t is not None)
    rows_qo = None if q_out is None else _norm_rows("q_out", q_out, q)
    rows_ko = None if k_out is None else _norm_rows("k_out", k_out, k)
    if q_out is None or (k_out is None and k is not None):
        with _allocating_on(stream, q.device) if stream is not None and q.is_cuda else _NOTHING:
            if q_out is None:
                q_out, rows_qo = _new_rows(q)
            if k is not None and k_out is None:
                k_out, rows_ko = _new_rows(k)
    handle, current = _on_device(q, stream)
    with current:
        st = _words_entry("rope_qk_norm_fwd")(q.shape[0], q.shape[1], code, rows_qo, rows_ko, rows_q, rows_k, *ptrs, eps,
                                              *turn, handle)
    if st != ROPE_OK:
        raise RopeError(st, last_error())
    if given:
        _TORCH[2](written)
    return q_out, k_out


def rope_qk_norm_workspace(dim: int) -> int:
    """Bytes of workspace that :func:`rope_qk_norm_bwd` needs for heads of
    ``dim`` lanes."""
    return library().rope_qk_norm_workspace(dim)


def rope_qk_norm_bwd(q_grad, k_grad, q, k, q_weight=None, k_weight=None, positions=None, inv_freq=None,
                     rotary_mode="interleave", partial_slice=None, eps: float = 1e-6, dq=None, dk=None,
                     weight_grads: bool = True, pair_axes=None, table_dtype=None, workspace=None, stream=None):
    """Backward of :func:`rope_qk_norm_fwd`: for the gradients q_grad and k_grad
    of its results, (dq, dk, dq_weight, dk_weight). q and k are the forward's
    inputs. dq and dk may be given, q_grad and k_grad themselves among them; a
    weight's gradient is None where the weight is, or without ``weight_grads``.
    workspace: a contiguous GPU tensor of ``rope_qk_norm_workspace(dim)`` bytes,
    16-byte aligned, that no other call uses meanwhile; None allocates one. Not
    recorded by autograd."""
    import torch
    _norm_args(q, k)
    ptrs = _norm_weights(q, k, q_weight, k_weight)
    if k is None and not (k_grad is None and dk is None):
        raise ValueError("k_grad and dk go with k")
    given = dq is not None or dk is not None
    code, dev, none = _dtype_code(q), q.device, k is None
    rows_q, rows_k = _rows("q", q), None if none else _rows("k", k)
    rows_qg, rows_kg = _norm_rows("q_grad", q_grad, q), None if none else _norm_rows("k_grad", k_grad, k)
    rows_dq = None if dq is None else _norm_rows("dq", dq, q)
    rows_dk = None if dk is None else _norm_rows("dk", dk, k)
    turn = _turn_args(positions, inv_freq, pair_axes, rotary_mode, partial_slice, table_dtype, code, dev)
    written = () if not given else tuple(t for t in (dq, dk) if t is not None)
    dw_q = dw_k = None
    at_dq = at_dk = at_space = None
    space = 0
    with _allocating_on(stream, dev) if stream is not None and q.is_cuda else _NOTHING:
        if dq is None:
            dq, rows_dq = _new_rows(q)
        if dk is None and not none:
            dk, rows_dk = _new_rows(k)
        if weight_grads:
            if q_weight is not None:
                dw_q = q_weight.new_empty(q_weight.shape)
                at_dq = dw_q.data_ptr() or None
            if k_weight is not None:
                dw_k = k_weight.new_empty(k_weight.shape)
                at_dk = dw_k.data_ptr() or None
            if dw_q is not None or dw_k is not None:
                if workspace is None:
                    workspace = q.new_empty(rope_qk_norm_workspace(q.shape[3]), dtype=torch.uint8)
                elif not isinstance(workspace, torch.Tensor) or not workspace.is_contiguous() or workspace.device != dev:
                    raise ValueError(f"workspace must be a contiguous tensor on {dev}")
                at_space, space = workspace.data_ptr() or None, workspace.nbytes
    handle, current = _on_device(q, stream)
    with current:
        st = _words_entry("rope_qk_norm_bwd")(q.shape[0], q.shape[1], code, rows_dq, rows_dk, at_dq, at_dk, rows_qg, rows_kg,
                                              rows_q, rows_k, *ptrs, eps, *turn, at_space, space, handle)
    if st != ROPE_OK:
        raise RopeError(st, last_error())
    if given:
        (_TORCH or _autograd())[2](written)
    return dq, dk, dw_q, dw_k


_QK_NORM_FN = None


def _qk_norm_fn():
    """The autograd function of the norms. Its arguments: q, k, their weights,
    positions, inv_freq, and what else the calls take."""
    global _QK_NORM_FN
    if _QK_NORM_FN is not None:
        return _QK_NORM_FN
    import torch

    def lanes(t):
        return t if t is None or t.shape[3] < 2 or t.stride(3) == 1 else t.contiguous()

    class QkNormFn(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, q_weight, k_weight, positions, inv_freq, how):
            ctx.save_for_backward(q, k, q_weight, k_weight, positions, inv_freq)
            ctx.how = how
            mode, sl, eps, pair_axes, table_dtype = how
            return rope_qk_norm_fwd(q, k, q_weight, k_weight, positions, inv_freq, mode, sl, eps, pair_axes=pair_axes,
                                    table_dtype=table_dtype)

        @staticmethod
        @torch.autograd.function.once_differentiable
        def backward(ctx, q_grad, k_grad):
            q, k, q_weight, k_weight, positions, inv_freq = ctx.saved_tensors
            mode, sl, eps, pair_axes, table_dtype = ctx.how
            need = ctx.needs_input_grad
            got = rope_qk_norm_bwd(lanes(q_grad), None if k is None else lanes(k_grad), q, k, q_weight, k_weight,
                                   positions, inv_freq, mode, sl, eps, weight_grads=need[2] or need[3],
                                   pair_axes=pair_axes, table_dtype=table_dtype)
            return *(g if n else None for g, n in zip(got, need)), None, None, None

    _QK_NORM_FN = QkNormFn
    return QkNormFn


def qk_norm_rotary(q, k, q_weight=None, k_weight=None, positions=None, inv_freq=None, rotary_mode="interleave",
                   partial_slice=None, eps: float = 1e-6, pair_axes=None, table_dtype=None):
    """:func:`rope_qk_norm_fwd` recorded for autograd: returns new tensors
    (q, k); gradients go to q, k and both weights, and not to positions and
    inv_freq. Differentiable once, not in forward mode."""
    how = (rotary_mode, None if partial_slice is None else (int(partial_slice[0]), int(partial_slice[1])), eps,
           None if pair_axes is None else tuple(pair_axes), table_dtype)
    return _qk_norm_fn().apply(q, k, q_weight, k_weight, positions, inv_freq, how)


def rope_proj_fwd(x, w, r1, r2, heads: int, rotary_mode="interleave", partial_slice=None, out=None,
                  out_dtype=None, stream=None):
    """Head projection with a rotary epilogue (the C ABI's rope_proj_fwd):
    ``y[b,s,h,:] = rotate(x[b,s,:] @ w[h*Dh:(h+1)*Dh, :].T)`` with each head's
    lanes ``[start, end)`` rotated by the tables, the projection accumulated
    in fp32 and rounded once, after the rotation, to ``out_dtype`` ("ascend-
    transformer-boost 的 MlaPreprocessOperation：MLA 预处理四阶段融合算子深度解析",
    section 3: the Q projection and RoPE stages, fused).

    x: (B, S, K) or (M, K) bf16/fp16; w: (H*Dh, K) of x's dtype (a linear
    layer's weight); r1/r2: 4-D tables broadcasting against (B, S, H, L).
    Returns ``out`` (allocated when None): (B, S, H, Dh) of ``out_dtype``
    (x's dtype by default, or torch.float32). The call is not recorded by
    autograd: the result gives x and w no gradient."""
    import torch
    if isinstance(rotary_mode, str):
        if rotary_mode not in MODES:
            raise ValueError(f"rotary_mode must be one of {sorted(MODES)}")
        rotary_mode = MODES[rotary_mode]
    for name, t in (("x", x), ("w", w), ("r1", r1), ("r2", r2)):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
    if x.dim() not in (2, 3) or w.dim() != 2:
        raise ValueError("x must be (B, S, K) or (M, K) and w (H*Dh, K)")
    B, S = (1, x.shape[0]) if x.dim() == 2 else (x.shape[0], x.shape[1])
    K = x.shape[-1]
    N = w.shape[0]
    if w.shape[1] != K or heads <= 0 or N % heads:
        raise ValueError(f"w must be (heads*Dh, K={K}), got {tuple(w.shape)} for {heads} heads")
    if w.dtype != x.dtype:
        raise ValueError("x and w must share a dtype")
    if not (x.is_contiguous() and w.is_contiguous()):
        raise ValueError("x and w must be contiguous")
    y_shape = (B, S, heads, N // heads)
    if out is None:
        out = torch.empty(y_shape, dtype=out_dtype or x.dtype, device=x.device)
    elif tuple(out.shape) != y_shape or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous {y_shape} tensor")
    for name, t in (("x", x), ("w", w), ("out", out)):
        if t.numel() and not t.is_cuda:
            raise ValueError(f"{name} must be a GPU tensor")
    dev = x.device
    handle = (torch.cuda.current_stream(dev).cuda_stream if x.is_cuda else None) if stream is None else \
        getattr(stream, "cuda_stream", stream)
    switch = x.is_cuda and dev.index != torch.cuda.current_device()
    with torch.cuda.device(dev) if switch else _nullcontext():
        st = raw_proj_call(out.data_ptr() or None, _dtype_code(out), x.data_ptr() or None, w.data_ptr() or None,
                           _dtype_code(x), y_shape, K, r1.data_ptr() or None, tuple(r1.shape), tuple(r1.stride()),
                           r2.data_ptr() or None, tuple(r2.shape), tuple(r2.stride()),
                           _dtype_code(r1) if r1.dtype == r2.dtype else -1, rotary_mode, partial_slice, handle)
    if st != ROPE_OK:
        raise RopeError(st, last_error())
    return out


def rope_proj_lora_workspace(tokens: int, K: int, rank: int) -> int:
    """Bytes of workspace that :func:`rope_proj_lora_fwd` needs for this many
    tokens."""
    return library().rope_proj_lora_workspace(_I64x4(1, tokens, 1, 1), K, rank)


def _allocating_on(stream, dev):
    """A context in which tensors are allocated for `stream` (a torch stream
    or a raw hipStream_t)."""
    import torch
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream, device=dev) if stream else torch.cuda.default_stream(dev)
    return torch.cuda.stream(stream)


def rope_proj_lora_fwd(x, w, a, b, adapters, r1, r2, heads: int, rotary_mode="interleave", partial_slice=None,
                       scales=None, out=None, out_dtype=None, workspace=None, stream=None):
    """:func:`rope_proj_fwd` for tokens of many requests, each with its own
    low-rank adapter beside the shared weight: ``y[m] = rotate(x[m] @ w.T +
    scales[i] * (x[m] @ a[i].T) @ b[i].T)`` for the token's adapter i.

    x, w, r1, r2, heads, rotary_mode, partial_slice, out, out_dtype: as in
    :func:`rope_proj_fwd`.
    a: (count, rank, K) and b: (count, heads * Dh, rank) contiguous, of x's
    dtype; rank a multiple of 8, at most LORA_RANK_MAX (pad with zeros).
    adapters: int32, one per token (x's shape without K): an index into a and
    b; one outside [0, count), such as -1, adds nothing. Any order.
    scales: float32 (count) or None for ones.
    workspace: a contiguous GPU tensor of at least
    ``rope_proj_lora_workspace(tokens, K, rank)`` bytes, 16-byte aligned, that
    no other call uses meanwhile; None allocates one.
    Returns ``out`` (allocated when None). No gradient passes through the call:
    tensors that need one are refused (while gradients are enabled)."""
    import torch
    if isinstance(rotary_mode, str):
        if rotary_mode not in MODES:
            raise ValueError(f"rotary_mode must be one of {sorted(MODES)}")
        rotary_mode = MODES[rotary_mode]
    for name, t in (("x", x), ("w", w), ("a", a), ("b", b), ("adapters", adapters), ("r1", r1), ("r2", r2)):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
    if x.dim() not in (2, 3) or w.dim() != 2:
        raise ValueError("x must be (B, S, K) or (M, K) and w (H*Dh, K)")
    B, S = (1, x.shape[0]) if x.dim() == 2 else (x.shape[0], x.shape[1])
    K, N = x.shape[-1], w.shape[0]
    if w.shape[1] != K or heads <= 0 or N % heads:
        raise ValueError(f"w must be (heads*Dh, K={K}), got {tuple(w.shape)} for {heads} heads")
    if a.dim() != 3 or b.dim() != 3 or a.shape[2] != K or b.shape[1] != N or a.shape[0] != b.shape[0] or \
            a.shape[1] != b.shape[2]:
        raise ValueError(f"a must be (count, rank, {K}) and b (count, {N}, rank), got {tuple(a.shape)} and "
                         f"{tuple(b.shape)}")
    if w.dtype != x.dtype or a.dtype != x.dtype or b.dtype != x.dtype:
        raise ValueError("x, w, a and b must share a dtype")
    if adapters.dtype != torch.int32 or adapters.numel() != B * S:
        raise ValueError("adapters must be an int32 tensor, one per token")
    if scales is not None and (not isinstance(scales, torch.Tensor) or scales.dtype != torch.float32 or
                               scales.shape != a.shape[:1]):
        raise ValueError("scales must be a float32 tensor (count)")
    _refuse_differentiated("rope_proj_lora_fwd", ("x", "w", "a", "b", "r1", "r2", "scales", "out"),
                           (x, w, a, b, r1, r2, scales, out))
    y_shape = (B, S, heads, N // heads)
    dev = x.device
    count, rank = a.shape[0], a.shape[1]
    if out is not None and tuple(out.shape) != y_shape:
        raise ValueError(f"out must be a contiguous {y_shape} tensor")
    given = out is not None
    # memory made here belongs to the call's stream: the allocator then hands
    # it on only to work behind this call's
    with _allocating_on(stream, dev) if stream is not None and x.is_cuda else _nullcontext():
        if out is None:
            out = torch.empty(y_shape, dtype=out_dtype or x.dtype, device=dev)
        if workspace is None:
            workspace = torch.empty(rope_proj_lora_workspace(B * S, K, rank) if count else 0, dtype=torch.uint8, device=dev)
    for i, t in enumerate((x, w, a, b, adapters, out, workspace, scales)):
        if t is None or (t.is_contiguous() and t.is_cuda and t.device == dev):
            continue
        name = ("x", "w", "a", "b", "adapters", "out", "workspace", "scales")[i]
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if not t.is_cuda and t.numel():
            raise ValueError(f"{name} must be a GPU tensor")
        if t.device != dev:
            raise ValueError(f"{name} must be on {dev}")
    for name, t in (("r1", r1), ("r2", r2)):
        if t.numel() and out.numel() and t.device != dev:
            raise ValueError(f"{name} must be on {dev}")
    lora = RopeLora(a.data_ptr() or None, b.data_ptr() or None, adapters.data_ptr() or None,
                    None if scales is None else scales.data_ptr() or None, count, rank)
    handle, current = _on_device(x, stream)
    sl = None if partial_slice is None else _I64x2(*partial_slice)
    with current:
        st = library().rope_proj_lora_fwd(
            out.data_ptr() or None, _dtype_code(out), x.data_ptr() or None, w.data_ptr() or None, _dtype_code(x),
            _I64x4(*y_shape), K, lora, r1.data_ptr() or None, _arr4(r1.shape), _arr4(r1.stride()),
            r2.data_ptr() or None, _arr4(r2.shape), _arr4(r2.stride()),
            _dtype_code(r1) if r1.dtype == r2.dtype else -1, rotary_mode, sl, workspace.data_ptr() or None,
            workspace.nbytes, handle)
    if st != ROPE_OK:
        raise RopeError(st, last_error())
    if given:
        _TORCH[2]((out,))
    return out
