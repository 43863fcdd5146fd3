"""Python binding of libpkv -- the paged-KV-cache hot path for GB300.

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  PyTorch supplies device memory and the current stream.  If the
shared library has not been built, importing works but every call raises
``PkvUnavailable``: there is no fallback.

    import paged_kv_cache_pkv_gb300 as pkv
    pkv.write(k_new, v_new, slot_mapping, k_cache, v_cache)
    out = pkv.attend(q, k_cache, v_cache, block_tables, seq_lens, query_start_loc, scale)
"""

from __future__ import annotations

import ctypes
import os

import torch

__all__ = [
    "PkvError", "PkvUnavailable", "lib", "open_library", "library_path", "Desc", "write", "attend",
    "workspace_size", "get_last_error", "launch_count", "Trace", "PagePool", "KERNELS",
    "export_pages", "import_pages", "write_fp8", "attend_fp8", "workspace_size_fp8",
    "write_rope", "write_rope_fp8", "write_latent", "attend_latent", "workspace_size_latent",
    "make_desc", "make_latent_desc", "Rope",
    "STATUS_BAD_SLOT", "STATUS_BAD_BLOCK", "STATUS_BAD_QUERY", "STATUS_TIMEOUT", "STATUS_BAD_POSITION",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
library_path = os.environ.get("PKV_LIBRARY", os.path.join(_HERE, "libpkv.so"))

STATUS_BAD_SLOT, STATUS_BAD_BLOCK, STATUS_BAD_QUERY, STATUS_TIMEOUT = 0x1, 0x2, 0x4, 0x8
STATUS_BAD_POSITION = 0x10
KERNELS = {"write": 0, "plan": 1, "decode": 2, "merge": 3, "prefill": 4, "latent": 5}
LATENT_DIM, LATENT_ROPE = 512, 64
LATENT_ROW = LATENT_DIM + LATENT_ROPE


class PkvError(RuntimeError):
    def __init__(self, code, what=""):
        self.code = code
        msg = _lib.pkv_strerror(code).decode() if _lib is not None else str(code)
        super().__init__(f"{what}: {msg} (code {code})" if what else f"{msg} (code {code})")


class PkvUnavailable(RuntimeError):
    pass


class Desc(ctypes.Structure):
    _fields_ = [("num_blocks", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("num_q_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("max_blocks_per_seq", ctypes.c_int32)]


class Rope(ctypes.Structure):
    _fields_ = [("cos_sin", ctypes.c_void_p), ("max_position", ctypes.c_int32),
                ("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32)]


_vp, _i32, _i64, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
_SIGS = {
    "pkv_write": (ctypes.c_int, [_vp, _vp, _vp, _i64, _vp, _vp, ctypes.POINTER(Desc), _vp]),
    "pkv_attend_workspace_size": (ctypes.c_int, [ctypes.POINTER(Desc), _i32, _i32, _i32, ctypes.POINTER(_sz)]),
    "pkv_attend": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, ctypes.c_float,
                                  _vp, _vp, _sz, ctypes.POINTER(Desc), _vp]),
    "pkv_attend_static": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32,
                                         ctypes.c_float, _vp, ctypes.POINTER(Desc), _vp]),
    "pkv_write_fp8": (ctypes.c_int, [_vp, _vp, _vp, _i64, _vp, _vp, _vp, _vp, ctypes.POINTER(Desc), _vp]),
    "pkv_attend_fp8_workspace_size": (ctypes.c_int, [ctypes.POINTER(Desc), _i32, _i32, _i32, ctypes.POINTER(_sz)]),
    "pkv_attend_fp8": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, ctypes.c_float,
                                      _vp, _vp, _sz, ctypes.POINTER(Desc), _vp]),
    "pkv_write_rope": (ctypes.c_int, [_vp, _vp, _vp, _i64, _i64, _i64, _vp, _vp, _i64, ctypes.POINTER(Rope), _vp,
                                      _vp, _vp, ctypes.POINTER(Desc), _vp]),
    "pkv_write_rope_fp8": (ctypes.c_int, [_vp, _vp, _vp, _i64, _i64, _i64, _vp, _vp, _i64, ctypes.POINTER(Rope), _vp,
                                          _vp, _vp, _vp, _vp, ctypes.POINTER(Desc), _vp]),
    "pkv_write_latent": (ctypes.c_int, [_vp, _vp, _vp, _i64, _i64, _i64, _i64, _vp, _vp, _i64, ctypes.POINTER(Rope),
                                        _vp, _vp, ctypes.POINTER(Desc), _vp]),
    "pkv_attend_latent_workspace_size": (ctypes.c_int, [ctypes.POINTER(Desc), _i32, _i32, ctypes.POINTER(_sz)]),
    "pkv_attend_latent": (ctypes.c_int, [_vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, ctypes.c_float, _vp, _vp, _sz,
                                         ctypes.POINTER(Desc), _vp]),
    "pkv_get_last_error": (ctypes.c_int, [_vp, ctypes.POINTER(ctypes.c_uint32)]),
    "pkv_strerror": (ctypes.c_char_p, [ctypes.c_int]),
    "pkv_launch_count": (ctypes.c_uint64, []),
    "pkv_trace_create": (ctypes.c_int, [_i32, ctypes.POINTER(_vp)]),
    "pkv_trace_attach": (ctypes.c_int, [_vp]),
    "pkv_trace_detach": (ctypes.c_int, []),
    "pkv_trace_read": (ctypes.c_int, [_vp, _i32, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(_i64)]),
    "pkv_trace_reset": (ctypes.c_int, [_vp]),
    "pkv_trace_destroy": (ctypes.c_int, [_vp]),
    "pkv_export_pages": (ctypes.c_int, [_vp, _vp, _vp, _i32, _vp, ctypes.POINTER(Desc), _vp]),
    "pkv_import_pages": (ctypes.c_int, [_vp, _vp, _i32, _vp, _vp, ctypes.POINTER(Desc), _vp]),
    "pkv_pool_create": (ctypes.c_int, [_i32, ctypes.POINTER(_vp)]),
    "pkv_pool_destroy": (ctypes.c_int, [_vp]),
    "pkv_pool_alloc": (ctypes.c_int, [_vp, _i32, ctypes.POINTER(_i32)]),
    "pkv_pool_retain": (ctypes.c_int, [_vp, ctypes.POINTER(_i32), _i32]),
    "pkv_pool_release": (ctypes.c_int, [_vp, ctypes.POINTER(_i32), _i32]),
    "pkv_pool_refcount": (ctypes.c_int, [_vp, _i32, ctypes.POINTER(_i32)]),
    "pkv_pool_usage": (ctypes.c_int, [_vp, ctypes.POINTER(_i32), ctypes.POINTER(_i32)]),
    "pkv_pool_make_writable": (ctypes.c_int, [_vp, _i32, _i32, _vp, _vp, ctypes.POINTER(Desc), _vp,
                                              ctypes.POINTER(_i32)]),
}

_lib = None


def open_library(path):
    """A ctypes handle of a build of the library at ``path``, with every
    entry point's signature declared.  Each build loaded this way keeps its
    own device status word, launch count and caches."""
    if not os.path.exists(path):
        raise PkvUnavailable(
            f"{path} is missing: build it with "
            "`python -m paged_kv_cache_pkv_gb300.build` (nvcc, sm_103a)")
    handle = ctypes.CDLL(path)
    for name, (res, args) in _SIGS.items():
        fn = getattr(handle, name)
        fn.restype, fn.argtypes = res, args
    return handle


def lib():
    """The loaded shared library (raises PkvUnavailable if it is not built)."""
    global _lib
    if _lib is None:
        _lib = open_library(library_path)
    return _lib


def _check(code, what):
    if code != 0:
        raise PkvError(code, what)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _stream(device, stream):
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return ctypes.c_void_p(s.cuda_stream)


def _need(t, name, dtype, ndim=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions, got shape {tuple(t.shape)}")


def make_desc(k_cache, num_q_heads, max_blocks_per_seq):
    nb, hkv, p, d = k_cache.shape
    return Desc(nb, p, hkv, num_q_heads, d, max_blocks_per_seq)


def write(k_new, v_new, slot_mapping, k_cache, v_cache, stream=None):
    """Scatter new K/V rows [T, Hkv, D] into the pools [NB, Hkv, P, D] at
    ``slot_mapping`` (int64 [T]; negative = skip).  In place, stream-ordered."""
    for t, n in ((k_new, "k_new"), (v_new, "v_new"), (k_cache, "k_cache"), (v_cache, "v_cache")):
        _need(t, n, torch.bfloat16)
    _need(slot_mapping, "slot_mapping", torch.int64, 1)
    if k_cache.shape != v_cache.shape or k_new.shape != v_new.shape or k_cache.dim() != 4:
        raise ValueError("k/v shapes disagree")
    T = k_new.shape[0]
    if slot_mapping.shape[0] != T or k_new.shape[1:] != (k_cache.shape[1], k_cache.shape[3]):
        raise ValueError("k_new must be [T, Hkv, D] matching the pool and slot_mapping")
    desc = make_desc(k_cache, k_cache.shape[1], 1)
    with torch.cuda.device(k_cache.device):
        _check(lib().pkv_write(_ptr(k_new), _ptr(v_new), _ptr(slot_mapping), T, _ptr(k_cache),
                               _ptr(v_cache), ctypes.byref(desc), _stream(k_cache.device, stream)),
               "pkv_write")


def workspace_size(desc, num_seqs, num_tokens, device=None, shared_prefix_pages=0):
    n = ctypes.c_size_t(0)
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        _check(lib().pkv_attend_workspace_size(ctypes.byref(desc), num_seqs, num_tokens,
                                               int(shared_prefix_pages), ctypes.byref(n)),
               "pkv_attend_workspace_size")
    return n.value


def attend(q, k_cache, v_cache, block_tables, seq_lens, query_start_loc, scale, out=None,
           workspace=None, stream=None, max_query_len=0, shared_prefix_pages=0):
    """Paged GQA attention of one continuous batch; returns ``out`` [T, Hq, D].

    ``workspace`` (uint8 CUDA tensor) may be passed to avoid an allocation by
    PyTorch's caching allocator on every call.  ``max_query_len`` is an
    optional host-side upper bound on query rows per sequence (0 = unknown);
    it only selects kernels, never results.  ``shared_prefix_pages`` > 0 says
    the first that many block-table entries of every row are the same pages
    (a common prefix), attended once for all rows (cascade)."""
    _need(q, "q", torch.bfloat16, 3)
    _need(k_cache, "k_cache", torch.bfloat16, 4)
    _need(v_cache, "v_cache", torch.bfloat16, 4)
    _need(block_tables, "block_tables", torch.int32, 2)
    _need(seq_lens, "seq_lens", torch.int32, 1)
    _need(query_start_loc, "query_start_loc", torch.int32, 1)
    T, Hq, D = q.shape
    B = seq_lens.shape[0]
    if query_start_loc.shape[0] != B + 1 or block_tables.shape[0] != B:
        raise ValueError("seq_lens [B], query_start_loc [B+1] and block_tables [B, M] disagree")
    if k_cache.shape != v_cache.shape or k_cache.shape[3] != D:
        raise ValueError("k_cache/v_cache/q shapes disagree")
    desc = make_desc(k_cache, Hq, block_tables.shape[1])
    if out is None:
        out = torch.empty_like(q)
    else:
        _need(out, "out", torch.bfloat16, 3)
        if out.shape != q.shape:
            raise ValueError("out must have q's shape")
    need = workspace_size(desc, B, T, q.device, shared_prefix_pages)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    else:
        _need(workspace, "workspace", torch.uint8)
        if workspace.numel() < need:
            raise ValueError(f"workspace needs {need} bytes, got {workspace.numel()}")
    with torch.cuda.device(q.device):
        _check(lib().pkv_attend(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), _ptr(seq_lens),
                                _ptr(query_start_loc), B, T, int(max_query_len), int(shared_prefix_pages),
                                float(scale), _ptr(out),
                                _ptr(workspace), workspace.numel(), ctypes.byref(desc),
                                _stream(q.device, stream)),
               "pkv_attend")
    return out


def _need_fp8_pool(k_cache, v_cache, k_scale, v_scale):
    for t, n in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        _need(t, n, torch.uint8, 4)
    for t, n in ((k_scale, "k_scale"), (v_scale, "v_scale")):
        _need(t, n, torch.uint8, 3)
    if k_cache.shape != v_cache.shape or k_scale.shape != v_scale.shape or \
            tuple(k_scale.shape) != tuple(k_cache.shape[:3]):
        raise ValueError("FP8 pools must be codes [NB, Hkv, P, D] and scales [NB, Hkv, P]")


def write_fp8(k_new, v_new, slot_mapping, k_cache, v_cache, k_scale, v_scale, stream=None):
    """pkv_write into FP8 pages: new bf16 rows [T, Hkv, D] are encoded as E4M3
    codes (uint8 pools [NB, Hkv, P, D]) with one power-of-two scale byte per
    row (uint8 [NB, Hkv, P]).  In place, stream-ordered."""
    _need(k_new, "k_new", torch.bfloat16, 3)
    _need(v_new, "v_new", torch.bfloat16, 3)
    _need(slot_mapping, "slot_mapping", torch.int64, 1)
    _need_fp8_pool(k_cache, v_cache, k_scale, v_scale)
    T = k_new.shape[0]
    if k_new.shape != v_new.shape or slot_mapping.shape[0] != T or \
            k_new.shape[1:] != (k_cache.shape[1], k_cache.shape[3]):
        raise ValueError("k_new must be [T, Hkv, D] matching the pool and slot_mapping")
    desc = make_desc(k_cache, k_cache.shape[1], 1)
    with torch.cuda.device(k_cache.device):
        _check(lib().pkv_write_fp8(_ptr(k_new), _ptr(v_new), _ptr(slot_mapping), T, _ptr(k_cache),
                                   _ptr(v_cache), _ptr(k_scale), _ptr(v_scale), ctypes.byref(desc),
                                   _stream(k_cache.device, stream)),
               "pkv_write_fp8")


def workspace_size_fp8(desc, num_seqs, num_tokens, device=None, shared_prefix_pages=0):
    """Workspace bytes attend_fp8 needs for a batch of this size."""
    n = _sz(0)
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        _check(lib().pkv_attend_fp8_workspace_size(ctypes.byref(desc), int(num_seqs), int(num_tokens),
                                                   int(shared_prefix_pages), ctypes.byref(n)),
               "pkv_attend_fp8_workspace_size")
    return n.value


def attend_fp8(q, k_cache, v_cache, k_scale, v_scale, block_tables, seq_lens, query_start_loc, scale,
               out=None, workspace=None, stream=None, max_query_len=0, shared_prefix_pages=0):
    """attend() over FP8 pages (codes and per-row scale bytes as written by
    write_fp8): long query chunks on the tensor-core prefill kernel, the rest
    on split-KV; max_query_len and shared_prefix_pages as in attend()."""
    _need(q, "q", torch.bfloat16, 3)
    _need_fp8_pool(k_cache, v_cache, k_scale, v_scale)
    _need(block_tables, "block_tables", torch.int32, 2)
    _need(seq_lens, "seq_lens", torch.int32, 1)
    _need(query_start_loc, "query_start_loc", torch.int32, 1)
    T, Hq, D = q.shape
    B = seq_lens.shape[0]
    if query_start_loc.shape[0] != B + 1 or block_tables.shape[0] != B:
        raise ValueError("seq_lens [B], query_start_loc [B+1] and block_tables [B, M] disagree")
    if k_cache.shape[3] != D:
        raise ValueError("k_cache/q shapes disagree")
    desc = make_desc(k_cache, Hq, block_tables.shape[1])
    if out is None:
        out = torch.empty_like(q)
    else:
        _need(out, "out", torch.bfloat16, 3)
        if out.shape != q.shape:
            raise ValueError("out must have q's shape")
    need = workspace_size_fp8(desc, B, T, q.device, shared_prefix_pages)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
    else:
        _need(workspace, "workspace", torch.uint8)
        if workspace.numel() < need:
            raise ValueError(f"workspace needs {need} bytes, got {workspace.numel()}")
    with torch.cuda.device(q.device):
        _check(lib().pkv_attend_fp8(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale),
                                    _ptr(block_tables), _ptr(seq_lens), _ptr(query_start_loc), B, T,
                                    int(max_query_len), int(shared_prefix_pages), float(scale), _ptr(out),
                                    _ptr(workspace), workspace.numel(), ctypes.byref(desc),
                                    _stream(q.device, stream)),
               "pkv_attend_fp8")
    return out


# The calls below are a few microseconds of GPU work for small batches, so
# their checks are made for speed: one short test a tensor, and the words for
# what is wrong with it only where it fails.


def _index(t, name):
    """The CUDA device that ``t`` is on."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    index = t.get_device()
    if index < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return index


def _take(t, name, dtype, ndim, index):
    """The address of ``t``, a contiguous tensor of this type on device ``index``."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == index and t.dim() == ndim
            and t.is_contiguous()):
        return t.data_ptr()
    _need(t, name, dtype, ndim)
    raise ValueError(f"{name} is on {t.device}, not on device {index} like the cache")


def _take_rows(t, name, tokens, heads, dim, index):
    """(address, token stride) of a bf16 tensor [tokens, heads, dim], or
    [tokens, dim] where heads is 0: a token's elements contiguous, any token
    stride that keeps 16-byte alignment."""
    shape = (tokens, heads, dim) if heads else (tokens, dim)
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} must be a CUDA tensor on the cache's device, got {t.device}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got shape {tuple(t.shape)}")
    stride = t.stride()
    if stride[-1] != 1 or (heads > 1 and stride[1] != dim):
        raise ValueError(f"a token's elements of {name} must be contiguous")
    row = dim * (heads or 1)
    if tokens < 2:
        return t.data_ptr(), row
    if stride[0] < row or stride[0] % 8:
        raise ValueError(f"{name}'s token stride must be a multiple of 8 elements and no less than a token")
    return t.data_ptr(), stride[0]


def _new(shape, dtype, device, stream):
    """An uninitialised tensor that belongs to the stream it is used on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _run(what, fn, index, stream, *args):
    """fn(*args, stream) with device ``index`` current."""
    # the current stream's handle, without the Stream object around it
    handle = torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream
    if torch.cuda.current_device() == index:
        code = fn(*args, handle)
    else:
        with torch.cuda.device(index):
            code = fn(*args, handle)
    if code:
        raise PkvError(code, what)


def _rope(cos_sin, interleaved, index):
    at = _take(cos_sin, "cos_sin", torch.float32, 2, index)
    max_position, dim = cos_sin.shape
    return Rope(at, max_position, dim, 1 if interleaved else 0)


def _write_rope(what, k_new, v_new, positions, cos_sin, slot_mapping, k_cache, pools, index, q, q_out, interleaved,
                stream):
    blocks, hkv, page, D = k_cache.shape
    T = k_new.shape[0] if isinstance(k_new, torch.Tensor) and k_new.dim() else -1
    k, ks = _take_rows(k_new, "k_new", T, hkv, D, index)
    v, vs = _take_rows(v_new, "v_new", T, hkv, D, index)
    pos = _take(positions, "positions", torch.int64, 1, index)
    slots = _take(slot_mapping, "slot_mapping", torch.int64, 1, index)
    if positions.shape[0] != T or slot_mapping.shape[0] != T:
        raise ValueError("k_new, positions and slot_mapping disagree on the number of tokens")
    hq, qs, qp, qo = hkv, 0, None, None
    if q is not None:
        hq = q.shape[1] if isinstance(q, torch.Tensor) and q.dim() == 3 else -1
        qp, qs = _take_rows(q, "q", T, hq, D, index)
        if q_out is None:
            q_out = _new(q.shape, q.dtype, q.device, stream)
        elif q_out.shape != q.shape:
            raise ValueError("q_out must have q's shape")
        qo = _take(q_out, "q_out", torch.bfloat16, 3, index)
    elif q_out is not None:
        raise ValueError("q_out without q")
    rope, desc = _rope(cos_sin, interleaved, index), Desc(blocks, page, hkv, hq, D, 1)
    _run(what, getattr(lib(), what), index, stream, qp, k, v, qs, ks, vs, pos, slots, T, ctypes.byref(rope), qo, *pools,
         ctypes.byref(desc))
    return q_out


def write_rope(k_new, v_new, positions, cos_sin, slot_mapping, k_cache, v_cache, q=None, q_out=None,
               interleaved=False, stream=None):
    """write() with the position rotation on the way: K rows (and the queries
    ``q`` [T, Hq, D], if given) are rotated by their ``positions`` (int64 [T])
    through ``cos_sin`` (fp32 [max_position, rotary_dim]: cosines, then sines;
    rotary_dim a multiple of 16, elements behind it are copied).  Pairs are
    (i, i + rotary_dim/2), or (2i, 2i + 1) with ``interleaved``.  k_new, v_new
    and q may be slices of one projection's output.  Returns the rotated
    queries (``q_out``, which may be a contiguous ``q`` itself), or None."""
    index = _index(k_cache, "k_cache")
    pools = (_take(k_cache, "k_cache", torch.bfloat16, 4, index), _take(v_cache, "v_cache", torch.bfloat16, 4, index))
    if k_cache.shape != v_cache.shape:
        raise ValueError("k_cache and v_cache shapes disagree")
    return _write_rope("pkv_write_rope", k_new, v_new, positions, cos_sin, slot_mapping, k_cache, pools, index, q,
                       q_out, interleaved, stream)


def write_rope_fp8(k_new, v_new, positions, cos_sin, slot_mapping, k_cache, v_cache, k_scale, v_scale, q=None,
                   q_out=None, interleaved=False, stream=None):
    """write_rope into FP8 pages (codes and scale bytes as in write_fp8): the
    rotated fp32 values are rounded once, to E4M3."""
    index = _index(k_cache, "k_cache")
    pools = (_take(k_cache, "k_cache", torch.uint8, 4, index), _take(v_cache, "v_cache", torch.uint8, 4, index),
             _take(k_scale, "k_scale", torch.uint8, 3, index), _take(v_scale, "v_scale", torch.uint8, 3, index))
    shape = k_cache.shape
    if v_cache.shape != shape or k_scale.shape != shape[:3] or v_scale.shape != shape[:3]:
        raise ValueError("FP8 pools must be codes [NB, Hkv, P, D] and scales [NB, Hkv, P]")
    return _write_rope("pkv_write_rope_fp8", k_new, v_new, positions, cos_sin, slot_mapping, k_cache, pools, index, q,
                       q_out, interleaved, stream)


def make_latent_desc(latent_cache, num_heads, max_blocks_per_seq):
    nb, page, row = latent_cache.shape
    return Desc(nb, page, 1, num_heads, row, max_blocks_per_seq)


def write_latent(c_new, k_pe, positions, cos_sin, slot_mapping, latent_cache, q_pe=None, q_out=None,
                 interleaved=False, stream=None):
    """Append one row a token to latent pages [NB, 16, 576]: the latent
    ``c_new`` [T, 512] as it is, and the shared key part ``k_pe`` [T, 64]
    rotated by its position (see write_rope; cos_sin [max_position, 64]).
    With ``q_pe`` [T, H, 64] the queries' rotated part goes into the last 64
    values of ``q_out`` [T, H, 576], whose first 512 are left alone.  c_new,
    k_pe and q_pe may be slices.  Returns q_out, or None."""
    index = _index(latent_cache, "latent_cache")
    pool = _take(latent_cache, "latent_cache", torch.bfloat16, 3, index)
    T = c_new.shape[0] if isinstance(c_new, torch.Tensor) and c_new.dim() else -1
    c, cs = _take_rows(c_new, "c_new", T, 0, LATENT_DIM, index)
    k, ks = _take_rows(k_pe, "k_pe", T, 0, LATENT_ROPE, index)
    pos = _take(positions, "positions", torch.int64, 1, index)
    slots = _take(slot_mapping, "slot_mapping", torch.int64, 1, index)
    if positions.shape[0] != T or slot_mapping.shape[0] != T:
        raise ValueError("c_new, positions and slot_mapping disagree on the number of tokens")
    heads, qs, hs, qp, qo = 1, 0, 0, None, None
    if q_pe is not None:
        if not isinstance(q_pe, torch.Tensor) or q_pe.dtype is not torch.bfloat16:
            raise TypeError(f"q_pe must be a {torch.bfloat16} tensor")
        if q_pe.get_device() != index:
            raise ValueError(f"q_pe must be a CUDA tensor on the cache's device, got {q_pe.device}")
        if q_pe.dim() != 3 or q_pe.shape[0] != T or q_pe.shape[2] != LATENT_ROPE or q_pe.stride(2) != 1:
            raise ValueError(f"q_pe must be [tokens, H, {LATENT_ROPE}] with contiguous rows, got shape "
                             f"{tuple(q_pe.shape)}")
        heads = q_pe.shape[1]
        hs = q_pe.stride(1) if heads > 1 else LATENT_ROPE
        qs = q_pe.stride(0) if T > 1 else heads * hs
        if hs < LATENT_ROPE or hs % 8 or qs < (heads - 1) * hs + LATENT_ROPE or qs % 8:
            raise ValueError("q_pe's strides must be multiples of 8 elements and its rows must not overlap")
        if q_out is None:
            q_out = _new((T, heads, LATENT_ROW), torch.bfloat16, q_pe.device, stream)
        elif q_out.shape != (T, heads, LATENT_ROW):
            raise ValueError(f"q_out must be [tokens, H, {LATENT_ROW}]")
        qp, qo = q_pe.data_ptr(), _take(q_out, "q_out", torch.bfloat16, 3, index)
    elif q_out is not None:
        raise ValueError("q_out without q_pe")
    rope, desc = _rope(cos_sin, interleaved, index), make_latent_desc(latent_cache, heads, 1)
    _run("pkv_write_latent", lib().pkv_write_latent, index, stream, c, k, qp, cs, ks, qs, hs, pos, slots, T,
         ctypes.byref(rope), qo, pool, ctypes.byref(desc))
    return q_out


def workspace_size_latent(desc, num_seqs, num_tokens, device=None):
    """Workspace bytes attend_latent needs (make_latent_desc describes the pool)."""
    n = _sz(0)
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        _check(lib().pkv_attend_latent_workspace_size(ctypes.byref(desc), int(num_seqs), int(num_tokens),
                                                      ctypes.byref(n)), "pkv_attend_latent_workspace_size")
    return n.value


def attend_latent(q, latent_cache, block_tables, seq_lens, query_start_loc, scale, out=None, workspace=None,
                  stream=None, max_query_len=0):
    """Absorbed attention over latent pages [NB, 16, 576]: every head of
    ``q`` [T, H, 576] against the one shared row a token, whose first 512
    values are the value.  Returns ``out`` [T, H, 512].  The other arguments
    are as in attend(); max_query_len (0 = unknown) selects tile sizes, which
    may change results in their last bits, never which rows are right."""
    index = _index(latent_cache, "latent_cache")
    pool = _take(latent_cache, "latent_cache", torch.bfloat16, 3, index)
    qp = _take(q, "q", torch.bfloat16, 3, index)
    tables = _take(block_tables, "block_tables", torch.int32, 2, index)
    lens = _take(seq_lens, "seq_lens", torch.int32, 1, index)
    qsl = _take(query_start_loc, "query_start_loc", torch.int32, 1, index)
    T, H, row = q.shape
    B = seq_lens.shape[0]
    if query_start_loc.shape[0] != B + 1 or block_tables.shape[0] != B:
        raise ValueError("seq_lens [B], query_start_loc [B+1] and block_tables [B, M] disagree")
    if latent_cache.shape[2] != row:
        raise ValueError("latent_cache and q rows disagree")
    desc = make_latent_desc(latent_cache, H, block_tables.shape[1])
    if out is None:
        out = _new((T, H, LATENT_DIM), torch.bfloat16, q.device, stream)
    elif out.shape != (T, H, LATENT_DIM):
        raise ValueError(f"out must be [tokens, H, {LATENT_DIM}]")
    if workspace is None:
        workspace = _new((workspace_size_latent(desc, B, T, index),), torch.uint8, q.device, stream)
    _run("pkv_attend_latent", lib().pkv_attend_latent, index, stream, qp, pool, tables, lens, qsl, B, T,
         int(max_query_len), scale, _take(out, "out", torch.bfloat16, 3, index),
         _take(workspace, "workspace", torch.uint8, 1, index), workspace.numel(), ctypes.byref(desc))
    return out


def export_pages(k_cache, v_cache, pages, out=None, stream=None):
    """Copy whole pages into a contiguous buffer [n, 2, Hkv, 16, 128] bf16
    (device or pinned host tensor); returns it."""
    _need(pages, "pages", torch.int32, 1)
    n = pages.shape[0]
    if out is None:
        out = torch.empty((n, 2) + tuple(k_cache.shape[1:]), dtype=torch.bfloat16, device=k_cache.device)
    if out.dtype != torch.bfloat16 or not out.is_contiguous() or out.numel() != n * 2 * k_cache[0].numel():
        raise ValueError("out must be a contiguous bf16 tensor of n * 2 pages")
    desc = make_desc(k_cache, k_cache.shape[1], 1)
    with torch.cuda.device(k_cache.device):
        _check(lib().pkv_export_pages(_ptr(k_cache), _ptr(v_cache), _ptr(pages), n, _ptr(out),
                                      ctypes.byref(desc), _stream(k_cache.device, stream)), "pkv_export_pages")
    return out


def import_pages(src, pages, k_cache, v_cache, stream=None):
    """Copy a buffer written by export_pages into the listed pool pages."""
    _need(pages, "pages", torch.int32, 1)
    n = pages.shape[0]
    if src.dtype != torch.bfloat16 or not src.is_contiguous() or src.numel() != n * 2 * k_cache[0].numel():
        raise ValueError("src must be a contiguous bf16 tensor of n * 2 pages")
    desc = make_desc(k_cache, k_cache.shape[1], 1)
    with torch.cuda.device(k_cache.device):
        _check(lib().pkv_import_pages(_ptr(src), _ptr(pages), n, _ptr(k_cache), _ptr(v_cache),
                                      ctypes.byref(desc), _stream(k_cache.device, stream)), "pkv_import_pages")


def get_last_error(device=None, stream=None):
    """Wait for the stream; read and clear the device status bits."""
    flags = ctypes.c_uint32(0)
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with torch.cuda.device(dev):
        _check(lib().pkv_get_last_error(_stream(dev, stream), ctypes.byref(flags)), "pkv_get_last_error")
    return flags.value


def launch_count():
    return int(lib().pkv_launch_count())


class PagePool:
    """Host-side page allocator with reference counts (see pkv_pool_* in pkv.h)."""

    def __init__(self, num_blocks):
        h = ctypes.c_void_p()
        _check(lib().pkv_pool_create(int(num_blocks), ctypes.byref(h)), "pkv_pool_create")
        self._h, self.num_blocks = h, int(num_blocks)

    @staticmethod
    def _arr(pages):
        pages = [int(x) for x in pages]
        return (ctypes.c_int32 * max(1, len(pages)))(*pages), len(pages)

    def alloc(self, n):
        buf = (ctypes.c_int32 * max(1, n))()
        _check(lib().pkv_pool_alloc(self._h, int(n), buf), "pkv_pool_alloc")
        return list(buf)[:n]

    def retain(self, pages):
        a, n = self._arr(pages)
        _check(lib().pkv_pool_retain(self._h, a, n), "pkv_pool_retain")

    def release(self, pages):
        a, n = self._arr(pages)
        _check(lib().pkv_pool_release(self._h, a, n), "pkv_pool_release")

    def refcount(self, page):
        c = ctypes.c_int32(0)
        _check(lib().pkv_pool_refcount(self._h, int(page), ctypes.byref(c)), "pkv_pool_refcount")
        return c.value

    def usage(self):
        u, t = ctypes.c_int32(0), ctypes.c_int32(0)
        _check(lib().pkv_pool_usage(self._h, ctypes.byref(u), ctypes.byref(t)), "pkv_pool_usage")
        return u.value, t.value

    def make_writable(self, page, rows, k_cache, v_cache, stream=None):
        """Private copy of a shared page (copy-on-write); returns the page to write."""
        desc = make_desc(k_cache, k_cache.shape[1], 1)
        out = ctypes.c_int32(-1)
        with torch.cuda.device(k_cache.device):
            _check(lib().pkv_pool_make_writable(self._h, int(page), int(rows), _ptr(k_cache), _ptr(v_cache),
                                                ctypes.byref(desc), _stream(k_cache.device, stream),
                                                ctypes.byref(out)), "pkv_pool_make_writable")
        return out.value

    def close(self):
        if self._h:
            lib().pkv_pool_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Trace:
    """Per-kernel device time of the library's launches on this thread."""

    def __init__(self, capacity=4096):
        h = ctypes.c_void_p()
        _check(lib().pkv_trace_create(capacity, ctypes.byref(h)), "pkv_trace_create")
        self._h = h

    def __enter__(self):
        _check(lib().pkv_trace_attach(self._h), "pkv_trace_attach")
        return self

    def __exit__(self, *exc):
        lib().pkv_trace_detach()
        return False

    def read(self, kernel):
        ms, n = ctypes.c_double(0), ctypes.c_int64(0)
        kid = KERNELS[kernel] if isinstance(kernel, str) else int(kernel)
        _check(lib().pkv_trace_read(self._h, kid, ctypes.byref(ms), ctypes.byref(n)), "pkv_trace_read")
        return ms.value, n.value

    def reset(self):
        _check(lib().pkv_trace_reset(self._h), "pkv_trace_reset")

    def close(self):
        if self._h:
            lib().pkv_trace_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
