"""Python binding of the ``il`` C ABI (``include/il.h``): argument marshalling only.

Every computation runs in ``libil.so``'s CUDA kernels.  There is no CPU
fallback: if the library is missing or no sm_103a device is current, the calls
raise :class:`ILError`.

The names follow the C ABI: :func:`upload_weight` (oxinfer ``Backend::upload``),
:func:`matmul_batch` (``Backend::matmul``: all jobs over one shared ``x``),
:func:`free_weight`, :func:`weight_bytes` (``WeightRef::bytes``),
:func:`dequantize_weight` (test hook), :func:`get_stats`.
"""
from __future__ import annotations

import ctypes
import os
import threading

import numpy as np

__all__ = ["ILError", "Weight", "FORMATS", "IL_BF16", "IL_Q8", "IL_Q4", "load", "build",
           "upload_weight", "matmul_batch", "matmul_batch_ptr", "matmul_batch_noalloc_ptr", "free_weight", "weight_bytes",
           "dequantize_weight", "check_device_status", "release_scratch", "get_stats", "reset_stats", "last_error",
           "version", "LIB_PATH", "STATUS", "KVCache", "kv_cache", "kv_extend", "kv_append", "kv_read", "kv_attend"]

IL_BF16, IL_Q8, IL_Q4 = 0, 1, 2
FORMATS = {"bf16": IL_BF16, "q8": IL_Q8, "q4": IL_Q4}
STATUS = {0: "IL_OK", -1: "IL_ERR_ARG", -2: "IL_ERR_SHAPE", -3: "IL_ERR_FORMAT",
          -4: "IL_ERR_HANDLE", -5: "IL_ERR_OOM", -6: "IL_ERR_CUDA",
          -7: "IL_ERR_DEVICE_TIMEOUT", -8: "IL_ERR_UNSUPPORTED"}

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libil.so")


class ILError(RuntimeError):
    """An ``il_*`` call failed; ``code`` is the negative ``il_status``."""

    def __init__(self, code: int, msg: str):
        super().__init__(f"{STATUS.get(code, code)}: {msg}")
        self.code = code


class _Job(ctypes.Structure):
    _fields_ = [("w", ctypes.c_void_p), ("n_out", ctypes.c_int64), ("y", ctypes.c_void_p)]


class _Stats(ctypes.Structure):
    _fields_ = [(n, ctypes.c_uint64) for n in
                ("uploads", "upload_bytes", "batches", "jobs", "launches", "weight_bytes",
                 "flops", "errors", "profiled_batches", "device_ns")]


class _KV(ctypes.Structure):
    _fields_ = ([("format", ctypes.c_int32), ("page_size", ctypes.c_int32), ("n_pages", ctypes.c_int64),
                 ("n_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32)]
                + [(n, ctypes.c_void_p) for n in ("k", "v", "k_scale", "v_scale")]
                + [(n, ctypes.c_int64) for n in ("page_stride", "token_stride", "head_stride", "scale_page_stride",
                                                 "scale_token_stride", "scale_head_stride")])


_lib = None
_lock = threading.Lock()


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile ``libil.so`` in-tree with nvcc (sm_103a)."""
    from . import _build
    return _build.build(force=force, verbose=verbose)


def load() -> ctypes.CDLL:
    """Load ``libil.so``; raises :class:`ILError` when it has not been built."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise ILError(-8, f"{LIB_PATH} is missing: build it with "
                              "shared_input_linear_gb300.build() (nvcc, sm_103a)")
        lib = ctypes.CDLL(LIB_PATH)
        i64, vp, ci = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
        lib.il_upload_weight.argtypes = [ci, vp, i64, i64]
        lib.il_upload_weight.restype = vp
        lib.il_matmul_batch.argtypes = [vp, i64, i64, ctypes.POINTER(_Job), ci, vp]
        lib.il_matmul_batch.restype = ci
        lib.il_matmul_batch_noalloc.argtypes = [vp, i64, i64, ctypes.POINTER(_Job), ci, vp]
        lib.il_matmul_batch_noalloc.restype = ci
        lib.il_matmul_batch_host.argtypes = [vp, i64, i64, ctypes.POINTER(_Job), ci, vp]
        lib.il_matmul_batch_host.restype = ci
        lib.il_upload_gate_up.argtypes = [ci, vp, vp, i64, i64]
        lib.il_upload_gate_up.restype = vp
        lib.il_centroid_head.argtypes = [vp, i64, vp, vp, vp, i64, vp, vp, vp, vp, vp]
        lib.il_centroid_head.restype = ci
        lib.il_kv_extend.argtypes = [i64, i64, vp, vp, vp, i64, i64, vp, i64, vp, vp, vp, vp, i64, vp, vp, vp, vp]
        lib.il_kv_extend.restype = ci
        lib.il_kv_append.argtypes = [vp, vp, i64, vp, i64, vp, i64, vp]
        lib.il_kv_append.restype = ci
        lib.il_kv_read.argtypes = [vp, vp, i64, vp, i64, vp, i64, vp]
        lib.il_kv_read.restype = ci
        lib.il_kv_attend.argtypes = [vp, vp, i64, vp, i64, i64, vp, i64, i64, ctypes.c_float, i64, vp, i64, vp, vp]
        lib.il_kv_attend.restype = ci
        lib.il_weight_is_gate_up.argtypes = [vp]
        lib.il_weight_is_gate_up.restype = ci
        lib.il_free_weight.argtypes = [vp]
        lib.il_free_weight.restype = None
        lib.il_weight_bytes.argtypes = [vp]
        lib.il_weight_bytes.restype = i64
        lib.il_weight_info.argtypes = [vp, ctypes.POINTER(ci), ctypes.POINTER(i64),
                                       ctypes.POINTER(i64)]
        lib.il_weight_info.restype = ci
        lib.il_dequantize_weight.argtypes = [vp, vp, vp]
        lib.il_dequantize_weight.restype = ci
        lib.il_check_device_status.argtypes = [vp]
        lib.il_check_device_status.restype = ci
        lib.il_release_scratch.argtypes = [vp]
        lib.il_release_scratch.restype = ci
        lib.il_last_error.argtypes = []
        lib.il_last_error.restype = ctypes.c_char_p
        lib.il_last_status.argtypes = []
        lib.il_last_status.restype = ci
        lib.il_get_stats.argtypes = [ctypes.POINTER(_Stats)]
        lib.il_get_stats.restype = ci
        lib.il_reset_stats.argtypes = []
        lib.il_reset_stats.restype = None
        lib.il_version.argtypes = []
        lib.il_version.restype = ci
        _lib = lib
        return lib


def last_error() -> str:
    return load().il_last_error().decode()


def _check(rc: int) -> int:
    if rc != 0:
        raise ILError(rc, last_error())
    return rc


def version() -> int:
    return load().il_version()


class Weight:
    """Owner of one device weight handle (freed on :meth:`free` or garbage collection)."""

    def __init__(self, handle: int, fmt: int, n_out: int, n_in: int, gate_up: bool = False):
        self.handle = handle
        self.fmt = fmt
        self.n_out = n_out      # columns of a job's output (the width of h for gate+up)
        self.n_in = n_in
        self.gate_up = gate_up

    @property
    def bytes(self) -> int:
        return weight_bytes(self)

    def free(self) -> None:
        if self.handle:
            load().il_free_weight(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


def _fmt(fmt) -> int:
    return FORMATS[fmt] if isinstance(fmt, str) else int(fmt)


def upload_weight(fmt, host, n_out: int, n_in: int) -> Weight:
    """``il_upload_weight``: ``host`` is a host buffer (numpy) in the documented layout."""
    buf = np.ascontiguousarray(host)
    lib = load()
    h = lib.il_upload_weight(_fmt(fmt), buf.ctypes.data, int(n_out), int(n_in))
    if not h:
        raise ILError(lib.il_last_status(), last_error())
    return Weight(h, _fmt(fmt), int(n_out), int(n_in))


def upload_gate_up(fmt, gate, up, n_out: int, n_in: int) -> Weight:
    """``il_upload_gate_up``: ``gate`` and ``up`` are host buffers of one shape in the
    layout of :func:`upload_weight`; a job of the result writes ``h = gelu(g) * u``,
    ``[t][n_out]``."""
    g = np.ascontiguousarray(gate)
    u = np.ascontiguousarray(up)
    lib = load()
    h = lib.il_upload_gate_up(_fmt(fmt), g.ctypes.data, u.ctypes.data, int(n_out), int(n_in))
    if not h:
        raise ILError(lib.il_last_status(), last_error())
    return Weight(h, _fmt(fmt), int(n_out), int(n_in), gate_up=True)


def is_gate_up(w) -> int:
    """``il_weight_is_gate_up``: 1, 0, or -1 for an invalid handle."""
    return int(load().il_weight_is_gate_up(w.handle if isinstance(w, Weight) else w))


def centroid_head(x, centroids: Weight, embed: Weight, ordering, top_k: int, token_out, score_out=None,
                  selected_out=None, scores_out=None, stream=None) -> None:
    """``il_centroid_head`` on torch CUDA tensors: ``x`` fp32 ``[h]``, ``ordering`` int32/uint32
    ``[vocab]``, ``token_out`` 32-bit ``[1]``; the optional outputs as documented in
    ``include/il.h``.  Enqueued on ``stream`` (default: the current torch stream)."""
    def ptr(t):
        return 0 if t is None else t.data_ptr()
    if not x.is_contiguous() or not ordering.is_contiguous():
        raise ILError(-1, "x and ordering must be contiguous")
    _check(load().il_centroid_head(ptr(x), int(x.numel()), centroids.handle, embed.handle, ptr(ordering),
                                   int(top_k), ptr(token_out), ptr(score_out), ptr(selected_out),
                                   ptr(scores_out), _stream_ptr(stream)))


def free_weight(w: Weight) -> None:
    w.free()


def weight_bytes(w: Weight) -> int:
    return int(load().il_weight_bytes(w.handle))


def _stream_ptr(stream) -> int:
    if stream is None:
        import torch
        # the handle of torch.cuda.current_stream() without the object (3 us on the host)
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        return torch.cuda.current_stream().cuda_stream if raw is None else raw(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def matmul_batch_ptr(x_ptr: int, t: int, n_in: int, jobs, stream_ptr: int) -> int:
    """``il_matmul_batch`` on raw device pointers; ``jobs`` is ``[(Weight|handle, n_out, y_ptr)]``."""
    arr = (_Job * max(1, len(jobs)))()
    for i, (w, n_out, y) in enumerate(jobs):
        arr[i].w = w.handle if isinstance(w, Weight) else w
        arr[i].n_out = int(n_out)
        arr[i].y = int(y)
    return _check(load().il_matmul_batch(x_ptr, int(t), int(n_in), arr, len(jobs), stream_ptr))


def prepare_jobs(jobs):
    """A reusable ``il_job`` array for ``[(Weight|handle, n_out, y_ptr)]``: marshal once,
    call :func:`matmul_batch_prepared` many times."""
    arr = (_Job * max(1, len(jobs)))()
    for i, (w, n_out, y) in enumerate(jobs):
        arr[i].w = w.handle if isinstance(w, Weight) else w
        arr[i].n_out = int(n_out)
        arr[i].y = int(y)
    return arr, len(jobs)


def matmul_batch_prepared(x_ptr: int, t: int, n_in: int, prepared, stream_ptr: int) -> int:
    """``il_matmul_batch`` with a job array from :func:`prepare_jobs`."""
    arr, n = prepared
    return _check(load().il_matmul_batch(x_ptr, int(t), int(n_in), arr, n, stream_ptr))


def matmul_batch_noalloc_ptr(x_ptr: int, t: int, n_in: int, jobs, stream_ptr: int) -> int:
    """``il_matmul_batch_noalloc`` on raw device pointers (same ``jobs`` form as
    :func:`matmul_batch_ptr`).  The library allocates no device memory for it;
    see ``include/il.h`` for the fixed scratch limit."""
    arr = (_Job * max(1, len(jobs)))()
    for i, (w, n_out, y) in enumerate(jobs):
        arr[i].w = w.handle if isinstance(w, Weight) else w
        arr[i].n_out = int(n_out)
        arr[i].y = int(y)
    return _check(load().il_matmul_batch_noalloc(x_ptr, int(t), int(n_in), arr, len(jobs), stream_ptr))


def matmul_batch(x, jobs, stream=None) -> None:
    """``il_matmul_batch`` on torch CUDA tensors.

    ``x``: fp32 ``[t][n_in]`` contiguous; ``jobs``: ``[(Weight, y)]`` with ``y``
    fp32 ``[t][n_out]`` contiguous, overwritten.  Enqueued on ``stream`` (default:
    the current torch stream).
    """
    if x.dim() != 2 or not x.is_contiguous():
        raise ILError(-1, "x must be a contiguous [t][n_in] tensor")
    t, n_in = x.shape
    lst = []
    for w, y in jobs:
        if not y.is_contiguous():
            raise ILError(-1, "y must be contiguous")
        lst.append((w, w.n_out, y.data_ptr()))
    matmul_batch_ptr(x.data_ptr(), t, n_in, lst, _stream_ptr(stream))


def matmul_batch_host_prepared(x_ptr: int, t: int, n_in: int, prepared, stream_ptr: int) -> int:
    """``il_matmul_batch_host`` with a job array from :func:`prepare_jobs` whose y
    pointers are host addresses; ``x_ptr`` is a host address too."""
    arr, n = prepared
    return _check(load().il_matmul_batch_host(x_ptr, int(t), int(n_in), arr, n, stream_ptr))


def matmul_batch_host(x, jobs, stream=None, sync: bool = True) -> None:
    """``il_matmul_batch_host`` on CPU torch tensors (pinned or not).

    ``x``: fp32 ``[t][n_in]`` contiguous; ``jobs``: ``[(Weight, y)]`` with ``y``
    fp32 ``[t][n_out]`` contiguous on the CPU, overwritten.  Enqueued on
    ``stream`` (default: the current torch stream); with ``sync`` the call waits
    for the stream, so ``y`` holds the results when it returns.
    """
    if x.device.type != "cpu" or x.dim() != 2 or not x.is_contiguous():
        raise ILError(-1, "x must be a contiguous [t][n_in] CPU tensor")
    t, n_in = x.shape
    lst = []
    for w, y in jobs:
        if y.device.type != "cpu" or not y.is_contiguous():
            raise ILError(-1, "y must be a contiguous CPU tensor")
        lst.append((w, w.n_out, y.data_ptr()))
    sp = _stream_ptr(stream)
    arr = (_Job * max(1, len(lst)))()
    for i, (w, n_out, y) in enumerate(lst):
        arr[i].w = w.handle if isinstance(w, Weight) else w
        arr[i].n_out = int(n_out)
        arr[i].y = int(y)
    _check(load().il_matmul_batch_host(x.data_ptr(), int(t), int(n_in), arr, len(lst), sp))
    if sync:
        import torch
        if sp:
            torch.cuda.ExternalStream(sp).synchronize()
        else:
            torch.cuda.synchronize()


def dequantize_weight(w: Weight, out, stream=None) -> None:
    """Test hook: every element of ``w`` as fp32 into ``out`` ([n_out][n_in], CUDA;
    [2*n_out][n_in] with gate/up rows interleaved for a gate+up weight)."""
    _check(load().il_dequantize_weight(w.handle, out.data_ptr(), _stream_ptr(stream)))


# ---------------------------------------------------------------------------
# Paged K/V cache
# ---------------------------------------------------------------------------
def _steps(t):
    """Strides of ``t``; 0 for a dimension of one entry, whose stride means nothing."""
    return [st if n > 1 else 0 for n, st in zip(t.shape, t.stride())]


class KVCache:
    """A paged K/V cache in the caller's tensors (``il_kv``); holds references to them.

    ``k``, ``v``: CUDA ``[n_pages][page_size][n_heads][head_dim]`` of one shape and one set of
    strides, the last dimension contiguous; pass ``pool.transpose(1, 2)`` of a pool stored
    head-major.  ``torch.bfloat16`` is IL_BF16; ``torch.int8`` is IL_Q8 with fp32 ``k_scale``,
    ``v_scale`` ``[n_pages][page_size][n_heads][head_dim / 32]``.  :func:`kv_cache` allocates one.
    """

    def __init__(self, k, v, k_scale=None, v_scale=None):
        import torch
        if k.dim() != 4 or k.shape != v.shape or _steps(k) != _steps(v) or k.dtype != v.dtype:
            raise ILError(-1, "k and v must be [n_pages][page_size][n_heads][head_dim] of one shape, stride and dtype")
        if k.dtype not in (torch.bfloat16, torch.int8):
            raise ILError(-3, "the cache must be bfloat16 or int8")
        if k.stride(3) != 1:
            raise ILError(-1, "the last dimension of k and v must be contiguous")
        if not (k.is_cuda and v.is_cuda):
            raise ILError(-1, "k and v must be CUDA tensors")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.n_pages, self.page_size, self.n_heads, self.head_dim = k.shape
        self.format = IL_BF16 if k.dtype == torch.bfloat16 else IL_Q8
        c = self._c = _KV(self.format, self.page_size, self.n_pages, self.n_heads, self.head_dim, k.data_ptr(),
                          v.data_ptr(), None, None, *k.stride()[:3], 0, 0, 0)
        if (self.format == IL_Q8) != (k_scale is not None) or (k_scale is None) != (v_scale is None):
            raise ILError(-1, "an int8 cache needs k_scale and v_scale, a bfloat16 cache has none")
        if k_scale is not None:
            shape = (*k.shape[:3], self.head_dim // 32)
            for t in (k_scale, v_scale):
                if (tuple(t.shape) != shape or t.dtype != torch.float32 or not t.is_cuda
                        or (shape[3] > 1 and t.stride(3) != 1)):
                    raise ILError(-1, f"scales must be CUDA float32 {list(shape)}, the last dimension contiguous")
            if _steps(k_scale)[:3] != _steps(v_scale)[:3]:
                raise ILError(-1, "k_scale and v_scale must have the same strides")
            c.k_scale, c.v_scale = k_scale.data_ptr(), v_scale.data_ptr()
            c.scale_page_stride, c.scale_token_stride, c.scale_head_stride = k_scale.stride()[:3]
        self._ref = ctypes.addressof(c)

    @property
    def bytes(self) -> int:
        """Bytes of the cache's elements and scales."""
        return sum(t.numel() * t.element_size() for t in (self.k, self.v, self.k_scale, self.v_scale) if t is not None)


def kv_cache(fmt, n_pages: int, page_size: int, n_heads: int, head_dim: int, device="cuda") -> KVCache:
    """A zeroed :class:`KVCache`, stored head-major within a page: a head's tokens of one page
    are one contiguous run."""
    import torch
    q8 = _fmt(fmt) == IL_Q8
    if not q8 and _fmt(fmt) != IL_BF16:
        raise ILError(-3, "the cache must be bf16 or q8")

    def pool(last, dtype):
        return torch.zeros((n_pages, n_heads, page_size, last), dtype=dtype, device=device).transpose(1, 2)
    kv = [pool(head_dim, torch.int8 if q8 else torch.bfloat16) for _ in range(2)]
    return KVCache(*kv, *([pool(head_dim // 32, torch.float32) for _ in range(2)] if q8 else []))


def _ptr(t, dtype, numel, what: str):
    """Address of a contiguous CUDA tensor of ``dtype`` and ``numel`` elements (0 for None)."""
    if t is None:
        return 0
    if t.dtype is not dtype or not t.is_cuda or not t.is_contiguous() or t.numel() != numel:
        raise ILError(-1, f"{what} must be a contiguous CUDA {dtype} tensor of {numel} elements")
    return t.data_ptr()


def _rows(t, n: int, heads: int, dim: int, f32, what: str):
    """(address, row stride) of fp32 ``[n][heads][dim]`` (or ``[n][heads*dim]``) whose rows are contiguous."""
    shape, st = t.shape, t.stride()
    if shape == (n, heads, dim):
        ok = st[2] == 1 and (st[1] == dim or heads == 1)
    else:
        ok = shape == (n, heads * dim) and st[1] == 1
    if not ok or t.dtype is not f32 or not t.is_cuda:
        if shape[1:] in ((heads, dim), (heads * dim,)) and shape[0] != n:
            raise ILError(-2, f"{what} has {shape[0]} rows, not {n}")
        raise ILError(-1, f"{what} must be CUDA float32 [{n}][{heads}][{dim}] with contiguous rows")
    return t.data_ptr(), st[0]


def _table(t, n_seq: int, i32):
    """(address, row stride, width) of an int32 block table."""
    shape, st = t.shape, t.stride()
    if len(shape) != 2 or shape[0] != n_seq or (st[1] != 1 and shape[1] > 1) or t.dtype is not i32 or not t.is_cuda:
        raise ILError(-1, f"table must be CUDA int32 [{n_seq}][width] with contiguous rows")
    return t.data_ptr(), st[0], shape[1]


def kv_extend(lens, add, table, ring, cursor, page_size: int, slots, lens_out=None, cursor_out=None, positions=None,
              first=None, info=None, stream=None) -> None:
    """``il_kv_extend``: sequences of ``lens`` grow by ``add`` tokens (or lose ``-add``): pages move
    between the free ``ring`` and ``table``, ``slots`` (and ``positions``) get the new tokens' places.

    All tensors are CUDA and contiguous (``table`` rows may be apart): ``lens``, ``add`` int32
    ``[n_seq]``; ``table`` int32 ``[n_seq][width]``; ``ring`` int32; ``cursor`` int64 ``[2]``; ``slots``,
    ``positions`` int32 ``[max_slots]``; ``first`` int32 ``[n_seq + 1]``; ``info`` int64 ``[4]``.
    ``lens_out`` and ``cursor_out`` default to ``lens`` and ``cursor`` themselves.
    """
    import torch
    i32, i64 = torch.int32, torch.int64
    n, most = lens.numel(), slots.numel()
    tp, ts, tw = _table(table, n, i32)
    size = ring.numel()
    lp, cp = _ptr(lens, i32, n, "lens"), _ptr(cursor, i64, 2, "cursor")
    rc = (_lib or load()).il_kv_extend(
        n, page_size, lp, _ptr(add, i32, n, "add"), tp, ts, tw, _ptr(ring, i32, size, "ring"), size, cp,
        lp if lens_out is None else _ptr(lens_out, i32, n, "lens_out"),
        cp if cursor_out is None else _ptr(cursor_out, i64, 2, "cursor_out"),
        _ptr(slots, i32, most, "slots"), most, _ptr(positions, i32, most, "positions"), _ptr(first, i32, n + 1, "first"),
        _ptr(info, i64, 4, "info"), _stream_ptr(stream))
    if rc:
        _check(rc)


def kv_append(cache: KVCache, k, v, slots, stream=None) -> None:
    """``il_kv_append``: fp32 rows ``k``, ``v`` ``[n][n_heads][head_dim]`` into the cache's ``slots``
    (int32 ``[n]``; a negative one is skipped).  The rows may be columns of a wider tensor."""
    import torch
    n, heads, dim, f32 = slots.numel(), cache.n_heads, cache.head_dim, torch.float32
    kp, ks = _rows(k, n, heads, dim, f32, "k")
    vp, vs = _rows(v, n, heads, dim, f32, "v")
    rc = (_lib or load()).il_kv_append(cache._ref, kp, ks, vp, vs, _ptr(slots, torch.int32, n, "slots"), n,
                                       _stream_ptr(stream))
    if rc:
        _check(rc)


def kv_read(cache: KVCache, slots, k, v, stream=None) -> None:
    """``il_kv_read``: the cached values of ``slots`` as fp32 into ``k`` and ``v`` (as for :func:`kv_append`)."""
    import torch
    n, heads, dim, f32 = slots.numel(), cache.n_heads, cache.head_dim, torch.float32
    kp, ks = _rows(k, n, heads, dim, f32, "k")
    vp, vs = _rows(v, n, heads, dim, f32, "v")
    rc = (_lib or load()).il_kv_read(cache._ref, _ptr(slots, torch.int32, n, "slots"), n, kp, ks, vp, vs,
                                     _stream_ptr(stream))
    if rc:
        _check(rc)


def kv_attend(cache: KVCache, q, table, lens, out, lse=None, scale=None, window: int = 0, stream=None) -> None:
    """``il_kv_attend``: attention of one token per sequence over its cached tokens.

    ``q``, ``out``: fp32 ``[n_seq][n_q_heads][head_dim]`` (sequences may be apart); ``table``, ``lens`` as
    :func:`kv_extend` leaves them; ``lse``: fp32 ``[n_seq][n_q_heads]`` or None; ``scale`` defaults
    to ``head_dim ** -0.5``; ``window``: tokens seen, counted from the end (0: all).

    A captured call uses the workspace of the stream it was captured on: graphs of one capture stream, and calls
    on that stream, must not run side by side."""
    import torch
    if q.dim() != 3:
        raise ILError(-1, "q must be [n_seq][n_q_heads][head_dim]")
    n, heads, _ = q.shape
    dim, f32, i32 = cache.head_dim, torch.float32, torch.int32
    qp, qs = _rows(q, n, heads, dim, f32, "q")
    op, os_ = _rows(out, n, heads, dim, f32, "out")
    tp, ts, tw = _table(table, n, i32)
    rc = (_lib or load()).il_kv_attend(cache._ref, qp, qs, tp, ts, tw, _ptr(lens, i32, n, "lens"), n, heads,
                                       dim ** -0.5 if scale is None else scale, window, op, os_,
                                       _ptr(lse, f32, n * heads, "lse"), _stream_ptr(stream))
    if rc:
        _check(rc)


def check_device_status(stream=None) -> None:
    _check(load().il_check_device_status(_stream_ptr(stream)))


def release_scratch(stream=None) -> None:
    """``il_release_scratch``: frees the library's scratch for ``stream`` (stream-ordered); graphs captured on
    the stream must not be replayed any more."""
    _check(load().il_release_scratch(_stream_ptr(stream)))


def get_stats() -> dict:
    s = _Stats()
    _check(load().il_get_stats(ctypes.byref(s)))
    return {name: getattr(s, name) for name, _ in _Stats._fields_}


def reset_stats() -> None:
    load().il_reset_stats()
