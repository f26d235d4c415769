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

__all__ = ["ILError", "Weight", "FORMATS", "KV_FORMATS", "IL_BF16", "IL_Q8", "IL_Q4", "IL_A4", "load", "build",
           "upload_weight", "matmul_batch", "matmul_batch_ptr", "matmul_batch_noalloc_ptr", "free_weight", "weight_bytes",
           "dequantize_weight", "check_device_status", "release_scratch", "get_stats", "reset_stats", "last_error",
           "version", "LIB_PATH", "STATUS", "KVCache", "kv_cache", "kv_extend", "kv_append", "kv_read", "kv_attend", "kv_weigh",
           "kv_evict"]

IL_BF16, IL_Q8, IL_Q4, IL_A4 = 0, 1, 2, 3
FORMATS = {"bf16": IL_BF16, "q8": IL_Q8, "q4": IL_Q4}
KV_FORMATS = {"bf16": IL_BF16, "q8": IL_Q8, "a4": IL_A4}
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


class _Score(ctypes.Structure):
    _fields_ = ([("cap", ctypes.c_float)] + [(n, ctypes.c_void_p) for n in ("slopes", "starts", "positions")]
                + [(n, ctypes.c_int64) for n in ("positions_stride", "positions_width")])


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
        lib.il_kv_attend_scored.argtypes = [vp, vp, i64, vp, i64, i64, vp, i64, i64, ctypes.c_float, i64, vp, vp, i64, vp, vp]
        lib.il_kv_attend_scored.restype = ci
        lib.il_kv_weigh.argtypes = [vp, vp, i64, vp, i64, i64, vp, i64, i64, ctypes.c_float, i64, vp, vp, vp, vp, vp, i64, i64, vp]
        lib.il_kv_weigh.restype = ci
        lib.il_kv_evict.argtypes = [vp, vp, i64, i64, vp, i64, i64, i64, i64, vp, vp, i64, i64, vp, vp, i64, i64, vp, i64, vp, vp]
        lib.il_kv_evict.restype = ci
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


_raw = None  # (raw current stream of a device, current device), once CUDA is up


def _stream_ptr(stream) -> int:
    global _raw
    if stream is None:
        if _raw is None:
            import torch
            raw, device = (getattr(torch._C, name, None) for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"))
            if raw is None or device is None:
                return torch.cuda.current_stream().cuda_stream
            torch.cuda.current_device()
            _raw = raw, device
        # the handle of torch.cuda.current_stream() without the object (3 us on the host)
        return _raw[0](_raw[1]())
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
_dtypes = None


def _types():
    """float32, int32, int64 (an import statement a call takes 0.3 us)."""
    global _dtypes
    import torch
    _dtypes = torch.float32, torch.int32, torch.int64
    return _dtypes


def _steps(t):
    """Strides of ``t``; 0 for a dimension of one entry, whose stride means nothing."""
    return [st if n > 1 else 0 for n, st in zip(t.shape, t.stride())]


class KVCache:
    """A paged K/V cache in the caller's tensors (``il_kv``); holds references to them.

    ``k``, ``v``: CUDA ``[n_pages][page_size][n_heads][head_dim]`` of one shape and one set of
    strides, the last dimension contiguous; pass ``pool.transpose(1, 2)`` of a pool stored
    head-major.  ``torch.bfloat16`` is IL_BF16; ``torch.int8`` is IL_Q8 with fp32 ``k_scale``,
    ``v_scale`` ``[n_pages][page_size][n_heads][head_dim / 32]``; ``torch.uint8`` is IL_A4, two elements a byte
    (a last dimension of ``head_dim / 2``), with bfloat16 ``k_scale``, ``v_scale``
    ``[n_pages][page_size][n_heads][head_dim / 32][2]``, the pairs (d, m).  :func:`kv_cache` allocates one.
    """

    def __init__(self, k, v, k_scale=None, v_scale=None):
        import torch
        if k.dim() != 4 or k.shape != v.shape or _steps(k) != _steps(v) or k.dtype != v.dtype:
            raise ILError(-1, "k and v must be [n_pages][page_size][n_heads][head_dim] of one shape, stride and dtype")
        formats = {torch.bfloat16: IL_BF16, torch.int8: IL_Q8, torch.uint8: IL_A4}
        if k.dtype not in formats:
            raise ILError(-3, "the cache must be bfloat16, int8 or uint8")
        if k.stride(3) != 1:
            raise ILError(-1, "the last dimension of k and v must be contiguous")
        if not (k.is_cuda and v.is_cuda):
            raise ILError(-1, "k and v must be CUDA tensors")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.n_pages, self.page_size, self.n_heads, self.head_dim = k.shape
        self.format = formats[k.dtype]
        pairs = self.format == IL_A4
        if pairs:
            self.head_dim *= 2
        c = self._c = _KV(self.format, self.page_size, self.n_pages, self.n_heads, self.head_dim, k.data_ptr(),
                          v.data_ptr(), None, None, *k.stride()[:3], 0, 0, 0)
        if (self.format != IL_BF16) != (k_scale is not None) or (k_scale is None) != (v_scale is None):
            raise ILError(-1, "an int8 or uint8 cache needs k_scale and v_scale, a bfloat16 cache has none")
        if k_scale is not None:
            shape = (*k.shape[:3], self.head_dim // 32) + ((2,) if pairs else ())
            dtype = torch.bfloat16 if pairs else torch.float32
            for t in (k_scale, v_scale):
                if (tuple(t.shape) != shape or t.dtype != dtype or not t.is_cuda or (shape[3] > 1 and t.stride(3) != len(shape) - 3)
                        or (pairs and (t.stride(4) != 1 or any(s % 2 for s in _steps(t)[:3])))):
                    raise ILError(-1, f"scales must be CUDA {dtype} {list(shape)}, the last dimension{'s' * pairs} contiguous")
            if _steps(k_scale)[:3] != _steps(v_scale)[:3]:
                raise ILError(-1, "k_scale and v_scale must have the same strides")
            c.k_scale, c.v_scale = k_scale.data_ptr(), v_scale.data_ptr()
            c.scale_page_stride, c.scale_token_stride, c.scale_head_stride = (s >> pairs for s in k_scale.stride()[:3])
        self._ref = ctypes.addressof(c)

    @property
    def bytes(self) -> int:
        """Bytes of the cache's elements and scales."""
        return sum(t.numel() * t.element_size() for t in (self.k, self.v, self.k_scale, self.v_scale) if t is not None)


def kv_cache(fmt, n_pages: int, page_size: int, n_heads: int, head_dim: int, device="cuda") -> KVCache:
    """A zeroed :class:`KVCache`, stored head-major within a page: a head's tokens of one page
    are one contiguous run."""
    import torch
    f = KV_FORMATS.get(fmt, fmt) if isinstance(fmt, str) else fmt
    if f not in KV_FORMATS.values():
        raise ILError(-3, "the cache must be bf16, q8 or a4")
    if f == IL_A4 and head_dim % 32:
        raise ILError(-2, "head_dim of a 4-bit cache must be a multiple of 32")

    def pool(dtype, *last):
        return torch.zeros((n_pages, n_heads, page_size, *last), dtype=dtype, device=device).transpose(1, 2)
    row = {IL_BF16: (torch.bfloat16, head_dim), IL_Q8: (torch.int8, head_dim), IL_A4: (torch.uint8, head_dim // 2)}[f]
    scales = {IL_BF16: None, IL_Q8: (torch.float32, head_dim // 32), IL_A4: (torch.bfloat16, head_dim // 32, 2)}[f]
    return KVCache(*(pool(*row) for _ in range(2)), *(pool(*scales) for _ in range(2) if scales))


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


def _table(t, n_seq: int, dtype, what: str = "table"):
    """(address, row stride, width) of a row a sequence: a block table, positions, weights."""
    shape, st = t.shape, t.stride()
    if len(shape) != 2 or shape[0] != n_seq or (st[1] != 1 and shape[1] > 1) or t.dtype is not dtype or not t.is_cuda:
        raise ILError(-1, f"{what} must be CUDA {dtype} [{n_seq}][width] with contiguous rows")
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
    _, i32, i64 = _dtypes or _types()
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
    f32, i32, _ = _dtypes or _types()
    n, heads, dim = slots.numel(), cache.n_heads, cache.head_dim
    kp, ks = _rows(k, n, heads, dim, f32, "k")
    vp, vs = _rows(v, n, heads, dim, f32, "v")
    rc = (_lib or load()).il_kv_append(cache._ref, kp, ks, vp, vs, _ptr(slots, i32, n, "slots"), n,
                                       _stream_ptr(stream))
    if rc:
        _check(rc)


def kv_read(cache: KVCache, slots, k, v, stream=None) -> None:
    """``il_kv_read``: the cached values of ``slots`` as fp32 into ``k`` and ``v`` (as for :func:`kv_append`)."""
    f32, i32, _ = _dtypes or _types()
    n, heads, dim = slots.numel(), cache.n_heads, cache.head_dim
    kp, ks = _rows(k, n, heads, dim, f32, "k")
    vp, vs = _rows(v, n, heads, dim, f32, "v")
    rc = (_lib or load()).il_kv_read(cache._ref, _ptr(slots, i32, n, "slots"), n, kp, ks, vp, vs,
                                     _stream_ptr(stream))
    if rc:
        _check(rc)


def _score(n: int, heads: int, cap: float, slopes, starts, positions):
    """An ``il_kv_score``, or None where nothing of it is given."""
    if not cap and slopes is None and starts is None and positions is None:
        return None
    f32, i32, _ = _dtypes or _types()
    c = _Score(cap, _ptr(slopes, f32, heads, "slopes"), _ptr(starts, i32, n, "starts"), 0, 0, 0)
    if positions is not None:
        c.positions, c.positions_stride, c.positions_width = _table(positions, n, i32, "positions")
    return c


def kv_attend(cache: KVCache, q, table, lens, out, lse=None, scale=None, window: int = 0, stream=None, cap: float = 0.0,
              slopes=None, starts=None, positions=None) -> None:
    """``il_kv_attend``: attention of one token per sequence over its cached tokens.

    ``q``, ``out``: fp32 ``[n_seq][n_q_heads][head_dim]`` (sequences may be apart); ``table``, ``lens`` as
    :func:`kv_extend` leaves them; ``lse``: fp32 ``[n_seq][n_q_heads]`` or None; ``scale`` defaults
    to ``head_dim ** -0.5``; ``window``: tokens seen, counted from the end (0: all).

    ``il_kv_attend_scored`` with one of these: ``cap``: logits are ``cap * tanh(s / cap)``; ``slopes`` fp32
    ``[n_q_heads]``: a bias of ``slopes[h]`` times the distance from the last token (a negative number), by index or by
    ``positions`` int32 ``[n_seq][width]``; ``starts`` int32 ``[n_seq]``: the first token seen.  ``window`` and ``starts`` count
    indices: not for sequences that :func:`kv_evict` has cut.

    A captured call uses the workspace of the stream it was captured on: graphs of one capture stream, and calls
    on that stream, must not run side by side."""
    f32, i32, _ = _dtypes or _types()
    if q.dim() != 3:
        raise ILError(-1, "q must be [n_seq][n_q_heads][head_dim]")
    (n, heads, _), dim = q.shape, cache.head_dim
    qp, qs = _rows(q, n, heads, dim, f32, "q")
    op, os_ = _rows(out, n, heads, dim, f32, "out")
    tp, ts, tw = _table(table, n, i32)
    lp, ep, stream = _ptr(lens, i32, n, "lens"), _ptr(lse, f32, n * heads, "lse"), _stream_ptr(stream)
    scale = dim ** -0.5 if scale is None else scale
    score = _score(n, heads, cap, slopes, starts, positions)
    if score is None:
        rc = (_lib or load()).il_kv_attend(cache._ref, qp, qs, tp, ts, tw, lp, n, heads, scale, window, op, os_, ep, stream)
    else:
        rc = (_lib or load()).il_kv_attend_scored(cache._ref, qp, qs, tp, ts, tw, lp, n, heads, scale, window,
                                                  ctypes.addressof(score), op, os_, ep, stream)
    if rc:
        _check(rc)


def _in_out(t, out, n: int, dtype, what: str):
    """(address, address of the output, row stride, width) of a row a sequence that is updated, in place or beside."""
    if t is None:
        raise ILError(-1, f"{what} must not be None")
    tp, ts, tw = _table(t, n, dtype, what)
    if out is None or out is t:
        return tp, tp, ts, tw
    if out.dtype is dtype and out.is_cuda and out.shape == t.shape and out.stride() == t.stride():
        return tp, out.data_ptr(), ts, tw
    op, os_, ow = _table(out, n, dtype, what + "_out")
    if ow != tw or (n > 1 and os_ != ts):
        raise ILError(-2, f"{what}_out must have the shape and strides of {what}")
    return tp, op, ts, tw


def kv_weigh(cache: KVCache, q, table, lens, lse, weights, weights_out=None, add=None, scale=None, window: int = 0, stream=None,
             cap: float = 0.0, slopes=None, starts=None, positions=None) -> None:
    """``il_kv_weigh``: adds to ``weights`` fp32 ``[n_seq][width]`` (rows may be apart) what each cached token gets of
    the attention of ``q`` over all query heads; ``weights_out`` defaults to ``weights`` itself.

    ``lse`` is what :func:`kv_attend` gave for the same arguments; the last ``add`` (int32 ``[n_seq]``) tokens are
    new and start from 0."""
    f32, i32, _ = _dtypes or _types()
    if q.dim() != 3:
        raise ILError(-1, "q must be [n_seq][n_q_heads][head_dim]")
    (n, heads, _), dim = q.shape, cache.head_dim
    qp, qs = _rows(q, n, heads, dim, f32, "q")
    tp, ts, tw = _table(table, n, i32)
    if lse is None:
        raise ILError(-1, "lse must not be None")
    score = _score(n, heads, cap, slopes, starts, positions)
    rc = (_lib or load()).il_kv_weigh(cache._ref, qp, qs, tp, ts, tw, _ptr(lens, i32, n, "lens"), n, heads,
                                      dim ** -0.5 if scale is None else scale, window,
                                      0 if score is None else ctypes.addressof(score), _ptr(lse, f32, n * heads, "lse"),
                                      _ptr(add, i32, n, "add"), *_in_out(weights, weights_out, n, f32, "weights"),
                                      _stream_ptr(stream))
    if rc:
        _check(rc)


def kv_evict(cache: KVCache, table, lens, weights, kept, drop, first: int = 0, recent: int = 0, weights_out=None, positions=None,
             positions_out=None, stream=None) -> None:
    """``il_kv_evict``: cuts each sequence to ``keep = kept.shape[1]`` tokens: those of the ``first`` and the ``recent``
    positions and the heaviest of the others.  ``kept`` int32 ``[n_seq][keep]`` gets the old index of each token, ``drop`` int32
    ``[n_seq]`` the changes of length, for :func:`kv_extend`.

    ``weights`` fp32 and ``positions`` int32 (or None: positions are indices) ``[n_seq][width]`` are updated, in place or
    into ``weights_out`` and ``positions_out``.  The caller writes the position of each new token, the newest of its sequence,
    before the next call; a sequence is not cut twice without a new token in between."""
    f32, i32, _ = _dtypes or _types()
    n = lens.numel()
    tp, ts, tw = _table(table, n, i32)
    kp, ks, keep = _table(kept, n, i32, "kept")
    places = (0, 0, 0, 0) if positions is None and positions_out is None else _in_out(positions, positions_out, n, i32, "positions")
    rc = (_lib or load()).il_kv_evict(cache._ref, tp, ts, tw, _ptr(lens, i32, n, "lens"), n, keep, first, recent,
                                      *_in_out(weights, weights_out, n, f32, "weights"), *places, kp, ks,
                                      _ptr(drop, i32, n, "drop"), _stream_ptr(stream))
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
