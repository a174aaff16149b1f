"""Binding of the 4-bit key/value cache (include/qknorm_kv4.h): argument
marshalling only, like ``_binding``; every step runs in the library's kernels.

Tensors live on one device, which need not be the current one.  Work is put on
``stream`` (default: the current stream of the tensors' device), and outputs
that are allocated here belong to that stream.
"""
from __future__ import annotations

import ctypes
import threading

from . import _binding
from ._binding import QKNormError, _dtype_code, _gamma_ptr

_lock = threading.Lock()
_kv4_lib = None
PAGE_SIZES = (16, 32, 64, 128, 256)
HEAD_DIMS = (64, 128, 256)


def _lib():
    """libqknorm.so with the prototypes of include/qknorm_kv4.h declared."""
    global _kv4_lib
    if _kv4_lib is not None:
        return _kv4_lib
    lib = _binding.load_library()
    with _lock:
        vp, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
        protos = {
            "qknorm_kv4_append": [vp, i32, i64, i32, i32, i32, i64, vp, vp, f32, vp, vp, i64, i32,
                                  vp, vp],
            "qknorm_kv4_read": [vp, i64, i32, i32, i32, vp, i64, vp, vp, i32, i64, vp],
            "qknorm_kv4_attention": [vp, i32, i64, i32, i32, i32, i64, vp, i64, i32, vp, i64, i64,
                                     vp, i64, vp, i32, f32, vp, i64, vp, vp, vp, i64, vp],
            "qknorm_kv4_attention_workspace": [i64, i32, i32, i32, i32, i32, i64, i32,
                                               ctypes.POINTER(i64)],
            "qknorm_kv4_evict": [vp, i64, i32, i32, i32, vp, vp, i64, i64, vp, i64, vp, i64, i64,
                                 i64, i64, vp, vp, vp],
            "qknorm_kv4_bad_pages": [ctypes.POINTER(ctypes.c_uint)],
            "qknorm_kv4_last_cuda_error": [],
            "qknorm_kv4_version": [],
        }
        for name, args in protos.items():
            fn = getattr(lib, name)
            fn.argtypes, fn.restype = args, i32
        _kv4_lib = lib
    return lib


def _check(fn, rc):
    if rc != 0:
        lib = _lib()
        raise QKNormError(fn, rc, lib.qknorm_status_string(rc).decode(),
                          lib.qknorm_kv4_last_cuda_error())


class _On:
    """Makes a device and, where one is given, a stream current for a call."""

    def __init__(self, device, stream):
        import torch

        if stream is not None:
            if stream.device != device:
                raise ValueError("stream belongs to %s, the tensors live on %s"
                                 % (stream.device, device))
            self._ctx = torch.cuda.stream(stream)
        elif torch.cuda.current_device() != device.index:
            self._ctx = torch.cuda.device(device)
        else:
            self._ctx = None

    def __enter__(self):
        if self._ctx is not None:
            self._ctx.__enter__()

    def __exit__(self, *exc):
        if self._ctx is not None:
            self._ctx.__exit__(*exc)


def _stream_of(device):
    import torch

    return torch.cuda.current_stream(device).cuda_stream


class KV4Cache:
    """A paged key/value cache held in 4 bits: ``pool`` (uint8 [num_pages, Hk,
    page_size // 16, 16 * D + 128], the layout of include/qknorm_kv4.h) and,
    for eviction, ``scores`` (float32 [num_pages, Hk, page_size]).  The tensors
    are the caller's; ``KV4Cache.empty`` allocates them, scores zeroed."""

    __slots__ = ("pool", "scores", "Hk", "D", "page_size", "num_pages")

    def __init__(self, pool, Hk, D, page_size=64, scores=None):
        import torch

        if D not in HEAD_DIMS:
            raise ValueError("D must be 64, 128 or 256, got %r" % (D,))
        if page_size not in PAGE_SIZES:
            raise ValueError("page_size must be one of %s, got %r" % (PAGE_SIZES, page_size))
        if not pool.is_cuda:
            raise ValueError("pool must be a CUDA tensor (QK-Norm runs only on the GPU)")
        shape = (pool.shape[0], Hk, page_size // 16, 16 * D + 128)
        if pool.dtype != torch.uint8 or tuple(pool.shape) != shape or not pool.is_contiguous():
            raise ValueError("pool must be a contiguous uint8 tensor [num_pages, Hk, "
                             "page_size // 16, 16 * D + 128]")
        if scores is not None:
            if (scores.dtype != torch.float32 or not scores.is_contiguous()
                    or tuple(scores.shape) != (shape[0], Hk, page_size)
                    or scores.device != pool.device):
                raise ValueError("scores must be a contiguous float32 tensor [num_pages, Hk, "
                                 "page_size] on the pool's device")
        self.pool, self.scores = pool, scores
        self.Hk, self.D, self.page_size, self.num_pages = Hk, D, page_size, shape[0]

    @classmethod
    def empty(cls, num_pages, Hk, D, page_size=64, scores=False, device="cuda"):
        import torch

        if D not in HEAD_DIMS or page_size not in PAGE_SIZES:
            raise ValueError("D must be one of %s and page_size one of %s"
                             % (HEAD_DIMS, PAGE_SIZES))
        pool = torch.zeros((num_pages, Hk, page_size // 16, 16 * D + 128), dtype=torch.uint8,
                           device=device)
        sums = None
        if scores:
            sums = torch.zeros((num_pages, Hk, page_size), dtype=torch.float32, device=device)
        return cls(pool, Hk, D, page_size, sums)


def _vec(t, name, dtype, n, device):
    """A device vector of ``n`` elements with unit stride."""
    if t.dtype != dtype or t.dim() != 1 or t.shape[0] != n or (n > 1 and t.stride(0) != 1):
        raise ValueError("%s must be a contiguous %s vector of %d elements" % (name, dtype, n))
    if t.device != device:
        raise ValueError("%s must live on the cache's device" % name)
    return t.data_ptr()


def _table(t, name, B, device):
    import torch

    if t.dtype != torch.int32 or t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError("%s must be an int32 tensor [B, pages] with unit column stride" % name)
    if t.shape[0] != B or t.device != device:
        raise ValueError("%s must have one row for each sequence, on the cache's device" % name)
    # One row (or one column) may come with any stride in torch.
    stride = t.stride(0) if B > 1 else t.shape[1]
    return t.data_ptr(), stride, t.shape[1]


def _fused(t, name, device):
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor (QK-Norm runs only on the GPU)" % name)
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError("%s must be a 2-D [T, row_stride] view with unit column stride" % name)
    if t.device != device:
        raise ValueError("%s must live on the cache's device" % name)
    return t.shape[0], t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _ptr(t):
    return None if t is None else t.data_ptr()


def kv4_bad_pages() -> int:
    """Pages and slots outside a pool that kernels on the current device met
    (qknorm_kv4_bad_pages)."""
    count = ctypes.c_uint(0)
    _check("qknorm_kv4_bad_pages", _lib().qknorm_kv4_bad_pages(ctypes.byref(count)))
    return int(count.value)


def qknorm_kv4_append(cache, qkv, slots, Hq, gamma_q=None, gamma_k=None, eps=1e-6, stream=None):
    """Per-head QK-Norm in place on ``qkv`` [T, row_stride] with its key and
    value rows stored in the cache, token t at slot ``slots[t]`` (int64; a
    negative slot stores nothing).  Without weights nothing is normalised."""
    import torch

    dev = cache.pool.device
    T, stride = _fused(qkv, "qkv", dev)
    sp = _vec(slots, "slots", torch.int64, T, dev)
    for g in (gamma_q, gamma_k):
        if g is not None and (g.device != dev or g.numel() != cache.D):
            raise ValueError("gamma_q and gamma_k must have D elements on the cache's device")
    with _On(dev, stream):
        rc = _lib().qknorm_kv4_append(
            qkv.data_ptr(), _dtype_code(qkv), T, Hq, cache.Hk, cache.D, stride,
            _gamma_ptr(gamma_q, "gamma_q"), _gamma_ptr(gamma_k, "gamma_k"), eps, sp,
            cache.pool.data_ptr(), cache.num_pages, cache.page_size, _ptr(cache.scores),
            _stream_of(dev))
    _check("qknorm_kv4_append", rc)
    return qkv


def qknorm_kv4_read(cache, slots, dtype=None, stream=None):
    """The rows that ``slots`` (int64 [N]) hold, as values of ``dtype``
    (default bfloat16): ``(k, v)``, each [N, Hk * D].  A slot outside the pool
    reads as zeros."""
    import torch

    dev = cache.pool.device
    if slots.dim() != 1:
        raise ValueError("slots must be a vector")
    N, width = slots.shape[0], cache.Hk * cache.D
    sp = _vec(slots, "slots", torch.int64, N, dev)
    with _On(dev, stream):
        k = torch.empty((N, width), dtype=dtype or torch.bfloat16, device=dev)
        v = torch.empty_like(k)
        rc = _lib().qknorm_kv4_read(
            cache.pool.data_ptr(), cache.num_pages, cache.page_size, cache.Hk, cache.D, sp, N,
            k.data_ptr(), v.data_ptr(), _dtype_code(k), width, _stream_of(dev))
    _check("qknorm_kv4_read", rc)
    return k, v


def _workspace_bytes(B, dtype, Hq, cache, max_q, max_kv, with_scores):
    n = ctypes.c_int64(0)
    _check("qknorm_kv4_attention_workspace", _lib().qknorm_kv4_attention_workspace(
        B, dtype, Hq, cache.Hk, cache.D, max_q, max_kv, int(with_scores), ctypes.byref(n)))
    return n.value


def kv4_attention_workspace(cache, qkv, Hq, page_table, max_q=1, add_scores=False):
    """A workspace for ``qknorm_kv4_attention`` with these arguments, to keep
    for calls that do not overlap on the GPU."""
    import torch

    n = _workspace_bytes(page_table.shape[0], _dtype_code(qkv), Hq, cache, max_q,
                         page_table.shape[1] * cache.page_size, add_scores)
    return torch.empty(n, dtype=torch.uint8, device=cache.pool.device)


def qknorm_kv4_attention(cache, qkv, Hq, page_table, kv_lens, q_starts=None, max_q=1, scale=None,
                         add_scores=False, out=None, lse=None, workspace=None, stream=None):
    """Attention of ``qkv``'s query heads over the cached rows; returns ``(out
    [T, Hq * D], lse [T, Hq])``.

    ``page_table`` int32 [B, pages], ``kv_lens`` int32 [B].  Without
    ``q_starts`` there is one query token for each sequence; with it (int32
    [B + 1]) sequence b has the rows ``q_starts[b]`` to ``q_starts[b + 1]``, at
    most ``max_q``.  ``scale`` defaults to D ** -0.5.  ``add_scores`` adds each
    cached row's weight to ``cache.scores``.  ``out`` and ``lse`` may be given;
    rows of no sequence are left as they are in them, and are undefined in
    outputs that are allocated here.  See include/qknorm_kv4.h."""
    import torch

    dev, D = cache.pool.device, cache.D
    T, stride = _fused(qkv, "qkv", dev)
    B = kv_lens.shape[0]
    tp, t_stride, pages = _table(page_table, "page_table", B, dev)
    lp = _vec(kv_lens, "kv_lens", torch.int32, B, dev)
    qp = None if q_starts is None else _vec(q_starts, "q_starts", torch.int32, B + 1, dev)
    if qkv.shape[1] < Hq * D:
        raise ValueError("qkv has fewer than Hq * D columns")
    if add_scores and cache.scores is None:
        raise ValueError("add_scores needs a cache with scores")
    code = _dtype_code(qkv)
    with _On(dev, stream):
        if out is None:
            out = torch.empty((T, Hq * D), dtype=qkv.dtype, device=dev)
        elif out.dtype != qkv.dtype or out.shape != (T, Hq * D):
            raise ValueError("out must be [T, Hq * D] in qkv's type")
        _, out_stride = _fused(out, "out", dev)
        if lse is None:
            lse = torch.empty((T, Hq), dtype=torch.float32, device=dev)
        elif (lse.dtype != torch.float32 or lse.shape != (T, Hq) or not lse.is_contiguous()
              or lse.device != dev):
            raise ValueError("lse must be a contiguous float32 tensor [T, Hq]")
        if workspace is None:
            workspace = torch.empty(_workspace_bytes(B, code, Hq, cache, max_q,
                                                     pages * cache.page_size, add_scores),
                                    dtype=torch.uint8, device=dev)
        elif workspace.device != dev or not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous, on the cache's device")
        rc = _lib().qknorm_kv4_attention(
            qkv.data_ptr(), code, T, Hq, cache.Hk, D, stride, cache.pool.data_ptr(),
            cache.num_pages, cache.page_size, tp, t_stride, pages, lp, B, qp, max_q,
            D ** -0.5 if scale is None else scale, out.data_ptr(), out_stride, lse.data_ptr(),
            cache.scores.data_ptr() if add_scores else None, workspace.data_ptr(),
            workspace.nbytes, _stream_of(dev))
    _check("qknorm_kv4_attention", rc)
    return out, lse


def qknorm_kv4_evict(cache, page_table, kv_lens, dst_table, budget, recent, stream=None):
    """Keep, of each sequence's and head's rows, the ``recent`` newest and the
    highest-scored others, ``budget`` in all, copied in order to the pages of
    ``dst_table`` (int32 [B, pages]; none of them read).  Returns ``(new_lens
    int32 [B], kept int32 [B, Hk, budget])``, the kept rows' numbers with -1
    behind the last."""
    import torch

    dev = cache.pool.device
    if cache.scores is None:
        raise ValueError("eviction needs a cache with scores")
    B = kv_lens.shape[0]
    tp, t_stride, pages = _table(page_table, "page_table", B, dev)
    dp, d_stride, d_pages = _table(dst_table, "dst_table", B, dev)
    lp = _vec(kv_lens, "kv_lens", torch.int32, B, dev)
    if not 1 <= budget <= d_pages * cache.page_size or not 0 <= recent <= budget:
        raise ValueError("1 <= budget <= dst_table's rows and 0 <= recent <= budget are required")
    with _On(dev, stream):
        new_lens = torch.empty(B, dtype=torch.int32, device=dev)
        kept = torch.empty((B, cache.Hk, budget), dtype=torch.int32, device=dev)
        rc = _lib().qknorm_kv4_evict(
            cache.pool.data_ptr(), cache.num_pages, cache.page_size, cache.Hk, cache.D,
            cache.scores.data_ptr(), tp, t_stride, pages, lp, B, dp, d_stride, d_pages, budget,
            recent, new_lens.data_ptr(), kept.data_ptr(), _stream_of(dev))
    _check("qknorm_kv4_evict", rc)
    return new_lens, kept
