"""Python binding of libkvq.so: rotated-INT4 paged KV cache for NVIDIA B200 (sm_100a).

Argument marshalling only -- every step of the path runs in the library's CUDA kernels.
The names mirror the C ABI in ``include/kvq.h``:

* ``kvq_alloc_pages``          -> :func:`alloc_pages`
* ``kvq_rotate_quant_append``  -> :func:`rotate_quant_append`
* ``kvq_decode_attention``     -> :func:`decode_attention`
* ``kvq_append_decode_attention`` -> :func:`append_decode_attention`
* ``kvq_prefill_attention``    -> :func:`prefill_attention`
* ``kvq_rope_quant_append``    -> :func:`rope_quant_append`
* ``kvq_gather_rows``          -> :func:`gather_rows`
* ``kvq_update_block_bounds``  -> :func:`update_block_bounds`
* ``kvq_select_blocks``        -> :func:`select_blocks`
* ``kvq_sparse_attention``     -> :func:`sparse_attention`
* ``kvq_free``                 -> :func:`free`
* ``kvq_assign_pages``, ``kvq_pool_bytes``, ``kvq_get_device_status`` likewise.

PyTorch provides device memory and streams (tensors are passed by ``data_ptr()``, the
stream by ``torch.cuda.current_stream().cuda_stream``).  There is no CPU fallback: if
``libkvq.so`` is missing and cannot be built, importing :func:`lib` raises.
"""
import ctypes
import os

import numpy as np

from . import build as _build

__all__ = [
    "KVQError", "Desc", "Cache", "lib", "pool_bytes", "assign_pages", "alloc_pages",
    "rotate_quant_append", "decode_attention", "append_decode_attention", "prefill_attention",
    "decode_attention_noalloc", "free",
    "Rope", "BlockBounds", "rope_quant_append", "gather_rows", "update_block_bounds",
    "select_blocks", "sparse_attention",
    "get_device_status", "status_string",
    "EXPORTED",
]

KVQ_OK, KVQ_EINVAL, KVQ_EUNSUPPORTED, KVQ_ENOPAGES, KVQ_ECUDA = 0, -1, -2, -3, -4
KVQ_DEV_BAD_PAGE, KVQ_DEV_BAD_POS, KVQ_DEV_TIMEOUT = 1, 2, 4

EXPORTED = (
    "kvq_pool_bytes", "kvq_assign_pages", "kvq_alloc_pages", "kvq_rotate_quant_append",
    "kvq_decode_attention", "kvq_pool_ptr", "kvq_get_device_status", "kvq_free",
    "kvq_status_string", "kvq_decode_attention_noalloc", "kvq_append_decode_attention",
    "kvq_prefill_attention", "kvq_rope_quant_append", "kvq_gather_rows",
    "kvq_update_block_bounds", "kvq_select_blocks", "kvq_sparse_attention",
)


class KVQError(RuntimeError):
    def __init__(self, what, status):
        super().__init__(f"{what}: {status_string(status)} ({status})")
        self.status = status


FORMAT_INT4 = 0
FORMAT_NVFP4 = 1


class Desc(ctypes.Structure):
    """``kvq_desc``: cache geometry (host integers); ``kv_format`` 0 = rotated INT4,
    1 = NVFP4 (``FORMAT_NVFP4``); omitted trailing fields are 0."""
    _fields_ = [(n, ctypes.c_int32) for n in (
        "num_layers", "num_kv_heads", "num_q_heads", "head_dim", "hadamard_block",
        "page_size", "num_pages", "max_batch", "max_pages_per_seq", "kv_format")]

    def __repr__(self):
        return "Desc(" + ", ".join(f"{n}={getattr(self, n)}" for n, _ in self._fields_) + ")"


_lib = None
_torch = None  # the torch module, imported with the first cache


def lib() -> ctypes.CDLL:
    """Load libkvq.so (building it first with nvcc if it is missing or stale)."""
    global _lib
    if _lib is None:
        path = _build.build()
        L = ctypes.CDLL(path)
        vp, i32, i32p = ctypes.c_void_p, ctypes.c_int32, ctypes.POINTER(ctypes.c_int32)
        i64 = ctypes.c_int64
        dp = ctypes.POINTER(Desc)
        sig = {
            "kvq_pool_bytes": (ctypes.c_size_t, [dp]),
            "kvq_assign_pages": (ctypes.c_int, [dp, i32, i32p, i32p, i32p]),
            "kvq_alloc_pages": (ctypes.c_int, [dp, vp, ctypes.c_size_t, i32, i32p, i32p, i32p,
                                               ctypes.POINTER(vp)]),
            "kvq_rotate_quant_append": (ctypes.c_int, [vp, i32, vp, vp, vp, vp, vp, i32, i32, vp]),
            "kvq_decode_attention": (ctypes.c_int, [vp, i32, vp, vp, vp, i32, ctypes.c_float, vp,
                                                    vp]),
            "kvq_pool_ptr": (vp, [vp]),
            "kvq_get_device_status": (ctypes.c_int, [vp, i32p, vp]),
            "kvq_free": (ctypes.c_int, [vp]),
            "kvq_status_string": (ctypes.c_char_p, [ctypes.c_int]),
            "kvq_decode_attention_noalloc": (ctypes.c_int, [dp, vp, ctypes.c_size_t, i32, vp, vp,
                                                            vp, i32, ctypes.c_float, vp, vp, vp]),
            "kvq_append_decode_attention": (ctypes.c_int, [vp, i32, vp, vp, vp, vp, vp, i32,
                                                           ctypes.c_float, vp, vp]),
            "kvq_prefill_attention": (ctypes.c_int, [vp, i32, vp, vp, vp, vp, i32, i32,
                                                     ctypes.c_float, vp, vp]),
            "kvq_rope_quant_append": (ctypes.c_int, [vp, i32, i32, vp, i64, vp, i64, vp, i64, vp, vp,
                                                     vp, vp, i32, i32, vp, i32, i32,
                                                     ctypes.c_double, vp, vp]),
            "kvq_gather_rows": (ctypes.c_int, [vp, i32, vp, vp, vp, i32, i32, i32, vp, vp, vp]),
            "kvq_update_block_bounds": (ctypes.c_int, [vp, i32, vp, vp, vp, vp, vp, i32, i32, vp]),
            "kvq_select_blocks": (ctypes.c_int, [vp, i32, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32,
                                                 i32, vp, vp]),
            "kvq_sparse_attention": (ctypes.c_int, [vp, i32, vp, vp, vp, vp, vp, i32, i32, i32,
                                                    ctypes.c_float, vp, vp]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().kvq_status_string(int(status)).decode()


def _check(rc, what):
    if rc != KVQ_OK:
        raise KVQError(what, rc)


def _i32(a):
    a = np.ascontiguousarray(a, dtype=np.int32)
    return a, a.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))


def pool_bytes(desc: Desc) -> int:
    return int(lib().kvq_pool_bytes(ctypes.byref(desc)))


def assign_pages(desc: Desc, capacity_tokens, page_order=None) -> np.ndarray:
    """Host-only deterministic page table [batch][max_pages_per_seq] (unused = -1)."""
    cap, capp = _i32(capacity_tokens)
    order, orderp = (None, None) if page_order is None else _i32(page_order)
    pt = np.full((cap.shape[0], desc.max_pages_per_seq), -7, np.int32)
    rc = lib().kvq_assign_pages(ctypes.byref(desc), cap.shape[0], capp, orderp,
                                pt.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)))
    _check(rc, "kvq_assign_pages")
    return pt


def _stream_ptr(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _dev_ptr(t, what, dtype=None):
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{what} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return t.data_ptr()


class Cache:
    """Owner of a ``kvq_cache*`` handle.  ``pool`` is the torch tensor backing the pool
    when the caller supplied one (kept alive here)."""

    def __init__(self, handle, desc, pool_tensor, device=None):
        global _torch
        import torch as _torch
        self.handle = handle
        self.desc = desc
        self.pool = pool_tensor
        self.device = device  # index of the CUDA device that the handle was made on
        # Plain values that every call reads (a ctypes field costs an attribute lookup and a box).
        self.kv_heads, self.q_heads = desc.num_kv_heads, desc.num_q_heads
        self.table_width = desc.max_pages_per_seq
        self.page_shape = (desc.num_layers, desc.num_pages, desc.num_kv_heads)
        self.torch_device = None if device is None else _torch.device("cuda", device)

    @property
    def pool_ptr(self) -> int:
        return int(lib().kvq_pool_ptr(self.handle) or 0)

    def close(self):
        if self.handle:
            rc = lib().kvq_free(self.handle)
            self.handle = None
            _check(rc, "kvq_free")

    def __del__(self):
        try:
            if self.handle:
                lib().kvq_free(self.handle)
                self.handle = None
        except Exception:
            pass


def alloc_pages(desc: Desc, capacity_tokens=None, page_order=None, pool=None):
    """Create a cache handle; returns ``(cache, page_table)`` with the host page table
    (np.int32 [batch][max_pages_per_seq]).  ``pool``: optional torch uint8 CUDA tensor of
    at least :func:`pool_bytes` bytes (the library allocates one otherwise)."""
    cap = np.zeros(0, np.int32) if capacity_tokens is None else capacity_tokens
    cap, capp = _i32(cap)
    order, orderp = (None, None) if page_order is None else _i32(page_order)
    pt = np.full((cap.shape[0], desc.max_pages_per_seq), -7, np.int32)
    pool_ptr, nbytes = None, 0
    if pool is not None:
        import torch
        pool_ptr = _dev_ptr(pool, "pool", torch.uint8)
        nbytes = pool.numel()
    h = ctypes.c_void_p()
    rc = lib().kvq_alloc_pages(ctypes.byref(desc), pool_ptr, nbytes, cap.shape[0], capp,
                               orderp, pt.ctypes.data_as(ctypes.POINTER(ctypes.c_int32)),
                               ctypes.byref(h))
    _check(rc, "kvq_alloc_pages")
    import torch
    return Cache(h, desc, pool, torch.cuda.current_device()), pt


def rotate_quant_append(cache: Cache, layer: int, k, v, cu_new_tokens, seq_lens, page_table,
                        stream=None) -> None:
    """Fused rotate + quantise + paged append of fp16 k, v [T][Hkv][128] (CUDA): INT4 rows,
    or NVFP4 rows for a cache made with kv_format = FORMAT_NVFP4.  Token t of sequence b
    (cu_new_tokens[b] <= t < cu_new_tokens[b+1]) lands at position seq_lens[b] + t -
    cu_new_tokens[b]; seq_lens is not updated."""
    import torch
    T = int(k.shape[0])
    batch = int(seq_lens.shape[0])
    rc = lib().kvq_rotate_quant_append(
        cache.handle, int(layer), _dev_ptr(k, "k", torch.float16), _dev_ptr(v, "v", torch.float16),
        _dev_ptr(cu_new_tokens, "cu_new_tokens", torch.int32),
        _dev_ptr(seq_lens, "seq_lens", torch.int32), _dev_ptr(page_table, "page_table", torch.int32),
        batch, T, _stream_ptr(stream))
    _check(rc, "kvq_rotate_quant_append")


def decode_attention(cache: Cache, layer: int, q, seq_lens, page_table, softmax_scale=0.0,
                     out=None, stream=None):
    """Paged GQA decode attention; q fp16 [batch][Hq][128] -> out fp16 (same shape)."""
    import torch
    if out is None:
        out = torch.empty_like(q)
    batch = int(seq_lens.shape[0])
    rc = lib().kvq_decode_attention(
        cache.handle, int(layer), _dev_ptr(q, "q", torch.float16),
        _dev_ptr(seq_lens, "seq_lens", torch.int32), _dev_ptr(page_table, "page_table", torch.int32),
        batch, float(softmax_scale), _dev_ptr(out, "out", torch.float16), _stream_ptr(stream))
    _check(rc, "kvq_decode_attention")
    return out


def append_decode_attention(cache: Cache, layer: int, k_new, v_new, q, seq_lens, page_table,
                            softmax_scale=0.0, out=None, stream=None):
    """One new token per sequence appended at seq_lens[b] (lengths before the append) and
    decode attention over seq_lens[b] + 1 tokens, in one launch."""
    import torch
    if out is None:
        out = torch.empty_like(q)
    batch = int(seq_lens.shape[0])
    rc = lib().kvq_append_decode_attention(
        cache.handle, int(layer), _dev_ptr(k_new, "k_new", torch.float16),
        _dev_ptr(v_new, "v_new", torch.float16), _dev_ptr(q, "q", torch.float16),
        _dev_ptr(seq_lens, "seq_lens", torch.int32), _dev_ptr(page_table, "page_table", torch.int32),
        batch, float(softmax_scale), _dev_ptr(out, "out", torch.float16), _stream_ptr(stream))
    _check(rc, "kvq_append_decode_attention")
    return out


def prefill_attention(cache: Cache, layer: int, q, cu_q, seq_lens, page_table, softmax_scale=0.0,
                      out=None, stream=None, total_q=None):
    """Causal chunked-prefill attention: q fp16 [total_q][Hq][128] (chunks concatenated),
    cu_q int32 [batch+1], seq_lens int32 [batch] (lengths with the chunk appended)."""
    import torch
    if out is None:
        out = torch.empty_like(q)
    batch = int(seq_lens.shape[0])
    tq = int(q.shape[0]) if total_q is None else int(total_q)
    rc = lib().kvq_prefill_attention(
        cache.handle, int(layer), _dev_ptr(q, "q", torch.float16),
        _dev_ptr(cu_q, "cu_q", torch.int32), _dev_ptr(seq_lens, "seq_lens", torch.int32),
        _dev_ptr(page_table, "page_table", torch.int32), batch, tq, float(softmax_scale),
        _dev_ptr(out, "out", torch.float16), _stream_ptr(stream))
    _check(rc, "kvq_prefill_attention")
    return out


def decode_attention_noalloc(desc: Desc, pool, layer: int, q, seq_lens, page_table,
                             softmax_scale=0.0, out=None, status=None, stream=None):
    """Decode attention without a handle and without any device allocation by the library
    (its scratch lives in a fixed device array; limits in include/kvq.h).  ``status``: an
    optional int32 CUDA tensor of one element that receives the KVQ_DEV_* bits."""
    import torch
    if out is None:
        out = torch.empty_like(q)
    batch = int(seq_lens.shape[0])
    st = None if status is None else _dev_ptr(status, "status", torch.int32)
    rc = lib().kvq_decode_attention_noalloc(
        ctypes.byref(desc), _dev_ptr(pool, "pool", torch.uint8), int(pool.numel()), int(layer),
        _dev_ptr(q, "q", torch.float16), _dev_ptr(seq_lens, "seq_lens", torch.int32),
        _dev_ptr(page_table, "page_table", torch.int32), batch, float(softmax_scale),
        _dev_ptr(out, "out", torch.float16), st, _stream_ptr(stream))
    _check(rc, "kvq_decode_attention_noalloc")
    return out


class Rope:
    """The position rotation of :func:`rope_quant_append`: ``inv_freq`` fp32 CUDA
    [rotary_dim / 2] (kept alive here), channel pairs (i, i + rotary_dim / 2) or, interleaved,
    (2i, 2i + 1); ``factor`` multiplies every cosine and sine.  ``inv_freq`` may be set again (or
    given other data in place) between calls; ``rotary_dim`` follows its length."""

    def __init__(self, inv_freq, interleaved=False, factor=1.0):
        self.inv_freq = inv_freq
        self.interleaved = bool(interleaved)
        self.factor = float(factor)

    @property
    def inv_freq(self):
        return self._inv_freq

    @inv_freq.setter
    def inv_freq(self, t):
        import torch
        ptr = _dev_ptr(t, "inv_freq", torch.float32)
        if t.dim() != 1:
            raise ValueError("inv_freq must have one dimension")
        self._inv_freq, self._ptr, self._device = t, ptr, t.get_device()
        self.rotary_dim = 2 * int(t.shape[0])

    def pointer(self, cache):
        """Address of the frequencies for a call on ``cache``.  The tensor was checked when it was
        set; it is checked again when its data has moved since."""
        t = self._inv_freq
        if t.data_ptr() != self._ptr:
            self.inv_freq = t
        if self.rotary_dim != 2 * t.numel():
            raise ValueError(f"rotary_dim {self.rotary_dim} with {t.numel()} frequencies")
        if self._device != cache.device:
            raise ValueError(f"inv_freq must be on cuda:{cache.device}")
        return self._ptr


class BlockBounds:
    """Per-page key bounds of a cache, by pool page: ``codes`` int8 CUDA
    [num_layers][num_pages][num_kv_heads][2][128] (lower, then upper bounds) in units of
    ``scale`` fp32 [num_layers][num_pages][num_kv_heads].  Filled by
    :func:`update_block_bounds`, read by :func:`select_blocks`.  Either may be set again to a tensor
    that fits the other."""

    def __init__(self, codes, scale):
        self._take(codes, scale)

    def _take(self, codes, scale):
        import torch
        ptrs = _dev_ptr(codes, "codes", torch.int8), _dev_ptr(scale, "scale", torch.float32)
        if tuple(codes.shape) != (*scale.shape, 2, 128) or scale.dim() != 3:
            raise ValueError("codes must be [layers][pages][heads][2][128], scale [layers][pages][heads]")
        self._codes, self._scale, self._ptrs = codes, scale, ptrs
        self._shape = tuple(scale.shape)
        self._device = codes.get_device() if codes.get_device() == scale.get_device() else -1

    @property
    def codes(self):
        return self._codes

    @codes.setter
    def codes(self, t):
        self._take(t, self._scale)

    @property
    def scale(self):
        return self._scale

    @scale.setter
    def scale(self, t):
        self._take(self._codes, t)

    @classmethod
    def alloc(cls, cache):
        """Bounds for every page of ``cache`` (260 bytes per page, KV head and layer)."""
        import torch
        shape, dev = cache.page_shape, cache.torch_device
        return cls(torch.zeros(*shape, 2, 128, dtype=torch.int8, device=dev),
                   torch.zeros(*shape, dtype=torch.float32, device=dev))

    def pointers(self, cache):
        """Addresses for a call on ``cache``.  Both tensors were checked when they were set; they
        are checked again when their data has moved since."""
        codes, scale = self._codes, self._scale
        at = self._ptrs
        if codes.data_ptr() != at[0] or scale.data_ptr() != at[1]:
            self._take(codes, scale)
        if self._shape != cache.page_shape:
            raise ValueError(f"bounds of {self._shape} for a cache of {cache.page_shape}")
        if self._device != cache.device:
            raise ValueError(f"bounds must be on cuda:{cache.device}")
        return self._ptrs


def _arg(cache, t, what, dtype, shape):
    """Pointer of a contiguous CUDA tensor on the cache's device, of the given type and shape."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == cache.device and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _dev_ptr(t, what, dtype)
    _refuse(cache, t, what, shape)


def _refuse(cache, t, what, shape):
    if t.get_device() != cache.device:
        raise ValueError(f"{what} is on cuda:{t.get_device()}, the cache on cuda:{cache.device}")
    raise ValueError(f"{what} must have shape {shape}, got {tuple(t.shape)}")


def _seqs(cache, seq_lens, page_table, cu, cu_name):
    """(batch, pointers of seq_lens, page_table and cu) of a call, checked."""
    i32, batch = _torch.int32, seq_lens.shape[0]
    return (batch, _arg(cache, seq_lens, "seq_lens", i32, (batch,)),
            _arg(cache, page_table, "page_table", i32, (batch, cache.table_width)),
            None if cu is None else _arg(cache, cu, cu_name, i32, (batch + 1,)))


def _run(cache, stream, name, *args):
    """Call the library on the cache's device and the given (default: current) stream."""
    fn = getattr(_lib, name)
    if stream is None:
        stream = _torch._C._cuda_getCurrentRawStream(cache.device)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    if _torch._C._cuda_getDevice() == cache.device:
        rc = fn(cache.handle, *args, stream)
    else:
        with _torch.cuda.device(cache.device):
            rc = fn(cache.handle, *args, stream)
    if rc != KVQ_OK:
        raise KVQError(name, rc)


def _empty(cache, shape, dtype, stream):
    """An output of the call's stream (so that the allocator orders its reuse after the call)."""
    if stream is None:
        return _torch.empty(shape, dtype=dtype, device=cache.torch_device)
    if isinstance(stream, int):
        stream = _torch.cuda.ExternalStream(stream, device=cache.torch_device)
    with _torch.cuda.stream(stream):
        return _torch.empty(shape, dtype=dtype, device=cache.torch_device)


def _tokens(cache, t, what, dtype, shape):
    """(pointer, token stride) of token rows whose heads are contiguous within a token."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == cache.device:
            s = t.stride()
            if (s[2] == 1 and (s[1] == 128 or shape[1] == 1)) or shape[0] == 0:
                return t.data_ptr(), s[0] if shape[0] > 1 else shape[1] * 128
            raise ValueError(f"{what}: the heads of a token must be contiguous")
    except AttributeError:
        pass
    if getattr(t, "is_cuda", False):
        if t.dtype != dtype:
            raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
        _refuse(cache, t, what, shape)
    raise TypeError(f"{what} must be a CUDA tensor")


def _dtype_code(dtype):
    if dtype == _torch.float16:
        return 0
    if dtype == _torch.bfloat16:
        return 1
    raise TypeError(f"rows must be float16 or bfloat16, got {dtype}")


def rope_quant_append(cache: Cache, layer: int, k, v, cu_new_tokens, seq_lens, page_table, rope: Rope,
                      q=None, positions=None, q_out=None, stream=None):
    """:func:`rotate_quant_append` with the position rotation of q and k applied on the way.
    k, v [T][Hkv][128] and q [T][Hq][128], all fp16 or all bf16, may be slices of one qkv buffer
    (a token's heads contiguous, any token stride).  Angles use the cache positions, or
    ``positions`` int32 [T].  Returns the rotated q in fp16 [T][Hq][128] (None without q)."""
    T, dtype = k.shape[0], k.dtype
    code = _dtype_code(dtype)
    kp, ks = _tokens(cache, k, "k", dtype, (T, cache.kv_heads, 128))
    vp, vs = _tokens(cache, v, "v", dtype, (T, cache.kv_heads, 128))
    batch, sl, pt, cu = _seqs(cache, seq_lens, page_table, cu_new_tokens, "cu_new_tokens")
    pos = None if positions is None else _arg(cache, positions, "positions", _torch.int32, (T,))
    freq = rope.pointer(cache)
    qp, qs, op = None, 0, None
    if q is not None:
        shape = (T, cache.q_heads, 128)
        qp, qs = _tokens(cache, q, "q", dtype, shape)
        if q_out is None:
            q_out = _empty(cache, shape, _torch.float16, stream)
            op = q_out.data_ptr()
        else:
            op = _arg(cache, q_out, "q_out", _torch.float16, shape)
    elif q_out is not None:
        raise ValueError("q_out without q")
    _run(cache, stream, "kvq_rope_quant_append", int(layer), code, qp, qs, kp, ks, vp, vs, cu, sl, pos, pt,
         batch, T, freq, rope.rotary_dim, int(rope.interleaved), rope.factor, op)
    return q_out


def gather_rows(cache: Cache, layer: int, cu_rows, starts, page_table, total_rows: int, dtype=None,
                k_out=None, v_out=None, stream=None):
    """Cached K and V rows in the model's basis: positions starts[b] .. starts[b] + cu_rows[b+1] -
    cu_rows[b] - 1 of every sequence, as two tensors [total_rows][Hkv][128] of ``dtype`` (fp16
    unless given; bf16).  Always both; the C call can leave out either."""
    dtype = _torch.float16 if dtype is None else dtype
    code = _dtype_code(dtype)
    shape = (int(total_rows), cache.kv_heads, 128)
    batch, st, pt, cu = _seqs(cache, starts, page_table, cu_rows, "cu_rows")
    if k_out is None and v_out is None and stream is None:
        k_out = _empty(cache, shape, dtype, stream)
        v_out = _torch.empty_like(k_out)
        kp, vp = k_out.data_ptr(), v_out.data_ptr()
    else:
        if k_out is None:
            k_out = _empty(cache, shape, dtype, stream)
        if v_out is None:
            v_out = _empty(cache, shape, dtype, stream)
        kp, vp = _arg(cache, k_out, "k_out", dtype, shape), _arg(cache, v_out, "v_out", dtype, shape)
    _run(cache, stream, "kvq_gather_rows", int(layer), cu, st, pt, batch, shape[0], code, kp, vp)
    return k_out, v_out


def update_block_bounds(cache: Cache, layer: int, bounds: BlockBounds, cu_new_tokens, seq_lens, page_table,
                        total_new_tokens: int, stream=None) -> None:
    """Bounds of every page that an append touched, after that append and with its arguments
    (seq_lens: the lengths before it)."""
    batch, sl, pt, cu = _seqs(cache, seq_lens, page_table, cu_new_tokens, "cu_new_tokens")
    codes, scale = bounds.pointers(cache)
    _run(cache, stream, "kvq_update_block_bounds", int(layer), codes, scale, cu, sl, pt, batch,
         int(total_new_tokens))


def select_blocks(cache: Cache, layer: int, q, seq_lens, page_table, bounds: BlockBounds, num_blocks: int,
                  cu_q=None, sink=1, recent=1, blocks=None, stream=None):
    """Pages to attend per query and KV head: the first ``sink``, the last ``recent`` and the best
    others by the bounds' score; int32 [total_q][Hkv][num_blocks], ascending, then -1.  q fp16
    [total_q][Hq][128]; one query per sequence, or the chunks of ``cu_q``.  seq_lens counts the
    queries' own tokens."""
    tq, nb = q.shape[0], int(num_blocks)
    batch, sl, pt, cu = _seqs(cache, seq_lens, page_table, cu_q, "cu_q")
    codes, scale = bounds.pointers(cache)
    qp = _arg(cache, q, "q", _torch.float16, (tq, cache.q_heads, 128))
    shape = (tq, cache.kv_heads, max(nb, 0))
    if blocks is None:
        blocks = _empty(cache, shape, _torch.int32, stream)
        bp = blocks.data_ptr()
    else:
        bp = _arg(cache, blocks, "blocks", _torch.int32, shape)
    _run(cache, stream, "kvq_select_blocks", int(layer), codes, scale, qp, cu, sl, pt, batch, tq, nb,
         int(sink), int(recent), bp)
    return blocks


def sparse_attention(cache: Cache, layer: int, q, seq_lens, page_table, blocks, cu_q=None,
                     softmax_scale=0.0, out=None, stream=None):
    """Attention of every query over the pages in its own list: blocks int32
    [total_q][Hkv][num_blocks] (negative: empty), as :func:`select_blocks` returns it or the
    caller's own; q, seq_lens, cu_q as there.  Returns fp16 [total_q][Hq][128]."""
    tq = q.shape[0]
    batch, sl, pt, cu = _seqs(cache, seq_lens, page_table, cu_q, "cu_q")
    qp = _arg(cache, q, "q", _torch.float16, (tq, cache.q_heads, 128))
    if blocks.dim() != 3:
        raise ValueError("blocks must be [total_q][num_kv_heads][num_blocks]")
    nb = int(blocks.shape[2])
    bp = _arg(cache, blocks, "blocks", _torch.int32, (tq, cache.kv_heads, nb))
    if out is None:
        out = _torch.empty_like(q) if stream is None else _empty(cache, q.shape, _torch.float16, stream)
        op = out.data_ptr()
    else:
        op = _arg(cache, out, "out", _torch.float16, (tq, cache.q_heads, 128))
    _run(cache, stream, "kvq_sparse_attention", int(layer), qp, cu, sl, pt, bp, nb, batch, tq,
         float(softmax_scale), op)
    return out


def get_device_status(cache: Cache, stream=None) -> int:
    """Read and clear the device status word (KVQ_DEV_* bits); synchronises the stream."""
    v = ctypes.c_int32(0)
    rc = lib().kvq_get_device_status(cache.handle, ctypes.byref(v), _stream_ptr(stream))
    _check(rc, "kvq_get_device_status")
    return int(v.value)


def free(cache: Cache) -> None:
    cache.close()
