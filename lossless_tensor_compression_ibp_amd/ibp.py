"""Python binding of libibp (include/ibp.h): argument marshalling only.

Every function forwards torch tensors (device memory, or pinned host memory
where the C ABI allows it) as raw pointers together with the HIP stream of
torch's current stream.  All codec work runs in the gfx950 kernels of
libibp.so; if the library is missing this module raises on first use.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np
import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libibp.so")

IBP_OK = 0
IBP_ERR_INVALID_ARG = -1
IBP_ERR_UNSUPPORTED = -2
IBP_ERR_DEVICE = -3
IBP_ERR_NOMEM = -4
IBP_ERR_CORRUPT = -5
IBP_ERR_RANGE = -6
IBP_ERR_TOO_LARGE = -7

# ibp_decompress_noalloc's static scratch (include/ibp.h)
NOALLOC_SCRATCH_BYTES = 1 << 20
NOALLOC_MAX_TILES = NOALLOC_SCRATCH_BYTES // 8 - 32

# every function the header declares (checked by the tests)
ABI_FUNCTIONS = (
    "ibp_build_metadata", "ibp_meta_create", "ibp_meta_get", "ibp_meta_get_info",
    "ibp_meta_set_first_read", "ibp_meta_destroy", "ibp_compress", "ibp_decompress", "ibp_gather_decompress",
    "ibp_check", "ibp_status_string",
    "ibp_packed_offsets", "ibp_compress_packed", "ibp_decompress_packed", "ibp_gather_decompress_packed",
    "ibp_compress_split", "ibp_decompress_split", "ibp_gather_decompress_split",
    "ibp_decompress_noalloc",
    "ibp_pages_copy", "ibp_pages_workspace", "ibp_pages_alloc", "ibp_pages_alloc_raw", "ibp_pages_fork", "ibp_pages_free",
    "ibp_pages_compact", "ibp_tree_attention_workspace", "ibp_tree_attention", "ibp_page_bounds",
    "ibp_select_pages_workspace", "ibp_select_pages", "ibp_sparse_attention_workspace", "ibp_sparse_attention",
)


class ibp_params(ctypes.Structure):
    _fields_ = [("tensor_bytes", ctypes.c_uint64), ("chunk_bits", ctypes.c_uint32),
                ("period_bits", ctypes.c_uint32), ("threshold", ctypes.c_double)]


class ibp_meta_info(ctypes.Structure):
    _fields_ = [("invariant_bits", ctypes.c_uint64), ("min_record_bytes", ctypes.c_uint64),
                ("max_runs", ctypes.c_uint32), ("uniform", ctypes.c_uint32)]


class ibp_pages(ctypes.Structure):
    _fields_ = [("meta", ctypes.c_void_p), ("slots", ctypes.c_void_p), ("n_slots", ctypes.c_uint64),
                ("bitmask", ctypes.c_void_p)]


class ibp_attention(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_uint32), ("head_dim", ctypes.c_uint32), ("page_tokens", ctypes.c_uint32),
                ("n_q_heads", ctypes.c_uint32), ("n_kv_heads", ctypes.c_uint32), ("scale", ctypes.c_float),
                ("n_rows", ctypes.c_uint64), ("n_seqs", ctypes.c_uint64), ("table_blocks", ctypes.c_uint64),
                ("max_len", ctypes.c_uint64), ("max_new", ctypes.c_uint32), ("q_row_stride", ctypes.c_int64),
                ("q_head_stride", ctypes.c_int64), ("new_row_stride", ctypes.c_int64),
                ("new_head_stride", ctypes.c_int64)]


class IBPError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {status_string(status)} ({status})")
        self.status = status


_lib = None


def lib():
    """Load libibp.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "python -m lossless_tensor_compression_ibp_amd.build_lib")
        L = ctypes.CDLL(LIB_PATH)
        p, u64, st = ctypes.c_void_p, ctypes.c_uint64, ctypes.c_int
        P = ctypes.POINTER
        L.ibp_build_metadata.argtypes = [P(ibp_params), p, u64, P(p), p]
        L.ibp_meta_create.argtypes = [P(ibp_params), p, p, P(p), p]
        L.ibp_meta_get.argtypes = [p, P(ibp_params), p, p]
        L.ibp_meta_get_info.argtypes = [p, P(ibp_meta_info)]
        L.ibp_meta_set_first_read.argtypes = [p, u64]
        L.ibp_meta_destroy.argtypes = [p]
        L.ibp_compress.argtypes = [p, p, u64, p, p, p, p]
        L.ibp_decompress.argtypes = [p, p, p, u64, p, p]
        L.ibp_decompress_noalloc.argtypes = [p, p, p, u64, p, p]
        L.ibp_gather_decompress.argtypes = [p, p, u64, p, p, u64, p, p]
        L.ibp_check.argtypes = [p, p]
        L.ibp_packed_offsets.argtypes = [p, p, u64, p, p]
        L.ibp_compress_packed.argtypes = [p, p, u64, p, p, u64, p, p]
        L.ibp_decompress_packed.argtypes = [p, p, u64, p, p, u64, p, p]
        L.ibp_gather_decompress_packed.argtypes = [p, p, u64, p, u64, p, p, u64, p, p]
        L.ibp_compress_split.argtypes = [p, p, u64, p, p, p, p, p]
        L.ibp_decompress_split.argtypes = [p, p, p, p, u64, p, p]
        L.ibp_gather_decompress_split.argtypes = [p, p, u64, p, p, p, u64, p, p]
        u32, A, G = ctypes.c_uint32, P(ibp_attention), P(ibp_pages)
        L.ibp_pages_copy.argtypes = [p, p, u64, p, p, p, u64, p, p, u64, p]
        L.ibp_pages_workspace.argtypes = [u64, u64]
        L.ibp_pages_alloc.argtypes = [p, p, u64, p, u64, p, u64, p]
        L.ibp_pages_alloc_raw.argtypes = [p, p, u64, p, p, u64, p, u64, p]
        L.ibp_pages_fork.argtypes = [p, p, u64, p, p, p, u64, u32, u64, p, u32, p, p, u64, p, u64, p]
        L.ibp_pages_free.argtypes = [p, p, u64, p, u64, u32, u64, p, u64, p]
        L.ibp_pages_compact.argtypes = [p, p, u64, p, p, p, p, p, u64, p, u64, p]
        L.ibp_tree_attention_workspace.argtypes = [A]
        L.ibp_tree_attention.argtypes = [G, G, A, p, p, p, p, p, p, p, p, u32, p, p, p, u64, p]
        L.ibp_page_bounds.argtypes = [G, u32, u32, p, p, u64, p, p]
        L.ibp_select_pages_workspace.argtypes = [A]
        L.ibp_select_pages.argtypes = [p, A, p, p, u64, p, p, p, u32, u32, p, u32, p, u64, p]
        L.ibp_sparse_attention_workspace.argtypes = [A, u32]
        L.ibp_sparse_attention.argtypes = [G, G, A, p, p, p, p, p, p, u32, p, p, p, u64, p]
        L.ibp_status_string.argtypes = [st]
        L.ibp_status_string.restype = ctypes.c_char_p
        for f in ABI_FUNCTIONS:
            if f != "ibp_status_string":
                getattr(L, f).restype = u64 if f.endswith("_workspace") else st
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().ibp_status_string(int(status)).decode()


def _check(status: int, what: str):
    if status != IBP_OK:
        raise IBPError(status, what)


def _need(t: torch.Tensor | None, nbytes: int, what: str):
    """Buffers reach the library as plain pointers: check here that each one
    holds what the call will read or write."""
    if t is not None and t.nbytes < nbytes:
        raise ValueError(f"{what} holds {t.nbytes} bytes, the call needs {nbytes}")


def _bitmask_bytes(n: int) -> int:
    return 4 * ((int(n) + 31) // 32)


def _need_all(*checks):
    """(tensor, bytes, name) triples; raises for the first buffer that is too
    small.  Called only after a combined test failed, so the common path of a
    hot call costs one comparison per buffer."""
    for t, nbytes, what in checks:
        _need(t, nbytes, what)


def _ptr(t: torch.Tensor | None):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to libibp must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> ctypes.c_void_p:
    """HIP stream handle: the given torch stream, else torch's current stream
    on the current device (read without building a Stream object)."""
    if stream is not None:
        return ctypes.c_void_p(stream.cuda_stream)
    if _raw_stream is not None:
        return ctypes.c_void_p(_raw_stream(torch.cuda.current_device()))
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


class Meta:
    """Owns an ibp_meta_t handle; keeps the tensor length L and chunk width W
    so that the calls below can check buffer sizes before the library sees
    plain pointers."""

    def __init__(self, handle: ctypes.c_void_p, tensor_bytes: int = 0, chunk_bits: int = 0):
        self.handle = handle
        self.tensor_bytes = int(tensor_bytes)
        self.chunk_bits = int(chunk_bits)
        self.hdr_words = (8 * self.tensor_bytes // self.chunk_bits + 31) // 32 if self.chunk_bits else 0

    @property
    def _as_parameter_(self):
        return self.handle

    def close(self):
        if self.handle:
            _check(lib().ibp_meta_destroy(self.handle), "ibp_meta_destroy")
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _params(tensor_bytes, chunk_bits, period_bits, threshold=0.0):
    return ibp_params(int(tensor_bytes), int(chunk_bits), int(period_bits), float(threshold))


def ibp_build_metadata(sample: torch.Tensor, n_sample: int, tensor_bytes: int, chunk_bits: int,
                       period_bits: int, threshold: float, stream=None) -> Meta:
    prm = _params(tensor_bytes, chunk_bits, period_bits, threshold)
    out = ctypes.c_void_p()
    _need(sample, int(n_sample) * int(tensor_bytes), "sample")
    _check(lib().ibp_build_metadata(ctypes.byref(prm), _ptr(sample), int(n_sample), ctypes.byref(out),
                                    _stream(stream)), "ibp_build_metadata")
    return Meta(out, tensor_bytes, chunk_bits)


def ibp_meta_create(tensor_bytes: int, chunk_bits: int, period_bits: int, mask, bitval, stream=None) -> Meta:
    mask = np.ascontiguousarray(mask, dtype=np.uint32)
    bitval = np.ascontiguousarray(bitval, dtype=np.uint32)
    prm = _params(tensor_bytes, chunk_bits, period_bits)
    out = ctypes.c_void_p()
    if mask.size < period_bits // 32 or bitval.size < period_bits // 32:
        raise ValueError("mask and bitval need period_bits / 32 words each")
    _check(lib().ibp_meta_create(ctypes.byref(prm), ctypes.c_void_p(mask.ctypes.data),
                                 ctypes.c_void_p(bitval.ctypes.data), ctypes.byref(out), _stream(stream)),
           "ibp_meta_create")
    return Meta(out, tensor_bytes, chunk_bits)


def ibp_meta_get(meta: Meta):
    prm = ibp_params()
    _check(lib().ibp_meta_get(meta, ctypes.byref(prm), None, None), "ibp_meta_get")
    mw = prm.period_bits // 32
    mask = np.zeros(mw, np.uint32)
    bitval = np.zeros(mw, np.uint32)
    _check(lib().ibp_meta_get(meta, None, ctypes.c_void_p(mask.ctypes.data),
                              ctypes.c_void_p(bitval.ctypes.data)), "ibp_meta_get")
    params = dict(tensor_bytes=prm.tensor_bytes, chunk_bits=prm.chunk_bits,
                  period_bits=prm.period_bits, threshold=prm.threshold)
    return params, mask, bitval


def ibp_meta_get_info(meta: Meta) -> dict:
    info = ibp_meta_info()
    _check(lib().ibp_meta_get_info(meta, ctypes.byref(info)), "ibp_meta_get_info")
    return dict(invariant_bits=info.invariant_bits, min_record_bytes=info.min_record_bytes,
                max_runs=info.max_runs, uniform=info.uniform)


def ibp_meta_set_first_read(meta: Meta, nbytes: int):
    _check(lib().ibp_meta_set_first_read(meta, int(nbytes)), "ibp_meta_set_first_read")


def ibp_meta_destroy(meta: Meta):
    meta.close()


def ibp_compress(meta: Meta, src: torch.Tensor, n_tensors: int, dst_slots: torch.Tensor,
                 bitmask: torch.Tensor, stored_bytes: torch.Tensor | None = None, stream=None):
    L, n = meta.tensor_bytes, int(n_tensors)
    _need(src, n * L, "src")
    _need(dst_slots, n * L, "dst_slots")
    _need(bitmask, _bitmask_bytes(n), "bitmask")
    _need(stored_bytes, 8 * n, "stored_bytes")
    _check(lib().ibp_compress(meta, _ptr(src), int(n_tensors), _ptr(dst_slots), _ptr(bitmask),
                              _ptr(stored_bytes), _stream(stream)), "ibp_compress")


def ibp_decompress(meta: Meta, slots: torch.Tensor, bitmask: torch.Tensor, n_tensors: int,
                   dst: torch.Tensor, stream=None):
    L, n = meta.tensor_bytes, int(n_tensors)
    _need(slots, n * L, "slots")
    _need(bitmask, _bitmask_bytes(n), "bitmask")
    _need(dst, n * L, "dst")
    _check(lib().ibp_decompress(meta, _ptr(slots), _ptr(bitmask), int(n_tensors), _ptr(dst),
                                _stream(stream)), "ibp_decompress")


def ibp_decompress_noalloc(meta: Meta, slots: torch.Tensor, bitmask: torch.Tensor, n_tensors: int,
                           dst: torch.Tensor, stream=None):
    """ibp_decompress without device allocation (the library's static
    scratch); the same output."""
    L, n = meta.tensor_bytes, int(n_tensors)
    _need(slots, n * L, "slots")
    _need(bitmask, _bitmask_bytes(n), "bitmask")
    _need(dst, n * L, "dst")
    _check(lib().ibp_decompress_noalloc(meta, _ptr(slots), _ptr(bitmask), int(n_tensors), _ptr(dst),
                                        _stream(stream)), "ibp_decompress_noalloc")


def ibp_gather_decompress(meta: Meta, slots: torch.Tensor, n_slots: int, bitmask: torch.Tensor,
                          ids: torch.Tensor, dst: torch.Tensor, stream=None):
    if ids.dtype != torch.int64:
        raise ValueError("ids must be int64")
    L, n, k = meta.tensor_bytes, int(n_slots), ids.numel()
    if slots.nbytes < n * L or bitmask.nbytes < 4 * ((n + 31) // 32) or dst.nbytes < k * L:
        _need_all((slots, n * L, "slots"), (bitmask, _bitmask_bytes(n), "bitmask"), (dst, k * L, "dst"))
    _check(lib().ibp_gather_decompress(meta, _ptr(slots), int(n_slots), _ptr(bitmask), _ptr(ids),
                                       int(ids.numel()), _ptr(dst), _stream(stream)),
           "ibp_gather_decompress")


def ibp_check(meta: Meta, stream=None) -> int:
    """Synchronises the stream; returns the latched device status (0 = ok)."""
    return int(lib().ibp_check(meta, _stream(stream)))


# ---------------------------------------------------------------------------
# Packed cache: items back to back at 16-byte aligned offsets.
# ---------------------------------------------------------------------------
def ibp_packed_offsets(meta: Meta, src: torch.Tensor, n_tensors: int, offsets: torch.Tensor, stream=None):
    """offsets: device int64 tensor of n_tensors + 1 entries (written)."""
    if offsets.dtype != torch.int64 or offsets.numel() < n_tensors + 1:
        raise ValueError("offsets must be int64 with n_tensors + 1 entries")
    if n_tensors:
        _need(src, int(n_tensors) * meta.tensor_bytes, "src")
    _check(lib().ibp_packed_offsets(meta, _ptr(src) if n_tensors else None, int(n_tensors), _ptr(offsets),
                                    _stream(stream)), "ibp_packed_offsets")


def ibp_compress_packed(meta: Meta, src: torch.Tensor, n_tensors: int, offsets: torch.Tensor, dst: torch.Tensor,
                        bitmask: torch.Tensor, capacity: int | None = None, stream=None):
    if capacity is None:
        capacity = dst.nbytes
    elif capacity > dst.nbytes:
        raise ValueError(f"capacity {capacity} exceeds dst ({dst.nbytes} bytes)")
    n = int(n_tensors)
    _need(src, n * meta.tensor_bytes, "src")
    _need(offsets, 8 * (n + 1), "offsets")
    _need(bitmask, _bitmask_bytes(n), "bitmask")
    _check(lib().ibp_compress_packed(meta, _ptr(src), int(n_tensors), _ptr(offsets), _ptr(dst), int(capacity),
                                     _ptr(bitmask), _stream(stream)), "ibp_compress_packed")


def ibp_decompress_packed(meta: Meta, buf: torch.Tensor, offsets: torch.Tensor, bitmask: torch.Tensor,
                          n_items: int, dst: torch.Tensor, buf_bytes: int | None = None, stream=None):
    if buf_bytes is None:
        buf_bytes = buf.nbytes
    elif buf_bytes > buf.nbytes:
        raise ValueError(f"buf_bytes {buf_bytes} exceeds buf ({buf.nbytes} bytes)")
    n = int(n_items)
    _need(offsets, 8 * (n + 1), "offsets")
    _need(bitmask, _bitmask_bytes(n), "bitmask")
    _need(dst, n * meta.tensor_bytes, "dst")
    _check(lib().ibp_decompress_packed(meta, _ptr(buf), int(buf_bytes), _ptr(offsets), _ptr(bitmask),
                                       int(n_items), _ptr(dst), _stream(stream)), "ibp_decompress_packed")


def ibp_gather_decompress_packed(meta: Meta, buf: torch.Tensor, offsets: torch.Tensor, n_items: int,
                                 bitmask: torch.Tensor, ids: torch.Tensor, dst: torch.Tensor,
                                 buf_bytes: int | None = None, stream=None):
    if ids.dtype != torch.int64:
        raise ValueError("ids must be int64")
    if buf_bytes is None:
        buf_bytes = buf.nbytes
    elif buf_bytes > buf.nbytes:
        raise ValueError(f"buf_bytes {buf_bytes} exceeds buf ({buf.nbytes} bytes)")
    n, k = int(n_items), ids.numel() * meta.tensor_bytes
    if offsets.nbytes < 8 * (n + 1) or bitmask.nbytes < 4 * ((n + 31) // 32) or dst.nbytes < k:
        _need_all((offsets, 8 * (n + 1), "offsets"), (bitmask, _bitmask_bytes(n), "bitmask"), (dst, k, "dst"))
    _check(lib().ibp_gather_decompress_packed(meta, _ptr(buf), int(buf_bytes), _ptr(offsets), int(n_items),
                                              _ptr(bitmask), _ptr(ids), int(ids.numel()), _ptr(dst),
                                              _stream(stream)), "ibp_gather_decompress_packed")


# ---------------------------------------------------------------------------
# Headers in GPU memory: header words beside the bitmask, payload in the slot.
# ---------------------------------------------------------------------------
def _header_words(meta: Meta) -> int:
    return meta.hdr_words


def header_words(meta: Meta) -> int:
    prm, _, _ = ibp_meta_get(meta)
    return (8 * prm["tensor_bytes"] // prm["chunk_bits"] + 31) // 32


def ibp_compress_split(meta: Meta, src: torch.Tensor, n_tensors: int, dst_slots: torch.Tensor,
                       headers: torch.Tensor, bitmask: torch.Tensor, stored_bytes: torch.Tensor | None = None,
                       stream=None):
    L, n = meta.tensor_bytes, int(n_tensors)
    _need(src, n * L, "src")
    _need(dst_slots, n * L, "dst_slots")
    _need(headers, 4 * n * _header_words(meta), "headers")
    _need(bitmask, _bitmask_bytes(n), "bitmask")
    _need(stored_bytes, 8 * n, "stored_bytes")
    _check(lib().ibp_compress_split(meta, _ptr(src), int(n_tensors), _ptr(dst_slots), _ptr(headers),
                                    _ptr(bitmask), _ptr(stored_bytes), _stream(stream)), "ibp_compress_split")


def ibp_decompress_split(meta: Meta, slots: torch.Tensor, headers: torch.Tensor, bitmask: torch.Tensor,
                         n_tensors: int, dst: torch.Tensor, stream=None):
    L, n = meta.tensor_bytes, int(n_tensors)
    _need(slots, n * L, "slots")
    _need(headers, 4 * n * _header_words(meta), "headers")
    _need(bitmask, _bitmask_bytes(n), "bitmask")
    _need(dst, n * L, "dst")
    _check(lib().ibp_decompress_split(meta, _ptr(slots), _ptr(headers), _ptr(bitmask), int(n_tensors), _ptr(dst),
                                      _stream(stream)), "ibp_decompress_split")


def ibp_gather_decompress_split(meta: Meta, slots: torch.Tensor, n_slots: int, headers: torch.Tensor,
                                bitmask: torch.Tensor, ids: torch.Tensor, dst: torch.Tensor, stream=None):
    if ids.dtype != torch.int64:
        raise ValueError("ids must be int64")
    L, n, k = meta.tensor_bytes, int(n_slots), ids.numel()
    hb = 4 * n * _header_words(meta)
    if (slots.nbytes < n * L or headers.nbytes < hb or bitmask.nbytes < 4 * ((n + 31) // 32)
            or dst.nbytes < k * L):
        _need_all((slots, n * L, "slots"), (headers, hb, "headers"), (bitmask, _bitmask_bytes(n), "bitmask"),
                  (dst, k * L, "dst"))
    _check(lib().ibp_gather_decompress_split(meta, _ptr(slots), int(n_slots), _ptr(headers), _ptr(bitmask),
                                             _ptr(ids), int(ids.numel()), _ptr(dst), _stream(stream)),
           "ibp_gather_decompress_split")


# ---------------------------------------------------------------------------
# Pages of a key/value cache: management without decoding, attention that
# reads them where they lie.  Every call takes an optional torch stream and
# queues on it (default: torch's current stream of the tensors' device).
# ---------------------------------------------------------------------------
_DTYPES = {torch.bfloat16: 0, torch.float16: 1}


def _addr(t: torch.Tensor | None):
    """Address of a tensor whose layout the call describes; an int, which
    ctypes takes for a pointer without an object of its own."""
    return None if t is None else t.data_ptr()


def _flat(t: torch.Tensor | None):
    """Address of a contiguous tensor."""
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to libibp must be contiguous")
    return t.data_ptr()


class Pages:
    """A pool of pages: the slots and bitmask that ibp_compress writes, and
    the handle of their format.  Keeps the tensors alive; `slots` may be any
    contiguous tensor of at least n_slots * L bytes, on the GPU or pinned."""

    def __init__(self, meta: Meta, slots: torch.Tensor, n_slots: int, bitmask: torch.Tensor):
        _need(slots, int(n_slots) * meta.tensor_bytes, "slots")
        _need(bitmask, _bitmask_bytes(n_slots), "bitmask")
        self.meta, self.slots, self.n_slots, self.bitmask = meta, slots, int(n_slots), bitmask
        self.tensor_bytes = meta.tensor_bytes
        self._struct = ibp_pages(meta.handle, _flat(slots), self.n_slots, _flat(bitmask))

    @property
    def _as_parameter_(self):
        if not self.meta.handle:
            raise ValueError("the pool's handle has been closed")
        return ctypes.byref(self._struct)


def _typed(t: torch.Tensor, dtype: torch.dtype, what: str, numel: int | None = None):
    if t.dtype != dtype:
        raise ValueError(f"{what} must be {dtype}, not {t.dtype}")
    if numel is not None and t.numel() < numel:
        raise ValueError(f"{what} holds {t.numel()} entries, the call needs {numel}")


def _stream_of(stream, t: torch.Tensor):
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None and t.is_cuda:
        return _raw_stream(t.get_device())
    return _stream(None)


def _workspace(given: torch.Tensor | None, nbytes: int, like: torch.Tensor, stream):
    """The caller's workspace, or one of torch's allocator that outlives the
    call on the stream it is used on."""
    if given is not None:
        _need(given, nbytes, "workspace")
        return given
    if nbytes == 0:
        return None
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device=like.device)


def _bytes_of(t: torch.Tensor | None) -> int:
    return 0 if t is None else t.nbytes


def ibp_pages_copy(meta: Meta, src_slots: torch.Tensor, n_src: int, src_bitmask: torch.Tensor, src_ids: torch.Tensor,
                   dst_slots: torch.Tensor, n_dst: int, dst_bitmask: torch.Tensor, dst_ids: torch.Tensor,
                   stream=None):
    """Item and bit of slot src_ids[i] -> slot dst_ids[i], without decoding
    (-1 on either side: skipped)."""
    _typed(src_ids, torch.int64, "src_ids")
    _typed(dst_ids, torch.int64, "dst_ids", src_ids.numel())
    L = meta.tensor_bytes
    _need_all((src_slots, int(n_src) * L, "src_slots"), (dst_slots, int(n_dst) * L, "dst_slots"),
              (src_bitmask, _bitmask_bytes(n_src), "src_bitmask"), (dst_bitmask, _bitmask_bytes(n_dst), "dst_bitmask"))
    _check(lib().ibp_pages_copy(meta, _flat(src_slots), int(n_src), _flat(src_bitmask), _flat(src_ids), _flat(dst_slots),
                                int(n_dst), _flat(dst_bitmask), _flat(dst_ids), src_ids.numel(),
                                _stream_of(stream, src_ids)), "ibp_pages_copy")


def ibp_pages_workspace(n_slots: int, n: int = 0) -> int:
    return int(lib().ibp_pages_workspace(int(n_slots), int(n)))


def ibp_pages_alloc(meta: Meta, refs: torch.Tensor, n_slots: int, ids: torch.Tensor, workspace=None, stream=None):
    """ids <- the lowest free slots, in order; their counts become 1.  Their
    bitmask bits stay: see ibp_pages_alloc_raw."""
    _typed(refs, torch.int32, "refs", int(n_slots))
    _typed(ids, torch.int64, "ids")
    ws = _workspace(workspace, ibp_pages_workspace(n_slots), refs, stream)
    _check(lib().ibp_pages_alloc(meta, _flat(refs), int(n_slots), _flat(ids), ids.numel(), _flat(ws), _bytes_of(ws),
                                 _stream_of(stream, refs)), "ibp_pages_alloc")


def ibp_pages_alloc_raw(meta: Meta, refs: torch.Tensor, n_slots: int, bitmask: torch.Tensor, ids: torch.Tensor,
                        workspace=None, stream=None):
    """The same for pages that are written in place: the slots' bits in bitmask
    become 0 (raw)."""
    _typed(refs, torch.int32, "refs", int(n_slots))
    _typed(ids, torch.int64, "ids")
    _need(bitmask, _bitmask_bytes(n_slots), "bitmask")
    ws = _workspace(workspace, ibp_pages_workspace(n_slots), refs, stream)
    _check(lib().ibp_pages_alloc_raw(meta, _flat(refs), int(n_slots), _flat(bitmask), _flat(ids), ids.numel(), _flat(ws),
                                     _bytes_of(ws), _stream_of(stream, refs)), "ibp_pages_alloc_raw")


def _table_shape(table: torch.Tensor):
    _typed(table, torch.int64, "table")
    if table.dim() != 3:
        raise ValueError("a block table has the shape (sequences, heads, blocks)")
    return table.shape


def ibp_pages_fork(meta: Meta, slots: torch.Tensor, n_slots: int, bitmask: torch.Tensor, refs: torch.Tensor,
                   table: torch.Tensor, lens: torch.Tensor, parents: torch.Tensor, children: torch.Tensor, *,
                   page_tokens: int, workspace=None, stream=None):
    """Sequence children[i] of the table becomes a fork of parents[i]: full
    pages shared, the partly filled one copied into a free slot."""
    n_seqs, heads, blocks = _table_shape(table)
    n = parents.numel()
    _typed(refs, torch.int32, "refs", int(n_slots))
    _typed(lens, torch.int32, "lens", n_seqs)
    _typed(parents, torch.int64, "parents")
    _typed(children, torch.int64, "children", n)
    _need_all((slots, int(n_slots) * meta.tensor_bytes, "slots"), (bitmask, _bitmask_bytes(n_slots), "bitmask"))
    ws = _workspace(workspace, ibp_pages_workspace(n_slots, n * heads), refs, stream)
    _check(lib().ibp_pages_fork(meta, _flat(slots), int(n_slots), _flat(bitmask), _flat(refs), _flat(table), n_seqs, heads,
                                blocks, _flat(lens), int(page_tokens), _flat(parents), _flat(children), n, _flat(ws),
                                _bytes_of(ws), _stream_of(stream, refs)), "ibp_pages_fork")


def ibp_pages_free(meta: Meta, refs: torch.Tensor, n_slots: int, table: torch.Tensor, seqs: torch.Tensor, stream=None):
    """Releases every page in the rows `seqs` of the table."""
    n_seqs, heads, blocks = _table_shape(table)
    _typed(refs, torch.int32, "refs", int(n_slots))
    _typed(seqs, torch.int64, "seqs")
    _check(lib().ibp_pages_free(meta, _flat(refs), int(n_slots), _flat(table), n_seqs, heads, blocks, _flat(seqs),
                                seqs.numel(), _stream_of(stream, refs)), "ibp_pages_free")


def ibp_pages_compact(meta: Meta, slots: torch.Tensor, n_slots: int, bitmask: torch.Tensor, refs: torch.Tensor,
                      map: torch.Tensor, n_live: torch.Tensor, table: torch.Tensor | None = None, workspace=None,
                      stream=None):
    """Live pages moved to slots [0, n_live); map: each slot's new id; the
    table's ids are rewritten."""
    _typed(refs, torch.int32, "refs", int(n_slots))
    _typed(map, torch.int64, "map", int(n_slots))
    _typed(n_live, torch.int64, "n_live", 1)
    if table is not None:
        _typed(table, torch.int64, "table")
    _need_all((slots, int(n_slots) * meta.tensor_bytes, "slots"), (bitmask, _bitmask_bytes(n_slots), "bitmask"))
    ws = _workspace(workspace, ibp_pages_workspace(n_slots), refs, stream)
    _check(lib().ibp_pages_compact(meta, _flat(slots), int(n_slots), _flat(bitmask), _flat(refs), _flat(map), _flat(n_live),
                                   _flat(table), 0 if table is None else table.numel(), _flat(ws), _bytes_of(ws),
                                   _stream_of(stream, refs)), "ibp_pages_compact")


def _queries(q: torch.Tensor, table: torch.Tensor, page_tokens: int, scale: float = 1.0) -> ibp_attention:
    """Shape and strides of the queries (rows, heads, dims), whose dims are
    contiguous."""
    if q.dtype not in _DTYPES:
        raise ValueError(f"q must be bfloat16 or float16, not {q.dtype}")
    n_seqs, kv_heads, blocks = _table_shape(table)
    if q.dim() != 3:
        raise ValueError("q has the shape (rows, heads, dims)")
    rows, heads, dim = q.shape
    row_stride, head_stride, dim_stride = q.stride()
    if dim > 1 and dim_stride != 1:
        raise ValueError("q's dims must be contiguous")
    return ibp_attention(_DTYPES[q.dtype], dim, int(page_tokens), heads, kv_heads, scale, rows, n_seqs, blocks, 0, 0,
                         row_stride, head_stride, 0, 0)


def _outputs(q, out, lse, k: Pages, v: Pages):
    if out.dtype != q.dtype:
        raise ValueError(f"out must be {q.dtype}, not {out.dtype}")
    _need(out, q.numel() * 2, "out")
    if lse is not None:
        _typed(lse, torch.float32, "lse", q.shape[0] * q.shape[1])
    if k.tensor_bytes != v.tensor_bytes:
        raise ValueError("pages of keys and of values differ in size")
    row = 2 * q.shape[2]
    if row == 0 or k.tensor_bytes % row:
        raise ValueError(f"a page of {k.tensor_bytes} bytes holds no whole rows of {q.shape[2]} numbers")
    return k.tensor_bytes // row




def ibp_tree_attention(k: Pages, v: Pages, q: torch.Tensor, k_table: torch.Tensor, v_table: torch.Tensor,
                       lens: torch.Tensor, new_rows: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                       mask: torch.Tensor, out: torch.Tensor, lse: torch.Tensor | None = None, *, scale: float,
                       max_len: int = 0, max_new: int, workspace=None, stream=None):
    """Attention of drafted tokens (rows new_rows[s] .. new_rows[s + 1] of q,
    k_new, v_new) over their sequence's pages and over the drafted tokens whose
    bits their mask row (int64 words) has.  One token per sequence with mask 1
    is a decoding step.  ibp_check of k's handle has the call's errors, that of
    v's handle those of the values' pages and ids."""
    a = _queries(q, k_table, _outputs(q, out, lse, k, v), scale)
    if v_table.shape != k_table.shape or v_table.dtype != torch.int64:
        raise ValueError("the block tables of keys and values differ in shape or type")
    _typed(lens, torch.int32, "lens", a.n_seqs)
    _typed(new_rows, torch.int32, "new_rows", a.n_seqs + 1)
    shape = (q.shape[0], a.n_kv_heads, q.shape[2])
    for t, what in ((k_new, "k_new"), (v_new, "v_new")):
        if t.dtype != q.dtype or tuple(t.shape) != shape or (shape[2] > 1 and t.stride(2) != 1):
            raise ValueError(f"{what} must be {q.dtype} of shape {shape} with contiguous dims")
    if k_new.stride() != v_new.stride():
        raise ValueError("k_new and v_new must have the same strides")
    _typed(mask, torch.int64, "mask")
    if mask.dim() != 2 or mask.shape[0] < q.shape[0]:
        raise ValueError("mask has a row of int64 words for each row of q")
    a.new_row_stride, a.new_head_stride = k_new.stride(0), k_new.stride(1)
    a.max_len, a.max_new = int(max_len), int(max_new)
    ref = ctypes.byref(a)
    ws = _workspace(workspace, int(lib().ibp_tree_attention_workspace(ref)), q, stream)
    _check(lib().ibp_tree_attention(k, v, ref, _addr(q), _flat(k_table), _flat(v_table), _flat(lens), _flat(new_rows),
                                    _addr(k_new), _addr(v_new), _flat(mask), mask.shape[1], _flat(out),
                                    _flat(lse), _flat(ws), _bytes_of(ws), _stream_of(stream, q)), "ibp_tree_attention")


def ibp_page_bounds(k: Pages, ids: torch.Tensor, tokens: torch.Tensor | None, bounds: torch.Tensor, stream=None):
    """bounds (n_slots, 2, dims): smallest and largest number of the first
    tokens[i] tokens of page ids[i]."""
    _typed(ids, torch.int64, "ids")
    if bounds.dtype not in _DTYPES or bounds.dim() != 3 or bounds.shape[1] != 2 or bounds.shape[0] < k.n_slots:
        raise ValueError("bounds must be bfloat16 or float16 of shape (slots, 2, dims)")
    if tokens is not None:
        _typed(tokens, torch.int32, "tokens", ids.numel())
    _check(lib().ibp_page_bounds(k, _DTYPES[bounds.dtype], bounds.shape[2], _flat(ids), _flat(tokens), ids.numel(),
                                 _flat(bounds), _stream_of(stream, ids)), "ibp_page_bounds")


def _rows_of(a: ibp_attention, lens, row_seq):
    _typed(lens, torch.int32, "lens", a.n_rows)
    if row_seq is not None:
        _typed(row_seq, torch.int32, "row_seq", a.n_rows)
    elif a.n_rows > a.n_seqs:
        raise ValueError("more rows than sequences need row_seq")


def _block_lists(a: ibp_attention, blocks: torch.Tensor) -> int:
    _typed(blocks, torch.int32, "blocks")
    if blocks.dim() != 3 or blocks.shape[0] != a.n_rows or blocks.shape[1] != a.n_kv_heads:
        raise ValueError("blocks has the shape (rows, key/value heads, blocks)")
    return blocks.shape[2]


def ibp_select_pages(q: torch.Tensor, bounds: torch.Tensor, k_table: torch.Tensor, lens: torch.Tensor,
                     blocks: torch.Tensor, *, meta: Meta, page_tokens: int, keep_first: int = 0, keep_last: int = 0,
                     row_seq: torch.Tensor | None = None, workspace=None, stream=None):
    """blocks (rows, key/value heads, n) <- the block numbers that each query
    reads: the first and last ones kept, and those with the highest bound on
    the score; ascending, -1 behind."""
    a = _queries(q, k_table, page_tokens)
    if bounds.dtype != q.dtype or bounds.dim() != 3 or bounds.shape[1] != 2 or bounds.shape[2] != q.shape[2]:
        raise ValueError("bounds must be of q's type and of shape (slots, 2, dims)")
    _rows_of(a, lens, row_seq)
    n = _block_lists(a, blocks)
    ref = ctypes.byref(a)
    ws = _workspace(workspace, int(lib().ibp_select_pages_workspace(ref)), q, stream)
    _check(lib().ibp_select_pages(meta, ref, _addr(q), _flat(bounds), bounds.shape[0], _flat(k_table), _flat(lens),
                                  _flat(row_seq), int(keep_first), int(keep_last), _flat(blocks), n, _flat(ws),
                                  _bytes_of(ws), _stream_of(stream, q)), "ibp_select_pages")


def ibp_sparse_attention(k: Pages, v: Pages, q: torch.Tensor, k_table: torch.Tensor, v_table: torch.Tensor,
                         lens: torch.Tensor, blocks: torch.Tensor, out: torch.Tensor,
                         lse: torch.Tensor | None = None, *, scale: float, row_seq: torch.Tensor | None = None,
                         workspace=None, stream=None):
    """Attention of each row over the pages that `blocks` lists for it.  Errors
    as in ibp_tree_attention."""
    a = _queries(q, k_table, _outputs(q, out, lse, k, v), scale)
    if v_table.shape != k_table.shape or v_table.dtype != torch.int64:
        raise ValueError("the block tables of keys and values differ in shape or type")
    _rows_of(a, lens, row_seq)
    n = _block_lists(a, blocks)
    ref = ctypes.byref(a)
    ws = _workspace(workspace, int(lib().ibp_sparse_attention_workspace(ref, n)), q, stream)
    _check(lib().ibp_sparse_attention(k, v, ref, _addr(q), _flat(k_table), _flat(v_table), _flat(lens),
                                      _flat(row_seq), _flat(blocks), n, _flat(out), _flat(lse), _flat(ws), _bytes_of(ws),
                                      _stream_of(stream, q)), "ibp_sparse_attention")
