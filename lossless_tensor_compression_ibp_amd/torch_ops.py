"""PyTorch operator registration over the C ABI (FR/KO summary, "Contributions
clés": the method ships as PyTorch extensions over GPU libraries, and a
framework integration takes a few lines of Python).

The ops live in the ``ibp`` namespace (``torch.ops.ibp.*``) and forward to the
binding in ``ibp.py``; every byte of codec work runs in libibp.so.  A handle
(``ibp.Meta``) cannot cross the operator boundary, so ``register(meta)``
returns an integer key that the ops take instead.  Each op also has a fake
(shape-only) implementation, so graphs that call it can be traced.

    from lossless_tensor_compression_ibp_amd import ibp, torch_ops
    key = torch_ops.register(ibp.ibp_build_metadata(sample, 1024, L, W, M, T))
    slots, bitmask, stored = torch.ops.ibp.compress(key, rows)
    batch = torch.ops.ibp.gather_decompress(key, slots, bitmask, ids)

A cache of pages is passed as the handle's key, the slots (n, L) and the
bitmask; the attention ops take one of keys and one of values.
"""
from __future__ import annotations

import itertools
import threading

import torch

from . import ibp

_lock = threading.Lock()
_handles: dict[int, ibp.Meta] = {}
_next = itertools.count(1)


def register(meta: ibp.Meta) -> int:
    """Key under which the ops find `meta` (kept alive until release())."""
    with _lock:
        key = next(_next)
        _handles[key] = meta
    return key


def release(key: int) -> None:
    with _lock:
        _handles.pop(key, None)


def _meta(key: int) -> ibp.Meta:
    try:
        return _handles[key]
    except KeyError:
        raise ValueError(f"no IBP handle registered under key {key}") from None


def _tensor_bytes(key: int) -> int:
    params, _, _ = ibp.ibp_meta_get(_meta(key))
    return int(params["tensor_bytes"])


def _check_status(meta: ibp.Meta) -> None:
    st = ibp.ibp_check(meta)
    if st != ibp.IBP_OK:
        raise ibp.IBPError(st, "device-side check")


@torch.library.custom_op("ibp::compress", mutates_args=())
def compress(key: int, src: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """src: uint8 (n, L) on the GPU or pinned.  Returns (slots (n, L) uint8 on
    src's side, bitmask int32 (ceil(n/32),) and stored bytes int64 (n,) on the
    GPU)."""
    meta = _meta(key)
    n = src.shape[0]
    dev = torch.device("cuda", torch.cuda.current_device())
    if src.is_cuda:
        slots = torch.empty_like(src)
    else:
        slots = torch.empty(src.shape, dtype=torch.uint8, pin_memory=True)
    bitmask = torch.zeros(max(1, (n + 31) // 32), dtype=torch.int32, device=dev)
    stored = torch.zeros(n, dtype=torch.int64, device=dev)
    ibp.ibp_compress(meta, src, n, slots, bitmask, stored)
    return slots, bitmask, stored


@compress.register_fake
def _(key: int, src: torch.Tensor):
    n = src.shape[0]
    dev = src.device if src.is_cuda else torch.device("cuda")
    return (torch.empty_like(src), torch.empty(max(1, (n + 31) // 32), dtype=torch.int32, device=dev),
            torch.empty(n, dtype=torch.int64, device=dev))


@torch.library.custom_op("ibp::decompress", mutates_args=())
def decompress(key: int, slots: torch.Tensor, bitmask: torch.Tensor) -> torch.Tensor:
    """All n slots decoded into a new (n, L) uint8 tensor on the GPU."""
    meta = _meta(key)
    n = slots.shape[0]
    out = torch.empty((n, _tensor_bytes(key)), dtype=torch.uint8, device=bitmask.device)
    ibp.ibp_decompress(meta, slots, bitmask, n, out)
    return out


@decompress.register_fake
def _(key: int, slots: torch.Tensor, bitmask: torch.Tensor):
    return torch.empty((slots.shape[0], slots.shape[1]), dtype=torch.uint8, device=bitmask.device)


@torch.library.custom_op("ibp::gather_decompress", mutates_args=())
def gather_decompress(key: int, slots: torch.Tensor, bitmask: torch.Tensor, ids: torch.Tensor) -> torch.Tensor:
    """Rows ids (int64, GPU) of the slots decoded into a new (len(ids), L)
    uint8 tensor on the GPU."""
    meta = _meta(key)
    out = torch.empty((ids.numel(), _tensor_bytes(key)), dtype=torch.uint8, device=ids.device)
    ibp.ibp_gather_decompress(meta, slots, slots.shape[0], bitmask, ids, out)
    return out


@gather_decompress.register_fake
def _(key: int, slots: torch.Tensor, bitmask: torch.Tensor, ids: torch.Tensor):
    return torch.empty((ids.numel(), slots.shape[1]), dtype=torch.uint8, device=ids.device)


def _pages(key: int, slots: torch.Tensor, bitmask: torch.Tensor) -> ibp.Pages:
    return ibp.Pages(_meta(key), slots, slots.shape[0], bitmask)


@torch.library.custom_op("ibp::pages_copy", mutates_args=("dst_slots", "dst_bitmask"))
def pages_copy(key: int, src_slots: torch.Tensor, src_bitmask: torch.Tensor, src_ids: torch.Tensor,
               dst_slots: torch.Tensor, dst_bitmask: torch.Tensor, dst_ids: torch.Tensor) -> None:
    """Items and bits of slots src_ids -> slots dst_ids, without decoding."""
    ibp.ibp_pages_copy(_meta(key), src_slots, src_slots.shape[0], src_bitmask, src_ids, dst_slots, dst_slots.shape[0],
                       dst_bitmask, dst_ids)


@pages_copy.register_fake
def _(key: int, src_slots: torch.Tensor, src_bitmask: torch.Tensor, src_ids: torch.Tensor, dst_slots: torch.Tensor,
      dst_bitmask: torch.Tensor, dst_ids: torch.Tensor):
    return None


@torch.library.custom_op("ibp::page_bounds", mutates_args=("bounds",))
def page_bounds(key: int, slots: torch.Tensor, bitmask: torch.Tensor, ids: torch.Tensor, tokens: torch.Tensor | None,
                bounds: torch.Tensor) -> None:
    """bounds[id] (2, dims) <- smallest and largest number of the first tokens
    of pages ids (tokens None: of whole pages)."""
    ibp.ibp_page_bounds(_pages(key, slots, bitmask), ids, tokens, bounds)


@page_bounds.register_fake
def _(key: int, slots: torch.Tensor, bitmask: torch.Tensor, ids: torch.Tensor, tokens: torch.Tensor | None,
      bounds: torch.Tensor):
    return None


@torch.library.custom_op("ibp::select_pages", mutates_args=())
def select_pages(key: int, q: torch.Tensor, bounds: torch.Tensor, k_table: torch.Tensor, lens: torch.Tensor, n: int,
                 page_tokens: int, keep_first: int = 0, keep_last: int = 0,
                 row_seq: torch.Tensor | None = None) -> torch.Tensor:
    """Block numbers (rows, key/value heads, n) that each query reads."""
    blocks = torch.empty((q.shape[0], k_table.shape[1], n), dtype=torch.int32, device=q.device)
    ibp.ibp_select_pages(q, bounds, k_table, lens, blocks, meta=_meta(key), page_tokens=page_tokens,
                         keep_first=keep_first, keep_last=keep_last, row_seq=row_seq)
    return blocks


@select_pages.register_fake
def _(key: int, q: torch.Tensor, bounds: torch.Tensor, k_table: torch.Tensor, lens: torch.Tensor, n: int,
      page_tokens: int, keep_first: int = 0, keep_last: int = 0, row_seq: torch.Tensor | None = None):
    return torch.empty((q.shape[0], k_table.shape[1], n), dtype=torch.int32, device=q.device)


def _out_and_lse(q: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor]:
    return (torch.empty(q.shape, dtype=q.dtype, device=q.device),
            torch.empty(q.shape[:2], dtype=torch.float32, device=q.device))


@torch.library.custom_op("ibp::sparse_attention", mutates_args=())
def sparse_attention(k_key: int, k_slots: torch.Tensor, k_bitmask: torch.Tensor, v_key: int, v_slots: torch.Tensor,
                     v_bitmask: torch.Tensor, q: torch.Tensor, k_table: torch.Tensor, v_table: torch.Tensor,
                     lens: torch.Tensor, blocks: torch.Tensor, scale: float,
                     row_seq: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """(out, log-sum-exp) of each row over the pages that blocks lists for it."""
    out, lse = _out_and_lse(q)
    ibp.ibp_sparse_attention(_pages(k_key, k_slots, k_bitmask), _pages(v_key, v_slots, v_bitmask), q, k_table, v_table,
                             lens, blocks, out, lse, scale=scale, row_seq=row_seq)
    return out, lse


@sparse_attention.register_fake
def _(k_key: int, k_slots: torch.Tensor, k_bitmask: torch.Tensor, v_key: int, v_slots: torch.Tensor,
      v_bitmask: torch.Tensor, q: torch.Tensor, k_table: torch.Tensor, v_table: torch.Tensor, lens: torch.Tensor,
      blocks: torch.Tensor, scale: float, row_seq: torch.Tensor | None = None):
    return _out_and_lse(q)


@torch.library.custom_op("ibp::tree_attention", mutates_args=())
def tree_attention(k_key: int, k_slots: torch.Tensor, k_bitmask: torch.Tensor, v_key: int, v_slots: torch.Tensor,
                   v_bitmask: torch.Tensor, q: torch.Tensor, k_table: torch.Tensor, v_table: torch.Tensor,
                   lens: torch.Tensor, new_rows: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor,
                   mask: torch.Tensor, scale: float, max_new: int,
                   max_len: int = 0) -> tuple[torch.Tensor, torch.Tensor]:
    """(out, log-sum-exp) of drafted tokens over their sequence's pages and the
    drafted tokens that mask has.  Rows that belong to no sequence are zero,
    and their log-sum-exp minus infinity."""
    out, lse = _out_and_lse(q)
    out.zero_()
    lse.fill_(float("-inf"))
    ibp.ibp_tree_attention(_pages(k_key, k_slots, k_bitmask), _pages(v_key, v_slots, v_bitmask), q, k_table, v_table,
                           lens, new_rows, k_new, v_new, mask, out, lse, scale=scale, max_len=max_len, max_new=max_new)
    return out, lse


@tree_attention.register_fake
def _(k_key: int, k_slots: torch.Tensor, k_bitmask: torch.Tensor, v_key: int, v_slots: torch.Tensor,
      v_bitmask: torch.Tensor, q: torch.Tensor, k_table: torch.Tensor, v_table: torch.Tensor, lens: torch.Tensor,
      new_rows: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor, mask: torch.Tensor, scale: float, max_new: int,
      max_len: int = 0):
    return _out_and_lse(q)


def check(key: int) -> None:
    """Raises if a kernel latched an error (an id out of range, a corrupt
    record) since the last check; waits for the current stream."""
    _check_status(_meta(key))
