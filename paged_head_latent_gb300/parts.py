"""Binding of the attention over parts of the cache: sliding windows with sinks, and prefixes
that several requests share, with the tables that name them.

Argument checks and marshalling only, like the package's other calls (include/mla_paged.h has
the definitions).  Every tensor is on one CUDA device, the call runs there on ``stream``
(default: that device's current stream), and nothing synchronises.  What a call allocates
(outputs and a workspace that are not given) belongs to that stream too.
"""

from __future__ import annotations

import ctypes
from typing import Tuple

import torch

from . import HEAD_DIM_CKV, HEAD_DIM_KPE, MlaDims, _cache_geometry, lib
from .cache import _BF16, _F32, _I32, _U8, _buffer, _call, _check, _fp8_cache, _scratch


# ---------------------------------------------------------------- the calls' common part
def _good(index, dtype, *tensors):
    """Whether these are contiguous tensors of ``dtype`` on CUDA device ``index``: the conditions that
    hold for good arguments, tested together (one check after the other took as long as the GPU's
    part of a small call)."""
    try:
        for t in tensors:
            if t.dtype is not dtype or t.get_device() != index or not t.is_contiguous():
                return False
    except AttributeError:
        return False
    return index >= 0


def _at(t):
    """The address of a tensor (what is none is refused by its check)."""
    return t.data_ptr() if isinstance(t, torch.Tensor) else None


def _numel(t):
    if not isinstance(t, torch.Tensor):
        raise TypeError("the lists must be torch.Tensors")
    return t.numel()


def _attend(name, q_nope, q_pe, cache, qo_indptr, ints, kv_indptr, kv_indices, middle, size, sm_scale, out, lse,
            workspace, flags, num_workers, stream):
    """``ints``: the names and tensors of the call's own lists; ``middle``: the arguments between the
    caches (and qo_indptr) and sm_scale; ``size``: (function, arguments) of the workspace size."""
    _check("q_nope", q_nope, _BF16)
    index = q_nope.get_device()
    shape = q_nope.shape
    fp8 = len(cache) == 1
    if not (_good(index, _BF16, q_pe, *(() if fp8 else cache))
            and _good(index, _I32, kv_indptr, kv_indices, *ints.values())
            and (not fp8 or _good(index, _U8, *cache)) and (qo_indptr is None or _good(index, _I32, qo_indptr))):
        _check("q_pe", q_pe, _BF16, index)
        for n, t in zip(("kv_fp8",) if fp8 else ("ckv_cache", "kpe_cache"), cache):
            _check(n, t, _U8 if fp8 else _BF16, index)
        for n, t in (("kv_indptr", kv_indptr), ("kv_indices", kv_indices), *ints.items()):
            _check(n, t, _I32, index)
        _check("qo_indptr", qo_indptr, _I32, index)
    if fp8:
        num_pages, page_size = _fp8_cache(cache[0], index)
    else:
        num_pages, page_size = _cache_geometry(*cache)
    if len(shape) != 3 or shape[2] != HEAD_DIM_CKV or q_pe.shape != (shape[0], shape[1], HEAD_DIM_KPE):
        raise ValueError("q_nope must be [rows, H, 512] and q_pe [rows, H, 64]")
    rows, heads, _ = shape
    batch = kv_indptr.numel() - 1
    if batch < 0:
        raise ValueError("kv_indptr must have batch + 1 entries")
    if qo_indptr is None:
        if "prefill" in name:
            raise TypeError("qo_indptr must be a torch.Tensor")
        if rows != batch:
            raise ValueError("decode: q_nope.shape[0] must equal len(kv_indptr) - 1")
        first = ()
    else:
        if qo_indptr.numel() != batch + 1:
            raise ValueError("qo_indptr and kv_indptr must both have batch + 1 entries")
        first = (qo_indptr.data_ptr(),)
    dims = MlaDims(batch, heads, HEAD_DIM_CKV, HEAD_DIM_KPE, num_pages, page_size, rows, kv_indices.numel(),
                   int(num_workers))
    if out is None and stream is None:
        out = torch.empty_like(q_nope)  # (quicker than by its shape)
    else:
        out = _buffer("out", out, shape, _BF16, q_nope, stream)
    lse = _buffer("lse", lse, (rows, heads), _F32, q_nope, stream)
    if workspace is None:
        with torch.cuda.device(index):
            need = size[0](dims, *size[1:])
        workspace = _scratch(torch.zeros, need, q_nope, stream, name + ": workspace size")
    elif not _good(index, _U8, workspace):  # (the library checks its size)
        _check("workspace", workspace, _U8, index)
    _call(name, index, stream, q_nope.data_ptr(), q_pe.data_ptr(), *[t.data_ptr() for t in cache], *first, *middle,
          float(sm_scale), out.data_ptr(), lse.data_ptr(), ctypes.byref(dims), workspace.data_ptr(), workspace.numel(),
          int(flags))
    return out, lse


# ---------------------------------------------------------------- sliding windows with sinks
def workspace_bytes_window(dims: MlaDims, window: int, sinks: int = 0, is_prefill: bool = False) -> int:
    """Workspace bytes of the window calls (0: such a call is refused).  ``is_prefill``: of the
    prefill calls, with dims.total_q query rows."""
    return int(lib().mla_workspace_bytes_window(ctypes.byref(dims), int(window), int(sinks), 1 if is_prefill else 0))


def _window(name, q_nope, q_pe, cache, qo_indptr, kv_indptr, kv_indices, window, sinks, sm_scale, out, lse, workspace,
            flags, num_workers, stream):
    window, sinks = int(window), int(sinks)
    if not 1 <= window < 2 ** 31 or not 0 <= sinks < 2 ** 31:
        raise ValueError("window must be at least 1 and sinks at least 0, both int32")
    return _attend(name, q_nope, q_pe, cache, qo_indptr, {}, kv_indptr, kv_indices,
                   (_at(kv_indptr), _at(kv_indices), window, sinks),
                   (workspace_bytes_window, window, sinks, qo_indptr is not None), sm_scale, out, lse, workspace, flags,
                   num_workers, stream)


def mla_paged_decode_window(q_nope, q_pe, ckv_cache, kpe_cache, kv_indptr, kv_indices, window, sinks, sm_scale,
                            out=None, lse=None, workspace=None, flags=0, num_workers=0,
                            stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """One query token per request over the last ``window`` and the first ``sinks`` of its keys.
    Arguments as for ``mla_paged_decode``; the lists name all keys of a request.  Returns (out, lse)."""
    return _window("mla_paged_decode_window", q_nope, q_pe, (ckv_cache, kpe_cache), None, kv_indptr,
                   kv_indices, window, sinks, sm_scale, out, lse, workspace, flags, num_workers, stream)


def mla_paged_decode_window_fp8(q_nope, q_pe, kv_fp8, kv_indptr, kv_indices, window, sinks, sm_scale, out=None, lse=None,
                                workspace=None, flags=0, num_workers=0,
                                stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """``mla_paged_decode_window`` over an FP8 cache kv_fp8 [num_pages, page_size, 656]."""
    return _window("mla_paged_decode_window_fp8", q_nope, q_pe, (kv_fp8,), None, kv_indptr, kv_indices,
                   window, sinks, sm_scale, out, lse, workspace, flags, num_workers, stream)


def mla_paged_prefill_window(q_nope, q_pe, ckv_cache, kpe_cache, qo_indptr, kv_indptr, kv_indices, window, sinks,
                             sm_scale, out=None, lse=None, workspace=None, flags=0, num_workers=0,
                             stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Causal attention of a chunk of new tokens in which every token sees the last ``window``
    keys up to its own and the first ``sinks``.  Arguments as for ``mla_paged_prefill_staged``."""
    return _window("mla_paged_prefill_window", q_nope, q_pe, (ckv_cache, kpe_cache), qo_indptr, kv_indptr,
                   kv_indices, window, sinks, sm_scale, out, lse, workspace, flags, num_workers, stream)


def mla_paged_prefill_window_fp8(q_nope, q_pe, kv_fp8, qo_indptr, kv_indptr, kv_indices, window, sinks, sm_scale,
                                 out=None, lse=None, workspace=None, flags=0, num_workers=0,
                                 stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """``mla_paged_prefill_window`` over an FP8 cache kv_fp8 [num_pages, page_size, 656]."""
    return _window("mla_paged_prefill_window_fp8", q_nope, q_pe, (kv_fp8,), qo_indptr, kv_indptr, kv_indices,
                   window, sinks, sm_scale, out, lse, workspace, flags, num_workers, stream)


# ---------------------------------------------------------------- prefixes shared by several requests
def workspace_bytes_shared(dims: MlaDims, groups: int, num_prefix_indices: int, is_prefill: bool = False) -> int:
    """Workspace bytes of the shared calls (0: such a call is refused).  ``is_prefill``: of the
    prefill calls, with dims.total_q query rows."""
    return int(lib().mla_workspace_bytes_shared(ctypes.byref(dims), int(groups), int(num_prefix_indices),
                                                1 if is_prefill else 0))


def _shared(name, q_nope, q_pe, cache, qo_indptr, group_indptr, prefix_indptr, prefix_indices, kv_indptr, kv_indices,
            sm_scale, out, lse, workspace, flags, num_workers, stream):
    groups, num_prefix = _numel(group_indptr) - 1, _numel(prefix_indices)
    if groups < 0 or _numel(prefix_indptr) != groups + 1:
        raise ValueError("group_indptr and prefix_indptr must both have groups + 1 entries")
    return _attend(name, q_nope, q_pe, cache, qo_indptr,
                   {"group_indptr": group_indptr, "prefix_indptr": prefix_indptr, "prefix_indices": prefix_indices},
                   kv_indptr, kv_indices, (group_indptr.data_ptr(), groups, prefix_indptr.data_ptr(),
                                           prefix_indices.data_ptr(), num_prefix, _at(kv_indptr), _at(kv_indices)),
                   (workspace_bytes_shared, groups, num_prefix, qo_indptr is not None), sm_scale, out, lse, workspace,
                   flags, num_workers, stream)


def mla_paged_decode_shared(q_nope, q_pe, ckv_cache, kpe_cache, group_indptr, prefix_indptr, prefix_indices, kv_indptr,
                            kv_indices, sm_scale, out=None, lse=None, workspace=None, flags=0, num_workers=0,
                            stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """One query token per request over the keys that its group shares (``prefix_*``) and those of
    its own (``kv_*``).  Group g: requests group_indptr[g] .. group_indptr[g + 1] - 1;
    ``block_table_to_shared_csr`` makes all five lists.  Rows of requests in no group are not
    written, neither in ``out`` and ``lse`` as given nor in new ones.  Returns (out, lse)."""
    return _shared("mla_paged_decode_shared", q_nope, q_pe, (ckv_cache, kpe_cache), None, group_indptr,
                   prefix_indptr, prefix_indices, kv_indptr, kv_indices, sm_scale, out, lse, workspace, flags,
                   num_workers, stream)


def mla_paged_decode_shared_fp8(q_nope, q_pe, kv_fp8, group_indptr, prefix_indptr, prefix_indices, kv_indptr,
                                kv_indices, sm_scale, out=None, lse=None, workspace=None, flags=0, num_workers=0,
                                stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """``mla_paged_decode_shared`` over an FP8 cache kv_fp8 [num_pages, page_size, 656]."""
    return _shared("mla_paged_decode_shared_fp8", q_nope, q_pe, (kv_fp8,), None, group_indptr, prefix_indptr,
                   prefix_indices, kv_indptr, kv_indices, sm_scale, out, lse, workspace, flags, num_workers, stream)


def mla_paged_prefill_shared(q_nope, q_pe, ckv_cache, kpe_cache, qo_indptr, group_indptr, prefix_indptr, prefix_indices,
                             kv_indptr, kv_indices, sm_scale, out=None, lse=None, workspace=None, flags=0,
                             num_workers=0, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Ragged chunks of new tokens behind a shared prefix: every token sees the whole prefix of
    its group, and causally the keys of its own request (``kv_*``: the new tokens' among them).
    Rows of requests in no group are not written."""
    return _shared("mla_paged_prefill_shared", q_nope, q_pe, (ckv_cache, kpe_cache), qo_indptr,
                   group_indptr, prefix_indptr, prefix_indices, kv_indptr, kv_indices, sm_scale, out, lse, workspace,
                   flags, num_workers, stream)


def mla_paged_prefill_shared_fp8(q_nope, q_pe, kv_fp8, qo_indptr, group_indptr, prefix_indptr, prefix_indices,
                                 kv_indptr, kv_indices, sm_scale, out=None, lse=None, workspace=None, flags=0,
                                 num_workers=0, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """``mla_paged_prefill_shared`` over an FP8 cache kv_fp8 [num_pages, page_size, 656]."""
    return _shared("mla_paged_prefill_shared_fp8", q_nope, q_pe, (kv_fp8,), qo_indptr, group_indptr,
                   prefix_indptr, prefix_indices, kv_indptr, kv_indices, sm_scale, out, lse, workspace, flags,
                   num_workers, stream)


# ---------------------------------------------------------------- the groups of a batch
def _room(name, capacity, t, most):
    if t is not None:
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.dim() != 1 or (capacity is not None and t.shape[0] != capacity):
            raise ValueError(f"{name} must be [capacity]")
        return t.shape[0]
    capacity = most if capacity is None else int(capacity)
    if capacity < 0:
        raise ValueError("capacities must not be negative")
    return capacity


def block_table_to_shared_csr(block_table, seq_lens, page_size, min_shared=1, prefix_capacity=None, capacity=None,
                              group_indptr=None, prefix_indptr=None, prefix_indices=None, kv_indptr=None,
                              kv_indices=None, stream=None):
    """The groups of neighbouring rows that share leading full pages, of a block table [batch,
    max_blocks] and seq_lens [batch] (int32, on the GPU).  A row joins its predecessor's group if
    they share at least ``min_shared`` keys (and one page).  Returns (group_indptr [batch + 1],
    prefix_indptr [batch + 1], prefix_indices [prefix_capacity], kv_indptr [batch + 1], kv_indices
    [capacity]), which ``mla_paged_decode_shared`` takes as they are.  The capacities default to what
    the table can name, and the attention's workspace follows them (1152 bytes an entry): smaller
    ones are fine where the lists fit.  Entries behind the end of a list are left as they were."""
    _check("block_table", block_table, _I32)
    index = block_table.get_device()
    _check("seq_lens", seq_lens, _I32, index)
    if block_table.dim() != 2 or seq_lens.shape != (block_table.shape[0],):
        raise ValueError("block_table must be [batch, max_blocks] and seq_lens [batch]")
    batch, max_blocks = block_table.shape
    page_size, min_shared = int(page_size), int(min_shared)
    if not 0 <= min_shared < 2 ** 31 or not 1 <= page_size < 2 ** 31:
        raise ValueError("page_size must be at least 1 and min_shared at least 0, both int32")
    most = max_blocks * page_size
    prefix_capacity = _room("prefix_indices", prefix_capacity, prefix_indices, batch // 2 * most)
    capacity = _room("kv_indices", capacity, kv_indices, batch * most)
    group_indptr = _buffer("group_indptr", group_indptr, (batch + 1,), _I32, block_table, stream)
    prefix_indptr = _buffer("prefix_indptr", prefix_indptr, (batch + 1,), _I32, block_table, stream)
    kv_indptr = _buffer("kv_indptr", kv_indptr, (batch + 1,), _I32, block_table, stream)
    prefix_indices = _buffer("prefix_indices", prefix_indices, (prefix_capacity,), _I32, block_table, stream)
    kv_indices = _buffer("kv_indices", kv_indices, (capacity,), _I32, block_table, stream)
    _call("mla_block_table_to_shared_csr", index, stream, block_table.data_ptr(), seq_lens.data_ptr(), batch,
          max_blocks, page_size, min_shared, group_indptr.data_ptr(), prefix_indptr.data_ptr(),
          prefix_indices.data_ptr(), prefix_capacity, kv_indptr.data_ptr(), kv_indices.data_ptr(), capacity)
    return group_indptr, prefix_indptr, prefix_indices, kv_indptr, kv_indices
