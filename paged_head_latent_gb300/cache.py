"""Binding of the cache's writers and readers, the staged chunk prefill and the page pool.

Argument checks and marshalling only, like the package's other calls (include/mla_paged.h
has the definitions).  Every tensor is on one CUDA device, the call runs there on ``stream``
(default: that device's current stream), and nothing synchronises.  What a call allocates
(outputs and a workspace that are not given) belongs to that stream too.
"""

from __future__ import annotations

import ctypes
from typing import Optional, Sequence, Tuple

import torch

from . import (FP8_TOKEN_BYTES, HEAD_DIM_CKV, HEAD_DIM_KPE, MlaDims, MlaError, MlaPool, MlaRopeDims, _cache_geometry,
               _new, lib, make_dims)

_BF16, _I32, _F32, _U8 = torch.bfloat16, torch.int32, torch.float32, torch.uint8
_raw_stream = torch._C._cuda_getCurrentRawStream
_entry = {}


def _check(name, t, dtype, index=None, contiguous=True):
    """Raise unless ``t`` is a (contiguous) CUDA tensor of ``dtype`` on device ``index``.
    The conditions that hold for every good argument are tested first and together: these
    calls take a few microseconds on the GPU, and so should their checks."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.is_cuda and (not contiguous or t.is_contiguous())
            and (index is None or t.get_device() == index)):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (there is no CPU path)")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if index is not None and t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, the other tensors on cuda:{index}")
    raise ValueError(f"{name} must be contiguous")


def _at(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _call(name, index, stream, *args):
    """The library's ``name`` on device ``index`` and ``stream`` (the last argument of every call)."""
    fn = _entry.get(name)
    if fn is None:
        fn = _entry[name] = getattr(lib(), name)
    raw = _raw_stream(index) if stream is None else stream.cuda_stream
    if torch.cuda.current_device() == index:
        st = fn(*args, raw)
    else:
        with torch.cuda.device(index):
            st = fn(*args, raw)
    if st != 0:
        raise MlaError(st, name)


def _bf16_caches(ckv_cache, kpe_cache, index=None):
    _check("ckv_cache", ckv_cache, _BF16, index)
    _check("kpe_cache", kpe_cache, _BF16, ckv_cache.get_device())
    return _cache_geometry(ckv_cache, kpe_cache)


def _fp8_cache(kv_fp8, index=None):
    _check("kv_fp8", kv_fp8, _U8, index)
    if kv_fp8.dim() != 3 or kv_fp8.shape[2] != FP8_TOKEN_BYTES:
        raise ValueError("kv_fp8 must be [num_pages, page_size, 656] uint8")
    return kv_fp8.shape[0], kv_fp8.shape[1]


def _ints(name, t, shape, index):
    _check(name, t, _I32, index)
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)} int32, got {list(t.shape)}")


def _buffer(name, t, shape, dtype, like, stream):
    """``t``, checked, or a new tensor on the device of ``like``."""
    if t is None:
        return _new(torch.empty, shape, dtype, like, stream)
    _check(name, t, dtype, like.get_device())
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    return t


def _scratch(make, need, like, stream, what):
    if need == 0:
        raise MlaError(-2, what)
    return _new(make, need, _U8, like, stream)


# ---------------------------------------------------------------- rotary positions and the cache write
def _rope_append(name, q_pe, ckv, k_pe, positions, inv_freq, slots, cache, geometry, q_out, sections, interleaved,
                 stream):
    index = ckv.get_device()
    _check("k_pe", k_pe, _BF16, index, False)
    tokens = ckv.shape[0]
    if ckv.shape != (tokens, HEAD_DIM_CKV) or k_pe.shape != (tokens, HEAD_DIM_KPE):
        raise ValueError("ckv must be [tokens, 512] and k_pe [tokens, 64]")
    _check("positions", positions, _I32, index)
    axes = positions.shape[0] if positions.dim() == 2 else positions.dim()
    if positions.dim() > 2 or not 1 <= axes <= 3 or positions.shape[-1] != tokens:
        raise ValueError("positions must be [tokens] or [axes, tokens] with one to three axes")
    if sections is None:
        if axes != 1:
            raise ValueError("sections (pairs of every axis) are needed with several axes")
        sections = (HEAD_DIM_KPE // 2,)
    if len(sections) != axes:
        raise ValueError("sections must name the pairs of every axis")
    _check("inv_freq", inv_freq, _F32, index)
    if inv_freq.shape != (HEAD_DIM_KPE // 2,):
        raise ValueError("inv_freq must be [32]")
    _ints("slots", slots, (tokens,), index)
    several = tokens > 1  # (the stride of a dimension of one element is never used)
    heads = q_token = q_head = 0
    if q_pe is None:
        if q_out is not None:
            raise ValueError("q_out without q_pe")
    else:
        _check("q_pe", q_pe, _BF16, index, False)
        if q_pe.dim() != 3 or q_pe.shape[0] != tokens or q_pe.shape[2] != HEAD_DIM_KPE:
            raise ValueError("q_pe must be [tokens, H, 64]")
        heads = q_pe.shape[1]
        q_token, q_head, last = q_pe.stride()
        if last != 1 and tokens and heads:
            raise ValueError("the last dimension of q_pe must be contiguous")
        q_out = _buffer("q_out", q_out, (tokens, heads, HEAD_DIM_KPE), _BF16, q_pe, stream)
    ckv_row, ckv_last = ckv.stride()
    kpe_row, kpe_last = k_pe.stride()
    if (ckv_last != 1 or kpe_last != 1) and tokens:
        raise ValueError("the last dimension of ckv and k_pe must be contiguous")
    dims = MlaRopeDims(tokens, heads, axes, tuple(sections), 1 if interleaved else 0, geometry[0], geometry[1],
                       q_token if several else 0, q_head if heads > 1 else 0, ckv_row if several else 0,
                       kpe_row if several else 0)
    _call(name, index, stream, _at(q_pe), ckv.data_ptr(), k_pe.data_ptr(), positions.data_ptr(), inv_freq.data_ptr(),
          slots.data_ptr(), _at(q_out), *cache, ctypes.byref(dims))
    return q_out


def mla_rope_append(q_pe, ckv, k_pe, positions, inv_freq, slots, ckv_cache, kpe_cache, q_out=None,
                    sections: Optional[Sequence[int]] = None, interleaved=True, stream=None):
    """Rotate q_pe [tokens, H, 64] (or None) and k_pe [tokens, 64] to ``positions`` ([tokens]
    or [axes, tokens] int32; ``sections``: pairs of each axis) and write ckv [tokens, 512] and
    the rotated keys to the bf16 cache's ``slots`` [tokens] (a slot outside the cache: not
    written).  inv_freq [32] float32.  The inputs may be slices of wider projections.
    Returns the rotated queries (q_out [tokens, H, 64]; None without q_pe)."""
    _check("ckv", ckv, _BF16, None, False)
    geometry = _bf16_caches(ckv_cache, kpe_cache, ckv.get_device())
    return _rope_append("mla_rope_append", q_pe, ckv, k_pe, positions, inv_freq, slots,
                        (ckv_cache.data_ptr(), kpe_cache.data_ptr()), geometry, q_out, sections, interleaved, stream)


def mla_rope_append_fp8(q_pe, ckv, k_pe, positions, inv_freq, slots, kv_fp8, q_out=None,
                        sections: Optional[Sequence[int]] = None, interleaved=True, stream=None):
    """``mla_rope_append`` into an FP8 cache: the latents are quantised in tiles of 128 (scale
    amax / 448, nearest E4M3), the rope part stays bf16."""
    _check("ckv", ckv, _BF16, None, False)
    geometry = _fp8_cache(kv_fp8, ckv.get_device())
    return _rope_append("mla_rope_append_fp8", q_pe, ckv, k_pe, positions, inv_freq, slots, (kv_fp8.data_ptr(),), geometry,
                        q_out, sections, interleaved, stream)


# ---------------------------------------------------------------- tokens read back, page copies
def _count(count, index):
    _check("count", count, _I32, index)
    if count.numel() != 1:
        raise ValueError("count must hold one int32")
    return count.data_ptr()


def _gather(name, cache, like, geometry, slots, ckv_out, kpe_out, count, stream):
    index = like.get_device()
    _check("slots", slots, _I32, index)
    if slots.dim() != 1:
        raise ValueError("slots must be [n]")
    n = slots.shape[0]
    ckv_out = _buffer("ckv_out", ckv_out, (n, HEAD_DIM_CKV), _BF16, like, stream)
    kpe_out = _buffer("kpe_out", kpe_out, (n, HEAD_DIM_KPE), _BF16, like, stream)
    _call(name, index, stream, *cache, slots.data_ptr(), n, None if count is None else _count(count, index),
          geometry[0], geometry[1], ckv_out.data_ptr(), kpe_out.data_ptr())
    return ckv_out, kpe_out


def mla_cache_gather(ckv_cache, kpe_cache, slots, ckv_out=None, kpe_out=None, count=None,
                     stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The cached tokens in ``slots`` [n] as contiguous rows (ckv [n, 512], kpe [n, 64]); zeros
    for a slot outside the cache.  ``count`` (one int32 on the device): rows at or past it are
    left as they were."""
    geometry = _bf16_caches(ckv_cache, kpe_cache)
    return _gather("mla_cache_gather", (ckv_cache.data_ptr(), kpe_cache.data_ptr()), ckv_cache, geometry, slots,
                   ckv_out, kpe_out, count, stream)


def mla_cache_gather_fp8(kv_fp8, slots, ckv_out=None, kpe_out=None, count=None,
                         stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """``mla_cache_gather`` from an FP8 cache: the bf16 values that the attention reads."""
    geometry = _fp8_cache(kv_fp8)
    return _gather("mla_cache_gather_fp8", (kv_fp8.data_ptr(),), kv_fp8, geometry, slots, ckv_out, kpe_out, count,
                   stream)


def _copy_pages(name, cache, index, geometry, src, dst, tokens, count, stream):
    _check("src", src, _I32, index)
    if src.dim() != 1:
        raise ValueError("src must be [n]")
    _ints("dst", dst, src.shape, index)
    if tokens is not None:
        _ints("tokens", tokens, src.shape, index)
    _call(name, index, stream, *cache, src.data_ptr(), dst.data_ptr(), _at(tokens), src.shape[0],
          None if count is None else _count(count, index), geometry[0], geometry[1])


def mla_cache_copy_pages(ckv_cache, kpe_cache, src, dst, tokens=None, count=None, stream=None) -> None:
    """Copy the first tokens[i] slots (all without ``tokens``) of page src[i] to page dst[i];
    entries with a page outside the cache copy nothing.  ``count`` (one int32 on the device):
    entries at or past it are not read."""
    geometry = _bf16_caches(ckv_cache, kpe_cache)
    _copy_pages("mla_cache_copy_pages", (ckv_cache.data_ptr(), kpe_cache.data_ptr()), ckv_cache.get_device(), geometry,
                src, dst, tokens, count, stream)


def mla_cache_copy_pages_fp8(kv_fp8, src, dst, tokens=None, count=None, stream=None) -> None:
    """``mla_cache_copy_pages`` for an FP8 cache."""
    geometry = _fp8_cache(kv_fp8)
    _copy_pages("mla_cache_copy_pages_fp8", (kv_fp8.data_ptr(),), kv_fp8.get_device(), geometry, src, dst, tokens,
                count, stream)


# ---------------------------------------------------------------- the staged chunk prefill
def workspace_bytes_prefill_staged(dims: MlaDims) -> int:
    return int(lib().mla_workspace_bytes_prefill_staged(ctypes.byref(dims)))


def workspace_bytes_prefill_fp8(dims: MlaDims) -> int:
    return int(lib().mla_workspace_bytes_prefill_fp8(ctypes.byref(dims)))


def _prefill(name, q_nope, q_pe, cache, geometry, qo_indptr, kv_indptr, kv_indices, sm_scale, out, lse, workspace, flags,
             num_workers, stream):
    index = q_nope.get_device()
    _check("q_pe", q_pe, _BF16, index)
    if q_nope.dim() != 3:
        raise ValueError("q_nope must be [total_q, H, 512]")
    rows, heads = q_nope.shape[0], q_nope.shape[1]
    if q_nope.shape != (rows, heads, HEAD_DIM_CKV) or q_pe.shape != (rows, heads, HEAD_DIM_KPE):
        raise ValueError("q_nope must be [total_q, H, 512] and q_pe [total_q, H, 64]")
    _check("qo_indptr", qo_indptr, _I32, index)
    _check("kv_indptr", kv_indptr, _I32, index)
    _check("kv_indices", kv_indices, _I32, index)
    batch = kv_indptr.numel() - 1
    if batch < 0 or qo_indptr.numel() != batch + 1:
        raise ValueError("qo_indptr and kv_indptr must both have batch + 1 entries")
    dims = make_dims(batch, heads, geometry[0], geometry[1], kv_indices.numel(), total_q=rows, num_workers=num_workers)
    out = _buffer("out", out, (rows, heads, HEAD_DIM_CKV), _BF16, q_nope, stream)
    lse = _buffer("lse", lse, (rows, heads), _F32, q_nope, stream)
    if workspace is None:
        with torch.cuda.device(index):
            need = workspace_bytes_prefill_staged(dims)
        workspace = _scratch(torch.zeros, need, q_nope, stream, "mla_workspace_bytes_prefill_staged")
    else:  # (the library checks its size)
        _check("workspace", workspace, _U8, index)
    _call(name, index, stream, q_nope.data_ptr(), q_pe.data_ptr(), *cache, qo_indptr.data_ptr(), kv_indptr.data_ptr(),
          kv_indices.data_ptr(), float(sm_scale), out.data_ptr(), lse.data_ptr(), ctypes.byref(dims), workspace.data_ptr(),
          workspace.numel(), int(flags))
    return out, lse


def mla_paged_prefill_staged(q_nope, q_pe, ckv_cache, kpe_cache, qo_indptr, kv_indptr, kv_indices, sm_scale, out=None,
                             lse=None, workspace=None, flags=0, num_workers=0,
                             stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Causal attention (bottom-right aligned) of a chunk of new tokens: what
    ``mla_paged_prefill`` computes, with the keys staged in the workspace and the query rows
    (token, head) in blocks of 128.  Returns (out, lse); rows behind qo_indptr's last request
    are left as they were."""
    _check("q_nope", q_nope, _BF16)
    geometry = _bf16_caches(ckv_cache, kpe_cache, q_nope.get_device())
    return _prefill("mla_paged_prefill_staged", q_nope, q_pe, (ckv_cache.data_ptr(), kpe_cache.data_ptr()), geometry,
                    qo_indptr, kv_indptr, kv_indices, sm_scale, out, lse, workspace, flags, num_workers, stream)


def mla_paged_prefill_fp8(q_nope, q_pe, kv_fp8, qo_indptr, kv_indptr, kv_indices, sm_scale, out=None, lse=None,
                          workspace=None, flags=0, num_workers=0,
                          stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """``mla_paged_prefill_staged`` over an FP8 cache kv_fp8 [num_pages, page_size, 656]."""
    _check("q_nope", q_nope, _BF16)
    geometry = _fp8_cache(kv_fp8, q_nope.get_device())
    return _prefill("mla_paged_prefill_fp8", q_nope, q_pe, (kv_fp8.data_ptr(),), geometry, qo_indptr, kv_indptr,
                    kv_indices, sm_scale, out, lse, workspace, flags, num_workers, stream)


# ---------------------------------------------------------------- the page pool
def workspace_bytes_pages(max_rows: int, num_pages: int, entries: int) -> int:
    """Workspace bytes of the pool's calls with up to ``entries`` entries."""
    pool = MlaPool(None, None, None, max_rows, 0, num_pages, 1)
    return int(lib().mla_workspace_bytes_pages(ctypes.byref(pool), int(entries)))


def _pool(block_table, seq_lens, ref_count, page_size):
    """The pool's description and device."""
    _check("block_table", block_table, _I32)
    index = block_table.get_device()
    if block_table.dim() != 2:
        raise ValueError("block_table must be [max_rows, max_blocks]")
    rows, blocks = block_table.shape
    _ints("seq_lens", seq_lens, (rows,), index)
    _check("ref_count", ref_count, _I32, index)
    if ref_count.dim() != 1:
        raise ValueError("ref_count must be [num_pages]")
    return MlaPool(block_table.data_ptr(), seq_lens.data_ptr(), ref_count.data_ptr(), rows, blocks, ref_count.shape[0],
                   page_size), index


def _entries(name, t, index):
    _check(name, t, _I32, index)
    if t.dim() != 1:
        raise ValueError(f"{name} must be [n]")
    return t.shape[0]


def _pool_scratch(workspace, pool, n, like, stream):
    if workspace is not None:  # (the library checks its size)
        _check("workspace", workspace, _U8, like.get_device())
        return workspace
    return _scratch(torch.empty, int(lib().mla_workspace_bytes_pages(ctypes.byref(pool), n)), like, stream,
                    "mla_workspace_bytes_pages")


def mla_pages_extend(block_table, seq_lens, ref_count, rows, new_tokens, page_size, capacity, new_indptr=None,
                     slots=None, results=None, workspace=None, stream=None):
    """Row rows[i] grows by new_tokens[i] tokens.  Returns (new_indptr [n + 1], slots
    [capacity], results [n]): where the granted tokens of every entry are in ``slots``, their
    token slots (-1 past the last), and 0 or the status of a refused entry (-6 bad index,
    -11 too few free pages).  A refused entry has no slots and the later ones move up: inputs
    packed by ``new_tokens`` have to be repacked by new_indptr before they go with ``slots``."""
    pool, index = _pool(block_table, seq_lens, ref_count, page_size)
    n = _entries("rows", rows, index)
    _ints("new_tokens", new_tokens, (n,), index)
    capacity = int(capacity)
    if capacity < 0:
        raise ValueError("capacity must not be negative")
    new_indptr = _buffer("new_indptr", new_indptr, (n + 1,), _I32, block_table, stream)
    slots = _buffer("slots", slots, (capacity,), _I32, block_table, stream)
    results = _buffer("results", results, (n,), _I32, block_table, stream)
    workspace = _pool_scratch(workspace, pool, n, block_table, stream)
    _call("mla_pages_extend", index, stream, ctypes.byref(pool), rows.data_ptr(), new_tokens.data_ptr(), n,
          new_indptr.data_ptr(), slots.data_ptr(), capacity, results.data_ptr(), workspace.data_ptr(),
          workspace.numel())
    return new_indptr, slots, results


def mla_pages_fork(block_table, seq_lens, ref_count, parents, children, page_size, src=None, dst=None,
                   copy_tokens=None, results=None, workspace=None, stream=None):
    """Row children[i] (empty) becomes a copy of row parents[i]; full pages are shared.
    Returns (results, src, dst, copy_tokens) [n]: the partly filled pages to copy with
    ``mla_cache_copy_pages(..., src, dst, tokens=copy_tokens)`` for every cache."""
    pool, index = _pool(block_table, seq_lens, ref_count, page_size)
    n = _entries("parents", parents, index)
    _ints("children", children, (n,), index)
    results = _buffer("results", results, (n,), _I32, block_table, stream)
    src = _buffer("src", src, (n,), _I32, block_table, stream)
    dst = _buffer("dst", dst, (n,), _I32, block_table, stream)
    copy_tokens = _buffer("copy_tokens", copy_tokens, (n,), _I32, block_table, stream)
    workspace = _pool_scratch(workspace, pool, n, block_table, stream)
    _call("mla_pages_fork", index, stream, ctypes.byref(pool), parents.data_ptr(), children.data_ptr(), n,
          src.data_ptr(), dst.data_ptr(), copy_tokens.data_ptr(), results.data_ptr(), workspace.data_ptr(),
          workspace.numel())
    return results, src, dst, copy_tokens


def mla_pages_free(block_table, seq_lens, ref_count, rows, page_size, stream=None) -> None:
    """The listed rows give up their pages and are empty."""
    pool, index = _pool(block_table, seq_lens, ref_count, page_size)
    n = _entries("rows", rows, index)
    _call("mla_pages_free", index, stream, ctypes.byref(pool), rows.data_ptr(), n)


def mla_pages_compact(block_table, seq_lens, ref_count, page_size, counts=None, src=None, dst=None, workspace=None,
                      stream=None):
    """Move the live pages to the front.  Returns (counts [2]: live pages and moves, src, dst
    [num_pages // 2]): the moves, to be copied with ``mla_cache_copy_pages(..., src, dst,
    count=counts[1:])`` for every cache."""
    pool, index = _pool(block_table, seq_lens, ref_count, page_size)
    moves = ref_count.shape[0] // 2
    counts = _buffer("counts", counts, (2,), _I32, block_table, stream)
    src = _buffer("src", src, (moves,), _I32, block_table, stream)
    dst = _buffer("dst", dst, (moves,), _I32, block_table, stream)
    workspace = _pool_scratch(workspace, pool, 0, block_table, stream)
    _call("mla_pages_compact", index, stream, ctypes.byref(pool), counts.data_ptr(), src.data_ptr(), dst.data_ptr(),
          workspace.data_ptr(), workspace.numel())
    return counts, src, dst
