"""Binding of the cache's writers and readers, the FP8 chunk prefill and the page pool.

Argument checks and marshalling only, like the package's other calls (include/mla_paged.h
has the definitions).  Every tensor is on one CUDA device, the call runs there on ``stream``
(default: that device's current stream), and nothing synchronises.
"""

from __future__ import annotations

import ctypes
from typing import Optional, Sequence, Tuple

import torch

from . import (FP8_TOKEN_BYTES, HEAD_DIM_CKV, HEAD_DIM_KPE, MlaDims, MlaError, MlaPool, MlaRopeDims, _cache_geometry,
               lib, make_dims)

_NULL = ctypes.c_void_p(None)


def _check(name, t, dtype, dev=None, contiguous=True):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (there is no CPU path)")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if dev is not None and t.device != dev:
        raise ValueError(f"{name} is on {t.device}, the other tensors on {dev}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _at(t: Optional[torch.Tensor]):
    return _NULL if t is None else ctypes.c_void_p(t.data_ptr())


def _call(name, dev, stream, *args):
    """The library's ``name`` on ``dev`` and ``stream`` (the last argument of every call)."""
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    handle = ctypes.c_void_p(stream.cuda_stream)
    if torch.cuda.current_device() == dev.index:
        st = getattr(lib(), name)(*args, handle)
    else:
        with torch.cuda.device(dev):
            st = getattr(lib(), name)(*args, handle)
    if st != 0:
        raise MlaError(st, name)


def _bf16_caches(ckv_cache, kpe_cache, dev=None):
    _check("ckv_cache", ckv_cache, torch.bfloat16, dev)
    _check("kpe_cache", kpe_cache, torch.bfloat16, ckv_cache.device)
    return _cache_geometry(ckv_cache, kpe_cache)


def _fp8_cache(kv_fp8, dev=None):
    _check("kv_fp8", kv_fp8, torch.uint8, dev)
    if kv_fp8.dim() != 3 or kv_fp8.shape[2] != FP8_TOKEN_BYTES:
        raise ValueError("kv_fp8 must be [num_pages, page_size, 656] uint8")
    return kv_fp8.shape[0], kv_fp8.shape[1]


def _ints(name, t, shape, dev):
    _check(name, t, torch.int32, dev)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)} int32, got {list(t.shape)}")


def _buffer(name, t, shape, dtype, dev):
    """``t``, checked, or a new tensor."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    _check(name, t, dtype, dev)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    return t


def _scratch(workspace, need, dev, what):
    if need == 0:
        raise MlaError(-2, what)
    if workspace is None:
        return torch.zeros(need, dtype=torch.uint8, device=dev)
    _check("workspace", workspace, torch.uint8, dev)
    return workspace


# ---------------------------------------------------------------- rotary positions and the cache write
def _rope_append(name, q_pe, ckv, k_pe, positions, inv_freq, slots, cache, geometry, q_out, sections, interleaved,
                 stream):
    dev = ckv.device
    for n, t in (("ckv", ckv), ("k_pe", k_pe)):
        _check(n, t, torch.bfloat16, dev, contiguous=False)
    tokens = ckv.shape[0]
    if ckv.shape != (tokens, HEAD_DIM_CKV) or k_pe.shape != (tokens, HEAD_DIM_KPE):
        raise ValueError("ckv must be [tokens, 512] and k_pe [tokens, 64]")
    _check("positions", positions, torch.int32, dev)
    if positions.dim() == 1:
        positions = positions[None]
    if positions.dim() != 2 or not 1 <= positions.shape[0] <= 3 or positions.shape[1] != tokens:
        raise ValueError("positions must be [tokens] or [axes, tokens] with one to three axes")
    axes = positions.shape[0]
    if sections is None:
        if axes != 1:
            raise ValueError("sections (pairs of every axis) are needed with several axes")
        sections = (HEAD_DIM_KPE // 2,)
    if len(sections) != axes:
        raise ValueError("sections must name the pairs of every axis")
    _check("inv_freq", inv_freq, torch.float32, dev)
    if inv_freq.shape != (HEAD_DIM_KPE // 2,):
        raise ValueError("inv_freq must be [32]")
    _ints("slots", slots, (tokens,), dev)
    heads, strides = 0, (0, 0)
    if q_pe is None:
        if q_out is not None:
            raise ValueError("q_out without q_pe")
    else:
        _check("q_pe", q_pe, torch.bfloat16, dev, contiguous=False)
        if q_pe.dim() != 3 or q_pe.shape[0] != tokens or q_pe.shape[2] != HEAD_DIM_KPE:
            raise ValueError("q_pe must be [tokens, H, 64]")
        heads = q_pe.shape[1]
        # (the stride of a dimension of one element is never used)
        strides = (q_pe.stride(0) if tokens > 1 else 0, q_pe.stride(1) if heads > 1 else 0)
        q_out = _buffer("q_out", q_out, (tokens, heads, HEAD_DIM_KPE), torch.bfloat16, dev)
    for n, t in (("q_pe", q_pe), ("ckv", ckv), ("k_pe", k_pe)):
        if t is not None and t.numel() and t.stride(-1) != 1:
            raise ValueError(f"the last dimension of {n} must be contiguous")
    row = [t.stride(0) if tokens > 1 else 0 for t in (ckv, k_pe)]
    dims = MlaRopeDims(tokens, heads, axes, (ctypes.c_int32 * 3)(*[int(x) for x in sections]), 1 if interleaved else 0,
                       geometry[0], geometry[1], strides[0], strides[1], row[0], row[1])
    _call(name, dev, stream, _at(q_pe), _at(ckv), _at(k_pe), _at(positions), _at(inv_freq), _at(slots), _at(q_out),
          *[_at(c) for c in cache], ctypes.byref(dims))
    return q_out


def mla_rope_append(q_pe, ckv, k_pe, positions, inv_freq, slots, ckv_cache, kpe_cache, q_out=None,
                    sections: Optional[Sequence[int]] = None, interleaved=True, stream=None):
    """Rotate q_pe [tokens, H, 64] (or None) and k_pe [tokens, 64] to ``positions`` ([tokens]
    or [axes, tokens] int32; ``sections``: pairs of each axis) and write ckv [tokens, 512] and
    the rotated keys to the bf16 cache's ``slots`` [tokens] (a slot outside the cache: not
    written).  inv_freq [32] float32.  The inputs may be slices of wider projections.
    Returns the rotated queries (q_out [tokens, H, 64]; None without q_pe)."""
    geometry = _bf16_caches(ckv_cache, kpe_cache, ckv.device)
    return _rope_append("mla_rope_append", q_pe, ckv, k_pe, positions, inv_freq, slots, (ckv_cache, kpe_cache),
                        geometry, q_out, sections, interleaved, stream)


def mla_rope_append_fp8(q_pe, ckv, k_pe, positions, inv_freq, slots, kv_fp8, q_out=None,
                        sections: Optional[Sequence[int]] = None, interleaved=True, stream=None):
    """``mla_rope_append`` into an FP8 cache: the latents are quantised in tiles of 128 (scale
    amax / 448, nearest E4M3), the rope part stays bf16."""
    geometry = _fp8_cache(kv_fp8, ckv.device)
    return _rope_append("mla_rope_append_fp8", q_pe, ckv, k_pe, positions, inv_freq, slots, (kv_fp8,), geometry, q_out,
                        sections, interleaved, stream)


# ---------------------------------------------------------------- tokens read back, page copies
def _gather(name, cache, geometry, slots, ckv_out, kpe_out, count, stream):
    dev = cache[0].device
    _check("slots", slots, torch.int32, dev)
    if slots.dim() != 1:
        raise ValueError("slots must be [n]")
    n = slots.shape[0]
    ckv_out = _buffer("ckv_out", ckv_out, (n, HEAD_DIM_CKV), torch.bfloat16, dev)
    kpe_out = _buffer("kpe_out", kpe_out, (n, HEAD_DIM_KPE), torch.bfloat16, dev)
    if count is not None:
        _count(count, dev)
    _call(name, dev, stream, *[_at(c) for c in cache], _at(slots), n, _at(count), geometry[0], geometry[1],
          _at(ckv_out), _at(kpe_out))
    return ckv_out, kpe_out


def _count(count, dev):
    _check("count", count, torch.int32, dev)
    if count.numel() != 1:
        raise ValueError("count must hold one int32")


def mla_cache_gather(ckv_cache, kpe_cache, slots, ckv_out=None, kpe_out=None, count=None,
                     stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The cached tokens in ``slots`` [n] as contiguous rows (ckv [n, 512], kpe [n, 64]); zeros
    for a slot outside the cache.  ``count`` (one int32 on the device): rows at or past it are
    left as they were."""
    geometry = _bf16_caches(ckv_cache, kpe_cache)
    return _gather("mla_cache_gather", (ckv_cache, kpe_cache), geometry, slots, ckv_out, kpe_out, count, stream)


def mla_cache_gather_fp8(kv_fp8, slots, ckv_out=None, kpe_out=None, count=None,
                         stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """``mla_cache_gather`` from an FP8 cache: the bf16 values that the attention reads."""
    return _gather("mla_cache_gather_fp8", (kv_fp8,), _fp8_cache(kv_fp8), slots, ckv_out, kpe_out, count, stream)


def _copy_pages(name, cache, geometry, src, dst, tokens, count, stream):
    dev = cache[0].device
    _check("src", src, torch.int32, dev)
    if src.dim() != 1:
        raise ValueError("src must be [n]")
    _ints("dst", dst, src.shape, dev)
    if tokens is not None:
        _ints("tokens", tokens, src.shape, dev)
    if count is not None:
        _count(count, dev)
    _call(name, dev, stream, *[_at(c) for c in cache], _at(src), _at(dst), _at(tokens), src.shape[0], _at(count),
          geometry[0], geometry[1])


def mla_cache_copy_pages(ckv_cache, kpe_cache, src, dst, tokens=None, count=None, stream=None) -> None:
    """Copy the first tokens[i] slots (all without ``tokens``) of page src[i] to page dst[i];
    entries with a page outside the cache copy nothing.  ``count`` (one int32 on the device):
    entries at or past it are not read."""
    geometry = _bf16_caches(ckv_cache, kpe_cache)
    _copy_pages("mla_cache_copy_pages", (ckv_cache, kpe_cache), geometry, src, dst, tokens, count, stream)


def mla_cache_copy_pages_fp8(kv_fp8, src, dst, tokens=None, count=None, stream=None) -> None:
    """``mla_cache_copy_pages`` for an FP8 cache."""
    _copy_pages("mla_cache_copy_pages_fp8", (kv_fp8,), _fp8_cache(kv_fp8), src, dst, tokens, count, stream)


# ---------------------------------------------------------------- the FP8 chunk prefill
def workspace_bytes_prefill_fp8(dims: MlaDims) -> int:
    return int(lib().mla_workspace_bytes_prefill_fp8(ctypes.byref(dims)))


def mla_paged_prefill_fp8(q_nope, q_pe, kv_fp8, qo_indptr, kv_indptr, kv_indices, sm_scale, out=None, lse=None,
                          workspace=None, flags=0, num_workers=0,
                          stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Causal attention (bottom-right aligned) of a chunk of new tokens over an FP8 cache:
    ``mla_paged_prefill`` with kv_fp8 [num_pages, page_size, 656].  Returns (out, lse); rows
    behind qo_indptr's last request are left as they were."""
    dev = q_nope.device
    for n, t in (("q_nope", q_nope), ("q_pe", q_pe)):
        _check(n, t, torch.bfloat16, dev)
    if q_nope.dim() != 3:
        raise ValueError("q_nope must be [total_q, H, 512]")
    rows, heads = q_nope.shape[0], q_nope.shape[1]
    if q_nope.shape != (rows, heads, HEAD_DIM_CKV) or q_pe.shape != (rows, heads, HEAD_DIM_KPE):
        raise ValueError("q_nope must be [total_q, H, 512] and q_pe [total_q, H, 64]")
    num_pages, page_size = _fp8_cache(kv_fp8, dev)
    for n, t in (("qo_indptr", qo_indptr), ("kv_indptr", kv_indptr), ("kv_indices", kv_indices)):
        _check(n, t, torch.int32, dev)
    batch = kv_indptr.numel() - 1
    if batch < 0 or qo_indptr.numel() != batch + 1:
        raise ValueError("qo_indptr and kv_indptr must both have batch + 1 entries")
    dims = make_dims(batch, heads, num_pages, page_size, kv_indices.numel(), total_q=rows, num_workers=num_workers)
    out = _buffer("out", out, (rows, heads, HEAD_DIM_CKV), torch.bfloat16, dev)
    lse = _buffer("lse", lse, (rows, heads), torch.float32, dev)
    with torch.cuda.device(dev):
        need = workspace_bytes_prefill_fp8(dims)
    workspace = _scratch(workspace, need, dev, "mla_workspace_bytes_prefill_fp8")
    _call("mla_paged_prefill_fp8", dev, stream, _at(q_nope), _at(q_pe), _at(kv_fp8), _at(qo_indptr), _at(kv_indptr),
          _at(kv_indices), float(sm_scale), _at(out), _at(lse), ctypes.byref(dims), _at(workspace), workspace.numel(),
          int(flags))
    return out, lse


# ---------------------------------------------------------------- the page pool
def workspace_bytes_pages(max_rows: int, num_pages: int, entries: int) -> int:
    """Workspace bytes of the pool's calls with up to ``entries`` entries."""
    pool = MlaPool(None, None, None, max_rows, 0, num_pages, 1)
    return int(lib().mla_workspace_bytes_pages(ctypes.byref(pool), int(entries)))


def _pool(block_table, seq_lens, ref_count, page_size) -> MlaPool:
    _check("block_table", block_table, torch.int32)
    if block_table.dim() != 2:
        raise ValueError("block_table must be [max_rows, max_blocks]")
    _ints("seq_lens", seq_lens, block_table.shape[:1], block_table.device)
    _check("ref_count", ref_count, torch.int32, block_table.device)
    if ref_count.dim() != 1:
        raise ValueError("ref_count must be [num_pages]")
    return MlaPool(block_table.data_ptr(), seq_lens.data_ptr(), ref_count.data_ptr(), block_table.shape[0],
                   block_table.shape[1], ref_count.shape[0], int(page_size))


def _pool_scratch(workspace, pool, n, dev):
    if workspace is not None:  # (the library checks its size)
        _check("workspace", workspace, torch.uint8, dev)
        return workspace
    return _scratch(None, int(lib().mla_workspace_bytes_pages(ctypes.byref(pool), n)), dev,
                    "mla_workspace_bytes_pages")


def mla_pages_extend(block_table, seq_lens, ref_count, rows, new_tokens, page_size, capacity, new_indptr=None,
                     slots=None, results=None, workspace=None, stream=None):
    """Row rows[i] grows by new_tokens[i] tokens.  Returns (new_indptr [n + 1], slots
    [capacity], results [n]): where the granted tokens of every entry are in ``slots``, their
    token slots (-1 past the last), and 0 or the status of a refused entry (-6 bad index,
    -11 too few free pages)."""
    dev = block_table.device
    pool = _pool(block_table, seq_lens, ref_count, page_size)
    _check("rows", rows, torch.int32, dev)
    n = rows.numel()
    _ints("rows", rows, (n,), dev)
    _ints("new_tokens", new_tokens, (n,), dev)
    capacity = int(capacity)
    if capacity < 0:
        raise ValueError("capacity must not be negative")
    new_indptr = _buffer("new_indptr", new_indptr, (n + 1,), torch.int32, dev)
    slots = _buffer("slots", slots, (capacity,), torch.int32, dev)
    results = _buffer("results", results, (n,), torch.int32, dev)
    workspace = _pool_scratch(workspace, pool, n, dev)
    _call("mla_pages_extend", dev, stream, ctypes.byref(pool), _at(rows), _at(new_tokens), n, _at(new_indptr),
          _at(slots), capacity, _at(results), _at(workspace), workspace.numel())
    return new_indptr, slots, results


def mla_pages_fork(block_table, seq_lens, ref_count, parents, children, page_size, src=None, dst=None,
                   copy_tokens=None, results=None, workspace=None, stream=None):
    """Row children[i] (empty) becomes a copy of row parents[i]; full pages are shared.
    Returns (results, src, dst, copy_tokens) [n]: the partly filled pages to copy with
    ``mla_cache_copy_pages(..., src, dst, tokens=copy_tokens)`` for every cache."""
    dev = block_table.device
    pool = _pool(block_table, seq_lens, ref_count, page_size)
    _check("parents", parents, torch.int32, dev)
    n = parents.numel()
    _ints("parents", parents, (n,), dev)
    _ints("children", children, (n,), dev)
    results = _buffer("results", results, (n,), torch.int32, dev)
    src = _buffer("src", src, (n,), torch.int32, dev)
    dst = _buffer("dst", dst, (n,), torch.int32, dev)
    copy_tokens = _buffer("copy_tokens", copy_tokens, (n,), torch.int32, dev)
    workspace = _pool_scratch(workspace, pool, n, dev)
    _call("mla_pages_fork", dev, stream, ctypes.byref(pool), _at(parents), _at(children), n, _at(src), _at(dst),
          _at(copy_tokens), _at(results), _at(workspace), workspace.numel())
    return results, src, dst, copy_tokens


def mla_pages_free(block_table, seq_lens, ref_count, rows, page_size, stream=None) -> None:
    """The listed rows give up their pages and are empty."""
    dev = block_table.device
    pool = _pool(block_table, seq_lens, ref_count, page_size)
    _check("rows", rows, torch.int32, dev)
    _call("mla_pages_free", dev, stream, ctypes.byref(pool), _at(rows), rows.numel())


def mla_pages_compact(block_table, seq_lens, ref_count, page_size, counts=None, src=None, dst=None, workspace=None,
                      stream=None):
    """Move the live pages to the front.  Returns (counts [2]: live pages and moves, src, dst
    [num_pages // 2]): the moves, to be copied with ``mla_cache_copy_pages(..., src, dst,
    count=counts[1:])`` for every cache."""
    dev = block_table.device
    pool = _pool(block_table, seq_lens, ref_count, page_size)
    moves = ref_count.shape[0] // 2
    counts = _buffer("counts", counts, (2,), torch.int32, dev)
    src = _buffer("src", src, (moves,), torch.int32, dev)
    dst = _buffer("dst", dst, (moves,), torch.int32, dev)
    workspace = _pool_scratch(workspace, pool, 0, dev)
    _call("mla_pages_compact", dev, stream, ctypes.byref(pool), _at(counts), _at(src), _at(dst), _at(workspace),
          workspace.numel())
    return counts, src, dst
