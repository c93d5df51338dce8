"""C-ABI refusals of the cache's writers, readers, chunk prefill and page pool; every case
fails (or is a no-op) on the host before any CUDA call."""

import ctypes

import pytest

FAKE = 0x10000  # never dereferenced
V = ctypes.c_void_p
NULL, DIMS, ALIGN, WORKSPACE = -1, -2, -3, -4


def _rope_dims(lib, **kw):
    d = dict(tokens=4, num_qo_heads=2, num_axes=1, section=(32, 0, 0), interleaved=1, num_pages=3, page_size=16,
             q_stride_token=128, q_stride_head=64, ckv_stride=512, kpe_stride=64)
    d.update(kw)
    d["section"] = (ctypes.c_int32 * 3)(*d["section"])
    return lib.MlaRopeDims(**d)


def _append(lib, fp8=False, null=(), off=(), **kw):
    names = ["q_pe", "ckv", "k_pe", "positions", "inv_freq", "slots", "q_out"] + (["kv"] if fp8 else ["ckv_c", "kpe_c"])
    ptrs = [V(0 if n in null else FAKE + (8 if n in off else 0)) for n in names]
    f = lib.lib().mla_rope_append_fp8 if fp8 else lib.lib().mla_rope_append
    dims = _rope_dims(lib, **kw)
    return f(*ptrs, ctypes.byref(dims), None)


@pytest.mark.parametrize("fp8", [False, True])
def test_rope_append_refusals(lib, fp8):
    bad = [dict(tokens=-1), dict(num_qo_heads=129), dict(num_qo_heads=-1), dict(num_axes=0), dict(num_axes=4),
           dict(section=(31, 0, 0)), dict(section=(32, 5, 0), num_axes=2), dict(section=(40, -8, 0), num_axes=2),
           dict(page_size=0), dict(num_pages=1 << 20, page_size=1 << 12), dict(ckv_stride=-8)]
    for kw in bad:
        assert _append(lib, fp8, **kw) == DIMS, kw
    for n in ("q_pe", "ckv", "k_pe", "positions", "inv_freq", "slots", "q_out", "kv" if fp8 else "kpe_c"):
        assert _append(lib, fp8, null=(n,)) == NULL, n
    for n in ("q_pe", "ckv", "k_pe", "q_out", "kv" if fp8 else "ckv_c"):
        assert _append(lib, fp8, off=(n,)) == ALIGN, n
    for kw in (dict(q_stride_token=130), dict(q_stride_head=68), dict(ckv_stride=516), dict(kpe_stride=65)):
        assert _append(lib, fp8, **kw) == ALIGN, kw
    assert _append(lib, fp8, tokens=0, null=("ckv", "slots")) == 0
    f = lib.lib().mla_rope_append_fp8 if fp8 else lib.lib().mla_rope_append
    assert f(*([V(FAKE)] * (8 if fp8 else 9)), None, None) == NULL


def test_gather_and_copy_refusals(lib):
    g = lib.lib().mla_cache_gather
    p, q = V(FAKE), V(FAKE + 8)
    assert g(p, p, p, -1, None, 4, 16, p, p, None) == DIMS
    assert g(p, p, p, 3, None, 4, 0, p, p, None) == DIMS
    assert g(None, p, p, 3, None, 4, 16, p, p, None) == NULL
    assert g(p, p, None, 3, None, 4, 16, p, p, None) == NULL
    assert g(p, p, p, 3, None, 4, 16, None, p, None) == NULL
    assert g(p, q, p, 3, None, 4, 16, p, p, None) == ALIGN
    assert g(p, p, p, 3, None, 4, 16, p, q, None) == ALIGN
    assert g(p, p, None, 0, None, 4, 16, None, None, None) == 0
    g = lib.lib().mla_cache_gather_fp8
    assert g(q, p, 3, None, 4, 16, p, p, None) == ALIGN
    assert g(None, p, 3, None, 4, 16, p, p, None) == NULL
    c = lib.lib().mla_cache_copy_pages
    assert c(p, p, p, p, None, -1, None, 4, 16, None) == DIMS
    assert c(p, None, p, p, None, 1, None, 4, 16, None) == NULL
    assert c(p, p, None, p, None, 1, None, 4, 16, None) == NULL
    assert c(p, q, p, p, None, 1, None, 4, 16, None) == ALIGN
    assert c(p, p, None, None, None, 0, None, 4, 16, None) == 0
    c = lib.lib().mla_cache_copy_pages_fp8
    assert c(None, p, p, None, 1, None, 4, 16, None) == NULL
    assert c(q, p, p, None, 1, None, 4, 16, None) == ALIGN


def _pool(lib, null=(), **kw):
    d = dict(block_table=FAKE, seq_lens=FAKE, ref_count=FAKE, max_rows=4, max_blocks=8, num_pages=32, page_size=16)
    d.update(kw)
    d.update({n: None for n in null})
    return lib.MlaPool(**d)


def test_pool_refusals(lib):
    L, p = lib.lib(), V(FAKE)
    by = ctypes.byref

    def extend(pool, n=2, cap=8, ws=p, size=1 << 20, rows=p, ptr=p, slots=p):
        return L.mla_pages_extend(by(pool) if pool else None, rows, p, n, ptr, slots, cap, p, ws, size, None)

    for kw in (dict(max_rows=-1), dict(max_blocks=-1), dict(page_size=0), dict(num_pages=1 << 27),
               dict(max_blocks=1 << 27)):
        assert extend(_pool(lib, **kw)) == DIMS, kw
        assert L.mla_pages_free(by(_pool(lib, **kw)), p, 1, None) == DIMS
        assert L.mla_pages_fork(by(_pool(lib, **kw)), p, p, 1, p, p, p, p, p, 1 << 20, None) == DIMS
        assert L.mla_pages_compact(by(_pool(lib, **kw)), p, p, p, p, 1 << 20, None) == DIMS
        assert L.mla_workspace_bytes_pages(by(_pool(lib, **kw)), 1) == 0
    for n in ("block_table", "seq_lens", "ref_count"):
        assert extend(_pool(lib, null=(n,))) == NULL
        assert L.mla_pages_free(by(_pool(lib, null=(n,))), p, 1, None) == NULL
        assert L.mla_pages_compact(by(_pool(lib, null=(n,))), p, p, p, p, 1 << 20, None) == NULL
    pool = _pool(lib)
    assert extend(None) == NULL
    assert extend(pool, n=-1) == DIMS
    assert extend(pool, cap=-1) == DIMS
    assert extend(pool, rows=None) == NULL and extend(pool, ptr=None) == NULL and extend(pool, slots=None) == NULL
    assert extend(pool, ws=None) == WORKSPACE and extend(pool, size=16) == WORKSPACE
    assert extend(pool, ws=V(FAKE + 8)) == ALIGN
    assert L.mla_pages_fork(by(pool), p, None, 1, p, p, p, p, p, 1 << 20, None) == NULL
    assert L.mla_pages_fork(by(pool), p, p, 1, p, p, p, p, p, 16, None) == WORKSPACE
    assert L.mla_pages_fork(by(pool), None, None, 0, None, None, None, None, None, 0, None) == 0
    assert L.mla_pages_free(by(pool), None, 1, None) == NULL
    assert L.mla_pages_free(by(pool), None, 0, None) == 0
    assert L.mla_pages_compact(by(pool), None, p, p, p, 1 << 20, None) == NULL
    assert L.mla_pages_compact(by(pool), p, None, p, p, 1 << 20, None) == NULL
    assert L.mla_pages_compact(by(pool), p, p, p, p, 16, None) == WORKSPACE


def test_workspace_of_more_entries_serves_fewer(lib):
    sizes = [lib.workspace_bytes_pages(100, 5000, n) for n in (0, 1, 100, 1000)]
    assert sizes == sorted(sizes) and sizes[0] > 0


def _prefill(lib, dims, null=(), off=(), ws=FAKE, size=1 << 40, flags=0):
    names = ["q_nope", "q_pe", "kv", "qo", "kp", "ki"]
    ptrs = [V(0 if n in null else FAKE + (8 if n in off else 0)) for n in names]
    out = [V(0 if n in null else FAKE) for n in ("out", "lse")]
    return lib.lib().mla_paged_prefill_fp8(*ptrs, 0.1, *out, ctypes.byref(dims), V(ws), size, flags, None)


def test_prefill_fp8_refusals(lib):
    def dims(**kw):
        d = dict(batch=2, num_qo_heads=16, num_pages=4, page_size=64, num_kv_indices=10, total_q=3, num_workers=4)
        d.update(kw)
        return lib.make_dims(**d)

    for kw in (dict(num_qo_heads=0), dict(num_qo_heads=129), dict(total_q=-1), dict(page_size=0),
               dict(num_pages=1 << 20, page_size=1 << 12), dict(num_workers=-1)):
        assert _prefill(lib, dims(**kw)) == DIMS, kw
    for n in ("q_nope", "q_pe", "kv", "qo", "kp", "ki", "out", "lse"):
        assert _prefill(lib, dims(), null=(n,)) == NULL, n
    for n in ("q_nope", "q_pe", "kv"):
        assert _prefill(lib, dims(), off=(n,)) == ALIGN, n
    assert _prefill(lib, dims(), ws=0) == WORKSPACE
    assert _prefill(lib, dims(), size=1000) == WORKSPACE
    assert _prefill(lib, dims(), ws=FAKE + 8) == ALIGN
    assert _prefill(lib, dims(total_q=0)) == 0
    small, large = (lib.workspace_bytes_prefill_fp8(dims(num_kv_indices=n)) for n in (64, 6400))
    assert large - small >= 1152 * (6400 - 128)
    assert lib.workspace_bytes_prefill_fp8(dims(num_qo_heads=0)) == 0


def test_prefill_staged_refusals(lib):
    dims = lib.make_dims(2, 16, 4, 64, 10, total_q=3, num_workers=4)
    names = ["q_nope", "q_pe", "ckv", "kpe", "qo", "kp", "ki", "out", "lse"]

    def call(null=None, off=None, d=dims, ws=FAKE, size=1 << 40, scale=0.1):
        p = [V(0 if n == null else FAKE + (8 if n == off else 0)) for n in names]
        return lib.lib().mla_paged_prefill_staged(*p[:7], scale, *p[7:], ctypes.byref(d), V(ws), size, 0, None)

    for n in names:
        assert call(null=n) == NULL, n
    for n in ("q_nope", "q_pe", "ckv", "kpe", "out"):
        assert call(off=n) == ALIGN, n
    assert call(scale=float("nan")) == DIMS
    assert call(ws=0) == WORKSPACE and call(size=4096) == WORKSPACE and call(ws=FAKE + 8) == ALIGN
    assert call(d=lib.make_dims(2, 16, 4, 64, 10, total_q=0)) == 0
    assert call(d=lib.make_dims(0, 16, 4, 64, 0, total_q=5)) == 0
    # Staged rows are 32-bit coordinates: too many requests or keys are refused.
    assert call(d=lib.make_dims(1 << 24, 1, 4, 64, 10, total_q=3, num_workers=4)) == DIMS
    assert lib.workspace_bytes_prefill_staged(dims) == lib.workspace_bytes_prefill_fp8(dims)
