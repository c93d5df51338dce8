"""C-ABI refusals of the window and the shared attention; every case fails (or is a no-op) on the
host before any CUDA call."""

import ctypes

import pytest

FAKE = 0x10000  # never dereferenced
V = ctypes.c_void_p
NULL, DIMS, ALIGN, WORKSPACE = -1, -2, -3, -4
KINDS = [(kind, prefill, fp8) for kind in ("window", "shared") for prefill in (False, True) for fp8 in (False, True)]


def _dims(lib, **kw):
    d = dict(batch=2, num_qo_heads=16, num_pages=4, page_size=64, num_kv_indices=10, total_q=3, num_workers=4)
    d.update(kw)
    return lib.make_dims(**d)


def _call(lib, kind, prefill, fp8, dims=None, null=(), off=(), ws=FAKE, size=1 << 40, scale=0.1, window=5, sinks=2,
          groups=2, num_prefix=7):
    def p(name):
        return V(0 if name in null else FAKE + (8 if name in off else 0))

    args = [p("q_nope"), p("q_pe")] + ([p("kv")] if fp8 else [p("ckv"), p("kpe")]) + ([p("qo")] if prefill else [])
    if kind == "window":
        args += [p("kp"), p("ki"), window, sinks]
    else:
        args += [p("gp"), groups, p("pp"), p("pi"), num_prefix, p("kp"), p("ki")]
    name = f"mla_paged_{'prefill' if prefill else 'decode'}_{kind}" + ("_fp8" if fp8 else "")
    return getattr(lib.lib(), name)(*args, scale, p("out"), p("lse"),
                                    ctypes.byref(dims) if dims is not None else None, V(ws), size, 0, None)


@pytest.mark.parametrize("kind,prefill,fp8", KINDS)
def test_refusals(lib, kind, prefill, fp8):
    good = _dims(lib)

    def call(dims=good, **kw):
        return _call(lib, kind, prefill, fp8, dims, **kw)

    assert call(dims=None) == NULL
    for kw in (dict(num_qo_heads=0), dict(num_qo_heads=129), dict(page_size=0), dict(batch=-1), dict(num_kv_indices=-1),
               dict(num_pages=1 << 20, page_size=1 << 12), dict(num_workers=-1)):
        assert call(dims=_dims(lib, **kw)) == DIMS, kw
    if prefill:
        assert call(dims=_dims(lib, total_q=-1)) == DIMS
    names = ["q_nope", "q_pe", "kp", "ki", "out", "lse"] + (["kv"] if fp8 else ["ckv", "kpe"]) + ["qo"] * prefill
    for n in names + (["gp", "pp", "pi"] if kind == "shared" else []):
        assert call(null=(n,)) == NULL, n
    for n in ["q_nope", "q_pe", "out"] + (["kv"] if fp8 else ["ckv", "kpe"]):
        assert call(off=(n,)) == ALIGN, n
    for scale in (float("nan"), float("inf")):
        assert call(scale=scale) == DIMS
    assert call(ws=0) == WORKSPACE and call(size=4096) == WORKSPACE and call(ws=FAKE + 8) == ALIGN
    assert call(dims=_dims(lib, batch=0, num_kv_indices=0)) == 0
    if prefill:
        assert call(dims=_dims(lib, total_q=0)) == 0
    if kind == "window":
        for kw in (dict(window=0), dict(window=-1), dict(window=-2 ** 31), dict(sinks=-1)):
            assert call(**kw) == DIMS, kw
    else:
        for kw in (dict(groups=-1), dict(num_prefix=-1)):
            assert call(**kw) == DIMS, kw
        assert call(groups=0) == 0
        # Staged rows are 32-bit coordinates.
        assert call(groups=1 << 24) == DIMS and call(num_prefix=2 ** 31 - 1) == DIMS
        assert call(dims=_dims(lib, num_kv_indices=2 ** 31 - 1)) == DIMS


def test_window_workspace(lib):
    """Long lists with a short window take the window's tiles, short ones their own."""
    def size(n, w, s=0, **kw):
        return lib.workspace_bytes_window(_dims(lib, num_kv_indices=n, **kw), w, s)

    tile = 128 * 1152 + 32
    assert size(10 ** 6, 100) == size(10 ** 7, 100) < size(10 ** 7, 1000) < size(10 ** 7, 1000, 500)
    assert size(10 ** 6, 100) <= size(0, 1) + 2 * 5 * tile + 4096
    assert size(1000, 2 ** 31 - 1, 2 ** 31 - 1) == size(1000, 10 ** 6)
    assert size(2 ** 31 - 1, 2 ** 31 - 1) == 0  # more staged keys than 32-bit coordinates
    assert size(2 ** 31 - 1, 1000) > 0
    assert size(10, 0) == 0 and size(10, 5, -1) == 0 and size(10, 5, num_qo_heads=0) == 0
    d = _dims(lib, num_kv_indices=10 ** 7, total_q=5000)
    assert lib.workspace_bytes_window(d, 100, 0, is_prefill=True) > lib.workspace_bytes_window(d, 100, 0)


def test_shared_workspace(lib):
    d = _dims(lib, num_kv_indices=1000)
    a, b = lib.workspace_bytes_shared(d, 2, 1000), lib.workspace_bytes_shared(d, 2, 11000)
    assert b - a >= 1152 * (10000 - 128)
    assert lib.workspace_bytes_shared(d, -1, 0) == 0 and lib.workspace_bytes_shared(d, 0, -1) == 0
    assert lib.workspace_bytes_shared(d, 1 << 24, 0) == 0
    assert lib.workspace_bytes_shared(d, 0, 0) > 0
