"""More C-ABI refusals of the cache's writers and the staged prefill; each is answered on the host
before any CUDA call."""

import ctypes

import pytest

from tests.test_cache_abi import ALIGN, DIMS, _append


@pytest.mark.parametrize("fp8", [False, True])
def test_rotation_in_place_needs_contiguous_queries(lib, fp8):
    """With q_out = q_pe and other strides, a head would be written over one that is not read yet."""
    for kw in (dict(q_stride_token=192), dict(q_stride_head=128), dict(q_stride_token=0),
               dict(q_stride_token=64, q_stride_head=256)):
        assert _append(lib, fp8, **kw) == DIMS, kw
    assert _append(lib, fp8, q_stride_token=130) == ALIGN
    # A stride that no second token or head uses does not matter: refused for another reason only.
    for kw in (dict(tokens=1, q_stride_token=8), dict(num_qo_heads=1, q_stride_token=64, q_stride_head=8)):
        assert _append(lib, fp8, off=("ckv",), **kw) == ALIGN, kw


def test_no_workspace_size_for_a_refused_staged_prefill(lib):
    """More staged rows than a 32-bit coordinate reaches: the call is refused, so its size is 0 too
    (a caller would allocate terabytes for it otherwise)."""
    for kw in (dict(batch=1 << 24, num_kv_indices=10), dict(batch=1, num_kv_indices=2 ** 31 - 1)):
        dims = lib.make_dims(num_qo_heads=1, num_pages=4, page_size=64, total_q=3, num_workers=4, **kw)
        p = [ctypes.c_void_p(0x10000)] * 7
        call = lib.lib().mla_paged_prefill_staged
        assert call(*p, 0.1, p[0], p[0], ctypes.byref(dims), p[0], 1 << 62, 0, None) == DIMS
        assert lib.workspace_bytes_prefill_staged(dims) == lib.workspace_bytes_prefill_fp8(dims) == 0
    largest = lib.make_dims(1, 1, 4, 64, (1 << 31) - 256, total_q=3, num_workers=4)
    assert lib.workspace_bytes_prefill_staged(largest) > 1152 * ((1 << 31) - 256)
