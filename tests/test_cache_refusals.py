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
