"""MLA_VALIDATE of the decode calls, and of shared calls whose requests are in no group."""

import pytest
import torch

from tests.conftest import require_gpu
from tests.test_parts_gpu import both, call, close, make_shared, on_gpu, plain

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("prefill", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
def test_no_group_at_all_is_reported(lib, prefill, fp8):
    """The status says so, no row is written, and without the flag nothing is reported."""
    require_gpu()
    x = make_shared([(50, [(1, 9), (1, 3)])], 16, 16, 9, fp8)
    x["gp"] = x["pp"] = torch.zeros(1, dtype=torch.int32)
    x["pi"] = x["pi"][:0]
    c = on_gpu(x)
    ws = torch.zeros(1 << 26, dtype=torch.uint8, device="cuda")
    out = torch.full((2, 16, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((2, 16), 7.0, device="cuda")
    for flags, status in ((0, 0), (1, -6), (0, 0)):
        call(lib, "shared", c, prefill, (), out=out, lse=lse, workspace=ws, flags=flags)
        assert lib.read_device_status(ws) == status
        assert (out == 7).all() and (lse == 7).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_decode(lib, fp8):
    """A token per request, without offsets of the queries."""
    require_gpu()
    ws = torch.zeros(1 << 27, dtype=torch.uint8, device="cuda")
    for kind, x, args in both(16, 64, fp8, 15, ((1, 90), (1, 200), (1, 130))):
        close(call(lib, kind, on_gpu(x), False, args, workspace=ws, flags=1), plain(x, *args))
        assert lib.read_device_status(ws) == 0
        for name, at, v in [("ki", 5, -1), ("kp", 1, 300)] + [("pi", 150, 1 << 30), ("gp", 1, 9)] * (kind == "shared"):
            y = {**x, name: x[name].clone()}
            y[name][at] = v
            call(lib, kind, on_gpu(y), False, args, workspace=ws, flags=1)
            assert lib.read_device_status(ws) == -6, (kind, name)
