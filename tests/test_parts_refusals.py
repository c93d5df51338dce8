"""More refusals of the shared-prefix calls on the host, before any CUDA call."""

import ctypes

import pytest

V = ctypes.c_void_p
FAKE = 0x10000  # never dereferenced


@pytest.mark.parametrize("batch", [2 ** 30 + 1, 2 ** 31 - 1])
def test_tables_of_more_rows_than_counters_hold(lib, batch):
    assert lib.lib().mla_block_table_to_shared_csr(V(FAKE), V(FAKE), batch, 1, 1, 1, V(FAKE), V(FAKE), None, 0, V(FAKE),
                                                   None, 0, None) == -2


@pytest.mark.parametrize("prefill", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
def test_validation_without_a_group_is_not_skipped(lib, prefill, fp8):
    """Requests in no group are what MLA_VALIDATE reports, so the call needs its workspace for the status."""
    name = f"mla_paged_{'prefill' if prefill else 'decode'}_shared" + ("_fp8" if fp8 else "")
    dims = lib.make_dims(2, 16, 4, 64, 10, total_q=3, num_workers=4)

    def call(flags, null=()):
        p = {n: V(0 if n in null else FAKE) for n in ("qn", "qp", "kv", "kpe", "qo", "gp", "pp", "pi", "kp", "ki", "out",
                                                      "lse", "ws")}
        args = [p["qn"], p["qp"], p["kv"]] + [p["kpe"]] * (not fp8) + [p["qo"]] * prefill
        return getattr(lib.lib(), name)(*args, p["gp"], 0, p["pp"], p["pi"], 7, p["kp"], p["ki"], 0.1, p["out"], p["lse"],
                                        ctypes.byref(dims), p["ws"], 1 << 40, flags, None)

    assert call(0) == 0 and call(0, ("ws",)) == 0
    assert call(1, ("ws",)) == -4
    for n in ("gp", "pp", "kp", "ki"):
        assert call(1, (n,)) == -1
