"""More refusals of the shared-prefix calls on the host, before any CUDA call."""

import ctypes

import pytest

V = ctypes.c_void_p
FAKE = 0x10000  # never dereferenced


@pytest.mark.parametrize("batch", [2 ** 30 + 1, 2 ** 31 - 1])
def test_tables_of_more_rows_than_counters_hold(lib, batch):
    assert lib.lib().mla_block_table_to_shared_csr(V(FAKE), V(FAKE), batch, 1, 1, 1, V(FAKE), V(FAKE), None, 0, V(FAKE),
                                                   None, 0, None) == -2
