"""Lists of the tables of shared prefixes that are no tensors."""

import pytest
import torch

from tests.conftest import require_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", ["group_indptr", "prefix_indptr", "prefix_indices", "kv_indptr", "kv_indices"])
def test_lists_that_are_no_tensors(lib, name):
    require_gpu()
    table = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError):
        lib.block_table_to_shared_csr(table, lens, 16, **{name: [1, 2, 3]})
