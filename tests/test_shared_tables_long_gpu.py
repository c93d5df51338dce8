"""Tables of shared prefixes whose offsets and lists reach the largest int, in batches of many warps."""

import numpy as np
import pytest
import torch

from tests.conftest import require_gpu
from tests.test_shared_tables import groups_of

pytestmark = pytest.mark.gpu

MOST = 2 ** 31 - 1


def counts(t):
    """Whether t holds 0, 1, 2, ... (looked at in parts, as the list fills 8.6 GB)."""
    return all(torch.equal(x, torch.arange(i * 2 ** 28, i * 2 ** 28 + x.numel(), dtype=torch.int32, device="cuda"))
               for i, x in enumerate(t.split(2 ** 28)))


@pytest.mark.parametrize("shared", [False, True])
def test_a_list_of_as_many_keys_as_an_int_counts(lib, shared):
    """A page of 2^31 - 1 tokens, as one row's own keys or as what two rows share."""
    require_gpu()
    rows = 2 if shared else 1
    table = torch.zeros(rows, 1, dtype=torch.int32, device="cuda")
    lens = torch.full((rows,), MOST, dtype=torch.int32, device="cuda")
    g, pp, pi, kp, ki = lib.block_table_to_shared_csr(table, lens, MOST, prefix_capacity=MOST if shared else 0,
                                                      capacity=0 if shared else MOST)
    assert (g.tolist(), pp.tolist(), kp.tolist()) == (([0, 2, 2], [0, MOST, MOST], [0, 0, 0]) if shared else
                                                      ([0, 1], [0, 0], [0, MOST]))
    assert counts(pi if shared else ki)


@pytest.mark.parametrize("n", [65, 700, 2100])
def test_offsets_of_many_rows_stay_at_the_largest_int(lib, n):
    """Long rows in groups of a few, so that the offsets reach 2^31 - 1 somewhere in the batch."""
    require_gpu()
    page, blocks = 1 << 18, 1000
    rng = np.random.default_rng(n)
    table = rng.integers(0, 30000, (n, blocks)).astype(np.int32)
    for i in range(1, n):
        if rng.random() < 0.7:
            k = rng.integers(1, blocks)
            table[i, :k] = table[i - 1, :k]
    lens = rng.integers(0, blocks * page + 1, n)
    # The definition, with offsets that stop at the largest int; a group shares what its offsets count.
    full = groups_of(table.tolist(), (lens // page).tolist(), 1)  # (in pages: the same groups)
    heads = [h for h in full[0] if h < n]
    pp, kp = [0], [0]
    shared = np.diff(full[1])[:len(heads)] * page
    for g, first in enumerate(heads):
        pp.append(min(pp[-1] + int(shared[g]), MOST) if pp[-1] < MOST else MOST)
        here = pp[-1] - pp[-2]
        for row in range(first, heads[g + 1] if g + 1 < len(heads) else n):
            kp.append(min(kp[-1] + int(lens[row]) - here, MOST))
    assert kp[-1] == MOST
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    got = lib.block_table_to_shared_csr(torch.from_numpy(table).cuda(), torch.from_numpy(lens.astype(np.int32)).cuda(), page,
                                        prefix_indices=e, kv_indices=e)
    assert got[0].tolist() == full[0]
    assert got[1].tolist() == pp + [pp[-1]] * (n + 1 - len(pp))
    assert got[3].tolist() == kp
