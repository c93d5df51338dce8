"""The groups of a batch from its block table: integer work, equal to a row-by-row oracle."""

import ctypes

import numpy as np
import pytest
import torch

from tests.conftest import require_gpu

FILL = -77


def groups_of(table, lens, page, min_shared=1):
    """(group_indptr, prefix_indptr, prefix slots, kv_indptr, own slots) as Python lists."""
    n, blocks = len(table), len(table[0]) if len(table) else 0
    lens = [min(max(v, 0), blocks * page) for v in lens]

    def common(i):
        most = min(lens[i - 1], lens[i]) // page
        k = 0
        while k < most and table[i - 1][k] == table[i][k]:
            k += 1
        return k * page

    heads, shared = [], []
    for i in range(n):
        if i == 0 or common(i) < max(1, min_shared):
            heads.append(i)
            shared.append(None)
        else:
            shared[-1] = common(i) if shared[-1] is None else min(shared[-1], common(i))
    shared = [s or 0 for s in shared]

    def slot(row, key):
        s = table[row][key // page] * page + key % page
        return s if 0 <= s < 2 ** 31 else -1

    prefix, pp, own, kp = [], [0], [], [0]
    for g, (first, keys) in enumerate(zip(heads, shared)):
        prefix += [slot(first, k) for k in range(keys)]
        pp.append(len(prefix))
        for row in range(first, heads[g + 1] if g + 1 < len(heads) else n):
            own += [slot(row, k) for k in range(keys, lens[row])]
            kp.append(len(own))
    pad = n + 1 - len(heads)
    return heads + [n] * pad, pp + [pp[-1]] * (n + 1 - len(pp)), prefix, kp, own


def test_the_oracle_on_a_worked_example():
    """Pages of 4: rows 0-2 share 7, 8 (row 1 only 7, its second page being partly filled), row 3
    shares nothing, row 4 is empty, rows 5 and 6 share page 3."""
    table = [[7, 8, 1], [7, 8, 0], [7, 8, 2], [9, 5, 6], [9, 5, 6], [3, 4, -1], [3, 0, -1]]
    lens = [9, 7, 12, 8, 0, 5, 4]
    g, pp, prefix, kp, own = groups_of(table, lens, 4)
    assert g == [0, 3, 4, 5, 7, 7, 7, 7]
    assert pp == [0, 4, 4, 4, 8, 8, 8, 8]
    assert prefix == [28, 29, 30, 31, 12, 13, 14, 15]
    assert kp == [0, 5, 8, 16, 24, 24, 25, 25]
    assert own[:8] == [32, 33, 34, 35, 4, 32, 33, 34] and own[24:] == [16]
    g, pp, prefix, kp, own = groups_of(table, lens, 4, min_shared=5)
    assert g == list(range(8)) and pp == [0] * 8 and kp[-1] == 45
    # A mistake planted in the comparison (a partly filled page counts) would give other lists.
    assert groups_of([[7, 8], [7, 8]], [8, 7], 4)[1] == [0, 4, 4]


def compare(lib, table, lens, page, min_shared=1, **kw):
    ref = groups_of(table.tolist(), lens.tolist(), page, min_shared)
    cap = kw.get("capacity", len(ref[4]) + 5)
    pcap = kw.get("prefix_capacity", len(ref[2]) + 5)
    bufs = dict(prefix_indices=torch.full((pcap + 64,), FILL, dtype=torch.int32, device="cuda"),
                kv_indices=torch.full((cap + 64,), FILL, dtype=torch.int32, device="cuda"))
    got = lib.block_table_to_shared_csr(table.cuda(), lens.cuda(), page, min_shared=min_shared,
                                        prefix_indices=bufs["prefix_indices"][:pcap], kv_indices=bufs["kv_indices"][:cap])
    g, pp, _, kp, _ = (t.tolist() for t in got)
    assert (g, pp, kp) == (ref[0], ref[1], ref[3])
    for name, want, room in (("prefix_indices", ref[2], pcap), ("kv_indices", ref[4], cap)):
        have = bufs[name].tolist()
        n = min(len(want), room)
        assert have[:n] == want[:n], name
        assert have[n:] == [FILL] * (len(have) - n), name  # nothing behind the list or the capacity
    return got


def random_table(rng, n, blocks, page, share, ids=50):
    """Rows that copy some leading pages of the row before with probability ``share``."""
    table = rng.integers(0, ids, (n, blocks))
    lens = rng.integers(0, blocks * page + 1, n)
    for i in range(1, n):
        if rng.random() < share:
            k = rng.integers(0, blocks + 1)
            table[i, :k] = table[i - 1, :k]
    return torch.tensor(table, dtype=torch.int32), torch.tensor(lens, dtype=torch.int32)


@pytest.mark.gpu
@pytest.mark.parametrize("n,blocks", [(1, 1), (2, 3), (33, 7), (64, 16), (64, 17), (65, 2), (100, 300), (1023, 4), (1025, 5),
                                      (2500, 3)])
@pytest.mark.parametrize("page", [1, 16, 64])
def test_tables_equal_the_oracle(lib, n, blocks, page):
    require_gpu()
    rng = np.random.default_rng(n + page)
    for share, min_shared in ((0.8, 1), (1.0, 0), (0.5, 3 * page), (0.9, 2 ** 31 - 1)):
        compare(lib, *random_table(rng, n, blocks, page, share), page, min_shared)


@pytest.mark.gpu
def test_lengths_and_ids_out_of_range(lib):
    """Negative and too large lengths are clamped; ids that give no int32 slot become -1."""
    require_gpu()
    table = torch.tensor([[3, -2, 5], [3, -2, 6], [3, 2 ** 30, 7], [3, 2 ** 30, 8], [-1, 4, 4], [-1, 4, 4]],
                         dtype=torch.int32)
    lens = torch.tensor([100, 12, 11, 2 ** 31 - 1, -5, 9], dtype=torch.int32)
    compare(lib, table, lens, 4)
    compare(lib, table.flip(0).contiguous(), lens, 4)


@pytest.mark.gpu
@pytest.mark.parametrize("capacity,prefix_capacity", [(0, 0), (100, 7), (1, 10 ** 4)])
def test_nothing_is_written_past_a_capacity(lib, capacity, prefix_capacity):
    require_gpu()
    rng = np.random.default_rng(5)
    compare(lib, *random_table(rng, 40, 20, 16, 0.9), 16, capacity=capacity, prefix_capacity=prefix_capacity)


@pytest.mark.gpu
def test_offsets_stay_at_the_largest_int(lib):
    """Rows of 2^30 keys each, none of which fit the lists: offsets stop at 2^31 - 1."""
    require_gpu()
    page, lens = 1 << 29, torch.full((6,), 1 << 30, dtype=torch.int32)
    table = torch.tensor([[1, 2], [3, 4], [5, 6], [5, 6], [7, 8], [7, 8]], dtype=torch.int32)
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    g, pp, _, kp, _ = lib.block_table_to_shared_csr(table.cuda(), lens.cuda(), page, prefix_indices=e, kv_indices=e)
    assert g.tolist() == [0, 1, 2, 4, 6, 6, 6]
    most = 2 ** 31 - 1
    assert pp.tolist() == [0, 0, 0, 1 << 30, most, most, most]
    # (the last group shares the keys that its offsets count; the rest is its rows' own)
    assert kp.tolist() == [0, 1 << 30, most, most, most, most, most]


@pytest.mark.gpu
def test_an_empty_batch(lib):
    require_gpu()
    got = lib.block_table_to_shared_csr(torch.zeros(0, 3, dtype=torch.int32, device="cuda"),
                                        torch.zeros(0, dtype=torch.int32, device="cuda"), 16)
    assert [t.tolist() for t in got] == [[0], [0], [], [0], []]
    got = lib.block_table_to_shared_csr(torch.zeros(3, 0, dtype=torch.int32, device="cuda"),
                                        torch.full((3,), 9, dtype=torch.int32, device="cuda"), 16)
    assert [t.tolist() for t in got] == [[0, 1, 2, 3], [0] * 4, [], [0] * 4, []]


@pytest.mark.gpu
def test_captured_and_replayed(lib):
    require_gpu()
    rng = np.random.default_rng(8)
    a, b = random_table(rng, 64, 12, 16, 0.9), random_table(rng, 64, 12, 16, 0.4)
    table, lens = a[0].cuda(), a[1].cuda()
    lib.block_table_to_shared_csr(table, lens, 16)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = lib.block_table_to_shared_csr(table, lens, 16)
    for t, n in (a, b, a):
        table.copy_(t)
        lens.copy_(n)
        graph.replay()
        torch.cuda.synchronize()
        g, pp, prefix, kp, own = groups_of(t.tolist(), n.tolist(), 16)
        assert (got[0].tolist(), got[1].tolist(), got[3].tolist()) == (g, pp, kp)
        assert got[2][:len(prefix)].tolist() == prefix and got[4][:len(own)].tolist() == own


V = ctypes.c_void_p
FAKE = 0x10000  # never dereferenced


def test_refusals(lib):
    f = lib.lib().mla_block_table_to_shared_csr
    names = ("table", "lens", "batch", "blocks", "page", "min", "gp", "pp", "pi", "pcap", "kp", "ki", "cap")
    good = dict(zip(names, (V(FAKE), V(FAKE), 2, 3, 16, 1, V(FAKE), V(FAKE), V(FAKE), 9, V(FAKE), V(FAKE), 9)))

    def call(**kw):
        return f(*{**good, **kw}.values(), None)

    for kw in (dict(batch=-1), dict(blocks=-1), dict(page=0), dict(min=-1), dict(cap=-1), dict(pcap=-1), dict(cap=2 ** 31),
               dict(pcap=2 ** 31), dict(blocks=1 << 27, page=16)):
        assert call(**kw) == -2, kw
    for name in ("table", "lens", "gp", "pp", "pi", "kp", "ki"):
        assert call(**{name: None}) == -1, name
