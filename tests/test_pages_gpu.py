"""The page pool on the GPU: integers, so every array has to equal the oracle's."""

import numpy as np
import pytest
import torch

from oracle import cache_oracle as co
from tests.conftest import require_gpu

pytestmark = pytest.mark.gpu


class Both:
    """The same pool on the GPU and in the oracle."""

    def __init__(self, lib, rows, blocks, pages, ps, entries=64):
        self.lib, self.ps = lib, ps
        self.table = torch.full((rows, blocks), -1, dtype=torch.int32).cuda()
        self.lens = torch.zeros(rows, dtype=torch.int32).cuda()
        self.refs = torch.zeros(pages, dtype=torch.int32).cuda()
        self.pool = co.Pool(self.table.tolist(), self.lens.tolist(), self.refs.tolist(), ps)
        self.ws = torch.full((lib.workspace_bytes_pages(rows, pages, entries),), 0xA5, dtype=torch.uint8).cuda()

    def arrays(self):
        return self.table, self.lens, self.refs

    def same(self):
        assert self.lens.tolist() == self.pool.lens
        assert self.refs.tolist() == self.pool.refs
        assert self.table.tolist() == self.pool.table

    def extend(self, rows, new, capacity):
        got = self.lib.mla_pages_extend(*self.arrays(), _i(rows), _i(new), self.ps, capacity, workspace=self.ws)
        want = self.pool.extend(rows, new, capacity)
        assert [t.tolist() for t in got] == [list(w) for w in want]
        self.same()

    def fork(self, parents, children):
        got = self.lib.mla_pages_fork(*self.arrays(), _i(parents), _i(children), self.ps, workspace=self.ws)
        assert [t.tolist() for t in got] == [list(w) for w in self.pool.fork(parents, children)]
        self.same()

    def free(self, rows):
        self.lib.mla_pages_free(*self.arrays(), _i(rows), self.ps)
        self.pool.free(rows)
        self.same()

    def compact(self):
        counts, src, dst = self.lib.mla_pages_compact(*self.arrays(), self.ps, workspace=self.ws)
        live, s, d = self.pool.compact()
        pad = [-1] * (self.refs.numel() // 2 - len(s))
        assert counts.tolist() == [live, len(s)] and src.tolist() == s + pad and dst.tolist() == d + pad
        self.same()


def _i(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


@pytest.mark.parametrize("rows,blocks,pages,ps", [(1, 1, 1, 1), (9, 6, 30, 4), (40, 11, 200, 1), (33, 5, 97, 64),
                                                  (300, 20, 5000, 16)])
@pytest.mark.parametrize("seed", range(3))
def test_random_calls(lib, rows, blocks, pages, ps, seed):
    """Long random sequences with bad rows, rows listed twice, negative counts and pools that run out."""
    require_gpu()
    rng = np.random.default_rng(1000 * seed + rows)
    b = Both(lib, rows, blocks, pages, ps)
    for _ in range(40):
        n = int(rng.integers(0, 50))
        some = rng.integers(-1, rows + 1, n).tolist()
        op = int(rng.integers(0, 6))
        if op <= 1:
            new = rng.integers(-1, max(2, blocks * ps // 2), n).tolist()
            b.extend(some, new, int(rng.integers(0, 1 + max(0, sum(new)))))
        elif op == 2:
            b.fork(some, rng.integers(-1, rows + 1, n).tolist())
        elif op == 3:
            b.free(some[:max(1, n // 4)])
        elif op == 4:
            b.compact()
        else:
            free_rows = [r for r in range(rows) if b.pool.lens[r] == 0][:20]
            full_rows = [r for r in range(rows) if b.pool.lens[r] > 0]
            if free_rows and full_rows:
                b.fork([full_rows[int(rng.integers(0, len(full_rows)))] for _ in free_rows], free_rows)


def test_large_pool(lib):
    """A pool of 300,000 pages and 3000 entries: many words of the bitmap, several rounds of the plan."""
    require_gpu()
    rng = np.random.default_rng(5)
    b = Both(lib, 4000, 70, 300000, 16, entries=4000)
    rows = rng.permutation(4000)[:3000].tolist()
    new = rng.integers(0, 1000, 3000).tolist()
    b.extend(rows, new, sum(new))
    b.free(rows[::3])
    b.compact()
    free = [r for r in range(4000) if b.pool.lens[r] == 0][:1500]
    b.fork([rows[1 + 3 * (i % 900)] for i in range(len(free))], free)
    b.extend(rows, [5] * 3000, 15000)


def test_every_page_free_and_none(lib):
    require_gpu()
    b = Both(lib, 3, 40, 64, 2)
    b.compact()                      # no live page
    b.extend([0, 1], [80, 48], 128)  # every page
    b.compact()
    b.extend([0, 2], [0, 1], 4)      # nothing needed; nothing left
    b.free([0])
    b.compact()
    b.extend([], [], 3)              # no entries: the slots are padding
    assert b.lib.mla_pages_fork(*b.arrays(), _i([]), _i([]), 2)[0].numel() == 0


def test_pages_held_by_the_caller(lib):
    """A page with a count that no row holds is live: it is not taken and it moves."""
    require_gpu()
    b = Both(lib, 3, 8, 16, 4)
    for p in (0, 9, 15):
        b.refs[p] = 1
        b.pool.refs[p] = 1
    b.extend([0, 1], [9, 30], 39)
    b.free([0])
    b.compact()


def test_captured_and_replayed_step(lib):
    """A step (free, fork, copy, extend) captured once and replayed with other entries, on a side stream."""
    require_gpu()
    ps, n = 4, 6
    b = Both(lib, 20, 10, 60, ps)
    kv = torch.randint(0, 256, (60, ps, 656), dtype=torch.uint8).cuda()
    b.extend(list(range(10)), [5, 9, 4, 17, 1, 30, 2, 2, 2, 2], 100)
    names = ("ended", "parents", "children", "rows", "new")
    now = {k: _i([-1] * n) for k in names}
    out = {}

    def step():
        lib.mla_pages_free(*b.arrays(), now["ended"], ps)
        out["fork"] = lib.mla_pages_fork(*b.arrays(), now["parents"], now["children"], ps, workspace=b.ws)
        lib.mla_cache_copy_pages_fp8(kv, out["fork"][1], out["fork"][2], tokens=out["fork"][3])
        out["extend"] = lib.mla_pages_extend(*b.arrays(), now["rows"], now["new"], ps, 64, workspace=b.ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()  # every entry is refused: nothing changes
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    b.same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    pages = kv.cpu()
    for todo in (dict(ended=[0, 1], parents=[3, 3, 5], children=[0, 11, 12], rows=[3, 0, 11, 5], new=[1, 7, 2, 3]),
                 dict(ended=[12, 3], parents=[11, 0], children=[13, 14], rows=[13, 14, 2], new=[9, 1, 0])):
        for k in names:
            now[k].copy_(_i((todo[k] + [-1] * n)[:n]))
        graph.replay()
        torch.cuda.synchronize()
        pad = {k: (todo[k] + [-1] * n)[:n] for k in names}
        b.pool.free(pad["ended"])
        want = b.pool.fork(pad["parents"], pad["children"])
        assert [t.tolist() for t in out["fork"]] == [list(w) for w in want]
        for s, d, t in zip(*want[1:]):
            if t:
                pages[d, :t] = pages[s, :t]
        assert torch.equal(kv.cpu(), pages)
        assert [t.tolist() for t in out["extend"]] == [list(w) for w in b.pool.extend(pad["rows"], pad["new"], 64)]
        b.same()


def test_python_refusals(lib):
    require_gpu()
    b = Both(lib, 4, 4, 16, 4)
    with pytest.raises(ValueError):
        lib.mla_pages_extend(*b.arrays(), _i([0]), _i([1, 2]), 4, 4)
    with pytest.raises(ValueError):
        lib.mla_pages_extend(*b.arrays(), _i([0]), _i([1]), 4, -1)
    with pytest.raises(TypeError):
        lib.mla_pages_free(*b.arrays(), _i([0]).long(), 4)
    with pytest.raises(ValueError):
        lib.mla_pages_free(b.table, b.lens[:2], b.refs, _i([0]), 4)
    with pytest.raises(lib.MlaError):
        lib.mla_pages_free(*b.arrays(), _i([0]), 0)
    with pytest.raises(lib.MlaError):
        lib.mla_pages_compact(*b.arrays(), 4, workspace=b.ws[:64])
