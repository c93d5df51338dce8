"""Lists and pools at which the kernels take another path: lists longer than a grid's first pass, and
pools around the sizes where the numbering of the free pages changes."""

import numpy as np
import pytest
import torch

from tests.conftest import require_gpu
from tests.test_pages_gpu import Both

pytestmark = pytest.mark.gpu


def _i(v):
    return torch.as_tensor(np.asarray(v), dtype=torch.int32).cuda()


@pytest.mark.parametrize("fp8", [False, True])
def test_gather_of_more_tokens_than_a_pass_of_the_grid(lib, fp8):
    """700,001 tokens (a pass takes 311,296), slots outside the cache among them."""
    require_gpu()
    pages, page, n = 90, 64, 700_001
    g = torch.Generator(device="cuda").manual_seed(4)
    slots = torch.randint(-20, pages * page + 20, (n,), generator=g, device="cuda", dtype=torch.int32)
    if fp8:
        kv = torch.randint(0, 0x7F, (pages, page, 656), generator=g, device="cuda", dtype=torch.uint8)
        kv[..., 512:528] = torch.tensor([2.0, 0.5, 0.75, 1.0], device="cuda").view(torch.uint8)
        every = torch.arange(pages * page, dtype=torch.int32, device="cuda")
        table = lib.mla_cache_gather_fp8(kv, every)  # (5760 tokens: one pass)
        got = lib.mla_cache_gather_fp8(kv, slots)
    else:
        table = [torch.randn(pages * page, d, generator=g, device="cuda").to(torch.bfloat16) for d in (512, 64)]
        got = lib.mla_cache_gather(*(t.view(pages, page, -1) for t in table), slots)
    inside = ((slots >= 0) & (slots < pages * page))[:, None]
    at = slots.clamp(0, pages * page - 1).long()
    for a, t in zip(got, table):
        assert torch.equal(a.view(torch.int16), torch.where(inside, t[at].view(torch.int16), 0))


def test_more_entries_than_a_pass_of_the_grid(lib):
    """9000 entries in extend, fork and free, whose grids end at 4096."""
    require_gpu()
    rng = np.random.default_rng(8)
    b = Both(lib, 20000, 4, 30000, 4, entries=9000)
    rows = rng.permutation(10000)[:9000].tolist()
    new = rng.integers(0, 12, 9000).tolist()
    b.extend(rows, new, sum(new) + 100)
    b.fork(rows, (10000 + rng.permutation(10000)[:9000]).tolist())
    b.extend(rows, [1] * 9000, 9000)   # (many of them hold a shared last page or find no page)
    b.free((rng.integers(-5, 20005, 9000)).tolist())
    b.compact()


@pytest.mark.parametrize("pages", [16352, 16383, 16384, 16385, 16416, 8192 * 3])
def test_pools_around_the_change_of_the_numbering(lib, pages):
    """The block numbers up to 16,384 pages by itself; a grid does beyond that, 8192 pages a span."""
    require_gpu()
    rng = np.random.default_rng(pages)
    b = Both(lib, 300, 200, pages, 1)
    held = rng.permutation(pages)[:pages // 3]
    b.refs[torch.from_numpy(held).cuda()] = 1
    for p in held:
        b.pool.refs[p] = 1
    b.extend(list(range(60)), rng.integers(0, 200, 60).tolist(), 12000)
    b.fork(list(range(40)), list(range(100, 140)))
    b.free(list(range(0, 60, 2)))
    b.compact()
    b.extend(list(range(150, 210)), [200] * 60, 12000)
    b.compact()
    b.extend([299], [1], 1)


def test_a_pool_of_more_spans_than_the_plan_has_threads(lib):
    """9.5 million pages (1160 spans), all held by the caller but 5000."""
    require_gpu()
    pages, rows, blocks = 9_500_000, 50, 120
    rng = np.random.default_rng(2)
    free = np.sort(rng.permutation(pages)[:5000])
    free[-1] = pages - 1
    refs = torch.ones(pages, dtype=torch.int32, device="cuda")
    refs[torch.from_numpy(free).cuda()] = 0
    table, lens = _i(np.full((rows, blocks), -1)), _i([0] * rows)
    ws = torch.full((lib.workspace_bytes_pages(rows, pages, 64),), 0xA5, dtype=torch.uint8).cuda()
    new = rng.integers(50, 110, 48)
    total = int(new.sum())
    assert total < 5000
    ptr, slots, results = lib.mla_pages_extend(table, lens, refs, _i(np.arange(48)), _i(new), 1, total, workspace=ws)
    assert not results.any() and ptr.tolist() == [0, *np.cumsum(new).tolist()]
    assert slots.tolist() == free[:total].tolist()
    want = np.full((rows, blocks), -1)
    at = 0
    for r, n in enumerate(new):
        want[r, :n] = free[at:at + n]
        at += n
    assert table.cpu().numpy().tolist() == want.tolist()
    # Give some back and compact: the live pages from the back fill the holes, in id order.
    lib.mla_pages_free(table, lens, refs, _i([3, 11, 40]), 1)
    state, before = refs.cpu().numpy().copy(), table.cpu().numpy().copy()
    counts, src, dst = lib.mla_pages_compact(table, lens, refs, 1, workspace=ws)
    live = int((state > 0).sum())
    from_back = live + np.flatnonzero(state[live:] > 0)
    holes = np.flatnonzero(state[:live] <= 0)
    assert counts.tolist() == [live, len(holes)] and len(holes) == len(from_back)
    assert src[:len(holes)].tolist() == from_back.tolist() and dst[:len(holes)].tolist() == holes.tolist()
    assert (src[len(holes):] == -1).all() and (dst[len(holes):] == -1).all()
    renamed = dict(zip(from_back.tolist(), holes.tolist()))
    assert table.tolist() == [[renamed.get(p, p) for p in row] for row in before.tolist()]
    assert (refs[:live] == 1).all() and not refs[live:].any()
