"""The staged prefill on inputs whose results are exact, so that one key lost, doubled or taken for
another shows whatever the length.

Token t of the cache is one at latent column t % 512 and at rope column t % 64, else zero.

* With queries of zeros every key weighs 1, so the row's sum and every output column's sum are
  integers that float32 (and bf16, for the weights) holds exactly: with v keys in sight, c_j of them
  one at column j, lse = log v and out_j = c_j / v.
* With a query of 2 at one column (latent or rope) a score is 2 or 0, exactly: with c of the v keys
  one there, lse = log(v - c + c e^2), and out_j is the sum of its keys' weights over that.

Tolerances.  lse: a weight is off by less than 2^-21 relative (a product and a sum in float32, an
exponential of two units), the sums of at most 2^16 weights in a few hundred pieces by 2^-16 at worst, a
piece's log2 (below 2^5) by 2^-19 absolute, the last logarithm by 2^-20: 2.5e-5 in all.  One key more
or less changes it by at least 1 / (the sum of the weights): 1 / 30,000 = 3.3e-5 for the longest flat
row here, 1 / 5000 for the longest peaked one (a column's keys are a 64th of all at most, so the sum is
below 1.11 v).  out: half a bf16 step for the output, another for the weights (none where all are 1),
and the lse's 2.5e-5, all relative; one key more or less is at least 1 / c_j, with c_j below 60 in
the flat rows, and e^-2 / c_j with c_j below 9 in the peaked ones.
"""

import math

import numpy as np
import pytest
import torch

from tests.conftest import require_gpu

HALF_STEP = 2.0 ** -8
LSE = 2.5e-5


def cache(pages, page):
    """The FP8 tokens as described above: E4M3 ones under scales of one."""
    n = pages * page
    t = torch.arange(n)
    kv = torch.zeros(n, 656, dtype=torch.uint8)
    kv[t, t % 512] = 0x38
    kv[:, 512:528] = torch.ones(n, 4).view(torch.uint8)
    rope = torch.zeros(n, 64, dtype=torch.bfloat16)
    rope[t, t % 64] = 1
    kv[:, 528:] = rope.view(torch.uint8)
    return kv.view(pages, page, 656)


def make(q_lens, kv_lens, page, seed):
    """(offsets of the queries, of the keys, slots in random order, pages)."""
    rng = np.random.default_rng(seed)
    pages = -(-sum(kv_lens) // page) + 3
    slots = rng.permutation(pages * page)[:sum(kv_lens)]
    return np.concatenate([[0], np.cumsum(q_lens)]), np.concatenate([[0], np.cumsum(kv_lens)]), slots, pages


def columns(rows, heads):
    """The column (0 .. 575) where every row's query is 2."""
    return (7 * np.arange(rows)[:, None] + 13 * np.arange(heads)) % 576


def reference(qo, kp, slots, heads, peaked, drop=None, double=None):
    """(out, lse) in float64; ``drop`` / ``double``: the position in ``slots`` of a key to leave out
    or to count twice."""
    rows = qo[-1]
    out, lse = np.zeros((rows, heads, 512)), np.full((rows, heads), -math.inf)
    where = columns(rows, heads)
    for b in range(len(qo) - 1):
        n, m = qo[b + 1] - qo[b], kp[b + 1] - kp[b]
        for i in range(n):
            see = np.arange(kp[b], kp[b] + max(0, m - n + i + 1))
            if double is not None and double in see:
                see = np.append(see, double)
            if drop is not None:
                see = see[see != drop]
            if not len(see):
                continue
            r, mine = qo[b] + i, slots[see]
            flat = np.bincount(mine % 512, minlength=512).astype(np.float64)
            if not peaked:
                out[r], lse[r] = flat / len(see), math.log(len(see))
                continue
            for h in range(heads):
                c = where[r, h]
                hit = mine % 512 == c if c < 512 else mine % 64 == c - 512
                w = np.where(hit, math.exp(2), 1.0)
                out[r, h] = np.bincount(mine % 512, weights=w, minlength=512) / w.sum()
                lse[r, h] = math.log(w.sum())
    return out, lse


def right(got, ref, peaked):
    out, lse = (np.asarray(t, np.float64) for t in got)
    none = np.isneginf(ref[1])
    if not np.array_equal(np.isneginf(lse), none) or not np.isfinite(out).all():
        return False
    if not (np.abs(lse[~none] - ref[1][~none]) <= LSE).all():
        return False
    return bool((np.abs(out - ref[0]) <= ((2 if peaked else 1) * HALF_STEP * 1.01 + LSE) * ref[0]).all())


CASES = [([9, 1, 20], [1500, 3000, 20]), ([1], [4400]), ([3, 1, 0, 8], [3, 64, 5, 129]), ([130, 2], [700, 1])]


@pytest.mark.parametrize("peaked", [False, True])
@pytest.mark.parametrize("q_lens,kv_lens", CASES)
def test_the_check_sees_a_single_key(q_lens, kv_lens, peaked):
    """On the CPU: the reference itself passes, rounded to bf16; with any one key dropped or counted
    twice it does not."""
    qo, kp, slots, _ = make(q_lens, kv_lens, 16, 3)

    def rounded(ref):
        return torch.from_numpy(ref[0]).to(torch.bfloat16).double().numpy(), ref[1].astype(np.float32)

    ref = reference(qo, kp, slots, 2, peaked)
    assert right(rounded(ref), ref, peaked)
    rng = np.random.default_rng(5)
    for b in range(len(q_lens)):
        if not q_lens[b]:
            continue
        some = {0, 127, 128, kv_lens[b] - 1, *rng.integers(0, kv_lens[b], 4).tolist()}
        for k in sorted(k for k in some if k < kv_lens[b]):
            for change in ("drop", "double"):
                other = reference(qo, kp, slots, 2, peaked, **{change: kp[b] + k})
                assert not right(rounded(other), ref, peaked), (b, k, change)


def run(lib, qo, kp, slots, pages, page, heads, peaked, **kw):
    rows = int(qo[-1])
    q = torch.zeros(rows, heads, 576, dtype=torch.bfloat16)
    if peaked:
        q.scatter_(2, torch.from_numpy(columns(rows, heads))[..., None], 2.0)
    to = lambda a: torch.tensor(a, dtype=torch.int32).cuda()  # noqa: E731
    got = lib.mla_paged_prefill_fp8(q[..., :512].contiguous().cuda(), q[..., 512:].contiguous().cuda(),
                                    cache(pages, page).cuda(), to(qo), to(kp), to(slots), 1.0, **kw)
    return [t.float().cpu().numpy() for t in got]


@pytest.mark.gpu
@pytest.mark.parametrize("peaked", [False, True])
@pytest.mark.parametrize("heads,workers", [(1, 0), (16, 0), (16, 1), (16, 2), (16, 7), (16, 150), (100, 40), (128, 0),
                                           (128, 11)])
@pytest.mark.parametrize("q_lens,kv_lens", CASES)
def test_every_key_counts_once(lib, q_lens, kv_lens, heads, workers, peaked):
    require_gpu()
    qo, kp, slots, pages = make(q_lens, kv_lens, 16, heads + workers)
    got = run(lib, qo, kp, slots, pages, 16, heads, peaked, num_workers=workers)
    assert right(got, reference(qo, kp, slots, heads, peaked), peaked)


@pytest.mark.gpu
@pytest.mark.parametrize("workers", [0, 3, 76, 300])
def test_long_rows(lib, workers):
    """One token over 25,000 keys and ten over 30,000, split over every worker."""
    require_gpu()
    qo, kp, slots, pages = make([1, 10], [25000, 30000], 64, workers)
    got = run(lib, qo, kp, slots, pages, 64, 16, False, num_workers=workers)
    assert right(got, reference(qo, kp, slots, 16, False), False)


@pytest.mark.gpu
@pytest.mark.parametrize("batch", [1023, 1024, 1025, 2600])
def test_more_requests_than_the_plan_keeps_near(lib, batch):
    """Around and far above the 1024 requests and row blocks that the plan keeps in shared memory."""
    require_gpu()
    rng = np.random.default_rng(batch)
    q_lens = rng.integers(0, 4, batch)
    q_lens[-1] = 30  # (the last request has several blocks)
    kv_lens = rng.integers(0, 150, batch)
    qo, kp, slots, pages = make(q_lens.tolist(), kv_lens.tolist(), 16, batch)
    got = run(lib, qo, kp, slots, pages, 16, 16, False)
    assert right(got, reference(qo, kp, slots, 16, False), False)
