"""Chunk prefill over an FP8 cache against a plain float64 attention.

Tolerances.  With keys exact (the cache's bf16 numbers), a score differs from the exact one
by at most d = 2^-14 scale (|q| . |k|) (float32 accumulation over 576 products, and partial
sums that may travel between SMs rounded to 16 bits, 2^-16 each); the weights are rounded
to bf16 (half a step, 2^-8) and the output once more.  So, with W = sum_t p_t |v_t|,
  |out - ref| <= 2^-8 |ref| + (2^-8 + 4 d) W,   |lse - ref| <= 2 d + 1e-5.
"""

import math

import numpy as np
import pytest
import torch

import oracle
from paged_head_latent_gb300 import workloads as wl
from tests.conftest import require_gpu

pytestmark = pytest.mark.gpu


def make(q_lens, kv_lens, heads, page, seed, q_scale=1.0):
    """FP8 workload with ragged chunks (kv_lens may be shorter than q_lens)."""
    g = torch.Generator().manual_seed(seed)
    w = wl.quantize_fp8(wl.make_decode(kv_lens, 1, page, seed=seed))
    total = sum(q_lens)
    qn = (torch.randn(total, heads, 512, generator=g) * q_scale).to(torch.bfloat16)
    qp = (torch.randn(total, heads, 64, generator=g) * q_scale).to(torch.bfloat16)
    ptr = torch.tensor([0] + np.cumsum(q_lens).tolist(), dtype=torch.int32)
    return dict(qn=qn, qp=qp, kv=w.kv_fp8, qo=ptr, kp=w.kv_indptr, ki=w.kv_indices, scale=w.sm_scale)


def plain(x, valid=None):
    """(out, lse, W, d) in float64; keys outside the cache are left out."""
    ckv, kpe = oracle.dequantize_fp8_cache(x["kv"].numpy())
    ckv, kpe = np.asarray(ckv, np.float64).reshape(-1, 512), np.asarray(kpe, np.float64).reshape(-1, 64)
    total, heads = x["qn"].shape[:2]
    out, lse = np.zeros((total, heads, 512)), np.full((total, heads), -math.inf)
    weight, slack = np.zeros((total, heads, 512)), np.zeros((total, heads))
    qn, qp = x["qn"].double().numpy(), x["qp"].double().numpy()
    qo, kp, ki = x["qo"].numpy(), x["kp"].numpy(), x["ki"].numpy()
    for b in range(len(qo) - 1):
        n, m = qo[b + 1] - qo[b], kp[b + 1] - kp[b]
        slots = ki[kp[b]:kp[b + 1]]
        for i in range(n):
            see = slots[:max(0, m - n + i + 1)]
            see = see[(see >= 0) & (see < len(ckv))]
            if not len(see):
                continue
            r = qo[b] + i
            k, p = ckv[see], kpe[see]
            s = (qn[r] @ k.T + qp[r] @ p.T) * x["scale"]
            top = s.max(-1, keepdims=True)
            e = np.exp(s - top)
            tot = e.sum(-1, keepdims=True)
            e /= tot
            lse[r] = (top + np.log(tot))[:, 0]
            out[r] = e @ k
            weight[r] = e @ np.abs(k)
            slack[r] = 2.0 ** -14 * x["scale"] * (np.abs(qn[r]) @ np.abs(k).T + np.abs(qp[r]) @ np.abs(p).T).max(-1)
    return out, lse, weight, slack


def run(lib, x, **kw):
    c = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in x.items()}
    return lib.mla_paged_prefill_fp8(c["qn"], c["qp"], c["kv"], c["qo"], c["kp"], c["ki"], c["scale"], **kw)


def close(got, ref, rows=None):
    out, lse = (t.float().cpu().numpy().astype(np.float64) for t in got)
    ro, rl, w, d = ref
    if rows is not None:
        out, lse = out[:rows], lse[:rows]
    none = np.isneginf(rl)
    assert np.array_equal(np.isneginf(lse), none)
    assert not out[none].any()
    err = np.abs(lse[~none] - rl[~none]) - (2 * d[~none] + 1e-5)
    assert err.size == 0 or err.max() <= 0, err.max()
    err = np.abs(out - ro) - (2.0 ** -8 * np.abs(ro) + (2.0 ** -8 + 4 * d[..., None]) * w)
    assert np.isfinite(out).all() and err.max() <= 0, err.max()


@pytest.mark.parametrize("heads,page", [(1, 64), (5, 7), (16, 16), (24, 64), (33, 1), (64, 32), (100, 128), (128, 64)])
@pytest.mark.parametrize("q_lens,kv_lens", [
    ([1], [1]), ([3, 1, 0, 8], [3, 64, 5, 65]), ([17, 2, 9], [200, 63, 9]), ([5, 4], [3, 0]), ([130], [700])])
def test_ragged_chunks(lib, heads, page, q_lens, kv_lens):
    require_gpu()
    x = make(q_lens, kv_lens, heads, page, seed=9 * heads + len(q_lens))
    ws = torch.zeros(1 << 28, dtype=torch.uint8, device="cuda")
    got = run(lib, x, workspace=ws)
    close(got, plain(x))
    assert lib.read_device_status(ws) == 0


@pytest.mark.parametrize("heads", [16, 128])
@pytest.mark.parametrize("workers", [1, 2, 7, 40, 150])
def test_split_counts(lib, heads, workers):
    require_gpu()
    x = make([9, 1, 20], [1500, 3000, 20], heads, 64, seed=workers)
    close(run(lib, x, num_workers=workers), plain(x))


def test_many_requests(lib):
    """More requests than workers, most of one token."""
    require_gpu()
    rng = np.random.default_rng(3)
    q = rng.integers(0, 4, 400).tolist()
    kv = [int(n + rng.integers(0, 150)) for n in q]
    x = make(q, kv, 16, 16, seed=77)
    close(run(lib, x), plain(x))


def test_large_scores_keep_their_order(lib):
    """Peaked softmaxes: scores of several hundred, so almost all weight is on one key."""
    require_gpu()
    x = make([6, 40], [300, 40], 16, 64, seed=5, q_scale=30.0)
    close(run(lib, x), plain(x))


def test_slots_outside_the_cache_and_unused_tokens(lib):
    require_gpu()
    x = make([4, 7, 3], [200, 70, 3], 16, 64, seed=6)
    tokens = x["kv"].view(-1, 656)
    unused = torch.ones(tokens.shape[0], dtype=torch.bool)
    unused[x["ki"].long()] = False
    tokens[unused] = 0x7F  # NaN codes and scales
    x["ki"][3], x["ki"][100], x["ki"][203] = -1, tokens.shape[0], 2 ** 31 - 1
    x["ki"][270:] = -5  # the last request has no key at all
    close(run(lib, x), plain(x))


def test_rows_behind_the_last_request_and_a_capacity(lib):
    """A padded step: more query rows and more key indices than the offsets use."""
    require_gpu()
    x = make([3, 20], [100, 90], 24, 16, seed=8)
    ref = plain(x)
    pad = dict(x)
    pad["qn"] = torch.cat([x["qn"], torch.full((5, 24, 512), float("nan"), dtype=torch.bfloat16)])
    pad["qp"] = torch.cat([x["qp"], torch.full((5, 24, 64), float("nan"), dtype=torch.bfloat16)])
    pad["ki"] = torch.cat([x["ki"], torch.full((300,), 2 ** 31 - 1, dtype=torch.int32)])
    out = torch.full((28, 24, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((28, 24), 7.0, device="cuda")
    got = run(lib, pad, out=out, lse=lse)
    close(got, ref, rows=23)
    assert (out[23:] == 7).all() and (lse[23:] == 7).all()


def test_captured_and_replayed_with_other_lengths(lib):
    """One graph, replayed with other offsets, indices and queries; two graphs share a workspace."""
    require_gpu()
    a, b = make([5, 60, 2], [64, 500, 129], 16, 64, seed=10), make([60, 1, 6], [500, 129, 64], 16, 64, seed=11)
    n = min(a["kv"].shape[0], b["kv"].shape[0])
    buf = {k: (torch.zeros_like(v) if k != "kv" else torch.zeros_like(v[:n])).cuda() for k, v in a.items()
           if isinstance(v, torch.Tensor)}
    ws = torch.zeros(1 << 27, dtype=torch.uint8, device="cuda")
    for k in buf:
        buf[k].copy_(a[k][:n] if k == "kv" else a[k])

    def call():
        return lib.mla_paged_prefill_fp8(buf["qn"], buf["qp"], buf["kv"], buf["qo"], buf["kp"], buf["ki"], a["scale"],
                                         workspace=ws)

    call()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call())
        graphs.append(g)
    for x in (a, b, a):
        x = dict(x, kv=x["kv"][:n].contiguous())
        x["ki"] = x["ki"].clamp(max=n * 64 - 1)
        ref = plain(x)
        for k in buf:
            buf[k].copy_(x[k])
        for g, o in zip(graphs, outs):
            g.replay()
            torch.cuda.synchronize()
            close(o, ref)


def test_repeats_exactly(lib):
    require_gpu()
    x = make([100, 3], [2000, 1000], 16, 64, seed=12)
    a, b = run(lib, x), run(lib, x)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_serving_steps_end_to_end(lib):
    """The operators as a serving program chains them: prompts extend the pool, are rotated
    and written, attend as a chunk; a fork, its page copies, a decode step, a free and a
    compaction; every attention output against the plain form on the cache as it then is."""
    require_gpu()
    ps, heads, rows, pages = 16, 16, 6, 40
    g = torch.Generator().manual_seed(1)
    kv = torch.zeros(pages, ps, 656, dtype=torch.uint8, device="cuda")
    table = torch.full((rows, 12), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(rows, dtype=torch.int32, device="cuda")
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    pool = (table, lens, refs)
    freq = (10000.0 ** (-torch.arange(32) / 32)).float().cuda()
    scale = 192 ** -0.5
    seen = {}

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    def step(which, new):
        before = lens.clone()
        ptr, slots, results = lib.mla_pages_extend(*pool, ints(which), ints(new), ps, sum(new))
        assert not results.any()
        total = sum(new)
        qn = torch.randn(total, heads, 512, generator=g).to(torch.bfloat16)
        qr = torch.randn(total, heads, 64, generator=g).to(torch.bfloat16)
        lat = torch.randn(total, 576, generator=g).to(torch.bfloat16).cuda()
        pos = torch.cat([before[r] + torch.arange(n, device="cuda") for r, n in zip(which, new)]).to(torch.int32)
        qp = lib.mla_rope_append_fp8(qr.cuda(), lat[:, :512], lat[:, 512:], pos, freq, slots, kv)
        some = ints(which).long()
        kp, ki = lib.block_table_to_csr(table[some].contiguous(), lens[some].contiguous(), ps)
        out, lse = lib.mla_paged_prefill_fp8(qn.cuda(), qp, kv, ptr, kp, ki, scale)
        x = dict(qn=qn, qp=qp.cpu(), kv=kv.cpu(), qo=ptr.cpu(), kp=kp.cpu(), ki=ki.cpu()[:int(kp[-1])], scale=scale)
        close((out, lse), plain(x))
        for r in which:
            seen[r] = lib.mla_cache_gather_fp8(kv, (table[r][:, None] * ps + torch.arange(ps, device="cuda")).flatten()[
                :int(lens[r])].to(torch.int32).contiguous())

    step([0, 1, 2], [37, 16, 5])
    res, src, dst, tokens = lib.mla_pages_fork(*pool, ints([0, 0, 1]), ints([3, 4, 5]), ps)
    assert not res.any() and tokens.tolist() == [5, 5, 0]
    lib.mla_cache_copy_pages_fp8(kv, src, dst, tokens=tokens)
    step([3, 4, 0, 5], [1, 1, 1, 1])
    assert torch.equal(seen[3][0][:37], seen[4][0][:37]) and not torch.equal(seen[3][0][37], seen[4][0][37])
    lib.mla_pages_free(*pool, ints([1, 0]), ps)
    counts, src, dst = lib.mla_pages_compact(*pool, ps)
    lib.mla_cache_copy_pages_fp8(kv, src, dst, count=counts[1:])
    kept = dict(seen)
    step([2, 3, 4, 5], [20, 2, 3, 4])
    for r in (2, 3, 4, 5):
        n = kept[r][0].shape[0]
        assert torch.equal(seen[r][0][:n], kept[r][0]) and torch.equal(seen[r][1][:n], kept[r][1])
