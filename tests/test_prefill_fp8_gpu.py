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


def bf16_caches(x):
    ckv, kpe = oracle.dequantize_fp8_cache(x["kv"].numpy())
    shape = x["kv"].shape[:2]
    return (torch.from_numpy(np.asarray(ckv)).reshape(*shape, 512).to(torch.bfloat16).cuda(),
            torch.from_numpy(np.asarray(kpe)).reshape(*shape, 64).to(torch.bfloat16).cuda())


@pytest.mark.parametrize("heads,page", [(1, 1), (16, 64), (100, 7), (128, 128)])
def test_staged_prefill_of_the_bf16_cache_is_the_same_bits(lib, heads, page):
    """The FP8 form stages the very numbers that the dequantised bf16 cache holds."""
    require_gpu()
    x = make([3, 0, 40, 1], [150, 9, 40, 700], heads, page, seed=20 + heads)
    x["ki"][5], x["ki"][160] = -3, 2 ** 31 - 1
    a = run(lib, x)
    c = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in x.items()}
    b = lib.mla_paged_prefill_staged(c["qn"], c["qp"], *bf16_caches(x), c["qo"], c["kp"], c["ki"], x["scale"])
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    close(b, plain(x))


def test_staged_prefill_agrees_with_the_row_by_row_prefill(lib):
    """Both within their bounds of the exact values, so within the sum of their bounds."""
    require_gpu()
    w = wl.make_prefill([33, 70, 1], [31, 0, 500], num_qo_heads=128, page_size=64, seed=99, name="staged").to("cuda")
    a = lib.run_workload(w)
    b = lib.mla_paged_prefill_staged(w.q_nope, w.q_pe, w.ckv_cache, w.kpe_cache, w.qo_indptr, w.kv_indptr, w.kv_indices,
                                     w.sm_scale)
    # 2^-8 (|ref| + W) each, W <= max |v| < 5.5; lse within 1e-3 of the row-by-row kernel's tolerance
    assert (a[0].float() - b[0].float()).abs().max() <= 4 * 2.0 ** -8 * 5.5
    assert (a[1] - b[1]).abs().max() <= 1e-3


@pytest.mark.parametrize("heads", [16, 128])
@pytest.mark.parametrize("workers", [0, 5])
def test_keys_that_are_not_finite(lib, heads, workers):
    """A NaN or infinite key makes the rows that see it NaN and no other: not the earlier tokens
    of the same block, not the other requests, not rows that end on the same tile."""
    require_gpu()
    x = make([6, 9, 4], [130, 300, 64], heads, 64, seed=30)
    tokens = x["kv"].view(-1, 656)
    keys = {b: x["ki"][x["kp"][b]:x["kp"][b + 1]].long() for b in range(3)}
    clean = plain(x)
    # Request 0: its last token's key has a NaN code, so only that token sees it.  Request 1: a
    # scale is infinite on the key of its token 5.  Request 2: an infinite rope value on key 0.
    tokens[keys[0][129], 100] = 0x7F
    tokens[keys[1][296], 512:516] = torch.tensor([float("inf")]).view(torch.uint8)
    tokens[keys[2][0], 528:530] = torch.tensor([float("-inf")], dtype=torch.bfloat16).view(torch.uint8)
    out, lse = (t.float().cpu() for t in run(lib, x, num_workers=workers))
    bad = torch.zeros(19, dtype=torch.bool)
    bad[5] = True            # request 0, token 5
    bad[6 + 5:15] = True     # request 1, tokens 5 .. 8 see key 296
    bad[15:] = True          # request 2, every token
    assert torch.isnan(out[bad]).all() and torch.isnan(lse[bad]).all()
    good = ~bad.numpy()
    close((out[~bad], lse[~bad]), tuple(t[good] for t in clean))


def test_queries_that_are_not_finite(lib):
    """A NaN query row spoils that row alone, not the rows of its block."""
    require_gpu()
    x = make([7, 5], [90, 200], 24, 16, seed=31)
    ref = plain(x)
    x["qn"][3, 7, 11] = float("nan")
    x["qp"][8, 0, 5] = float("inf")
    out, lse = (t.float().cpu() for t in run(lib, x))
    bad = torch.zeros(12, 24, dtype=torch.bool)
    bad[3, 7] = bad[8, 0] = True
    assert torch.isnan(out[bad]).all() and torch.isnan(lse[bad]).all()
    good = ~bad.numpy()
    close((out[~bad], lse[~bad]), tuple(t[good] for t in ref))


@pytest.mark.parametrize("scale", [0.0, -0.05, 1e-30, 3.0])
def test_softmax_scales(lib, scale):
    require_gpu()
    x = make([9, 2], [140, 77], 16, 64, seed=32)
    x["scale"] = scale
    ref = list(plain(x))
    ref[3] = np.abs(ref[3])
    close(run(lib, x), ref)


def test_same_slot_many_times(lib):
    require_gpu()
    x = make([8, 3], [200, 64], 16, 64, seed=33)
    x["ki"][:200] = x["ki"][:200][torch.arange(200) % 7]
    close(run(lib, x), plain(x))


def test_two_streams_with_their_own_workspaces(lib):
    require_gpu()
    xs = [make([60, 9], [500, 130], 16, 64, seed=40 + i) for i in range(2)]
    refs = [plain(x) for x in xs]
    on_gpu = [{k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in x.items()} for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    ws = [torch.zeros(1 << 27, dtype=torch.uint8, device="cuda") for _ in xs]
    torch.cuda.synchronize()
    outs = []
    for _ in range(5):
        outs = [lib.mla_paged_prefill_fp8(c["qn"], c["qp"], c["kv"], c["qo"], c["kp"], c["ki"], c["scale"], workspace=w,
                                          stream=s) for c, w, s in zip(on_gpu, ws, streams)]
    torch.cuda.synchronize()
    for o, r in zip(outs, refs):
        close(o, r)


def test_validate_reports_bad_offsets(lib):
    require_gpu()
    x = make([4, 7], [200, 70], 16, 64, seed=34)
    ws = torch.zeros(1 << 27, dtype=torch.uint8, device="cuda")
    run(lib, x, workspace=ws, flags=lib.MLA_VALIDATE)
    assert lib.read_device_status(ws) == 0
    x["ki"][3] = -1
    run(lib, x, workspace=ws, flags=lib.MLA_VALIDATE)
    assert lib.read_device_status(ws) == -6


@pytest.mark.parametrize("qo,kp", [([0, 11, 4], [0, 200, 270]), ([0, 4, 11], [0, 300, 270]), ([5, 2, 60], [-7, 900, 3]),
                                   ([0, 11, 0], [0, 270, 0])])
def test_corrupt_offsets_stay_in_bounds(lib, qo, kp):
    """Offsets that decrease or leave their arrays: the call returns, and nothing outside the
    outputs is written (guard rows keep their values)."""
    require_gpu()
    x = make([4, 7], [200, 70], 16, 64, seed=35)
    x["qo"], x["kp"] = torch.tensor(qo, dtype=torch.int32), torch.tensor(kp, dtype=torch.int32)
    guard = torch.full((11 + 64, 16, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((11 + 64, 16), 7.0, device="cuda")
    run(lib, x, out=guard[32:43], lse=lse[32:43])
    torch.cuda.synchronize()
    for t in (guard, lse):
        assert (t[:32] == 7).all() and (t[43:] == 7).all()


def test_bounded_waits(lib):
    """A load that never happens: the call returns, the status says timeout, the next call is right."""
    require_gpu()
    x = make([40], [2000], 16, 64, seed=36)
    ws = torch.zeros(1 << 28, dtype=torch.uint8, device="cuda")
    try:
        lib.lib().mla_debug_inject_timeout(1, 20_000_000)
        run(lib, x, workspace=ws, num_workers=1)
        assert lib.read_device_status(ws) == -7
    finally:
        lib.lib().mla_debug_inject_timeout(-1, 0)
    close(run(lib, x, workspace=ws, num_workers=1), plain(x))
    assert lib.read_device_status(ws) == 0


def test_long_cache(lib):
    """2.1 million keys of one request: staged rows past 2 GB, a row split over every worker."""
    require_gpu()
    n, page = 2_100_000, 64
    pages = -(-n // page)
    g = torch.Generator(device="cuda").manual_seed(3)
    kv = torch.zeros(pages, page, 656, dtype=torch.uint8, device="cuda")
    kv[..., :512] = torch.randint(0, 0x7F, (pages, page, 512), generator=g, device="cuda", dtype=torch.uint8)
    kv[..., 512:528] = torch.full((4,), 2.0 ** -6, device="cuda").view(torch.uint8)
    kv[..., 528:] = torch.randn(pages, page, 64, generator=g, device="cuda").to(torch.bfloat16).view(torch.uint8)
    q = [torch.randn(3, 5, d, generator=g, device="cuda").to(torch.bfloat16) for d in (512, 64)]
    ki = torch.randperm(pages * page, generator=g, device="cuda")[:n].to(torch.int32)
    scale = 0.02
    out, lse = lib.mla_paged_prefill_fp8(*q, kv, torch.tensor([0, 3], dtype=torch.int32, device="cuda"),
                                         torch.tensor([0, n], dtype=torch.int32, device="cuda"), ki, scale)
    tok = kv.view(-1, 656)
    top, acc, tot, wsum = None, 0, 0, 0
    for at in range(0, n, 300_000):
        rows = tok[ki[at:at + 300_000].long()]
        v = rows[:, :512].contiguous().view(torch.float8_e4m3fn).double() * 2.0 ** -6
        r = rows[:, 528:].contiguous().view(torch.bfloat16).double()
        s = (q[0].double() @ v.t() + q[1].double() @ r.t()) * scale
        idx = torch.arange(at, at + rows.shape[0], device="cuda")
        s = s.masked_fill((idx[None] >= (n - 3 + torch.arange(3, device="cuda") + 1)[:, None])[:, None], -math.inf)
        m = s.amax(-1, keepdim=True) if top is None else torch.maximum(top, s.amax(-1, keepdim=True))
        old = 1.0 if top is None else torch.exp(top - m)
        p = torch.exp(s - m)
        acc, tot, wsum = acc * old + p @ v, tot * old + p.sum(-1, keepdim=True), wsum * old + p @ v.abs()
        top = m
    ref, w = acc / tot, wsum / tot
    assert ((out.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 1e-3) * w).all()
    # (float32 sums of 2.1 million terms in tiles: 2^-24 for each of at most 220 partial sums a worker)
    assert ((lse.double() - (top + tot.log())[..., 0]).abs() <= 1e-4).all()


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


def test_what_a_call_allocates_belongs_to_its_stream(lib):
    """Memory of the current stream may still be in use there, or be zeroed too late, when a call
    runs on another stream: whatever the call allocates is that stream's."""
    require_gpu()
    x = make([60, 9], [500, 130], 16, 64, seed=44)
    ref = plain(x)
    c = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in x.items()}
    slots = torch.arange(500, dtype=torch.int32, device="cuda")
    table = torch.full((4, 2000), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(4, dtype=torch.int32, device="cuda")
    refs = torch.zeros(8000, dtype=torch.int32, device="cuda")
    rows = torch.arange(4, dtype=torch.int32, device="cuda")
    new = torch.full((4,), 2000, dtype=torch.int32, device="cuda")
    latent = torch.randn(69, 512, device="cuda").to(torch.bfloat16)
    key = torch.randn(69, 64, device="cuda").to(torch.bfloat16)
    pos = torch.zeros(69, dtype=torch.int32, device="cuda")
    freq = torch.ones(32, device="cuda")
    nowhere = torch.full((69,), -1, dtype=torch.int32, device="cuda")
    rows_ref = lib.mla_cache_gather_fp8(c["kv"], slots)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.memory._record_memory_history(context=None, max_entries=1000)
    try:
        got = lib.mla_paged_prefill_fp8(c["qn"], c["qp"], c["kv"], c["qo"], c["kp"], c["ki"], c["scale"], stream=side)
        gathered = lib.mla_cache_gather_fp8(c["kv"], slots, stream=side)
        indptr, taken, results = lib.mla_pages_extend(table, lens, refs, rows, new, 1, 8000, stream=side)
        rotated = lib.mla_rope_append_fp8(c["qp"], latent, key, pos, freq, nowhere, c["kv"], stream=side)
        moves = lib.mla_pages_compact(table, lens, refs, 1, stream=side)
        trace = torch.cuda.memory._snapshot()["device_traces"][torch.cuda.current_device()]
    finally:
        torch.cuda.memory._record_memory_history(enabled=None)
    streams = [e["stream"] for e in trace if e["action"] == "alloc"]
    # (outputs and workspaces: 2 + 1, 2, 3 + 1, 1, 3 + 1)
    assert len(streams) == 14 and set(streams) == {side.cuda_stream}
    torch.cuda.synchronize()
    close(got, ref)
    assert all(torch.equal(a, b) for a, b in zip(gathered, rows_ref))
    assert results.tolist() == [0] * 4 and indptr.tolist() == [0, 2000, 4000, 6000, 8000]
    assert torch.equal(taken.cpu(), torch.arange(8000, dtype=torch.int32))
    assert torch.equal(rotated, c["qp"])
    assert moves[0].tolist() == [8000, 0]


def test_two_graphs_share_a_workspace(lib):
    """Calls of other sizes captured into two graphs over one workspace, replayed in turn: nothing
    in it carries over.  A third call allocates its workspace inside the capture."""
    require_gpu()
    xs = [make([60, 9, 0], [500, 130, 64], 16, 64, seed=50), make([3, 1, 40, 7], [900, 1, 40, 333], 24, 16, seed=51)]
    cs = [{k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in x.items()} for x in xs]
    ws = torch.zeros(1 << 27, dtype=torch.uint8, device="cuda")

    def call(c, workspace):
        return lib.mla_paged_prefill_fp8(c["qn"], c["qp"], c["kv"], c["qo"], c["kp"], c["ki"], c["scale"],
                                         workspace=workspace)

    want = [call(c, ws) for c in cs]
    for w, x in zip(want, xs):
        close(w, plain(x))
    captured = []
    for c, workspace in ((cs[0], ws), (cs[1], ws), (cs[0], None)):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = call(c, workspace)
        captured.append((graph, got))
    for i in (0, 1, 2, 1, 0, 0, 2):
        graph, got = captured[i]
        for t in got:
            t.fill_(float("nan"))
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, want[i % 2]))
