"""Windowed attention with sinks and shared-prefix attention against a plain float64 attention.

Tolerances, as for the staged prefill, whose arithmetic this is.  With keys exact (the cache's
bf16 numbers), a score differs from the exact one by at most d = 2^-14 scale (|q| . |k|) (float32
accumulation over 576 products); the weights are rounded to bf16 (half a step, 2^-8) and the
output once more.  So, with W = sum_t p_t |v_t|,
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

SCALE = 192 ** -0.5


def offsets(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32)


def make(q_lens, lists, heads, page, seed, fp8, q_scale=1.0):
    """Queries, a cache, and the slots of lists (a list of lengths) on random pages."""
    g = torch.Generator().manual_seed(seed)
    w = wl.make_decode([max(n, 1) for n in lists], 1, page, seed=seed)
    x = dict(qn=(torch.randn(sum(q_lens), heads, 512, generator=g) * q_scale).to(torch.bfloat16),
             qp=(torch.randn(sum(q_lens), heads, 64, generator=g) * q_scale).to(torch.bfloat16), qo=offsets(q_lens))
    if fp8:
        x["kv"] = wl.quantize_fp8(w).kv_fp8
    else:
        x["ckv"], x["kpe"] = w.ckv_cache, w.kpe_cache
    at = w.kv_indptr.tolist()
    x["lists"] = [w.kv_indices[at[i]:at[i] + n].clone() for i, n in enumerate(lists)]
    return x


def make_window(q_lens, kv_lens, heads, page, seed, fp8=False, **kw):
    x = make(q_lens, kv_lens, heads, page, seed, fp8, **kw)
    x["ki"], x["kp"] = torch.cat(x["lists"]), offsets(kv_lens)
    return x


def make_shared(groups, heads, page, seed, fp8=False, **kw):
    """groups: (prefix keys, [(new tokens, own keys), ...]) each."""
    q = [n for _, m in groups for n, _ in m]
    own = [n for _, m in groups for _, n in m]
    prefix = [n for n, _ in groups]
    x = make(q, prefix + own, heads, page, seed, fp8, **kw)
    x.update(gp=offsets([len(m) for _, m in groups]), pp=offsets(prefix), kp=offsets(own))
    x["pi"] = torch.cat(x["lists"][:len(prefix)]) if prefix else torch.zeros(0, dtype=torch.int32)
    x["ki"] = torch.cat(x["lists"][len(prefix):])
    return x


def values(x):
    if "kv" in x:
        ckv, kpe = oracle.dequantize_fp8_cache(x["kv"].numpy())
    else:
        ckv, kpe = x["ckv"].double().numpy(), x["kpe"].double().numpy()
    return np.asarray(ckv, np.float64).reshape(-1, 512), np.asarray(kpe, np.float64).reshape(-1, 64)


def plain(x, window=None, sinks=0):
    """(out, lse, W, d) in float64; keys outside the cache are left out."""
    ckv, kpe = values(x)
    total, heads = x["qn"].shape[:2]
    out, lse = np.zeros((total, heads, 512)), np.full((total, heads), -math.inf)
    weight, slack = np.zeros((total, heads, 512)), np.zeros((total, heads))
    qn, qp = x["qn"].double().numpy(), x["qp"].double().numpy()
    qo, kp, ki = x["qo"].numpy(), x["kp"].numpy(), x["ki"].numpy()
    gp = x["gp"].numpy() if "gp" in x else None
    for b in range(len(qo) - 1):
        n, m = qo[b + 1] - qo[b], kp[b + 1] - kp[b]
        prefix = []
        if gp is not None:
            g = max(i for i in range(len(gp) - 1) if gp[i] <= b)
            prefix = x["pi"].numpy()[x["pp"][g]:x["pp"][g + 1]]
        for i in range(n):
            p = m - n + i
            own = [ki[kp[b] + t] for t in range(m) if t <= p and (window is None or t > p - window or t < sinks)]
            see = np.concatenate([prefix, own]).astype(np.int64)
            see = see[(see >= 0) & (see < len(ckv))]
            if not len(see):
                continue
            r = qo[b] + i
            k, e = ckv[see], kpe[see]
            s = (qn[r] @ k.T + qp[r] @ e.T) * SCALE
            top = s.max(-1, keepdims=True)
            e2 = np.exp(s - top)
            tot = e2.sum(-1, keepdims=True)
            e2 /= tot
            lse[r] = (top + np.log(tot))[:, 0]
            out[r] = e2 @ k
            weight[r] = e2 @ np.abs(k)
            slack[r] = 2.0 ** -14 * SCALE * (np.abs(qn[r]) @ np.abs(k).T + np.abs(qp[r]) @ np.abs(e).T).max(-1)
    return out, lse, weight, slack


def on_gpu(x):
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in x.items()}


def call(lib, kind, x, prefill, args, **kw):
    """The call of this kind ("window" or "shared") on x's tensors, on the GPU already."""
    name = f"mla_paged_{'prefill' if prefill else 'decode'}_{kind}" + ("_fp8" if "kv" in x else "")
    cache = (x["kv"],) if "kv" in x else (x["ckv"], x["kpe"])
    lists = (x["kp"], x["ki"]) if kind == "window" else (x["gp"], x["pp"], x["pi"], x["kp"], x["ki"])
    return getattr(lib, name)(x["qn"], x["qp"], *cache, *((x["qo"],) if prefill else ()), *lists, *args, SCALE, **kw)


def close(got, ref, rows=None):
    out, lse = (t.float().cpu().numpy().astype(np.float64) for t in got)
    ro, rl, w, d = ref
    if rows is not None:
        out, lse = out[rows], lse[rows]
        ro, rl, w, d = ro[rows], rl[rows], w[rows], d[rows]
    none = np.isneginf(rl)
    assert np.array_equal(np.isneginf(lse), none)
    assert not out[none].any()
    err = np.abs(lse[~none] - rl[~none]) - (2 * d[~none] + 1e-5)
    assert err.size == 0 or err.max() <= 0, err.max()
    err = np.abs(out - ro) - (2.0 ** -8 * np.abs(ro) + (2.0 ** -8 + 4 * d[..., None]) * w)
    assert np.isfinite(out).all() and (err.size == 0 or err.max() <= 0), err.max()


SIZES = [(1, 64), (5, 7), (16, 16), (24, 64), (33, 1), (64, 32), (100, 128), (128, 64)]


# ---------------------------------------------------------------- windows with sinks
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("heads,page", SIZES)
@pytest.mark.parametrize("window,sinks", [(1, 0), (64, 4), (100, 1), (128, 130), (5000, 7)])
def test_window_decode(lib, heads, page, window, sinks, fp8):
    require_gpu()
    x = make_window([1] * 9, [1, 0, 63, 64, 65, 129, 300, 101, 700], heads, page, heads + window, fp8)
    ws = torch.zeros(1 << 28, dtype=torch.uint8, device="cuda")
    close(call(lib, "window", on_gpu(x), False, (window, sinks), workspace=ws), plain(x, window, sinks))
    assert lib.read_device_status(ws) == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("heads,page", SIZES)
@pytest.mark.parametrize("window,sinks", [(1, 0), (3, 2), (64, 4), (129, 200)])
@pytest.mark.parametrize("q_lens,kv_lens", [([3, 1, 0, 8], [3, 64, 5, 265]), ([17, 2, 9], [200, 63, 9]), ([5, 4], [3, 0]),
                                            ([130], [500])])
def test_window_prefill(lib, heads, page, window, sinks, q_lens, kv_lens, fp8):
    require_gpu()
    if heads > 64 and q_lens == [130] and fp8:
        pytest.skip("the float64 reference takes long; the bf16 case has this size")
    x = make_window(q_lens, kv_lens, heads, page, 9 * heads + len(q_lens), fp8)
    close(call(lib, "window", on_gpu(x), True, (window, sinks)), plain(x, window, sinks))


@pytest.mark.parametrize("window", [2 ** 31 - 1, 4096])
def test_a_window_over_all_keys_is_plain_attention(lib, window):
    """The same tiles in the same order as the staged prefill: the same bits."""
    require_gpu()
    x = on_gpu(make_window([3, 40, 1], [150, 40, 700], 16, 7, 3))
    a = call(lib, "window", x, True, (window, 2 ** 31 - 1))
    b = lib.mla_paged_prefill_staged(x["qn"], x["qp"], x["ckv"], x["kpe"], x["qo"], x["kp"], x["ki"], SCALE)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("kind", ["window", "shared"])
@pytest.mark.parametrize("heads", [16, 128])
@pytest.mark.parametrize("workers", [1, 2, 7, 40, 150])
def test_split_counts(lib, kind, heads, workers):
    require_gpu()
    if kind == "window":
        x, args = make_window([9, 1, 20], [1500, 3000, 20], heads, 64, workers), (1000, 100)
        ref = plain(x, *args)
    else:
        x, args = make_shared([(1500, [(2, 300), (9, 20), (1, 700)]), (200, [(3, 3)] * 4)], heads, 64, workers), ()
        ref = plain(x)
    close(call(lib, kind, on_gpu(x), True, args, num_workers=workers), ref)


@pytest.mark.parametrize("kind", ["window", "shared"])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("heads,page", [(16, 16), (16, 64), (128, 64)])
@pytest.mark.parametrize("workers", [1, 2, 7])
def test_many_blocks_to_a_worker(lib, kind, fp8, heads, page, workers):
    """Decode with few workers: a worker walks through several blocks of several tiles each."""
    require_gpu()
    lens = [700, 1, 0, 300, 129, 64, 500, 65, 900, 128, 640, 7]
    if kind == "window":
        x, args = make_window([1] * len(lens), lens, heads, page, workers, fp8), (500, 3)
    else:
        members = [(1, n) for n in lens]
        x, args = make_shared([(700, members[:5]), (0, members[5:7]), (130, members[7:])], heads, page, workers, fp8), ()
    ws = torch.zeros(1 << 28, dtype=torch.uint8, device="cuda")
    close(call(lib, kind, on_gpu(x), False, args, num_workers=workers, workspace=ws), plain(x, *args))
    assert lib.read_device_status(ws) == 0


# ---------------------------------------------------------------- shared prefixes
GROUPS = [
    [(300, [(1, 5), (1, 1), (1, 130), (1, 0)])],
    [(0, [(1, 0), (1, 64), (1, 0)]), (129, [(1, 0)] * 2), (128, []), (1, [(1, 200)])],
    [(64, [(1, n) for n in range(40)]), (700, [(1, 3)])],
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("heads,page", SIZES)
@pytest.mark.parametrize("groups", GROUPS)
def test_shared_decode(lib, heads, page, groups, fp8):
    require_gpu()
    x = make_shared(groups, heads, page, heads, fp8)
    ws = torch.zeros(1 << 28, dtype=torch.uint8, device="cuda")
    close(call(lib, "shared", on_gpu(x), False, (), workspace=ws), plain(x))
    assert lib.read_device_status(ws) == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("heads,page", SIZES)
@pytest.mark.parametrize("groups", [
    [(300, [(3, 3), (1, 70), (0, 50), (9, 200)]), (0, [(2, 2), (0, 0), (1, 1)])],
    [(130, [(5, 3), (4, 0), (2, 2)])],                 # tokens that see no key of their own
    [(0, [(5, 3), (4, 0)]), (64, []), (0, [(0, 9)])],  # tokens that see none at all
    [(200, [(140, 150), (1, 1), (30, 300)])],
])
def test_shared_prefill(lib, heads, page, groups, fp8):
    require_gpu()
    if heads > 64 and groups[0][1][0][0] == 140 and fp8:
        pytest.skip("the float64 reference takes long; the bf16 case has this size")
    x = make_shared(groups, heads, page, heads + 1, fp8)
    close(call(lib, "shared", on_gpu(x), True, ()), plain(x))


def test_many_groups_and_requests(lib):
    """More groups, requests and blocks than the plan's near tables hold, most of them short."""
    require_gpu()
    rng = np.random.default_rng(3)
    groups = [(int(rng.integers(0, 40)), [(int(rng.integers(0, 3)), int(rng.integers(0, 9))) for _ in
                                          range(int(rng.integers(0, 3)))]) for _ in range(1300)]
    groups += [(150, [(1, 2)] * 300)]
    x = make_shared(groups, 100, 16, 77)
    assert x["kp"].numel() > 1026 and x["gp"].numel() > 1026
    close(call(lib, "shared", on_gpu(x), True, ()), plain(x))


def test_many_window_requests(lib):
    require_gpu()
    rng = np.random.default_rng(4)
    q = rng.integers(0, 3, 1500).tolist()
    kv = [int(n + rng.integers(0, 150)) for n in q]
    x = make_window(q, kv, 16, 16, 78)
    close(call(lib, "window", on_gpu(x), True, (60, 3)), plain(x, 60, 3))


# ---------------------------------------------------------------- both
def both(heads, page, fp8, seed, q=((3, 90), (7, 200), (1, 130))):
    """A window and a shared call with the same kind of rows: (kind, inputs, args)."""
    yield "window", make_window([n for n, _ in q], [m for _, m in q], heads, page, seed, fp8), (70, 5)
    yield "shared", make_shared([(140, [(n, m) for n, m in q[:2]]), (30, [(n, m) for n, m in q[2:]])], heads, page,
                                seed, fp8), ()


@pytest.mark.parametrize("fp8", [False, True])
def test_slots_outside_the_cache_and_unused_tokens(lib, fp8):
    require_gpu()
    for kind, x, args in both(16, 64, fp8, 6):
        slots = (x["kv"].shape[0] if fp8 else x["ckv"].shape[0]) * 64
        used = torch.cat([x["ki"], x.get("pi", x["ki"][:0])]).long()
        unused = torch.ones(slots, dtype=torch.bool)
        unused[used] = False
        for name, width in (("kv", 656),) if fp8 else (("ckv", 512), ("kpe", 64)):
            x[name].view(-1, width)[unused] = 0x7F if fp8 else float("nan")
        x["ki"][3], x["ki"][100], x["ki"][219] = -1, slots, 2 ** 31 - 1
        if kind == "shared":
            x["pi"][0], x["pi"][139], x["pi"][150] = -7, slots + 5, 2 ** 31 - 1
        close(call(lib, kind, on_gpu(x), True, args), plain(x, *args))


@pytest.mark.parametrize("heads", [16, 128])
@pytest.mark.parametrize("workers", [0, 5])
@pytest.mark.parametrize("prefill", [False, True])
def test_window_keys_that_are_not_finite(lib, heads, workers, prefill):
    """A NaN or infinite key makes the rows that see it NaN and no other; keys in front of every
    window, and slots behind a request's last key, may hold anything."""
    require_gpu()
    q = [6, 9, 4] if prefill else [1, 1, 1]
    x = make_window(q, [400, 300, 64], heads, 64, 30)
    clean = plain(x, 100, 10)
    ckv, kpe = x["ckv"].view(-1, 512), x["kpe"].view(-1, 64)
    key = lambda b, t: int(x["ki"][x["kp"][b] + t])  # noqa: E731
    for t in range(10, 400 - q[0] + 1 - 100):  # request 0: all that no token sees
        ckv[key(0, t)] = float("nan")
        kpe[key(0, t)] = float("inf")
    page = key(0, 399) // 64
    ckv[page * 64 + 400 % 64:(page + 1) * 64] = float("nan")
    ckv[key(1, 299), 100] = float("nan")  # request 1: its last token sees it
    kpe[key(2, 3), 7] = float("-inf")     # request 2: a sink, which all tokens see
    out, lse = (t.float().cpu() for t in call(lib, "window", on_gpu(x), prefill, (100, 10), num_workers=workers))
    bad = torch.zeros(sum(q), dtype=torch.bool)
    bad[q[0] + q[1] - 1:] = True
    assert torch.isnan(lse[bad]).all() and torch.isnan(out[bad]).all()
    good = ~bad.numpy()
    close((out[~bad], lse[~bad]), tuple(t[good] for t in clean))


@pytest.mark.parametrize("heads", [16, 128])
@pytest.mark.parametrize("prefill", [False, True])
def test_shared_keys_that_are_not_finite(lib, heads, prefill):
    """A key of one request's own spoils that request's rows (of them, the tokens that see it), a
    key of a prefix the rows of its group."""
    require_gpu()
    n = [5, 3, 2, 4] if prefill else [1] * 4
    x = make_shared([(200, [(n[0], 60), (n[1], 130), (n[2], 9)]), (70, [(n[3], 64)])], heads, 64, 31)
    clean = plain(x)
    ckv, kpe = x["ckv"].view(-1, 512), x["kpe"].view(-1, 64)
    ckv[int(x["ki"][60 + 129]), 3] = float("nan")  # request 1's last key
    kpe[int(x["pi"][200 + 69]), 3] = float("inf")  # the second group's prefix
    out, lse = (t.float().cpu() for t in call(lib, "shared", on_gpu(x), prefill, ()))
    bad = torch.zeros(sum(n), dtype=torch.bool)
    bad[n[0] + n[1] - 1] = True
    bad[n[0] + n[1] + n[2]:] = True
    assert torch.isnan(lse[bad]).all() and torch.isnan(out[bad]).all()
    good = ~bad.numpy()
    close((out[~bad], lse[~bad]), tuple(t[good] for t in clean))


@pytest.mark.parametrize("heads", [16, 128])
def test_fp8_keys_that_are_not_finite(lib, heads):
    """One token per request over an FP8 cache: NaN codes, infinite and NaN scales and rope values spoil
    the rows that see them alone, whether in the latent's first or last columns or in the rope part."""
    require_gpu()
    inf = torch.tensor([float("inf")]).view(torch.uint8)

    def spoil(tokens, slots):
        tokens[slots[0], 3] = 0x7F
        tokens[slots[1], 500] = 0xFF
        tokens[slots[2], 512 + 12:512 + 16] = inf
        tokens[slots[3], 512:516] = torch.tensor([float("nan")]).view(torch.uint8)
        tokens[slots[4], 528 + 20:528 + 22] = torch.tensor([float("-inf")], dtype=torch.bfloat16).view(torch.uint8)

    lens = [400, 300, 64, 100, 90, 200, 150]
    x = make_window([1] * 7, lens, heads, 16, 33, True)
    ref = plain(x, 60, 10)
    key = lambda b, t: int(x["ki"][x["kp"][b] + t])  # noqa: E731
    tokens = x["kv"].view(-1, 656)
    spoil(tokens, [key(0, t) for t in (10, 100, 200, 300, 339)])            # in front of the window, no sinks
    spoil(tokens, [key(1, 299), key(2, 3), key(3, 60), key(4, 30), key(5, 9)])  # the last, a sink, in the window
    out, lse = (t.float().cpu() for t in call(lib, "window", on_gpu(x), False, (60, 10)))
    bad = torch.tensor([False, True, True, True, True, True, False])
    assert torch.isnan(lse[bad]).all() and torch.isnan(out[bad]).all()
    close((out[~bad], lse[~bad]), tuple(t[~bad.numpy()] for t in ref))
    x = make_shared([(200, [(1, n) for n in (60, 130, 9, 70, 64, 100)]), (70, [(1, 64), (1, 3)])], heads, 16, 34, True)
    ref = plain(x)
    tokens, first = x["kv"].view(-1, 656), x["kp"].tolist()
    spoil(tokens, [int(x["ki"][first[b] + t]) for b, t in ((0, 59), (1, 0), (2, 8), (3, 64), (6, 63))])
    out, lse = (t.float().cpu() for t in call(lib, "shared", on_gpu(x), False, ()))
    bad = torch.tensor([True, True, True, True, False, False, True, False])
    assert torch.isnan(lse[bad]).all() and torch.isnan(out[bad]).all()
    close((out[~bad], lse[~bad]), tuple(t[~bad.numpy()] for t in ref))


@pytest.mark.parametrize("fp8", [False, True])
def test_rows_behind_the_last_request_and_capacities(lib, fp8):
    """A padded step: more query rows and indices than the offsets use, groups that are empty."""
    require_gpu()
    for kind, x, args in both(24, 16, fp8, 8):
        ref = plain(x, *args)
        n = x["qn"].shape[0]
        x["qn"] = torch.cat([x["qn"], torch.full((5, 24, 512), float("nan"), dtype=torch.bfloat16)])
        x["qp"] = torch.cat([x["qp"], torch.full((5, 24, 64), float("nan"), dtype=torch.bfloat16)])
        x["ki"] = torch.cat([x["ki"], torch.full((700,), 2 ** 31 - 1, dtype=torch.int32)])
        if kind == "shared":
            x["pi"] = torch.cat([x["pi"], torch.full((700,), 2 ** 31 - 1, dtype=torch.int32)])
            x["gp"], x["pp"] = (torch.cat([t, t[-1:], t[-1:]]) for t in (x["gp"], x["pp"]))
        out = torch.full((n + 5, 24, 512), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((n + 5, 24), 7.0, device="cuda")
        got = call(lib, kind, on_gpu(x), True, args, out=out, lse=lse)
        close((got[0][:n], got[1][:n]), ref)
        assert (out[n:] == 7).all() and (lse[n:] == 7).all()


def test_requests_in_no_group_stay_as_they_were(lib):
    require_gpu()
    x = make_shared([(50, [(2, 9), (1, 3)]), (64, [(3, 30)]), (0, [(2, 5)])], 16, 16, 9)
    ref = plain(x)
    x["gp"], x["pp"] = x["gp"][1:3].clone(), x["pp"][1:3].clone()  # the second group alone
    out = torch.full((8, 16, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((8, 16), 7.0, device="cuda")
    got = call(lib, "shared", on_gpu(x), True, (), out=out, lse=lse)
    close((got[0][3:6], got[1][3:6]), tuple(t[3:6] for t in ref))
    for t in (out, lse):
        assert (t[:3] == 7).all() and (t[6:] == 7).all()
    x["gp"] = x["pp"] = torch.zeros(1, dtype=torch.int32)  # no group at all
    got = call(lib, "shared", on_gpu(x), True, (), out=out.fill_(7), lse=lse.fill_(7))
    assert (got[0] == 7).all() and (got[1] == 7).all()


@pytest.mark.parametrize("prefill", [False, True])
def test_captured_and_replayed_with_other_lengths(lib, prefill):
    """One graph, replayed with other offsets, indices and queries; graphs of both kinds share a workspace."""
    require_gpu()
    q = ((1, 90), (1, 200), (1, 130)), ((1, 300), (1, 20), (1, 5))
    if prefill:
        q = ((3, 90), (7, 200), (1, 130)), ((5, 300), (1, 20), (5, 5))
    ws = torch.zeros(1 << 27, dtype=torch.uint8, device="cuda")
    graphs = []
    for a, b in zip(both(16, 64, False, 10, q[0]), both(16, 64, False, 11, q[1])):
        kind, args = a[0], a[2]
        buf = {}
        for k, v in a[1].items():
            if isinstance(v, torch.Tensor):
                big = a[1][k] if a[1][k].shape[0] >= b[1][k].shape[0] else b[1][k]
                buf[k] = torch.zeros_like(big).cuda()

        def fill(x, buf=buf):
            for k in buf:
                buf[k][:x[k].shape[0]].copy_(x[k])

        fill(a[1])
        call(lib, kind, buf, prefill, args, workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = call(lib, kind, buf, prefill, args, workspace=ws)
        graphs.append((g, out, fill, a[1], b[1], args))
    for turn in (3, 4, 3):
        for entry in graphs:
            g, out, fill, args = entry[0], entry[1], entry[2], entry[5]
            x = entry[turn]
            fill(x)
            g.replay()
            torch.cuda.synchronize()
            n = x["qn"].shape[0]
            close((out[0][:n], out[1][:n]), plain(x, *args))


@pytest.mark.parametrize("prefill", [False, True])
def test_repeats_exactly(lib, prefill):
    require_gpu()
    q = ((60, 2000), (3, 1000), (1, 5)) if prefill else ((1, 2000), (1, 1000), (1, 5))
    for kind, x, args in both(16, 64, False, 12, q):
        c = on_gpu(x)
        a, b = call(lib, kind, c, prefill, args), call(lib, kind, c, prefill, args)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_on_another_stream(lib):
    """Inputs made late on the call's stream; outputs and workspace belong to it."""
    require_gpu()
    s = torch.cuda.Stream()
    for kind, x, args in both(16, 64, False, 14):
        ref = plain(x, *args)
        c = on_gpu(x)
        torch.cuda.synchronize()
        late = {k: torch.zeros_like(v) if isinstance(v, torch.Tensor) else v for k, v in c.items()}
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            torch.cuda._sleep(20_000_000)
            for k, v in c.items():
                if isinstance(v, torch.Tensor):
                    late[k].copy_(v)
        got = call(lib, kind, late, True, args, stream=s)
        s.synchronize()
        close(got, ref)


def test_large_scores_keep_their_order(lib):
    """Scores of several hundred, so almost all weight is on one key; sinks and prefix first."""
    require_gpu()
    x = make_window([6, 40], [300, 40], 16, 64, 5, q_scale=30.0)
    close(call(lib, "window", on_gpu(x), True, (90, 20)), plain(x, 90, 20))
    x = make_shared([(300, [(1, 40), (6, 200)])], 16, 64, 5, q_scale=30.0)
    close(call(lib, "shared", on_gpu(x), True, ()), plain(x))


def test_validation(lib):
    """MLA_VALIDATE records bad lists and groups; good ones leave the status alone."""
    require_gpu()
    ws = torch.zeros(1 << 27, dtype=torch.uint8, device="cuda")
    for kind, x, args in both(16, 64, False, 15):
        call(lib, kind, on_gpu(x), True, args, workspace=ws, flags=1)
        assert lib.read_device_status(ws) == 0
        bad = [("ki", 5, -1), ("kp", 1, 300)]
        if kind == "shared":
            bad += [("pi", 150, 1 << 30), ("gp", 1, 9), ("gp", 2, 2), ("pp", 2, 150)]
        for name, at, v in bad:
            y = {**x, name: x[name].clone()}
            y[name][at] = v
            call(lib, kind, on_gpu(y), True, args, workspace=ws, flags=1)
            assert lib.read_device_status(ws) == -6, (kind, name)


@pytest.mark.parametrize("seed", range(6))
def test_corrupt_offsets_stay_inside_the_buffers(lib, seed):
    """Offsets of any values: the call ends, the status is clean, buffers around the outputs are whole."""
    require_gpu()
    rng = np.random.default_rng(seed)
    for kind, x, args in both(16, 64, False, 16):
        for name in ("qo", "kp") + (("gp", "pp") if kind == "shared" else ()):
            v = rng.choice([-5, 0, 1, 2, 3, 50, 400, 2 ** 31 - 1, -2 ** 31], x[name].numel())
            x[name] = torch.tensor(v, dtype=torch.int64).to(torch.int32)
        out = torch.full((33, 16, 512), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((33, 16), 7.0, device="cuda")
        dims = lib.make_dims(3, 16, x["ckv"].shape[0], 64, x["ki"].numel(), total_q=11)
        need = (lib.workspace_bytes_window(dims, *args, is_prefill=True) if kind == "window" else
                lib.workspace_bytes_shared(dims, 2, x["pi"].numel(), is_prefill=True))
        ws = torch.zeros(need + 4096, dtype=torch.uint8, device="cuda")
        ws[need:] = 0x5A
        call(lib, kind, on_gpu(x), True, args, out=out[11:22], lse=lse[11:22], workspace=ws[:need])
        torch.cuda.synchronize()
        assert (out[:11] == 7).all() and (out[22:] == 7).all() and (lse[:11] == 7).all() and (lse[22:] == 7).all()
        assert (ws[need:] == 0x5A).all()
        assert lib.read_device_status(ws) == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("prefill", [False, True])
@pytest.mark.parametrize("page", [16, 64])
def test_a_workspace_that_other_calls_have_filled(lib, fp8, prefill, page):
    """Whatever lies behind the status word (here NaN in every type) is written before it is read."""
    require_gpu()
    q = ((3, 90), (7, 200), (1, 130), (2, 0)) if prefill else ((1, 90), (1, 200), (1, 130), (1, 0))
    for kind, x, args in both(24, page, fp8, 21, q):
        ws = torch.full((1 << 28,), 0xFF, dtype=torch.uint8, device="cuda")
        ws[:256] = 0
        close(call(lib, kind, on_gpu(x), prefill, args, workspace=ws), plain(x, *args))
        assert lib.read_device_status(ws) == 0


@pytest.mark.parametrize("heads", [16, 128])
@pytest.mark.parametrize("prefill", [False, True])
def test_own_pages_that_are_not_finite(lib, heads, prefill):
    """A NaN key in a whole page of one request's own keys: the group's other requests, whose rows may
    share a block with that request's, stay as they are."""
    require_gpu()
    n = [2, 1, 3] if prefill else [1] * 3
    for members in ([(n[0], 128), (n[1], 200), (n[2], 70)], [(n[0], 200)]):
        x = make_shared([(64, members)], heads, 64, 35)
        clean = plain(x)
        at = int(x["kp"][int(len(members) > 1)]) + 70  # the second page of the second request, or of the only one
        x["ckv"].view(-1, 512)[int(x["ki"][at]), 9] = float("nan")
        out, lse = (t.float().cpu() for t in call(lib, "shared", on_gpu(x), prefill, ()))
        bad = torch.ones(len(out), dtype=torch.bool)
        if len(members) > 1:
            bad[:n[0]] = False
            bad[n[0] + n[1]:] = False
        assert torch.isnan(lse[bad]).all() and torch.isnan(out[bad]).all()
        good = ~bad.numpy()
        close((out[~bad], lse[~bad]), tuple(t[good] for t in clean))


@pytest.mark.parametrize("kind", ["window", "shared", "causal"])
def test_outputs_on_a_16_byte_boundary(lib, kind):
    """Rows of the output are written 32 bytes at a time where its address allows it, else 16."""
    require_gpu()
    x, args = make_window([3, 40], [150, 40], 16, 16, 41), (2 ** 31 - 1, 0)
    if kind == "shared":
        x, args = make_shared([(30, [(3, 50), (40, 70)])], 16, 16, 41), ()
    c, ref = on_gpu(x), plain(x)
    for skip in (8, 16):
        flat = torch.full((43 * 16 * 512 + 32,), 7.0, dtype=torch.bfloat16, device="cuda")
        out = flat[skip:skip + 43 * 16 * 512].view(43, 16, 512)
        assert out.data_ptr() % 32 == 2 * skip % 32
        if kind == "causal":
            got = lib.mla_paged_prefill_staged(c["qn"], c["qp"], c["ckv"], c["kpe"], c["qo"], c["kp"], c["ki"], SCALE,
                                               out=out)
        else:
            got = call(lib, kind, c, True, args, out=out)
        close(got, ref)
        assert (flat[:skip] == 7).all() and (flat[skip + 43 * 16 * 512:] == 7).all()


@pytest.mark.parametrize("kind", ["window", "shared"])
@pytest.mark.parametrize("page", [16, 64])
def test_bounded_waits(lib, kind, page):
    """A load that never happens: the call returns, the status says timeout, the next call is right."""
    require_gpu()
    if kind == "window":
        x, args = make_window([1] * 3, [2000, 700, 5], 16, page, 36), (1000, 100)
    else:
        x, args = make_shared([(700, [(1, 2000), (1, 5)])], 16, page, 36), ()
    ws = torch.zeros(1 << 28, dtype=torch.uint8, device="cuda")
    c = on_gpu(x)
    try:
        lib.lib().mla_debug_inject_timeout(1, 20_000_000)
        call(lib, kind, c, False, args, workspace=ws, num_workers=1)
        assert lib.read_device_status(ws) == -7
    finally:
        lib.lib().mla_debug_inject_timeout(-1, 0)
    close(call(lib, kind, c, False, args, workspace=ws, num_workers=1), plain(x, *args))
    assert lib.read_device_status(ws) == 0


def test_two_calls_at_once(lib):
    """On two streams, with a workspace each."""
    require_gpu()
    made = [entry for seed in (51, 52) for entry in both(16, 64, False, seed, ((40, 2000), (3, 1000), (1, 5)))]
    inputs = [on_gpu(x) for _, x, _ in made]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in made]
    got = [[call(lib, kind, c, True, args, stream=s) for _ in range(3)][-1]
           for s, (kind, _, args), c in zip(streams, made, inputs)]
    torch.cuda.synchronize()
    for g, (kind, x, args) in zip(got, made):
        close(g, plain(x, *args))


def test_far_slots(lib):
    """Slots past 2^31 bytes of the caches, staged and read where they lie."""
    require_gpu()
    pages, page = 36000, 64
    g = torch.Generator(device="cuda").manual_seed(5)
    ckv = torch.zeros(pages, page, 512, dtype=torch.bfloat16, device="cuda")
    kpe = torch.zeros(pages, page, 64, dtype=torch.bfloat16, device="cuda")
    far = pages - 8
    ckv[far:].normal_(generator=g)
    kpe[far:].normal_(generator=g)
    slots = torch.arange(far * page, pages * page, dtype=torch.int32)
    x = dict(qn=torch.randn(2, 16, 512, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16),
             qp=torch.randn(2, 16, 64, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16), qo=offsets([1, 1]))
    y = dict(x, ki=slots[:431], kp=offsets([300, 131]))
    z = dict(x, pi=slots[:200], pp=offsets([200]), gp=offsets([2]), ki=slots[200:431], kp=offsets([100, 131]))
    for kind, v, args in (("window", y, (200, 3)), ("shared", z, ())):
        got = call(lib, kind, {**on_gpu(v), "ckv": ckv, "kpe": kpe}, False, args)
        near = {**v, "ckv": ckv[far:].cpu(), "kpe": kpe[far:].cpu()}
        for name in ("ki", "pi"):
            if name in near:
                near[name] = near[name] - far * page
        close(got, plain(near, *args))


@pytest.mark.parametrize("kind", ["window", "shared"])
@pytest.mark.parametrize("page", [16, 64])
def test_a_million_keys(lib, kind, page):
    """Staged rows past 1 GB (page 16), a block split over every worker, halves read in place (page 64)."""
    require_gpu()
    n, own = 1_100_000, (77, 1)
    pages = -(-(n + sum(own)) // page) + 2
    g = torch.Generator(device="cuda").manual_seed(page)
    ckv = torch.randn(pages, page, 512, generator=g, device="cuda", dtype=torch.bfloat16)
    kpe = torch.randn(pages, page, 64, generator=g, device="cuda", dtype=torch.bfloat16)
    at = torch.randperm(pages, generator=g, device="cuda")
    slots = (at[:, None] * page + torch.arange(page, device="cuda")).view(-1).int()
    qn = torch.randn(2, 5, 512, generator=g, device="cuda", dtype=torch.bfloat16)
    qp = torch.randn(2, 5, 64, generator=g, device="cuda", dtype=torch.bfloat16)
    x = dict(qn=qn, qp=qp, ckv=ckv, kpe=kpe)
    a, b = slots[:n], slots[n:n + sum(own)]
    if kind == "shared":
        x.update(pi=a.contiguous(), pp=offsets([n]).cuda(), gp=offsets([2]).cuda(), ki=b.contiguous(), kp=offsets(own).cuda())
        lists, args = [torch.cat([a, b[:77]]), torch.cat([a, b[77:]])], ()
    else:  # the first request sees a window of 1,000,000 and 5 sinks, the second all of its keys
        x.update(ki=slots[:n + sum(own)].contiguous(), kp=offsets([n, sum(own)]).cuda())
        lists, args = [torch.cat([a[:5], a[n - 1_000_000:]]), b], (1_000_000, 5)
    ref = []
    for r, keys in enumerate(lists):
        s, w, parts = [], qn[r].double(), keys.long().split(200_000)
        k = [ckv.view(-1, 512)[i].double() for i in parts]
        e = [kpe.view(-1, 64)[i].double() for i in parts]
        s = torch.cat([w @ y.T + qp[r].double() @ z.T for y, z in zip(k, e)], 1) * SCALE
        size = torch.stack([(w.abs() @ y.abs().T + qp[r].double().abs() @ z.abs().T).amax(-1) for y, z in zip(k, e)]).amax(0)
        lse = torch.logsumexp(s, -1)
        p = torch.exp(s - lse[:, None]).split(200_000, 1)
        ref.append((sum(u @ y for u, y in zip(p, k)), lse, sum(u @ y.abs() for u, y in zip(p, k)), 2.0 ** -14 * SCALE * size))
    close(call(lib, kind, x, False, args), tuple(torch.stack(t).cpu().numpy() for t in zip(*ref)))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("prefill", [False, True])
@pytest.mark.parametrize("page", [16, 64])
def test_lists_without_entries(lib, fp8, prefill, page):
    """No prefix index, no own index, neither: null pointers on the C side."""
    require_gpu()
    n = 3 if prefill else 1
    close(call(lib, "window", on_gpu(make_window([n, n], [0, 0], 16, page, 1, fp8)), prefill, (5, 2)),
          plain(make_window([n, n], [0, 0], 16, page, 1, fp8), 5, 2))
    for groups in ([(0, [(n, 4), (n, 70)]), (0, [(n, 1)])], [(70, [(n, 0), (n, 0)])], [(0, [(n, 0), (n, 0)])]):
        x = make_shared(groups, 16, page, 2, fp8)
        assert not x["pi"].numel() or not x["ki"].numel()
        close(call(lib, "shared", on_gpu(x), prefill, ()), plain(x))


@pytest.mark.parametrize("kind", ["window", "shared"])
def test_a_negative_scale(lib, kind):
    require_gpu()
    for x, args in ((make_window([1, 1], [300, 20], 16, 64, 71), (128, 3)),
                    (make_shared([(200, [(1, 300), (1, 20)])], 16, 64, 71), ())):
        if ("gp" in x) != (kind == "shared"):
            continue
        c = on_gpu(x)
        got = getattr(lib, f"mla_paged_decode_{kind}")(
            c["qn"], c["qp"], c["ckv"], c["kpe"],
            *((c["kp"], c["ki"], *args) if kind == "window" else (c["gp"], c["pp"], c["pi"], c["kp"], c["ki"])), -SCALE)
        close(got, plain({**x, "qn": -x["qn"], "qp": -x["qp"]}, *args))
