"""The operators around the paged latent cache, as measured cases.

Four families, as a serving step uses them together:

  append  rotary positions (one to three axes) applied to q_pe and k_pe, and the new tokens
          written into the paged cache (bf16, or quantised to the 656-byte FP8 token)
  gather  cached tokens read back by slot as contiguous bf16 rows
  chunk   causal attention of a chunk of new tokens over an FP8 paged cache
  pool    the cache's pages: freeing, forking (shared full pages, a copied partial page) and
          extending sequences; compacting the live pages to the front

``own`` chooses between the plain form (elementary torch operations in 32 bits or more) and
the calls of this repository's package.
"""

import math
import random

import torch

own = False

CKV, KPE, PAIRS, TOKEN = 512, 64, 32, 656
SM_SCALE = 192 ** -0.5
DEV = "cuda"


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # One decode step of a batch of 64: a token per sequence, latency counts.
        {"name": "append_decode", "kind": "append", "tokens": 64, "heads": 128, "page": 64, "axes": 1,
         "interleaved": True, "fp8": False, "start": 4096},
        # A prefill step with image patches: three position axes, half-split pairs.
        {"name": "append_image_prefill", "kind": "append", "tokens": 8192, "heads": 128, "page": 64, "axes": 3,
         "interleaved": False, "fp8": False, "start": 20000},
        # A ragged mixed step of a head-sharded model into an FP8 cache, read back as bf16 rows.
        {"name": "append_fp8_ragged", "kind": "append", "tokens": 777, "heads": 16, "page": 16, "axes": 1,
         "interleaved": True, "fp8": True, "start": 900000},
        # Short contexts at page size 1 read back for the up-projection of their keys.
        {"name": "gather_small", "kind": "gather", "batch": 4, "kv_lo": 1, "kv_hi": 300, "page": 1, "fp8": False},
        # The benchmark batch's whole context, dequantised.
        {"name": "gather_fp8_context", "kind": "gather", "batch": 64, "kv_lo": 1024, "kv_hi": 8192, "page": 64,
         "fp8": True},
        # Verification of a few drafted tokens per sequence, head-sharded model.
        {"name": "chunk_verify", "kind": "chunk", "batch": 32, "heads": 16, "q_lo": 1, "q_hi": 8, "kv_lo": 64,
         "kv_hi": 1024, "page": 64},
        # One chunk of a long prompt of a head-sharded model.
        {"name": "chunk_h16", "kind": "chunk", "batch": 2, "heads": 16, "q_lo": 512, "q_hi": 512, "kv_lo": 4096,
         "kv_hi": 8192, "page": 16},
        # Chunks of four prompts, all 128 heads.
        {"name": "chunk_h128", "kind": "chunk", "batch": 4, "heads": 128, "q_lo": 256, "q_hi": 1024, "kv_lo": 1024,
         "kv_hi": 4096, "page": 64},
        # Bookkeeping of a decode step: a few sequences end, a few fork, every other one grows by a token.
        {"name": "pool_decode", "kind": "pool", "rows": 96, "ended": 8, "forks": 4, "fork_each": 2, "new_lo": 1,
         "new_hi": 1, "kv_lo": 16, "kv_hi": 2048, "page": 64, "pages": 4096, "fp8": False},
        # A beam step with many forks and prompts that grow by whole chunks, FP8 cache.
        {"name": "pool_beam_fp8", "kind": "pool", "rows": 512, "ended": 64, "forks": 128, "fork_each": 3,
         "new_lo": 0, "new_hi": 700, "kv_lo": 100, "kv_hi": 8000, "page": 64, "pages": 65536, "fp8": True},
        # A pool with holes everywhere, brought to the front.
        {"name": "compact_large", "kind": "compact", "rows": 200, "kv_lo": 1000, "kv_hi": 5000, "page": 64,
         "pages": 20000, "fp8": False},
        {"name": "compact_fp8_small_pages", "kind": "compact", "rows": 33, "kv_lo": 1, "kv_hi": 700, "page": 16,
         "pages": 1501, "fp8": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["append", "append", "gather", "chunk", "chunk", "pool", "compact"])
    page = rng.choice([1, 7, 16, 32, 64, 128])
    if kind == "append":
        heads = rng.choice([1, 7, 16, 33, 64, 100, 128])
        return {"kind": kind, "tokens": _log(rng, 1, 8000), "heads": heads, "page": page, "axes": rng.choice([1, 2, 3]),
                "interleaved": rng.random() < 0.5, "fp8": rng.random() < 0.5, "start": _log(rng, 1, 1000000)}
    if kind == "gather":
        hi = _log(rng, 8, 8000)
        return {"kind": kind, "batch": _log(rng, 1, 60), "kv_lo": rng.randint(0, hi // 2), "kv_hi": hi, "page": page,
                "fp8": rng.random() < 0.5}
    if kind == "chunk":
        heads = rng.choice([1, 5, 16, 24, 64, 128])
        batch = _log(rng, 1, 32)
        q_hi = _log(rng, 1, max(1, min(1000, 4096 // batch)))
        kv_hi = q_hi + _log(rng, 1, 3000)
        return {"kind": kind, "batch": batch, "heads": heads, "q_lo": rng.randint(1, q_hi), "q_hi": q_hi,
                "kv_lo": q_hi, "kv_hi": kv_hi, "page": page}
    page = rng.choice([16, 32, 64, 128])
    hi = _log(rng, 40, 4000)
    rows = _log(rng, 8, 300)
    pages = rows * (hi // page + 2) * 2 + rng.randint(0, 500)
    if kind == "pool":
        forks = rng.randint(1, rows // 4)
        return {"kind": kind, "rows": rows, "ended": rng.randint(1, rows // 4), "forks": forks,
                "fork_each": rng.randint(1, 3), "new_lo": 0, "new_hi": rng.choice([1, 4, 600]), "kv_lo": 1,
                "kv_hi": hi, "page": page, "pages": min(pages, 30000), "fp8": rng.random() < 0.5}
    return {"kind": kind, "rows": min(rows, 150), "kv_lo": 1, "kv_hi": hi, "page": page,
            "pages": min(pages, 1280000 // page), "fp8": rng.random() < 0.5}


def _rng_of(case):
    """Lengths are part of the case: the same for every seed."""
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _lens(case, n):
    r = _rng_of(case)
    return [r.randint(case["kv_lo"], case["kv_hi"]) for _ in range(n)]


def _chunk_lens(case):
    r = _rng_of(case)
    q = [r.randint(case["q_lo"], case["q_hi"]) for _ in range(case["batch"])]
    kv = [max(n, r.randint(case["kv_lo"], case["kv_hi"])) for n in q]
    return q, kv


def _ceil(a, b):
    return -(-a // b)


def _pool_plan(case):
    """What a step of the pool does, as host numbers: the live rows' lengths and pages (sequences
    beyond the pool's size are left out), the rows that end, fork and grow."""
    r = _rng_of(case)
    ps, rows = case["page"], case["rows"]
    lens, used = [], 0
    room = int(case["pages"] * 0.6)
    for _ in range(rows):
        n = r.randint(case["kv_lo"], case["kv_hi"])
        need = _ceil(n, ps)
        if used + need > room:
            n = need = 0
        lens.append(n)
        used += need
    if case["kind"] != "pool":
        return lens, [], [], [], [], []
    order = list(range(rows))
    r.shuffle(order)
    ended = order[: case["ended"]]
    parents, children, child = [], [], rows
    for p in order[case["ended"]: case["ended"] + case["forks"]]:
        for _ in range(case["fork_each"]):
            parents.append(p)
            children.append(child)
            child += 1
    grow = order[case["ended"]:]
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in grow]
    return lens, ended, parents, children, grow, new


def _token_bytes(case):
    return TOKEN if case["fp8"] else 2 * (CKV + KPE)


def work(case):
    k = case["kind"]
    if k == "append":
        t, h = case["tokens"], case["heads"]
        rows = t * (2 * 2 * h * KPE + 2 * (CKV + KPE) + _token_bytes(case) + 4 * (case["axes"] + 1))
        if case["fp8"]:
            rows += t * (TOKEN + 2 * (CKV + KPE))
        return {"bytes": rows, "flops": t * (6 * PAIRS * (h + 1) + (4 * CKV if case["fp8"] else 0))}
    if k == "gather":
        n = sum(_lens(case, case["batch"]))
        return {"bytes": max(1, n * (_token_bytes(case) + 2 * (CKV + KPE) + 4)), "flops": n * CKV if case["fp8"] else 0}
    if k == "chunk":
        q, kv = _chunk_lens(case)
        h = case["heads"]
        pairs = sum(n * (m - n) + n * (n + 1) // 2 for n, m in zip(q, kv))
        return {"bytes": sum(kv) * (TOKEN + 4) + sum(q) * h * (2 * (CKV + KPE) + 2 * CKV + 4),
                "flops": 2 * (2 * CKV + KPE) * h * pairs}
    lens, ended, parents, children, grow, new = _pool_plan(case)
    ps = case["page"]
    if k == "pool":
        touched = sum(_ceil(lens[r], ps) for r in ended) + 2 * sum(_ceil(lens[p], ps) for p in parents)
        copied = sum(lens[p] % ps for p in parents)
        return {"bytes": 4 * case["pages"] + 8 * touched + 2 * copied * _token_bytes(case) + 4 * sum(new),
                "flops": 0}
    live = sum(_ceil(n, ps) for n in lens)
    moved = live * (1 - live / case["pages"])  # pages are spread evenly: this share lies behind the first `live`
    return {"bytes": int(4 * case["pages"] + 8 * live + 2 * moved * ps * _token_bytes(case)), "flops": 0}


# ---------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(shape, g):
    return torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _quantised(ckv, kpe):
    """FP8 tokens of bf16 latents [..., 512] and rope parts [..., 64]: a scale of amax / 448 for each 128."""
    tiles = ckv.float().unflatten(-1, (4, 128))
    amax = tiles.abs().amax(-1)
    # (a division by a Python number would multiply by its reciprocal, a rounding off the quotient)
    scale = torch.where(amax > 0, amax / torch.full_like(amax, 448.0), torch.ones_like(amax))
    codes = (tiles / scale[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return torch.cat([codes.flatten(-2).view(torch.uint8), scale.view(torch.uint8), kpe.contiguous().view(torch.uint8)], -1)


def _cache(case, pages, g):
    ckv, kpe = _randn((pages, case["page"], CKV), g), _randn((pages, case["page"], KPE), g)
    if case.get("fp8", True):
        return {"kv_fp8": _quantised(ckv, kpe)}
    return {"ckv_cache": ckv, "kpe_cache": kpe}


def _paged_slots(lens, ps, pages, g):
    """Token slots of sequences on randomly permuted pages, packed, and their offsets."""
    perm = torch.randperm(pages, generator=g, device=DEV)
    parts, at, ptr = [], 0, [0]
    for n in lens:
        need = _ceil(n, ps)
        own_pages = perm[at: at + need]
        at += need
        parts.append((own_pages[:, None] * ps + torch.arange(ps, device=DEV)).flatten()[:n])
        ptr.append(ptr[-1] + n)
    slots = torch.cat(parts) if parts else perm[:0]
    return slots.to(torch.int32), _ints(ptr)


def _prepare_append(case, seed):
    g = _gen(seed)
    t, h, ps = case["tokens"], case["heads"], case["page"]
    pages = _ceil(t, ps) + 3
    s = _cache(case, pages, g)
    # q_pe and k_pe are slices of the projections' outputs, as a model has them.
    s["q"] = _randn((t, h, 192), g)
    s["kv"] = _randn((t, CKV + KPE), g)
    s["slots"] = _paged_slots([t], ps, pages, g)[0]
    if t > 100:
        s["slots"][-3:] = -1  # rows of padding behind the last sequence
    s["inv_freq"] = (10000.0 ** (-torch.arange(PAIRS, device=DEV, dtype=torch.float64) / PAIRS)).float()
    if case["axes"] == 1:
        s["positions"] = (torch.arange(t, device=DEV) + case["start"]).to(torch.int32)[None].contiguous()
    else:
        grid = torch.arange(t, device=DEV)
        axes = [torch.full_like(grid, case["start"]), case["start"] + grid // 37, case["start"] + grid % 37]
        s["positions"] = torch.stack(axes[: case["axes"]]).to(torch.int32).contiguous()
    s["sections"] = {1: [32], 2: [12, 20], 3: [8, 12, 12]}[case["axes"]]
    return s


def _prepare_gather(case, seed):
    g = _gen(seed)
    lens = _lens(case, case["batch"])
    pages = sum(_ceil(n, case["page"]) for n in lens) + 2
    s = _cache(case, pages, g)
    s["slots"], s["indptr"] = _paged_slots(lens, case["page"], pages, g)
    return s


def _prepare_chunk(case, seed):
    g = _gen(seed)
    q, kv = _chunk_lens(case)
    pages = sum(_ceil(n, case["page"]) for n in kv) + 2
    s = _cache(case, pages, g)
    s["q_nope"], s["q_pe"] = _randn((sum(q), case["heads"], CKV), g), _randn((sum(q), case["heads"], KPE), g)
    s["slots"], s["kv_indptr"] = _paged_slots(kv, case["page"], pages, g)
    ptr = [0]
    for n in q:
        ptr.append(ptr[-1] + n)
    s["qo_indptr"] = _ints(ptr)
    s["q_max"], s["kv_max"] = max(q), max(kv)
    return s


def _prepare_pool(case, seed):
    g = _gen(seed)
    lens, ended, parents, children, grow, new = _pool_plan(case)
    ps, pages = case["page"], case["pages"]
    rows = case["rows"] + len(children) + 1
    blocks = max(1, max(_ceil(n, ps) for n in lens) + _ceil(max(new, default=0), ps) + 1)
    # One buffer holds the pool's tables, so that a pass can start from the same state again.
    s = _cache(case, pages, g)
    pool = torch.empty(rows * blocks + rows + pages, dtype=torch.int32, device=DEV)
    s["pool"] = pool
    s["table"] = pool[: rows * blocks].view(rows, blocks)
    s["lens"] = pool[rows * blocks: rows * blocks + rows]
    s["ref"] = pool[rows * blocks + rows:]
    pool.zero_()
    s["table"].fill_(-1)
    s["lens"][: case["rows"]] = _ints(lens)
    perm = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    need = torch.tensor([_ceil(n, ps) for n in lens], device=DEV)
    used = torch.arange(blocks, device=DEV)[None] < need[:, None]
    s["table"][: case["rows"]][used] = perm[: int(need.sum())]
    s["ref"][perm[: int(need.sum())].long()] = 1
    s["before"] = pool.clone()
    s.update(ended=_ints(ended), parents=_ints(parents), children=_ints(children), grow=_ints(grow), new=_ints(new))
    s["capacity"] = sum(new)
    s["page"] = ps
    return s


def prepare(case, seed):
    k = case["kind"]
    s = (_prepare_append if k == "append" else _prepare_gather if k == "gather" else _prepare_chunk if k == "chunk"
         else _prepare_pool)(case, seed)
    s["case"] = case
    return s


# ---------------------------------------------------------------- the plain forms
def _rotate(x, positions, inv_freq, axis_of_pair, interleaved):
    """Rotary positions on x [T, heads, 64]; the angles in 64 bits, as far positions need."""
    angle = positions.double()[axis_of_pair].t() * inv_freq.double()
    c, s = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    y = x.float()
    if interleaved:
        a, b = y[..., 0::2], y[..., 1::2]
        return torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2).to(torch.bfloat16)
    a, b = y[..., :PAIRS], y[..., PAIRS:]
    return torch.cat([a * c - b * s, a * s + b * c], -1).to(torch.bfloat16)


def _axis_of_pair(sections):
    return torch.repeat_interleave(torch.arange(len(sections), device=DEV), torch.tensor(sections, device=DEV))


def _dequantised(tokens):
    codes = tokens[..., :CKV].contiguous().view(torch.float8_e4m3fn).float().unflatten(-1, (4, 128))
    scale = tokens[..., CKV: CKV + 16].contiguous().view(torch.float32)
    return (codes * scale[..., None]).flatten(-2).to(torch.bfloat16), tokens[..., CKV + 16:].contiguous().view(torch.bfloat16)


def _read(s, slots):
    if "kv_fp8" in s:
        ckv, kpe = _dequantised(s["kv_fp8"].view(-1, TOKEN)[slots.clamp(min=0).long()])
    else:
        at = slots.clamp(min=0).long()
        ckv, kpe = s["ckv_cache"].view(-1, CKV)[at], s["kpe_cache"].view(-1, KPE)[at]
    ok = (slots >= 0)[:, None]
    return torch.where(ok, ckv, torch.zeros_like(ckv)), torch.where(ok, kpe, torch.zeros_like(kpe))


def _append(s):
    pair_axis = _axis_of_pair(s["sections"])
    rot = (s["positions"], s["inv_freq"], pair_axis, s["case"]["interleaved"])
    q = _rotate(s["q"][..., 128:], *rot)
    k = _rotate(s["kv"][:, None, CKV:], *rot)[:, 0]
    ckv = s["kv"][:, :CKV]
    keep = torch.nonzero(s["slots"] >= 0)[:, 0]
    at = s["slots"][keep].long()
    if "kv_fp8" in s:
        s["kv_fp8"].view(-1, TOKEN)[at] = _quantised(ckv[keep], k[keep])
        return q, _read(s, s["slots"])
    s["ckv_cache"].view(-1, CKV)[at] = ckv[keep]
    s["kpe_cache"].view(-1, KPE)[at] = k[keep]
    return q, (s["ckv_cache"], s["kpe_cache"])


def _chunk(s):
    ckv, kpe = _read(s, s["slots"])
    h, qm, km = s["q_nope"].shape[1], s["q_max"], s["kv_max"]
    qp, kp = s["qo_indptr"].long(), s["kv_indptr"].long()
    qn, kn = qp.diff(), kp.diff()
    batch = qn.numel()
    # Queries and keys in padded rectangles, one for each sequence.
    qi, ki = torch.arange(qm, device=DEV), torch.arange(km, device=DEV)
    q_at = (qp[:-1, None] + torch.minimum(qi[None], qn[:, None] - 1)).clamp(min=0)
    k_at = (kp[:-1, None] + torch.minimum(ki[None], kn[:, None] - 1)).clamp(min=0)
    q = torch.cat([s["q_nope"], s["q_pe"]], -1).float()[q_at].view(batch, qm * h, CKV + KPE)
    k = torch.cat([ckv, kpe], -1).float()[k_at]
    v = k[..., :CKV]
    score = torch.bmm(q, k.transpose(1, 2)).mul_(SM_SCALE).view(batch, qm, h, km)
    seen = ki[None, None] < (kn - qn)[:, None, None] + qi[None, :, None] + 1
    score.masked_fill_(~seen[:, :, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.bmm(p.view(batch, qm * h, km), v).view(batch, qm, h, CKV) / total
    lse = (top + total.log())[..., 0]
    real = torch.nonzero((qi[None] < qn[:, None]).flatten())[:, 0]
    return out.view(-1, h, CKV)[real].to(torch.bfloat16), lse.view(-1, h)[real]


def _free_rows(s, rows):
    table, lens, ref, ps = s["table"], s["lens"], s["ref"], s["page"]
    rows = rows.long()
    used = torch.arange(table.shape[1], device=DEV)[None] < ((lens[rows] + ps - 1) // ps)[:, None]
    pages = torch.where(used, table[rows], torch.zeros_like(table[rows])).long().flatten()
    ref.index_add_(0, pages, -used.flatten().int())
    table[rows] = -1
    lens[rows] = 0


def _fork_rows(s):
    table, lens, ref, ps = s["table"], s["lens"], s["ref"], s["page"]
    parents, children = s["parents"].long(), s["children"].long()
    n = lens[parents]
    full, tail = n // ps, n % ps
    block = torch.arange(table.shape[1], device=DEV)[None]
    shared = block < full[:, None]
    rows = torch.where(shared, table[parents], torch.full_like(table[parents], -1))
    ref.index_add_(0, rows.clamp(min=0).long().flatten(), shared.flatten().int())
    # A partial page is copied to the lowest free page, in the order of the pairs.
    free = torch.nonzero(ref == 0)[:, 0].int()
    part = tail > 0
    rank = torch.cumsum(part, 0) - part.int()
    new = torch.where(part, free[rank.clamp(max=free.numel() - 1)], -1)
    src = torch.where(part, table[parents].gather(1, full.clamp(max=table.shape[1] - 1)[:, None].long())[:, 0], -1)
    ref[new[part].long()] = 1
    rows = torch.where(part[:, None] & (block == full[:, None]), new[:, None], rows)
    table[children] = rows.to(torch.int32)
    lens[children] = n
    return torch.zeros_like(s["parents"]), src.int(), new.int(), tail.int()


def _copy(s, src, dst, tokens):
    keep = torch.nonzero((src >= 0) & (tokens > 0))[:, 0]
    src, dst = src[keep].long(), dst[keep].long()
    take = (torch.arange(s["page"], device=DEV)[None] < tokens[keep][:, None])[..., None]
    for name in ("kv_fp8",) if "kv_fp8" in s else ("ckv_cache", "kpe_cache"):
        s[name][dst] = torch.where(take, s[name][src], s[name][dst])


def _extend_rows(s):
    table, lens, ref, ps = s["table"], s["lens"], s["ref"], s["page"]
    rows, new = s["grow"].long(), s["new"]
    n = lens[rows]
    have, want = (n + ps - 1) // ps, (n + new + ps - 1) // ps
    need = want - have
    first = torch.cumsum(need, 0) - need
    free = torch.nonzero(ref == 0)[:, 0].int()
    block = torch.arange(table.shape[1], device=DEV)[None]
    added = (block >= have[:, None]) & (block < want[:, None])
    pick = free[(first[:, None] + block - have[:, None]).clamp(0, free.numel() - 1)]
    table[rows] = torch.where(added, pick, table[rows])
    ref[pick[added].long()] = 1
    lens[rows] = n + new
    ptr = torch.cat([torch.zeros_like(new[:1]), torch.cumsum(new, 0).int()])
    owner = torch.repeat_interleave(torch.arange(rows.numel(), device=DEV), new.long())
    at = n[owner] + torch.arange(owner.numel(), device=DEV) - ptr[owner]
    slots = table[rows[owner], at // ps] * ps + at % ps
    return ptr, slots.int(), torch.zeros_like(s["grow"])


def _compact(s):
    table, lens, ref, ps = s["table"], s["lens"], s["ref"], s["page"]
    pages = ref.numel()
    live = ref > 0
    count = live.sum()
    page = torch.arange(pages, device=DEV)
    src = torch.nonzero(live & (page >= count))[:, 0]
    dst = torch.nonzero(~live & (page < count))[:, 0]
    remap = page.clone()
    remap[src] = dst
    used = torch.arange(table.shape[1], device=DEV)[None] < ((lens + ps - 1) // ps)[:, None]
    table.copy_(torch.where(used, remap[table.clamp(min=0).long()].int(), table))
    ref[dst] = ref[src]
    ref[src] = 0
    for name in ("kv_fp8",) if "kv_fp8" in s else ("ckv_cache", "kpe_cache"):
        s[name][dst] = s[name][src]
    lists = torch.full((2, max(1, pages // 2)), -1, dtype=torch.int32, device=DEV)
    lists[0, : src.numel()], lists[1, : src.numel()] = src.int(), dst.int()
    return torch.stack([count.int(), torch.full_like(count, src.numel()).int()]), lists[0], lists[1]


def _cache_out(s):
    """The cache's buffers; pages of an FP8 cache are only copied, and compared as words."""
    return s["kv_fp8"].view(torch.int32) if "kv_fp8" in s else (s["ckv_cache"], s["kpe_cache"])


# ---------------------------------------------------------------- one pass
def run(state):
    k = state["case"]["kind"]
    if own:
        return _run_own(state, k)
    if k == "append":
        return _append(state)
    if k == "gather":
        return _read(state, state["slots"])
    if k == "chunk":
        return _chunk(state)
    state["pool"].copy_(state["before"])
    if k == "compact":
        return _compact(state), state["table"], state["lens"], state["ref"], _cache_out(state)
    _free_rows(state, state["ended"])
    fork = _fork_rows(state)
    _copy(state, *fork[1:])
    return fork, _extend_rows(state), state["table"], state["lens"], state["ref"], _cache_out(state)


def _run_own(s, k):
    import paged_head_latent_gb300 as mla

    fp8 = "kv_fp8" in s
    cache = (s["kv_fp8"],) if fp8 else (s["ckv_cache"], s["kpe_cache"])
    if k == "append":
        call = mla.mla_rope_append_fp8 if fp8 else mla.mla_rope_append
        q = call(s["q"][..., 128:], s["kv"][:, :CKV], s["kv"][:, CKV:], s["positions"], s["inv_freq"], s["slots"],
                 *cache, sections=s["sections"], interleaved=s["case"]["interleaved"])
        return q, mla.mla_cache_gather_fp8(*cache, s["slots"]) if fp8 else cache
    if k == "gather":
        return (mla.mla_cache_gather_fp8 if fp8 else mla.mla_cache_gather)(*cache, s["slots"])
    if k == "chunk":
        if "workspace" not in s:  # kept, as a serving program keeps it
            s["workspace"] = torch.zeros(mla.workspace_bytes_prefill_fp8(mla.make_dims(
                s["qo_indptr"].numel() - 1, s["q_nope"].shape[1], s["kv_fp8"].shape[0], s["kv_fp8"].shape[1],
                s["slots"].numel(), total_q=s["q_nope"].shape[0])), dtype=torch.uint8, device=DEV)
        return mla.mla_paged_prefill_fp8(s["q_nope"], s["q_pe"], s["kv_fp8"], s["qo_indptr"], s["kv_indptr"],
                                         s["slots"], SM_SCALE, workspace=s["workspace"])
    copy = mla.mla_cache_copy_pages_fp8 if fp8 else mla.mla_cache_copy_pages
    if "workspace" not in s:
        s["workspace"] = torch.zeros(mla.workspace_bytes_pages(s["table"].shape[0], s["ref"].numel(), max(
            1, s["grow"].numel(), s["parents"].numel())), dtype=torch.uint8, device=DEV)
    tables, ws = (s["table"], s["lens"], s["ref"]), s["workspace"]
    s["pool"].copy_(s["before"])
    if k == "compact":
        counts, src, dst = mla.mla_pages_compact(*tables, s["page"], workspace=ws)
        copy(*cache, src, dst, count=counts[1:])
        return (counts, src, dst), *tables, _cache_out(s)
    mla.mla_pages_free(*tables, s["ended"], s["page"])
    fork = mla.mla_pages_fork(*tables, s["parents"], s["children"], s["page"], workspace=ws)
    copy(*cache, *fork[1:3], tokens=fork[3])
    extend = mla.mla_pages_extend(*tables, s["grow"], s["new"], s["page"], s["capacity"], workspace=ws)
    return fork, extend, *tables, _cache_out(s)


# ---------------------------------------------------------------- the definitions in 64 bits
def _exact_rotated(x, s):
    """x [T, heads, 64] as complex numbers, times e^(i angle)."""
    pair_axis = [a for a, n in enumerate(s["sections"]) for _ in range(n)]
    angle = torch.stack([s["positions"][a].double() * s["inv_freq"][i].double() for i, a in enumerate(pair_axis)], -1)
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]
    y = x.double()
    if s["case"]["interleaved"]:
        z = torch.view_as_complex(y.unflatten(-1, (PAIRS, 2)).contiguous()) * turn
        return torch.view_as_real(z).flatten(-2)
    z = torch.complex(y[..., :PAIRS].contiguous(), y[..., PAIRS:].contiguous()) * turn
    return torch.cat([z.real, z.imag], -1)


def _exact_e4m3(code):
    """The numbers that E4M3 codes stand for: sign, four exponent bits (bias 7), three mantissa bits."""
    c = code.long()
    e, m = (c >> 3) & 15, (c & 7).double()
    value = torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * torch.pow(2.0, (e - 7).double()))
    return torch.where(c >= 128, -value, value)


def _exact_tokens(tokens):
    """Latents (code times scale) and rope parts of FP8 tokens [n, 656]."""
    scale = tokens[:, CKV: CKV + 16].contiguous().view(torch.float32).double().repeat_interleave(128, 1)
    return _exact_e4m3(tokens[:, :CKV]) * scale, tokens[:, CKV + 16:].contiguous().view(torch.bfloat16).double()


def _exact_quantised(x):
    """x [n, 512] after the FP8 cache: scale amax / 448 and the quotient x / scale as the 32-bit numbers
    that the cache's format defines, then the nearest E4M3 number."""
    tiles = x.double().unflatten(-1, (4, 128))
    amax = tiles.abs().amax(-1, keepdim=True)
    scale = torch.where(amax > 0, amax / 448, 1.0).float().double()
    y = (tiles / scale).float().double().clamp(-448, 448)
    step = torch.pow(2.0, torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(y / step) * step * scale).flatten(-2)


def _exact_append(s):
    q, k = _exact_rotated(s["q"][..., 128:], s), _exact_rotated(s["kv"][:, None, CKV:], s)[:, 0]
    slots = s["slots"].tolist()
    at = [i for i, n in enumerate(slots) if n >= 0]
    if "kv_fp8" in s:
        ckv, kpe = torch.zeros(len(slots), CKV, device=DEV, dtype=torch.float64), torch.zeros_like(k)
        ckv[at], kpe[at] = _exact_quantised(s["kv"][at][:, :CKV]), k[at]
        return q, (ckv, kpe)
    ckv, kpe = s["ckv_cache"].double(), s["kpe_cache"].double()
    where = torch.tensor([slots[i] for i in at], device=DEV)
    ckv.view(-1, CKV)[where], kpe.view(-1, KPE)[where] = s["kv"][at][:, :CKV].double(), k[at]
    return q, (ckv, kpe)


def _exact_chunk(s):
    qp, kp = s["qo_indptr"].tolist(), s["kv_indptr"].tolist()
    outs, lses = [], []
    for b in range(len(qp) - 1):
        rows = s["kv_fp8"].view(-1, TOKEN)[s["slots"][kp[b]: kp[b + 1]].long()]
        latent, rope = _exact_tokens(rows)
        v = latent.float().to(torch.bfloat16).double()  # the cache's value of a token is a bf16 number
        n, m = qp[b + 1] - qp[b], kp[b + 1] - kp[b]
        hidden = torch.arange(m, device=DEV)[None] > torch.arange(m - n, m, device=DEV)[:, None]
        x = torch.einsum("qhd,kd->hqk", s["q_nope"][qp[b]: qp[b + 1]].double(), v)
        x = (x + torch.einsum("qhd,kd->hqk", s["q_pe"][qp[b]: qp[b + 1]].double(), rope)) * SM_SCALE
        x = x.masked_fill(hidden, -math.inf)
        lse = torch.logsumexp(x, -1)
        outs.append(torch.einsum("hqk,kd->qhd", torch.exp(x - lse[..., None]), v))
        lses.append(lse.t())
    return torch.cat(outs), torch.cat(lses)


def _exact_pool(s):
    """The tables as Python lists, one step after the other; what moved in a bf16 cache."""
    table, lens, ref, ps = s["table"].tolist(), s["lens"].tolist(), s["ref"].tolist(), s["page"]
    moves = []
    if s["case"]["kind"] == "compact":
        front = sum(1 for n in ref if n > 0)
        holes = iter([p for p in range(front) if ref[p] == 0])
        moves = [(p, next(holes), ps) for p in range(front, len(ref)) if ref[p] > 0]
    else:
        for r in s["ended"].tolist():
            for page in table[r][: _ceil(lens[r], ps)]:
                ref[page] -= 1
        free = iter([p for p, n in enumerate(ref) if n == 0])
        for parent in s["parents"].tolist():
            if lens[parent] % ps:
                moves.append((table[parent][lens[parent] // ps], next(free), lens[parent] % ps))
    if "kv_fp8" in s:
        return None
    found = []
    for cache in (s["ckv_cache"].double(), s["kpe_cache"].double()):
        for src, dst, n in moves:
            cache[dst, :n] = cache[src, :n]
        found.append(cache)
    return tuple(found)


def exact(case, seed):
    s = prepare(case, seed)
    k = case["kind"]
    if k == "append":
        return _exact_append(s)
    if k == "chunk":
        return _exact_chunk(s)
    if k == "gather":
        at = s["slots"].tolist()
        if "kv_fp8" in s:
            return _exact_tokens(s["kv_fp8"].view(-1, TOKEN)[at])
        return s["ckv_cache"].view(-1, CKV)[at].double(), s["kpe_cache"].view(-1, KPE)[at].double()
    cache = _exact_pool(s)
    if cache is None:
        return None
    return (None, None, None, None, cache) if k == "compact" else (None, None, None, None, None, cache)
