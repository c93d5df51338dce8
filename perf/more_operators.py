"""Attention over parts of the paged latent cache, as measured cases.

Three families, as a serving step uses them:

  window  attention that sees the last ``window`` keys and the first ``sinks`` keys of its
          sequence: one token per sequence, or a causal chunk of new tokens
  shared  attention of sequences that share a long prefix, whose keys are listed once for the
          group: one token per sequence, or a causal chunk of new tokens behind the prefix
  tables  the groups of sequences that share leading pages, found from the page pool's block
          table, with the key lists that the shared attention takes

``own`` chooses between the plain form (elementary torch operations in 32 bits or more) and
the calls of this repository's package.
"""

import math
import random

import torch

own = False

CKV, KPE, TOKEN = 512, 64, 656
SM_SCALE = 192 ** -0.5
DEV = "cuda"


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # A few short chats of a head-sharded model with a short window: latency counts.
        {"name": "window_decode_small", "kind": "window", "prefill": False, "batch": 4, "heads": 16, "kv_lo": 1,
         "kv_hi": 2000, "window": 512, "sinks": 4, "page": 64, "fp8": False},
        # A full batch with all 128 heads deep in long contexts: every sequence reads its whole window.
        {"name": "window_decode_h128", "kind": "window", "prefill": False, "batch": 64, "heads": 128, "kv_lo": 4096,
         "kv_hi": 16384, "window": 4096, "sinks": 64, "page": 64, "fp8": False},
        # A large head-sharded batch over an FP8 cache with small pages, some sequences shorter than the window.
        {"name": "window_decode_fp8", "kind": "window", "prefill": False, "batch": 96, "heads": 16, "kv_lo": 100,
         "kv_hi": 6000, "window": 1024, "sinks": 1, "page": 16, "fp8": True},
        # Chunks of four prompts through a windowed layer, all 128 heads.
        {"name": "window_prefill_h128", "kind": "window", "prefill": True, "batch": 4, "heads": 128, "q_lo": 256,
         "q_hi": 1024, "kv_lo": 1024, "kv_hi": 8192, "window": 1024, "sinks": 4, "page": 64, "fp8": False},
        # Verification of drafted tokens, FP8 cache at page size 1.
        {"name": "window_verify_fp8", "kind": "window", "prefill": True, "batch": 32, "heads": 16, "q_lo": 1, "q_hi": 8,
         "kv_lo": 64, "kv_hi": 4096, "window": 777, "sinks": 13, "page": 1, "fp8": True},
        # Eight beams of one prompt, head-sharded model: latency counts.
        {"name": "shared_beams", "kind": "shared", "prefill": False, "groups": 1, "members_lo": 8, "members_hi": 8,
         "heads": 16, "prefix_lo": 777, "prefix_hi": 777, "own_lo": 1, "own_hi": 60, "page": 16, "fp8": False},
        # A full batch behind one system prompt, all 128 heads.
        {"name": "shared_decode_h128", "kind": "shared", "prefill": False, "groups": 1, "members_lo": 64,
         "members_hi": 64, "heads": 128, "prefix_lo": 8192, "prefix_hi": 8192, "own_lo": 1, "own_hi": 1024, "page": 64,
         "fp8": False},
        # Several prompts sampled a few times each, head-sharded model, FP8 cache; some groups are single sequences.
        {"name": "shared_groups_fp8", "kind": "shared", "prefill": False, "groups": 12, "members_lo": 1,
         "members_hi": 20, "heads": 16, "prefix_lo": 1000, "prefix_hi": 16384, "own_lo": 1, "own_hi": 600, "page": 64,
         "fp8": True},
        # Short questions about one document, page size 1.
        {"name": "shared_questions", "kind": "shared", "prefill": True, "groups": 1, "members_lo": 24, "members_hi": 24,
         "heads": 16, "prefix_lo": 4096, "prefix_hi": 4096, "q_lo": 1, "q_hi": 60, "own_lo": 0, "own_hi": 200,
         "page": 1, "fp8": False},
        # Chunks behind two shared prompts, all 128 heads, FP8 cache.
        {"name": "shared_prefill_h128", "kind": "shared", "prefill": True, "groups": 2, "members_lo": 4,
         "members_hi": 4, "heads": 128, "prefix_lo": 1024, "prefix_hi": 4096, "q_lo": 16, "q_hi": 256, "own_lo": 0,
         "own_hi": 300, "page": 64, "fp8": True},
        # The groups of a small beam search.
        {"name": "tables_beams", "kind": "tables", "groups": 2, "members_lo": 8, "members_hi": 8, "prefix_lo": 300,
         "prefix_hi": 900, "own_lo": 1, "own_hi": 100, "min_shared": 16, "page": 16},
        # The groups of a large batch behind long documents.
        {"name": "tables_documents", "kind": "tables", "groups": 60, "members_lo": 1, "members_hi": 16,
         "prefix_lo": 500, "prefix_hi": 16384, "own_lo": 0, "own_hi": 2000, "min_shared": 128, "page": 64},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["window", "window", "shared", "shared", "tables"])
    page = rng.choice([1, 7, 16, 32, 64, 64, 128])
    heads = rng.choice([1, 5, 16, 24, 64, 100, 128])
    prefill = rng.random() < 0.5
    fp8 = rng.random() < 0.5
    if kind == "window":
        batch = _log(rng, 1, 96)
        window, sinks = _log(rng, 1, 4096), rng.choice([0, 1, 4, rng.randint(5, 300)])
        case = {"kind": kind, "prefill": prefill, "batch": batch, "heads": heads, "window": window, "sinks": sinks,
                "page": page, "fp8": fp8}
        if prefill:
            case["q_hi"] = _log(rng, 1, max(1, min(1000, 2048 // batch)))
            case["q_lo"] = rng.randint(1, case["q_hi"])
        hi = case.get("q_hi", 0) + _log(rng, 1, min(16000, 600000 // batch))
        return {**case, "kv_lo": rng.randint(case.get("q_hi", 1), hi), "kv_hi": hi}
    if kind == "shared":
        groups = _log(rng, 1, 12)
        members = _log(rng, 1, max(1, 96 // groups))
        case = {"kind": kind, "prefill": prefill, "groups": groups, "members_lo": rng.randint(1, members),
                "members_hi": members, "heads": heads, "page": page, "fp8": fp8}
        hi = _log(rng, 1, min(16000, 400000 // (groups * members)))
        if prefill:
            case["q_hi"] = _log(rng, 1, max(1, min(300, 1024 // (groups * members))))
            case["q_lo"] = rng.randint(1, case["q_hi"])
            hi = min(hi, 5000)
        own_hi = _log(rng, 1, 1000)
        return {**case, "prefix_lo": rng.randint(0, hi), "prefix_hi": hi, "own_lo": rng.randint(0, own_hi),
                "own_hi": own_hi}
    groups = _log(rng, 1, 60)
    hi = _log(rng, 1, 16000)
    return {"kind": kind, "groups": groups, "members_lo": 1, "members_hi": _log(rng, 1, 16),
            "prefix_lo": rng.randint(0, hi), "prefix_hi": hi, "own_lo": 0, "own_hi": _log(rng, 1, 2000),
            "min_shared": _log(rng, 1, 300), "page": page}


def _ceil(a, b):
    return -(-a // b)


def _rng_of(case):
    """Lengths are part of the case: the same for every seed."""
    return random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))


def _window_lens(case):
    """New tokens and keys of every sequence."""
    r = _rng_of(case)
    q = [r.randint(case["q_lo"], case["q_hi"]) if case["prefill"] else 1 for _ in range(case["batch"])]
    return q, [max(n, r.randint(case["kv_lo"], case["kv_hi"])) for n in q]


def _groups(case):
    """For every group its shared keys (whole pages, as the pool shares them), and for every member
    its new tokens and own keys (the new tokens' keys among them)."""
    r = _rng_of(case)
    found = []
    for _ in range(case["groups"]):
        members = r.randint(case["members_lo"], case["members_hi"])
        prefix = r.randint(case["prefix_lo"], case["prefix_hi"]) // case["page"] * case["page"]
        q = [r.randint(case["q_lo"], case["q_hi"]) if case.get("prefill") else 1 for _ in range(members)]
        more = [r.randint(case["own_lo"], case["own_hi"]) for _ in q]
        found.append((prefix, q, [n + m if case.get("prefill") else m for n, m in zip(q, more)]))
    return found


def work(case):
    if case["kind"] == "tables":
        entries = keys = 0
        for prefix, _, own_keys in _groups(case):
            entries += sum(_ceil(prefix + n, case["page"]) for n in own_keys)
            keys += prefix + sum(own_keys)
        return {"bytes": 4 * (entries + keys), "flops": 0}
    if case["kind"] == "window":
        w, s = case["window"], case["sinks"]
        q, kv = _window_lens(case)
        pairs = keys = 0
        for n, m in zip(q, kv):
            first = max(0, m - n + 1 - w)  # of the window of the sequence's first new token
            keys += min(s, first) + m - first
            pairs += sum(min(s, max(0, m - n + 1 + i - w)) + min(w, m - n + 1 + i) for i in range(n))
    else:
        q, pairs, keys = [], 0, 0
        for prefix, new, own_keys in _groups(case):
            q += new
            keys += prefix + sum(own_keys)
            for n, m in zip(new, own_keys):
                pairs += n * prefix + sum(max(0, m - n + 1 + i) for i in range(n))
    rows = sum(q) * case["heads"]
    return {"bytes": keys * ((TOKEN if case["fp8"] else 2 * (CKV + KPE)) + 4) + rows * (2 * (CKV + KPE) + 2 * CKV + 4),
            "flops": 2 * (2 * CKV + KPE) * case["heads"] * pairs}


# ---------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _randn(shape, g):
    return torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _offsets(counts):
    ptr = [0]
    for n in counts:
        ptr.append(ptr[-1] + n)
    return _ints(ptr)


def _quantised(ckv, kpe):
    """FP8 tokens of bf16 latents [..., 512] and rope parts [..., 64]: a scale of amax / 448 for each 128."""
    tiles = ckv.float().unflatten(-1, (4, 128))
    amax = tiles.abs().amax(-1)
    scale = torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))
    codes = (tiles / scale[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return torch.cat([codes.flatten(-2).view(torch.uint8), scale.view(torch.uint8), kpe.contiguous().view(torch.uint8)], -1)


def _cache(case, pages, g):
    ckv, kpe = _randn((pages, case["page"], CKV), g), _randn((pages, case["page"], KPE), g)
    if case["fp8"]:
        return {"kv_fp8": _quantised(ckv, kpe)}
    return {"ckv_cache": ckv, "kpe_cache": kpe}


def _paged_slots(lens, ps, g):
    """Token slots of lists on randomly permuted pages, packed, and the number of pages."""
    pages = sum(_ceil(n, ps) for n in lens) + 2
    perm = torch.randperm(pages, generator=g, device=DEV)
    parts, at = [perm[:0]], 0
    for n in lens:
        need = _ceil(n, ps)
        parts.append((perm[at: at + need][:, None] * ps + torch.arange(ps, device=DEV)).flatten()[:n])
        at += need
    return torch.cat(parts).to(torch.int32), pages


def _queries(case, tokens, g):
    return {"q_nope": _randn((tokens, case["heads"], CKV), g), "q_pe": _randn((tokens, case["heads"], KPE), g)}


def _prepare_window(case, seed):
    g = _gen(seed)
    q, kv = _window_lens(case)
    slots, pages = _paged_slots(kv, case["page"], g)
    return {**_cache(case, pages, g), **_queries(case, sum(q), g), "slots": slots, "kv_indptr": _offsets(kv),
            "qo_indptr": _offsets(q), "q_max": max(q)}


def _prepare_shared(case, seed):
    g = _gen(seed)
    groups = _groups(case)
    prefix, q = [p for p, _, _ in groups], [n for _, new, _ in groups for n in new]
    own_keys = [n for _, _, m in groups for n in m]
    slots, pages = _paged_slots(prefix + own_keys, case["page"], g)
    return {**_cache(case, pages, g), **_queries(case, sum(q), g), "prefix_slots": slots[: sum(prefix)].clone(),
            "slots": slots[sum(prefix):].clone(), "prefix_indptr": _offsets(prefix), "kv_indptr": _offsets(own_keys),
            "qo_indptr": _offsets(q), "group_indptr": _offsets([len(m) for _, _, m in groups]), "q_max": max(q),
            "prefix_max": max(prefix), "own_max": max(own_keys)}


def _prepare_tables(case, seed):
    g = _gen(seed)
    ps, groups = case["page"], _groups(case)
    rows = [(p, n) for p, _, own_keys in groups for n in own_keys]
    blocks = max(_ceil(p + n, ps) for p, n in rows) + 2
    table = torch.full((len(rows), blocks), -1, dtype=torch.int32, device=DEV)
    need = sum(p // ps for p, _, _ in groups) + sum(_ceil(n, ps) for _, n in rows)
    perm = torch.randperm(need + 5, generator=g, device=DEV).to(torch.int32)
    at = row = 0
    for prefix, _, own_keys in groups:
        shared = perm[at: at + prefix // ps]
        at += prefix // ps
        for n in own_keys:
            table[row, : prefix // ps] = shared
            table[row, prefix // ps: prefix // ps + _ceil(n, ps)] = perm[at: at + _ceil(n, ps)]
            at += _ceil(n, ps)
            row += 1
    # Room for the lists, as a program keeps it; what lies behind a list's end stays as it is.
    room = sum(p + n for p, n in rows)
    return {"table": table, "lens": _ints([p + n for p, n in rows]),
            "prefix_slots": torch.full((sum(p for p, _, _ in groups),), -1, dtype=torch.int32, device=DEV),
            "slots": torch.full((room,), -1, dtype=torch.int32, device=DEV)}


def prepare(case, seed):
    s = {"window": _prepare_window, "shared": _prepare_shared, "tables": _prepare_tables}[case["kind"]](case, seed)
    s["case"] = case
    return s


# ---------------------------------------------------------------- the plain forms
def _dequantised(tokens):
    codes = tokens[..., :CKV].contiguous().view(torch.float8_e4m3fn).float().unflatten(-1, (4, 128))
    scale = tokens[..., CKV: CKV + 16].contiguous().view(torch.float32)
    return (codes * scale[..., None]).flatten(-2).to(torch.bfloat16), tokens[..., CKV + 16:].contiguous().view(torch.bfloat16)


def _keys(s, slots):
    """The keys [..., 576] in these token slots, in 32 bits."""
    if "kv_fp8" in s:
        return torch.cat(_dequantised(s["kv_fp8"].view(-1, TOKEN)[slots]), -1).float()
    return torch.cat([s["ckv_cache"].view(-1, CKV)[slots], s["kpe_cache"].view(-1, KPE)[slots]], -1).float()


def _padded(ptr, width):
    """Positions of lists in a rectangle [lists, width] (those behind a list's end name its last entry)."""
    at, n = torch.arange(width, device=DEV), ptr.diff()
    return ptr[:-1, None] + torch.minimum(at[None], (n[:, None] - 1).clamp(min=0))


def _attend(s, k, seen):
    """Queries in a rectangle [lists, q_max] over keys k [lists, n, 576]; seen [lists, q_max, n]."""
    h, qm = s["q_nope"].shape[1], s["q_max"]
    qp = s["qo_indptr"].long()
    lists, n = k.shape[:2]
    at = _padded(qp, qm)
    q = torch.cat([s["q_nope"], s["q_pe"]], -1).float()[at].view(lists, qm * h, CKV + KPE)
    score = torch.bmm(q, k.transpose(1, 2)).mul_(SM_SCALE).view(lists, qm, h, n)
    score.masked_fill_(~seen[:, :, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = score.sub_(torch.where(torch.isfinite(top), top, torch.zeros_like(top))).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.bmm(p.view(lists, qm * h, n), k[..., :CKV]).view(lists, qm, h, CKV)
    out = torch.where(total > 0, out / total, torch.zeros_like(out))
    lse = (top + total.log())[..., 0]
    real = torch.nonzero((torch.arange(qm, device=DEV)[None] < qp.diff()[:, None]).flatten())[:, 0]
    return out.view(-1, h, CKV)[real].to(torch.bfloat16), lse.view(-1, h)[real]


def _window(s):
    c = s["case"]
    w, sinks, qm = c["window"], c["sinks"], s["q_max"]
    kp, qn = s["kv_indptr"].long(), s["qo_indptr"].long().diff()
    kn = kp.diff()
    # A rectangle of the first keys and of those from the first new token's window on.
    first = (kn - qn + 1 - w).clamp(min=0)
    j = torch.arange(sinks + w + qm - 1, device=DEV)
    pos = torch.where(j[None] < sinks, j[None], first[:, None] + j[None] - sinks)
    real = torch.where(j[None] < sinks, j[None] < first[:, None], pos < kn[:, None])
    at = torch.where(real, kp[:-1, None] + pos, torch.zeros_like(pos))
    k = _keys(s, s["slots"][at].long())
    end = (kn - qn + 1)[:, None] + torch.arange(qm, device=DEV)[None]  # keys up to each token's own
    seen = (pos[:, None] < end[..., None]) & ((pos[:, None] >= end[..., None] - w) | (pos[:, None] < sinks)) & real[:, None]
    return _attend(s, k, seen)


def _shared(s):
    qm = s["q_max"]
    members = s["group_indptr"].long().diff()
    group = torch.repeat_interleave(torch.arange(members.numel(), device=DEV), members)
    pp, kp, qn = s["prefix_indptr"].long(), s["kv_indptr"].long(), s["qo_indptr"].long().diff()
    pn, kn = pp.diff()[group], kp.diff()
    i, j = torch.arange(s["prefix_max"], device=DEV)[None], torch.arange(s["own_max"], device=DEV)[None]
    in_prefix, in_own = i < pn[:, None], j < kn[:, None]
    lists = torch.cat([s["prefix_slots"], s["slots"], torch.zeros_like(s["qo_indptr"][:1])])
    at = torch.cat([torch.where(in_prefix, pp[group][:, None] + i, torch.full_like(in_prefix, lists.numel() - 1, dtype=torch.long)),
                    torch.where(in_own, s["prefix_slots"].numel() + kp[:-1, None] + j,
                                torch.full_like(in_own, lists.numel() - 1, dtype=torch.long))], 1)
    k = _keys(s, lists[at].long())
    end = (kn - qn + 1)[:, None] + torch.arange(qm, device=DEV)[None]
    seen = torch.cat([in_prefix[:, None].expand(-1, qm, -1), in_own[:, None] & (j[None] < end[..., None])], 2)
    return _attend(s, k, seen)


def _tables(s):
    table, lens, ps = s["table"], s["lens"].long(), s["case"]["page"]
    n, blocks = table.shape
    full = lens // ps
    block = torch.arange(blocks, device=DEV)[None]
    same = (table[1:] == table[:-1]) & (block < torch.minimum(full[1:], full[:-1])[:, None])
    pages = torch.cat([torch.zeros_like(lens[:1]), same.int().cumprod(1).sum(1)])  # leading pages as the row before
    head = pages * ps < max(1, s["case"]["min_shared"])
    head[:1] = True
    group = head.long().cumsum(0) - 1
    # Shared keys of a group: what all its neighbours share; none in a group of one.
    least = torch.full((n,), blocks + 1, dtype=torch.long, device=DEV)
    least = least.scatter_reduce(0, group, torch.where(head, torch.full_like(pages, blocks + 1), pages), "amin")
    shared = torch.where(least <= blocks, least * ps, torch.zeros_like(least))
    rows = torch.arange(n, device=DEV)
    group_ptr = torch.full((n + 1,), n, dtype=torch.long, device=DEV)
    group_ptr.scatter_reduce_(0, group, rows, "amin")
    zero = torch.zeros_like(lens[:1])
    own_keys = lens - shared[group]
    prefix_ptr, kv_ptr = torch.cat([zero, shared.cumsum(0)]), torch.cat([zero, own_keys.cumsum(0)])
    owner = torch.repeat_interleave(rows, shared)
    at = torch.arange(owner.numel(), device=DEV) - prefix_ptr[owner]
    s["prefix_slots"][: owner.numel()] = table[group_ptr[owner], at // ps] * ps + (at % ps).int()
    owner = torch.repeat_interleave(rows, own_keys)
    at = torch.arange(owner.numel(), device=DEV) - kv_ptr[owner] + shared[group[owner]]
    s["slots"][: owner.numel()] = table[owner, at // ps] * ps + (at % ps).int()
    return group_ptr.int(), prefix_ptr.int(), s["prefix_slots"], kv_ptr.int(), s["slots"]


# ---------------------------------------------------------------- one pass
def run(state):
    k = state["case"]["kind"]
    if own:
        return _run_own(state, k)
    return {"window": _window, "shared": _shared, "tables": _tables}[k](state)


def _run_own(s, k):
    import paged_head_latent_gb300 as mla

    c = s["case"]
    if k == "tables":
        return mla.block_table_to_shared_csr(s["table"], s["lens"], c["page"], min_shared=c["min_shared"],
                                             prefix_indices=s["prefix_slots"], kv_indices=s["slots"])
    fp8 = "kv_fp8" in s
    cache = (s["kv_fp8"],) if fp8 else (s["ckv_cache"], s["kpe_cache"])
    queries = (s["qo_indptr"],) if c["prefill"] else ()
    if "workspace" not in s:  # kept, as a serving program keeps it
        dims = mla.make_dims(s["kv_indptr"].numel() - 1, s["q_nope"].shape[1], cache[0].shape[0], cache[0].shape[1],
                             s["slots"].numel(), total_q=s["q_nope"].shape[0])
        need = (mla.workspace_bytes_window(dims, c["window"], c["sinks"], is_prefill=c["prefill"]) if k == "window" else
                mla.workspace_bytes_shared(dims, s["group_indptr"].numel() - 1, s["prefix_slots"].numel(),
                                           is_prefill=c["prefill"]))
        s["workspace"] = torch.zeros(need, dtype=torch.uint8, device=DEV)
    if k == "window":
        call = ((mla.mla_paged_prefill_window_fp8 if fp8 else mla.mla_paged_prefill_window) if c["prefill"] else
                (mla.mla_paged_decode_window_fp8 if fp8 else mla.mla_paged_decode_window))
        return call(s["q_nope"], s["q_pe"], *cache, *queries, s["kv_indptr"], s["slots"], c["window"], c["sinks"],
                    SM_SCALE, workspace=s["workspace"])
    call = ((mla.mla_paged_prefill_shared_fp8 if fp8 else mla.mla_paged_prefill_shared) if c["prefill"] else
            (mla.mla_paged_decode_shared_fp8 if fp8 else mla.mla_paged_decode_shared))
    return call(s["q_nope"], s["q_pe"], *cache, *queries, s["group_indptr"], s["prefix_indptr"], s["prefix_slots"],
                s["kv_indptr"], s["slots"], SM_SCALE, workspace=s["workspace"])


# ---------------------------------------------------------------- the definitions in 64 bits
def _exact_e4m3(code):
    """The numbers that E4M3 codes stand for: sign, four exponent bits (bias 7), three mantissa bits."""
    c = code.long()
    e, m = (c >> 3) & 15, (c & 7).double()
    value = torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * torch.pow(2.0, (e - 7).double()))
    return torch.where(c >= 128, -value, value)


def _exact_rows(s, slots):
    """Latents and rope parts in these slots; a latent of an FP8 token is code times scale as a bf16 number."""
    at = torch.tensor(slots, dtype=torch.long, device=DEV)
    if "kv_fp8" not in s:
        return s["ckv_cache"].view(-1, CKV)[at].double(), s["kpe_cache"].view(-1, KPE)[at].double()
    tokens = s["kv_fp8"].view(-1, TOKEN)[at]
    scale = tokens[:, CKV: CKV + 16].contiguous().view(torch.float32).double().repeat_interleave(128, 1)
    latent = (_exact_e4m3(tokens[:, :CKV]) * scale).float().to(torch.bfloat16).double()
    return latent, tokens[:, CKV + 16:].contiguous().view(torch.bfloat16).double()


def _exact_row_block(s, first, last, latent, rope, hidden):
    """Query tokens first .. last - 1 over these keys; hidden [tokens, keys]."""
    x = torch.einsum("qhd,kd->hqk", s["q_nope"][first:last].double(), latent)
    x = (x + torch.einsum("qhd,kd->hqk", s["q_pe"][first:last].double(), rope)) * SM_SCALE
    x = x.masked_fill(hidden, -math.inf)
    lse = torch.logsumexp(x, -1)
    weight = torch.exp(x - torch.where(torch.isfinite(lse), lse, torch.zeros_like(lse))[..., None])
    return torch.einsum("hqk,kd->qhd", weight, latent), lse.t()


def exact(case, seed):
    if case["kind"] == "tables":
        return None
    s = prepare(case, seed)
    qp, kp, slots = s["qo_indptr"].tolist(), s["kv_indptr"].tolist(), s["slots"].tolist()
    found = []
    if case["kind"] == "window":
        for b in range(len(qp) - 1):
            n, m = qp[b + 1] - qp[b], kp[b + 1] - kp[b]
            keys = [t for t in range(m) if t < case["sinks"] or t > m - n - case["window"]]
            latent, rope = _exact_rows(s, [slots[kp[b] + t] for t in keys])
            t, p = torch.tensor(keys, device=DEV)[None], torch.arange(m - n, m, device=DEV)[:, None]
            hidden = (t > p) | ((t <= p - case["window"]) & (t >= case["sinks"]))
            found.append(_exact_row_block(s, qp[b], qp[b + 1], latent, rope, hidden))
    else:
        gp, pp, prefix = s["group_indptr"].tolist(), s["prefix_indptr"].tolist(), s["prefix_slots"].tolist()
        for g in range(len(gp) - 1):
            for b in range(gp[g], gp[g + 1]):
                n, m, shared = qp[b + 1] - qp[b], kp[b + 1] - kp[b], pp[g + 1] - pp[g]
                latent, rope = _exact_rows(s, prefix[pp[g]: pp[g + 1]] + slots[kp[b]: kp[b + 1]])
                t, p = torch.arange(-shared, m, device=DEV)[None], torch.arange(m - n, m, device=DEV)[:, None]
                found.append(_exact_row_block(s, qp[b], qp[b + 1], latent, rope, (t >= 0) & (t > p)))
    return torch.cat([out for out, _ in found]), torch.cat([lse for _, lse in found])
