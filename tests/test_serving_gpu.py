"""The serving step as the README prints it: the very lines are run, eagerly and captured, with
entries that the pool refuses in the middle of the step."""

import copy
import os

import numpy as np
import pytest
import torch

from oracle import cache_oracle as co
from tests.conftest import ROOT, require_gpu
from tests.test_prefill_fp8_gpu import close, plain

pytestmark = pytest.mark.gpu

PS, HEADS, PAGES, BLOCKS, ROWS = 4, 16, 60, 5, 8
FREQ = (10000.0 ** (-torch.arange(32) / 32)).float()


def readme_lines():
    """(the lines that run once, a step's lines) of the README's serving step."""
    with open(os.path.join(ROOT, "README.md")) as f:
        text = f.read()
    part = text[text.index("**A serving step.**"):text.index("**Where it stands")]
    code = [line[4:] if line.startswith("    ") else None for line in part.splitlines()]
    step = next(i for i, line in enumerate(code) if line and "mla_pages_extend" in line)
    return ["\n".join(line for line in lines if line is not None) for lines in (code[:step], code[step:])]


def _i(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


def _bf(g, *shape):
    return torch.randn(shape, generator=g).to(torch.bfloat16)


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("rows,new", [
    ([5, 2, 0], [4, 3, 2]),                  # some rows of the pool, in another order; nothing refused
    ([5, 1, 0], [4, 4, 4]),                  # row 1 is full: the middle entry is refused
    ([-1, 5, 99, 0, 5, 2], [3, 1, 2, 6, 5, 0]),  # rows that are none, a row named twice, no tokens
    ([0, 3, 2, 6], [1, 0, 2, 17]),           # an entry without tokens, a row that begins
])
def test_the_readmes_step(lib, rows, new, captured):
    require_gpu()
    once, step = readme_lines()
    g = torch.Generator().manual_seed(len(rows) + new[0])
    n, total = len(rows), 24
    lens0 = [9, 20, 4, 1, 0, 7, 0, 12]  # (row 1 fills its table)
    start = np.concatenate([[0], np.cumsum(new)])
    inputs = dict(q_nope=_bf(g, total, HEADS, 512), q_pe=_bf(g, total, HEADS, 64), ckv=_bf(g, total, 512),
                  k_pe=_bf(g, total, 64), positions=torch.zeros(total, dtype=torch.int32))
    for i, (r, c) in enumerate(zip(rows, new)):
        first = lens0[r] if 0 <= r < ROWS else 0
        inputs["positions"][start[i]:start[i + 1]] = first + torch.arange(c, dtype=torch.int32)
    ns = dict(torch=torch, mla=lib, n=n, total=total, heads=HEADS, num_pages=PAGES, page_size=PS,
              table=_i([[-1] * BLOCKS] * ROWS), lens=_i([0] * ROWS), refs=_i([0] * PAGES), rows=_i(rows),
              new_tokens=_i(new), parents=_i([5, 0, 2, 1]), children=_i([4, 6, 6, 2]), ended=_i([0, 7, -1]),
              inv_freq=FREQ.cuda(), sm_scale=192 ** -0.5,
              kv_fp8=torch.zeros(PAGES, PS, 656, dtype=torch.uint8).cuda(), **{k: v.cuda() for k, v in inputs.items()})
    pool = co.Pool(ns["table"].tolist(), ns["lens"].tolist(), ns["refs"].tolist(), PS)
    arrays = (ns["table"], ns["lens"], ns["refs"])
    order = [7, 3, 1, 0, 2, 5]
    # What was there before: random tokens.
    _, slots, _ = lib.mla_pages_extend(*arrays, _i(order), _i([lens0[r] for r in order]), PS, sum(lens0))
    pool.extend(order, [lens0[r] for r in order], sum(lens0))
    codes, scales = co.quantise(_bf(g, sum(lens0), 512).float().numpy())
    old = torch.cat([torch.from_numpy(codes), torch.from_numpy(scales).view(torch.uint8),
                     _bf(g, sum(lens0), 64).view(torch.uint8)], 1)
    ns["kv_fp8"].view(-1, 656)[slots.long()] = old.cuda()
    tokens, at = {}, 0
    for r in order:
        tokens[r] = old[at:at + lens0[r]]
        at += lens0[r]
    # Room for the keys of the granted entries and no more.
    dry = copy.deepcopy(pool)
    granted = [r for r, st in zip(rows, dry.extend(rows, new, total)[2]) if st == 0]
    ns["max_keys"] = sum(dry.lens[r] for r in granted)
    exec(once, ns)
    state = [t.clone() for t in (*arrays, ns["kv_fp8"])]
    given = dict(ns)
    exec(step, ns)
    if captured:
        def rewind():
            for t, s in zip((*arrays, given["kv_fp8"]), state):
                t.copy_(s)

        rewind()
        graph = torch.cuda.CUDAGraph()
        ns = dict(given)
        with torch.cuda.graph(graph):
            exec(step, ns)
        for t in (ns["out"], ns["lse"], ns["q_pe"], given["workspace"]):
            t.fill_(0)
        graph.replay()
    torch.cuda.synchronize()

    # The oracle: every granted entry with its own inputs, refused ones with nothing.
    ptr, slots, status = pool.extend(rows, new, total)
    assert ns["ok"].tolist() == status and ns["ptr"].tolist() == ptr and ns["slots"].tolist() == slots
    scratch = torch.zeros(1, total, 656, dtype=torch.uint8).cuda()
    rotated = lib.mla_rope_append_fp8(given["q_pe"], given["ckv"], given["k_pe"], given["positions"], given["inv_freq"],
                                      torch.arange(total, dtype=torch.int32).cuda(), scratch).cpu()
    q_nope, q_pe, kp, kv = [], [], [0], []
    for i, (r, st) in enumerate(zip(rows, status)):
        if st == 0:
            mine = slice(start[i], start[i + 1])
            tokens[r] = torch.cat([tokens.get(r, old[:0]), scratch[0, mine].cpu()])
            q_nope.append(inputs["q_nope"][mine])
            q_pe.append(rotated[mine])
        kv.append(tokens[r] if st == 0 else old[:0])
    for i, st in enumerate(status):
        kp.append(kp[-1] + len(kv[i]))
    x = dict(qn=torch.cat(q_nope), qp=torch.cat(q_pe), kv=torch.cat(kv)[:, None], qo=torch.tensor(ptr),
             kp=torch.tensor(kp), ki=torch.arange(kp[-1]), scale=192 ** -0.5)
    assert len(x["qn"]) == ptr[-1] and ptr[-1] > 0
    close((ns["out"], ns["lse"]), plain(x), rows=ptr[-1])
    res = pool.fork([5, 0, 2, 1], [4, 6, 6, 2])[0]
    for p, c, st in zip([5, 0, 2, 1], [4, 6, 6, 2], res):
        if st == 0:
            tokens[c] = tokens.get(p, old[:0])
    pool.free([0, 7, -1])
    tokens[0] = tokens[7] = old[:0]
    pool.compact()
    assert given["lens"].tolist() == pool.lens and given["refs"].tolist() == pool.refs
    assert given["table"].tolist() == pool.table
    cache = given["kv_fp8"].cpu().view(-1, 656)
    for r in range(ROWS):
        at = [pool.table[r][k // PS] * PS + k % PS for k in range(pool.lens[r])]
        assert torch.equal(cache[at], tokens.get(r, old[:0]))


@pytest.mark.parametrize("pages", [600, 40000])
def test_one_workspace_for_the_pool_and_the_attention(lib, pages):
    """The pool's calls leave the attention's status word alone: no error is read that no attention
    call made, and one that was made is still there."""
    require_gpu()
    ws = torch.zeros(1 << 26, dtype=torch.uint8, device="cuda")
    arrays = (_i([[-1] * 9] * 5), _i([0] * 5), _i([0] * pages))
    bad = torch.ones(1, 1, 512, dtype=torch.bfloat16).cuda()
    attend = (bad, bad[..., :64].contiguous(), torch.zeros(1, 4, 656, dtype=torch.uint8).cuda(), _i([0, 1]), _i([0, 2]),
              _i([0, -1]), 1.0)
    for flags, status in ((0, 0), (lib.MLA_VALIDATE, -6)):
        lib.mla_paged_prefill_fp8(*attend, workspace=ws, flags=flags)
        _, _, results = lib.mla_pages_extend(*arrays, _i([0, 3]), _i([9, 6]), PS, 15, workspace=ws)
        assert results.tolist() == [0, 0]
        lib.mla_pages_fork(*arrays, _i([0]), _i([4]), PS, workspace=ws)
        lib.mla_pages_free(*arrays, _i([0, 4]), PS)
        lib.mla_pages_compact(*arrays, PS, workspace=ws)
        assert lib.read_device_status(ws) == status
        lib.mla_pages_free(*arrays, _i([3]), PS)


def test_more_tokens_than_an_int_holds(lib):
    """Rows that all hold one page that is counted once, which no call of the pool makes: the
    offsets stay at the largest int, and no slot is written outside the buffer."""
    require_gpu()
    rows, ps = 3000, 1 << 20
    table, lens, refs = _i([[0]] * rows), _i([1] * rows), _i([1] + [0] * 1999)
    guard = torch.full((300,), 7, dtype=torch.int32, device="cuda")
    ptr, slots, results = lib.mla_pages_extend(table, lens, refs, torch.arange(rows, dtype=torch.int32, device="cuda"),
                                               _i([ps - 1] * rows), ps, 100, slots=guard[100:200])
    assert not results.any() and (lens == ps).all()
    assert ptr.tolist() == [min(i * (ps - 1), 2 ** 31 - 1) for i in range(rows + 1)]
    assert slots.tolist() == list(range(1, 101))
    assert (guard[:100] == 7).all() and (guard[200:] == 7).all()
