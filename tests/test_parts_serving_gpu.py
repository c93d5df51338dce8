"""The decode step over shared prompts and a window as the README prints it: the very lines are run over a
pool of forked rows, eagerly and captured; and what the binding of these calls refuses and allocates."""

import os

import numpy as np
import pytest
import torch

from tests.conftest import ROOT, require_gpu
from tests.test_parts_gpu import SCALE, both, close, on_gpu, plain

pytestmark = pytest.mark.gpu

FREQ = (10000.0 ** (-torch.arange(32) / 32)).float()
CKV, KPE = (512,), (64,)


def readme_lines():
    """(the lines that run once, a step's lines) of the README's step over shared prompts."""
    with open(os.path.join(ROOT, "README.md")) as f:
        text = f.read()
    part = text[text.index("**Shared prompts and windows.**"):text.index("**How it is checked")]
    code = [line[4:] if line.startswith("    ") else None for line in part.splitlines()]
    step = next(i for i, line in enumerate(code) if line and line.startswith("positions"))
    return ["\n".join(line for line in lines if line is not None) for lines in (code[:step], code[step:])]


def _i(v):
    return torch.tensor(v, dtype=torch.int32).cuda()


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("page,heads", [(4, 16), (64, 128), (16, 24)])
def test_the_readmes_step(lib, page, heads, captured):
    """Two prompts of several full pages, forked to beams, and a row of its own: five steps, between which
    a beam dies and another takes its row."""
    require_gpu()
    once, step = readme_lines()
    g = torch.Generator().manual_seed(page + heads)
    batch, blocks, pages = 8, 9, 80
    prompts = {0: 3 * page + 2, 4: 5 * page, 7: page - 1}
    ns = dict(torch=torch, mla=lib, batch=batch, heads=heads, num_pages=pages, page_size=page,
              table=_i([[-1] * blocks] * batch), lens=_i([0] * batch), refs=_i([0] * pages), rows=_i(list(range(batch))),
              one_each=_i([1] * batch), inv_freq=FREQ.cuda(), sm_scale=SCALE, window=page + 3, sinks=2)
    arrays = (ns["table"], ns["lens"], ns["refs"])
    cache = {name: torch.randn(pages, page, *dim, generator=g).to(torch.bfloat16).cuda()
             for name, dim in (("ckv_cache", CKV), ("kpe_cache", KPE))}
    ns.update(cache)

    def fork(parents, children):
        res, src, dst, m = lib.mla_pages_fork(*arrays, _i(parents), _i(children), page)
        assert res.tolist() == [0] * len(parents)
        lib.mla_cache_copy_pages(cache["ckv_cache"], cache["kpe_cache"], src, dst, tokens=m)

    _, _, ok = lib.mla_pages_extend(*arrays, _i(list(prompts)), _i(list(prompts.values())), page, sum(prompts.values()))
    assert ok.tolist() == [0, 0, 0]
    fork([0, 0, 0, 4, 4], [1, 2, 3, 5, 6])
    exec(once, ns)
    inputs = {name: torch.zeros(batch, *shape, dtype=torch.bfloat16, device="cuda")
              for name, shape in (("q_nope", (heads, 512)), ("q_pe", (heads, 64)), ("ckv", CKV), ("k_pe", KPE))}
    graph, got = None, None
    for turn in range(5):
        if turn == 3:  # beam 2 dies, a beam of row 1 takes its place
            lib.mla_pages_free(*arrays, _i([2]), page)
            fork([1], [2])
        for t in inputs.values():
            t.copy_(torch.randn(t.shape, generator=g).to(torch.bfloat16))
        if not captured or turn == 0:
            got = dict(ns, **inputs)
            exec(step, got)
        elif graph is None:
            graph = torch.cuda.CUDAGraph()
            got = dict(ns, **inputs)
            with torch.cuda.graph(graph):
                exec(step, got)
        if graph is not None:
            graph.replay()
        torch.cuda.synchronize()
        assert got["ok"].tolist() == [0] * batch
        lens, table = ns["lens"].tolist(), ns["table"].tolist()
        assert lens == [prompts[0 if r < 4 else 4 if r < 7 else 7] + turn + 1 for r in range(batch)]
        lists = [torch.tensor([table[r][k // page] * page + k % page for k in range(lens[r])], dtype=torch.int32)
                 for r in range(batch)]
        # The lists split into prefixes that several rows share and the rows' own.
        groups = got["groups"].tolist()
        assert groups[:4] == [0, 4, 7, 8]
        shared = np.diff(got["prefix_ptr"].tolist())[:3].tolist()
        assert shared == [3 * page, 5 * page, 0]
        x = dict(qn=inputs["q_nope"].cpu(), qp=got["q_pe"].cpu(), qo=torch.arange(batch + 1), ki=torch.cat(lists),
                 kp=torch.tensor(np.concatenate([[0], np.cumsum(lens)])), ckv=cache["ckv_cache"].cpu(),
                 kpe=cache["kpe_cache"].cpu())
        close((got["out"], got["lse"]), plain(x))
        close((got["out_w"], got["lse_w"]), plain(x, ns["window"], ns["sinks"]))
    assert lib.read_device_status(ns["workspace"]) == 0


def _names(kind):
    return ("kp", "ki") if kind == "window" else ("gp", "pp", "pi", "kp", "ki")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("prefill", [False, True])
def test_python_refusals(lib, fp8, prefill):
    require_gpu()
    q = ((2, 90), (3, 20), (1, 5)) if prefill else ((1, 90), (1, 20), (1, 5))
    for kind, x, args in both(16, 16, fp8, 61, q):
        name = f"mla_paged_{'prefill' if prefill else 'decode'}_{kind}" + ("_fp8" if fp8 else "")
        c = on_gpu(x)

        def call(args=args, scale=SCALE, kw={}, **new):
            y = {**c, **new}
            cache = (y["kv"],) if fp8 else (y["ckv"], y["kpe"])
            return getattr(lib, name)(y["qn"], y["qp"], *cache, *((y["qo"],) if prefill else ()),
                                      *(y[n] for n in _names(kind)), *args, scale, **kw)

        call()
        rows = c["qn"].shape[0]
        values = [dict(qn=c["qn"][..., :256].contiguous()), dict(qp=c["qp"][:, :8].contiguous()),
                  dict(qn=c["qn"].transpose(0, 1)), dict(qn=x["qn"]), dict(ki=x["ki"]), dict(kp=c["kp"][:0]),
                  dict(kp=torch.cat([c["kp"], c["kp"]])), dict(ki=c["ki"][::2]),
                  dict(kw=dict(out=torch.empty(rows + 1, 16, 512, dtype=torch.bfloat16, device="cuda"))),
                  dict(kw=dict(lse=torch.empty(rows, 8, device="cuda")))]
        values += [dict(kv=c["kv"][..., :640].contiguous())] if fp8 else [dict(kpe=c["kpe"][:1]), dict(ckv=x["ckv"])]
        types = [dict(qn=c["qn"].half()), dict(qp=c["qp"].float()), dict(ki=c["ki"].long()), dict(kp=c["kp"].long()),
                 dict(ki=[1, 2]), dict(kw=dict(lse=torch.empty(rows, 16, dtype=torch.bfloat16, device="cuda")))]
        types += [dict(kv=c["kv"].view(torch.int8))] if fp8 else [dict(ckv=c["ckv"].half())]
        if prefill:
            values.append(dict(qo=c["qo"][:-1].contiguous()))
            types.append(dict(qo=None))
        if kind == "window":
            values += [dict(args=(0, 0)), dict(args=(5, -1)), dict(args=(2 ** 31, 0)), dict(args=(5, 2 ** 31))]
        else:
            values += [dict(gp=c["gp"][:0]), dict(pp=c["pp"][:-1].contiguous()), dict(pi=x["pi"])]
            types += [dict(gp=None), dict(pi=c["pi"].long()), dict(pp=[0, 1])]
        for kw in values:
            with pytest.raises(ValueError):
                call(**kw)
        for kw in types:
            with pytest.raises(TypeError):
                call(**kw)
        small = torch.zeros(4096, dtype=torch.uint8, device="cuda")
        for kw in (dict(scale=float("nan")), dict(kw=dict(workspace=small)), dict(kw=dict(num_workers=-1))):
            with pytest.raises(lib.MlaError):
                call(**kw)


def test_python_refusals_of_the_tables(lib):
    require_gpu()
    table, lens = _i([[1, 2], [1, 3]]), _i([20, 30])
    call = lib.block_table_to_shared_csr
    call(table, lens, 16)
    for a, kw in (((table[0], lens, 16), {}), ((table, lens[:1], 16), {}), ((table, lens, 0), {}),
                  ((table, lens, 16), dict(min_shared=-1)), ((table, lens, 16), dict(capacity=-1)),
                  ((table, lens, 16), dict(kv_indices=_i([0, 0]), capacity=3)), ((table.cpu(), lens, 16), {}),
                  ((table, lens, 16), dict(group_indptr=_i([0, 0]))), ((table.t(), lens, 16), {})):
        with pytest.raises(ValueError):
            call(*a, **kw)
    for a, kw in (((table.long(), lens, 16), {}), ((table, lens.long(), 16), {}),
                  ((table, lens, 16), dict(prefix_indices=table.view(-1).float()))):
        with pytest.raises(TypeError):
            call(*a, **kw)
    with pytest.raises(lib.MlaError):
        call(table, lens, 1 << 30, capacity=0, prefix_capacity=0)


def test_allocations_belong_to_the_stream(lib):
    """Outputs and workspace of the attention, the five lists of the tables."""
    require_gpu()
    calls = []
    for fp8 in (False, True):
        for prefill in (False, True):
            q = ((2, 90), (3, 20), (1, 5)) if prefill else ((1, 90), (1, 20), (1, 5))
            for kind, x, args in both(16, 16, fp8, 62, q):
                name = f"mla_paged_{'prefill' if prefill else 'decode'}_{kind}" + ("_fp8" if fp8 else "")
                c = on_gpu(x)
                given = [c["qn"], c["qp"], *((c["kv"],) if fp8 else (c["ckv"], c["kpe"])),
                         *((c["qo"],) if prefill else ()), *(c[n] for n in _names(kind)), *args, SCALE]
                calls.append((lambda s, f=getattr(lib, name), given=given: f(*given, stream=s), 3))
    table, lens = _i([[1, 2], [1, 3]]), _i([20, 30])
    calls.append((lambda s: lib.block_table_to_shared_csr(table, lens, 16, stream=s), 5))
    want = [call(None) for call, _ in calls]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for (call, count), ref in zip(calls, want):
        torch.cuda.memory._record_memory_history(context=None, max_entries=100)
        try:
            got = call(side)
            trace = torch.cuda.memory._snapshot()["device_traces"][torch.cuda.current_device()]
        finally:
            torch.cuda.memory._record_memory_history(enabled=None)
        streams = [e["stream"] for e in trace if e["action"] == "alloc"]
        assert len(streams) == count and set(streams) == {side.cuda_stream}
        torch.cuda.synchronize()
        if count == 3:
            assert all(torch.equal(a, b) for a, b in zip(got, ref))
        else:
            assert all(torch.equal(got[i], ref[i]) for i in (0, 1, 3))
