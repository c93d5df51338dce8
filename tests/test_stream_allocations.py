"""Every binding call that takes a stream allocates its outputs and its workspace for that stream.

Memory of another stream may still be in use there, and a workspace that is zeroed on another
stream may be zeroed after the kernels have begun to write it.  No GPU: a library of fakes that
returns success, CPU tensors, and a record of the stream that was current at each allocation.
"""

import contextlib

import pytest
import torch

import paged_head_latent_gb300 as mla

BF16, I32 = torch.bfloat16, torch.int32


class FakeLibrary:
    def __getattr__(self, name):
        return (lambda *args: 4096) if name.startswith("mla_workspace_bytes") else (lambda *args: 0)


class FakeStream:
    cuda_stream = 7


@pytest.fixture
def allocations(monkeypatch):
    """[the stream that was current, or None] of every torch.empty / torch.zeros of a call."""
    current, made = [None], []

    @contextlib.contextmanager
    def on(stream):
        current.append(stream)
        yield
        current.pop()

    def recorded(make):
        def f(*args, **kw):
            made.append(current[-1])
            return make(*args, **kw)
        return f

    monkeypatch.setattr(mla, "_lib", FakeLibrary())
    monkeypatch.setattr(mla, "_check_cuda", lambda name, t, dtype: None)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: FakeStream())
    monkeypatch.setattr(torch, "empty", recorded(torch.empty))
    monkeypatch.setattr(torch, "zeros", recorded(torch.zeros))
    return made


def _bf(*shape):
    return torch.ones(shape, dtype=BF16)


def _ints(*values):
    return torch.tensor(values, dtype=I32)


CKV, KPE, FP8 = _bf(2, 4, 512), _bf(2, 4, 64), torch.full((2, 4, 656), 1, dtype=torch.uint8)
Q, QP = _bf(2, 3, 512), _bf(2, 3, 64)
TABLE, LENS = torch.ones(2, 5, dtype=I32), _ints(3, 4)
CALLS = {  # name: (the call with a stream, allocations: outputs and workspace)
    "decode": (lambda s: mla.mla_paged_decode(Q, QP, CKV, KPE, _ints(0, 1, 2), _ints(0, 1), 1.0, stream=s), 3),
    "prefill": (lambda s: mla.mla_paged_prefill(Q, QP, CKV, KPE, _ints(0, 2), _ints(0, 2), _ints(0, 1), 1.0,
                                                stream=s), 3),
    "mtp": (lambda s: mla.mla_paged_decode_mtp(Q[None], QP[None], CKV, KPE, _ints(0, 2), _ints(0, 1), 1.0,
                                               stream=s), 3),
    "sparse": (lambda s: mla.mla_paged_decode_sparse(Q, QP, CKV, KPE, TABLE, 1.0, stream=s), 3),
    "fp8": (lambda s: mla.mla_paged_decode_fp8(Q, QP, FP8, _ints(0, 1, 2), _ints(0, 1), 1.0, stream=s), 3),
    "sparse_fp8": (lambda s: mla.mla_paged_decode_sparse_fp8(Q, QP, FP8, TABLE, 1.0, stream=s), 3),
    "csr": (lambda s: mla.block_table_to_csr(TABLE, LENS, 4, stream=s), 2),
    "block_table": (lambda s: mla.mla_paged_decode_block_table(Q, QP, CKV, KPE, TABLE, LENS, 1.0, stream=s), 3),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_a_calls_allocations_follow_its_stream(allocations, name):
    call, count = CALLS[name]
    side = FakeStream()
    call(side)
    assert len(allocations) == count and all(s is side for s in allocations)
    del allocations[:]
    call(None)  # the current stream's, as ever
    assert allocations == [None] * count
