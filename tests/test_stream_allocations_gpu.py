"""What the attention calls and the block-table adapter allocate belongs to the stream that they are
given: the allocator's own trace, and results on a stream that waits for nothing else."""

import pytest
import torch

from paged_head_latent_gb300 import workloads as wl
from tests.conftest import require_gpu

pytestmark = pytest.mark.gpu


def test_the_allocators_trace_names_the_stream(lib):
    require_gpu()
    dec = wl.make_decode([300, 77], 16, 64, seed=3).to("cuda")
    pre = wl.make_prefill([33, 1], [31, 500], num_qo_heads=16, page_size=64, seed=4).to("cuda")
    f8 = wl.quantize_fp8(wl.make_decode([300, 77], 16, 64, seed=3)).to("cuda")
    table = torch.arange(12, dtype=torch.int32, device="cuda").view(2, 6)
    lens = torch.tensor([300, 77], dtype=torch.int32, device="cuda")
    top = torch.arange(40, dtype=torch.int32, device="cuda").view(2, 20)
    rows = (dec.q_nope, dec.q_pe, dec.ckv_cache, dec.kpe_cache)
    few = max(1, dec.num_pages)
    table = table % few
    calls = [
        (lambda s: lib.run_workload(dec, stream=s), 3),
        (lambda s: lib.run_workload(pre, stream=s), 3),
        (lambda s: lib.mla_paged_decode_mtp(dec.q_nope[:, None], dec.q_pe[:, None], *rows[2:], dec.kv_indptr,
                                            dec.kv_indices, dec.sm_scale, stream=s), 3),
        (lambda s: lib.mla_paged_decode_sparse(*rows, top, dec.sm_scale, stream=s), 3),
        (lambda s: lib.run_workload(f8, stream=s), 3),
        (lambda s: lib.mla_paged_decode_block_table(*rows, table, lens, dec.sm_scale, stream=s), 3),
        (lambda s: lib.block_table_to_csr(table, lens, 64, stream=s), 2),
    ]
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
            n = int(ref[0][-1])
            assert torch.equal(got[0], ref[0]) and torch.equal(got[1][:n], ref[1][:n])
