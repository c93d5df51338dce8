"""The kernels that find shared prefixes, run from their source on the CPU under chosen schedules
(cuda_on_host.h): their lists may not depend on which warp is ahead of which, nor on how early a kernel
begins that overlaps the one whose offsets it reads."""

import ctypes
import os
import re
import shutil
import subprocess
import sys

import numpy as np
import pytest

from tests.conftest import ROOT
from tests.test_shared_tables import groups_of

CSRC = os.path.join(ROOT, "paged_head_latent_gb300", "csrc")
FILL, GUARD = -77, 1024


class Params(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("block_table", "seq_lens")] + [
        (n, ctypes.c_int) for n in ("batch", "max_blocks", "page_size", "min_shared")] + [
        (n, ctypes.c_void_p) for n in ("group_indptr", "prefix_indptr", "prefix_indices", "kv_indptr", "kv_indices")] + [
        (n, ctypes.c_longlong) for n in ("prefix_capacity", "capacity")]


def kernels():
    """The kernels' source and that of their parameters, without includes, PTX and launches."""
    with open(os.path.join(CSRC, "launch.h")) as f:
        params = re.search(r"struct SharedTableParams \{.*?\n\};\n", f.read(), re.S).group(0)
    with open(os.path.join(CSRC, "mla_shared_tables.cu")) as f:
        text = f.read()
    text = text[:text.index("template <typename Kernel>")]
    text = re.sub(r"asm volatile\(\"griddepcontrol[^;]*;\" ::: \"memory\"\);", "", text)
    assert "asm" not in text
    return f"namespace mla {{\n{params}}}\n" + text.replace('#include "launch.h"', "") + "}\n}\n"


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    if not shutil.which("g++"):
        pytest.skip("no host compiler")
    at = tmp_path_factory.mktemp("host")
    (at / "kernels.h").write_text(kernels())
    out = at / "tables.so"
    subprocess.run(["g++", "-std=c++17", "-O2", "-fwrapv", "-shared", "-fPIC", "-w", f"-I{ROOT}/tests",
                    f'-DKERNELS="{at}/kernels.h"', f"{ROOT}/tests/shared_tables_on_host.cpp", "-o", str(out)], check=True)
    lib = ctypes.CDLL(str(out))
    lib.path = str(out)
    lib.tables_early_loads.restype = ctypes.c_longlong
    return lib


def buffer(n):
    return np.full(n + 2 * GUARD, FILL, np.int32)


def run(host, table, lens, page, min_shared, schedule, small, cap, pcap, later=None):
    """(group_indptr, prefix_indptr, prefix_indices, kv_indptr, kv_indices); nothing around them is written."""
    n = len(lens)
    bufs = [buffer(m) for m in (n + 1, n + 1, pcap, n + 1, cap)]
    at = [b[GUARD:].ctypes.data for b in bufs]
    p = Params(table.ctypes.data, lens.ctypes.data, n, table.shape[1], page, min_shared, *at, pcap, cap)
    later = ctypes.c_void_p(later.ctypes.data if later is not None else None)
    assert host.tables_run(ctypes.byref(p), int(small), schedule, later), "an offset is negative or falls"
    assert host.tables_early_loads() == 0, "offsets are read as if nothing wrote them while the kernel lives"
    for b, m in zip(bufs, (n + 1, n + 1, pcap, n + 1, cap)):
        assert (b[:GUARD] == FILL).all() and (b[GUARD + m:] == FILL).all()
    return [b[GUARD:len(b) - GUARD] for b in bufs]


def make(rng, n, blocks, page, share):
    table = rng.integers(0, 50, (n, blocks)).astype(np.int32)
    lens = rng.integers(0, blocks * page + 1, n).astype(np.int32)
    for i in range(1, n):
        if rng.random() < share:
            k = rng.integers(0, blocks + 1)
            table[i, :k] = table[i - 1, :k]
    return table, lens


@pytest.mark.parametrize("n,small,schedule", [
    *((n, small, s) for n, small in ((1, True), (40, True), (64, True), (1, False), (66, False)) for s in range(4)),
    (300, False, 1), (300, False, 2), (1100, False, 1)])
def test_lists_under_any_schedule(host, n, small, schedule):
    """Warps and lanes in ascending and descending order, and in two random ones."""
    rng = np.random.default_rng(n)
    blocks, page = 5, 2
    for share, min_shared in ((0.9, 1), (0.6, 3)) if n < 100 else ((0.9, 1),):
        table, lens = make(rng, n, blocks, page, share)
        ref = groups_of(table.tolist(), lens.tolist(), page, min_shared)
        got = run(host, table, lens, page, min_shared, schedule, small, len(ref[4]) + 3, len(ref[2]) + 3)
        for have, want in zip(got, ref):
            assert have[:len(want)].tolist() == want and (have[len(want):] == FILL).all()


@pytest.mark.parametrize("schedule", [0, 1])
@pytest.mark.parametrize("n,small", [(70, False), (50, True)])
def test_lengths_that_change_meanwhile_lead_nowhere_else(host, n, small, schedule):
    """Lengths rewritten between two launches of a call, or during its single one, make lists that mean nothing, inside
    their buffers."""
    rng = np.random.default_rng(5)
    table, lens = make(rng, n, 5, 2, 1.0)
    table[:] = table[0]
    lens[:] = 9
    run(host, table, lens, 2, 1, schedule, small, 300, 50, later=rng.integers(0, 11, n).astype(np.int32))
    run(host, table, lens, 2, 1, schedule, small, 300, 50, later=np.zeros(n, np.int32))


@pytest.mark.parametrize("what", ["prefix", "own keys", "pages"])
def test_lists_as_long_as_an_int_counts(host, what):
    """Counters that step past 2^31 - 1 end their loops there (in a process of its own: status 3 is an access
    outside the list or the table)."""
    n = ["prefix", "own keys", "pages"].index(what)
    code = f"import ctypes, sys; sys.exit(0 if ctypes.CDLL({host.path!r}).tables_far({n}) == 1 else 1)"
    assert subprocess.run([sys.executable, "-c", code]).returncode == 0
