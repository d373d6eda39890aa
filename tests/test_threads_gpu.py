"""Calls of the C ABI from two host threads at once, on a stream each: what one call
asks of a kernel (its shared memory) must not be taken back by the other's."""
from __future__ import annotations

import ctypes
import threading

import pytest
import torch

from mamba2_ssm_decode_gb300 import _abi

from .test_layer_gpu import DEV

pytestmark = pytest.mark.gpu
CALLS = 1500


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mamba2_ssm_decode_gb300 import build
    build.build()


def at_once(jobs):
    """Every job(stream) CALLS times from a thread of its own; the refused calls."""
    refused, lib = [], _abi.lib()
    start = threading.Barrier(len(jobs))
    torch.cuda.synchronize()

    def work(job, stream):
        start.wait()
        for n in range(CALLS):
            st = job(ctypes.c_void_p(stream.cuda_stream))
            if st != _abi.SSU_OK:
                refused.append((n, st, lib.ssu_last_error().decode()))

    threads = [threading.Thread(target=work, args=(j, torch.cuda.Stream())) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return refused


def ints(*shape, fill=0):
    return torch.full(shape, fill, dtype=torch.int32, device=DEV)


def test_assignment_of_two_pools_at_once():
    """20000 and 12000 slots (listed), then 2^20 and 300000 (searched)."""
    lib, keep, jobs, results = _abi.lib(), [], [], []

    def job(slots):
        table, counts, out, fresh = ints(9, 2, fill=-1), ints(9, fill=2), ints(9, 2), ints(9, 2)
        missing = ints(1, fill=7)
        keep.extend((table, counts))
        results.append((out, missing))
        args = [t.data_ptr() for t in (table, counts)] + [_abi.SSU_I32, 9, 2, slots, -1]
        args += [t.data_ptr() for t in (out, fresh, missing)]
        keep.append(fresh)
        return lambda stream: lib.ssu_slots_assign(*args, stream)

    for slots in ((20000, 12000), (1 << 20, 300000)):
        del jobs[:], results[:]
        jobs += [job(s) for s in slots]
        assert at_once(jobs) == []
        for out, missing in results:
            assert out.view(-1).tolist() == list(range(18)) and int(missing) == 0


def test_maps_of_two_batches_at_once():
    """16384 and 7000 sequences."""
    lib, keep, jobs, results = _abi.lib(), [], [], []
    for n in (16384, 7000):
        p, rows = _abi.PromptMapsParams(), 2 * n
        t = dict(lens=ints(n, fill=2), cu_seqlens=ints(n + 1), cu_chunk_seqlens=ints(3 * n + 1),
                 seq_idx=ints(3 * n), last_chunk_indices=ints(n), num_chunks=ints(1),
                 has_initial_state=torch.zeros(n, dtype=torch.uint8, device=DEV))
        for name, v in t.items():
            setattr(p, name, v.data_ptr())
        p.index_dtype, p.nseqs, p.rows, p.chunk_size, p.max_chunks = _abi.SSU_I32, n, rows, 16, 3 * n
        keep.append((p, t))
        results.append((n, t))
        jobs.append(lambda stream, p=p: lib.ssu_prompt_maps(ctypes.byref(p), stream))
    assert at_once(jobs) == []
    for n, t in results:
        assert torch.equal(t["cu_seqlens"].cpu(), torch.arange(0, 2 * n + 1, 2, dtype=torch.int32))
        assert int(t["num_chunks"]) == n


def test_compaction_of_two_pools_at_once():
    """2^20 and 300000 slots."""
    lib, keep, jobs, results = _abi.lib(), [], [], []
    for slots in (1 << 20, 300000):
        pool = torch.arange(slots, dtype=torch.int32, device=DEV)
        table, out, live = ints(8), ints(8), ints(1, fill=7)
        table.copy_(torch.arange(8, dtype=torch.int32) + slots - 8)
        pools = (_abi.Pool * 1)(_abi.Pool(pool.data_ptr(), 4, 4))
        size = lib.ssu_slots_compact_workspace_bytes(slots, 8, 0)
        ws = torch.empty(size, dtype=torch.uint8, device=DEV)
        keep.append((pool, table, pools, ws))
        results.append((out, live))
        args = [pools, 1, slots, table.data_ptr(), out.data_ptr(), _abi.SSU_I32, 8, -1,
                live.data_ptr(), ws.data_ptr(), size]
        jobs.append(lambda stream, args=args: lib.ssu_slots_compact(*args, stream))
    assert at_once(jobs) == []
    for out, live in results:
        assert sorted(out.tolist()) == list(range(8)) and int(live) == 8
