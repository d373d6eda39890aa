"""Linear attention over prompts: operands whose rows lie inside their heads, and a
workspace that calls in turn share."""
from __future__ import annotations

import pytest
import torch

import mamba2_ssm_decode_gb300 as ssu

from .test_layer_gpu import BF16, DEV, F16, F32, cu_of, same_bits
from .test_serving_gpu import lin_inputs, on_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mamba2_ssm_decode_gb300 import build
    build.build()
    yield
    assert ssu.ssu_device_error() == 0


@pytest.mark.parametrize("io,d", [(BF16, 64), (BF16, 128), (F16, 64)])
@pytest.mark.parametrize("lens", [[30, 100, 1], [1500]])
@pytest.mark.parametrize("first", ["q", "v", "qkv"])
def test_heads_first(io, d, lens, first):
    """[heads, rows, d] in memory, of q and k, of v, or of all: the bits of rows first."""
    T, S = sum(lens), len(lens)
    i = lin_inputs(T, 4, 2, d, d, S, io, F32, seed=3)
    d = on_gpu(i)
    cu, pools = cu_of(lens).to(DEV), [d["pool"].clone() for _ in range(2)]
    plain = [d[n].contiguous() for n in "qkv"]
    moved = [t.transpose(0, 1).contiguous().transpose(0, 1) if n in first else t
             for n, t in zip("qkv", plain)]
    got = [ssu.linattn_fwd_varlen(*ops, cu, log_decay=d["log_decay"], state=p)
           for ops, p in zip((plain, moved), pools)]
    same_bits(*got)
    same_bits(*pools)


def test_captured_prompts_in_turn_on_one_workspace():
    """Two graphs and an eager call, one behind the other on a stream, of other lengths and
    pieces, through one workspace."""
    d = [on_gpu(lin_inputs(n, 2, 2, 64, 64, 1, BF16, F32, seed=n)) for n in (1500, 900)]
    cus = [cu_of([n]).to(DEV) for n in (1500, 900)]
    size = max(ssu.linattn_workspace_bytes(n, 1, 2, 64, 64, BF16) for n in (1500, 900))
    ws = torch.empty(size, dtype=torch.uint8, device=DEV)

    def call(n, pool, out, ws):
        ssu.linattn_fwd_varlen(d[n]["q"], d[n]["k"], d[n]["v"], cus[n], log_decay=d[n]["log_decay"],
                               state=pool, out=out, workspace=ws)

    outs = [torch.empty(t["v"].shape, dtype=BF16, device=DEV) for t in d]
    pools = [t["pool"].clone() for t in d]
    graphs = []
    for n in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[n]):
            call(n, pools[n], outs[n], ws)
    want = [(t["pool"].clone(), torch.empty_like(o)) for t, o in zip(d, outs)]
    for step in range(3):
        for n in (0, 1):
            graphs[n].replay()
            call(n, want[n][0], want[n][1], ws if step % 2 else torch.empty_like(ws))
        for n in (0, 1):
            same_bits(outs[n], want[n][1])
            same_bits(pools[n], want[n][0])
