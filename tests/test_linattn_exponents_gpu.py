"""Linear attention over prompts: the weight between two rows is e^(the sum of the log
decays between them), however much was forgotten before.

Two values that cancel: with k_a = k_b, v_b = -5/8 v_a and ld_b = ln 5/8, row b's output
is zero.  A weight is off by what its exponent is (the difference of two sums: half
a unit in the last place of |log2 5/8| < 1, 2^-25, and twice that where it is taken in
two steps through a row in between), by two fast exponentials (2^-22 each), and by its
parts (2^-22 in fp16, 2^-17 in bf16), and 64 products add with at most 2^-23 each of
what has been added: below 2^-18 in fp16 and 2^-15 in bf16 of |scale q . k| |v|, which
is also how far sum and rounding of one output go.
"""
from __future__ import annotations

import math

import pytest
import torch

import mamba2_ssm_decode_gb300 as ssu

from .test_layer_gpu import BF16, DEV, F16, cu_of, gen

pytestmark = pytest.mark.gpu
ROOM = {F16: 2.0 ** -18, BF16: 2.0 ** -15}


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mamba2_ssm_decode_gb300 import build
    build.build()
    yield
    assert ssu.ssu_device_error() == 0


@pytest.mark.parametrize("io", [F16, BF16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("forgotten,at", [
    (list(range(63)), 63),              # all before the two rows
    (list(range(32)) + [40], 48),       # another sixteen's last row and its first
    ([0, 16, 32, 48], 50),              # the first row of each sixteen
    ([], 20),
    ([], 48)])
def test_weights_after_what_was_forgotten(io, d, forgotten, at):
    g, H, rows = gen(d + at), 2, 128
    q, k = (torch.rand(rows, 1, d, generator=g).add(0.5).to(io) for _ in range(2))
    v = torch.zeros(rows, H, d)
    v[at - 1] = (8 * torch.randint(1, 9, (H, d), generator=g)).float()
    v[at] = -0.625 * v[at - 1]
    k[at] = k[at - 1]
    ld = torch.zeros(rows, H)
    ld[forgotten] = -math.inf
    ld[[64 + r for r in forgotten]] = -math.inf     # and so in the chunk after
    ld[at] = math.log(0.625)
    v[64 + at - 1:64 + at + 1], ld[64 + at] = v[at - 1:at + 1], ld[at]
    k[64 + at - 1:64 + at + 1] = k[at - 1:at + 1]
    if not forgotten:
        ld[64] = -math.inf
    pool = torch.zeros(1, H, d, d, device=DEV)
    out = ssu.linattn_fwd_varlen(q.to(DEV), k.to(DEV), v.to(io).to(DEV), cu_of([rows]).to(DEV),
                                 log_decay=ld.to(DEV), state=pool)
    for r in (at, 64 + at):
        size = float((q[r, 0].double() * k[r, 0].double()).sum()) * d ** -0.5 * v[r].abs().double()
        assert bool((out[r].cpu().double().abs() <= ROOM[io] * size + 2.0 ** -25).all()), r


@pytest.mark.parametrize("io", [F16, BF16])
@pytest.mark.parametrize("last", [-math.inf, -1e4, -230.0])
@pytest.mark.parametrize("form", ["prompt", "tokens"])
def test_growth_brings_nothing_forgotten_back(io, last, form):
    """A state and rows that are forgotten, then growth by e^80 over the chunk's other rows:
    what is left of them is zero (e^-230 e^80 is below fp32's range)."""
    g, H, d, rows = gen(3), 2, 64, 64
    q, k = (torch.randn(rows, H, d, generator=g).to(io) for _ in range(2))
    v = torch.randn(rows, H, d, generator=g).to(io)
    v[10:] = 0.0
    ld = torch.full((rows, H), 80.0 / 53)
    ld[:10], ld[10] = 0.0, last
    pool = torch.randn(1, H, d, d, generator=g).to(DEV)
    args = [t.to(DEV) for t in (q, k, v)]
    cu = cu_of([rows]).to(DEV)
    if form == "prompt":
        out = ssu.linattn_fwd_varlen(*args, cu, log_decay=ld.to(DEV), state=pool)
    else:
        out = ssu.linattn_update_varlen(pool, *args, log_decay=ld.to(DEV), cu_seqlens=cu,
                                        state_batch_indices=torch.zeros(1, rows, dtype=torch.int32,
                                                                        device=DEV))
    assert bool(out[:10].any()) and not bool(out[10:].any())
    assert not bool(pool.any())


@pytest.mark.parametrize("io", [F16, BF16])
def test_growth_that_is_lost_again(io):
    """A value that grows by e^40 within 16 rows and shrinks by e^95 within the 46 after: what
    is left, e^-55, counts where the scale says so.  An exponent of 137 is held to 2^-16."""
    rows, d, scale = 64, 64, 2.0 ** 70
    q, k, v = (torch.zeros(rows, 1, d, dtype=io) for _ in range(3))
    q[:], k[0], v[0] = 0.125, 0.125, 1.0
    ld = torch.zeros(rows, 1)
    ld[1:16], ld[16:62] = 40.0 / 15, -95.0 / 46
    out = ssu.linattn_fwd_varlen(q.to(DEV), k.to(DEV), v.to(DEV), cu_of([rows]).to(DEV),
                                 log_decay=ld.to(DEV), scale=scale, state=torch.zeros(1, 1, d, d, device=DEV))
    want = scale * torch.exp(ld.double().cumsum(0))[:, :, None].expand(rows, 1, d)
    there = want < torch.finfo(io).max
    off = (out.cpu().double() / want - 1.0).abs()[there]
    assert there[61:].all() and float(off.max()) <= torch.finfo(io).eps / 2 + 2.0 ** -14
