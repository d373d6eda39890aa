"""Linear attention of sequences that are cut into pieces: the state that enters a
piece is the one that came before, decayed by all of the rows between.

A state alone (zero k and v) against exp(the sum of ld) S0 in fp64.  An element is
rounded twice a chunk of 64 rows and twice a piece, by at most 2^-24 each; with
start values of random digits those roundings favour no sign, so that the mean over
a head's n elements stays below 2^-24 sqrt(2 chunks / n), whatever the number of
rows allows: below 2^-24 here.  What all of a head's elements share is what a decay
itself is off by, in proportion to the sum of ld.
"""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import mamba2_ssm_decode_gb300 as ssu

from .test_layer_gpu import BF16, DEV, F16, cu_of, gen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mamba2_ssm_decode_gb300 import build
    build.build()
    yield
    assert ssu.ssu_device_error() == 0


def decayed(ld, pool, io=BF16, d=64, q=0.0, k=0.0, v=0.0):
    """Outputs and states of one sequence whose rows are all alike but for their decays."""
    H, rows = pool.shape[1], ld.shape[0] if ld.dim() == 2 else 131072
    one = lambda n, x: torch.full((rows, n, d), x, dtype=io, device=DEV)  # noqa: E731
    got = pool.to(DEV).clone()
    out = ssu.linattn_fwd_varlen(one(1, q), one(1, k), one(H, v), cu_of([rows]).to(DEV),
                                 log_decay=ld.to(DEV), state=got)
    return out, got


@pytest.mark.parametrize("io", [BF16, F16])
@pytest.mark.parametrize("each", [False, True])
def test_slow_decays_over_many_rows(io, each):
    """131072 rows of about e^-1e-6: the mean of a head is off by less than 2^-20 (e^-0.13
    to e^-0.42 in all: an error of 2^-22 of the sum, and the mean of the roundings)."""
    H, rows = 8, 131072
    ld = -1e-6 * (1.0 + 0.3 * torch.arange(H))
    s0 = 0.5 + torch.rand(1, H, 64, 64, generator=gen(1))
    _, got = decayed(ld.expand(rows, H).contiguous() if each else ld, s0, io)
    want = torch.exp(rows * ld.double())[None, :, None, None] * s0.double()
    off = (got.cpu().double() / want - 1.0).mean((0, 2, 3)).abs()
    assert float(off.max()) <= 2.0 ** -20, off.tolist()


@pytest.mark.parametrize("io", [BF16, F16])
def test_a_state_grows_and_shrinks_through_pieces(io):
    """e^100 within 128 rows, from 1e-30; what was nothing stays nothing.  The sum, 144 in
    units of log2, is held to 2^-17, its exponential to some 2^-20."""
    rows = 3000
    ld = torch.zeros(rows, 2)
    ld[600:728, 0], ld[1800:1928, 1] = 100.0 / 128, -100.0 / 128
    s0 = torch.rand(1, 2, 64, 64, generator=gen(2)) + 0.5
    s0[:, 0] *= 1e-30
    s0[:, 1] *= 1e30
    s0[:, :, 5] = 0.0
    out, got = decayed(ld, s0, io)
    want = torch.exp(ld.double().sum(0))[None, :, None, None] * s0.double()
    off = (got.cpu().double() - want).abs()
    assert bool((off <= 2.0 ** -15 * want).all())
    assert not bool(out.any())
    # every piece beyond fp32's range, and nothing in the state
    out, got = decayed(torch.full((rows, 2), 0.5), torch.zeros_like(s0), io)
    assert not bool(out.any()) and not bool(got.any())


@pytest.mark.parametrize("io", [BF16, F16])
def test_what_a_piece_forgets_stays_forgotten(io):
    """A decay of zero (or far below fp32's range), and growth by e^80 in a later piece."""
    rows = 3000
    ld = torch.zeros(rows, 2)
    ld[1000, 0] = -math.inf
    ld[900:1100, 1] = -5.0
    ld[1500:1564] = 80.0 / 64
    _, got = decayed(ld, torch.ones(1, 2, 64, 64), io)
    want = np.exp(ld.double().sum(0).numpy())
    assert want[0] == 0.0 and want[1] < 1e-300
    assert not bool(got.any())
