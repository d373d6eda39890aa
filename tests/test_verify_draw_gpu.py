"""The draw of the verification at the borders between two tokens: floor(u W) is that of
the exact product, for every u and every sum of weights."""
from __future__ import annotations

import pytest
import torch

import mamba2_ssm_decode_gb300 as ssu
from oracle import serving

from .test_layer_gpu import BF16, DEV, F32, gen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mamba2_ssm_decode_gb300 import build
    build.build()


def drawn(p, u):
    rows = p.shape[0]
    none = torch.zeros(rows, 0, dtype=torch.int64, device=DEV)
    return ssu.drafts_verify(p.to(DEV), none, u.view(rows, 1).to(DEV))[0][:, 0].tolist()


def split(w):
    """A weight below 2^44 as two that are fp32 numbers in units of 2^-44."""
    high = w >> 20 << 20
    return [high / 2.0 ** 44, (w - high) / 2.0 ** 44]


def test_the_product_is_not_rounded():
    """u W just below a whole number m that is also the border of two tokens: the lower one."""
    rows, us = [], []
    for k in (1, 3, 8388607, 8400943, 12345677, 16777215):  # u = k 2^-24, k odd
        W = (1 << 44) - (1 << 24) + (-pow(k, -1, 1 << 24)) % (1 << 24)
        m = (k * W + 1) >> 24
        assert (k * W + 1) % (1 << 24) == 0 and 0 < m < W
        rows.append(split(m) + split(W - m))
        us.append(k / 2.0 ** 24)
        assert all(float(torch.tensor(x, dtype=F32)) == x for x in rows[-1])
    # token 1 ends at m, unless it weighs nothing
    assert drawn(torch.tensor(rows), torch.tensor(us)) == [1 if r[1] else 0 for r in rows]


def test_small_uniforms():
    """u of any size: 2^-24 and far below draw the first token that weighs something."""
    p = torch.tensor([[0.0, 2.0 ** -44, 0.5, 0.5]]).repeat(5, 1)
    u = torch.tensor([2.0 ** -44, 2.0 ** -45, 2.0 ** -100, 1e-45, 0.0])
    # W = 2^44 + 1: u W is 1 + 2^-44 for the first one, below 1 for the others
    assert drawn(p, u) == [2, 1, 1, 1, 1]


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rows_whose_weights_come_to_2_63(dtype):
    """2^19 weights of 1: floor(u 2^63) lies in token floor(u 2^19)."""
    V = 1 << 19
    us = torch.tensor([0.25, 0.9974, 0.9976, 0.999, 1 - 2.0 ** -24])
    got = drawn(torch.ones(5, V, dtype=dtype), us)
    assert got == [int(float(u) * V) for u in us]


@pytest.mark.parametrize("seed", range(4))
def test_borders_of_random_rows(seed):
    """u at, just below and just above the borders of random rows, against the oracle."""
    g, V, per = gen(seed), 300, 12
    p = torch.softmax(2 * torch.randn(40, V, generator=g), 1)
    w = (p.double() * 2.0 ** 44).round()
    edge = (w.cumsum(1) / w.sum(1, keepdim=True)).float()
    rows, us = [], []
    for r in range(40):
        for t in torch.randint(0, V, (per // 3,), generator=g).tolist():
            x = edge[r, t:t + 1]
            for u in (torch.nextafter(x, torch.zeros(1)), x, torch.nextafter(x, torch.ones(1))):
                rows.append(r)
                us.append(float(u.clamp(0.0, 1 - 2.0 ** -24)))
    p, u = p[rows], torch.tensor(us)
    want, _ = serving.verify(p, torch.zeros(len(us), 0, dtype=torch.int64), u[:, None])
    assert drawn(p, u) == [t[0] for t in want]
