"""Pin of the verification's oracle: floor(u W) of the exact product."""
from __future__ import annotations

import torch

from oracle import serving


def test_the_draw_rounds_nothing():
    """u = k 2^-24 and W with k W = m 2^24 - 1: u W is just below m, where the first two
    tokens end, and an fp64 product is m."""
    for k in (8400943, 12345677):
        W = (1 << 44) - (1 << 24) + (-pow(k, -1, 1 << 24)) % (1 << 24)
        m = (k * W + 1) >> 24
        assert float(k / 2.0 ** 24) * float(W) == m and k * W < m << 24
        w = [m >> 20 << 20, m % (1 << 20), (W - m) >> 20 << 20, (W - m) % (1 << 20)]
        p = torch.tensor([[x / 2.0 ** 44 for x in w]])
        u = torch.tensor([[k / 2.0 ** 24]])
        none = torch.zeros(1, 0, dtype=torch.int64)
        assert serving.verify(p, none, u) == ([[1]], [1])
        assert serving.verify(p, none, u + 2.0 ** -24) == ([[2]], [1])
