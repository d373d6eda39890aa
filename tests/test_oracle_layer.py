"""Pins of the fp64 oracle of the calls around the state update (oracle/layer.py)."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from oracle import layer


def test_convolution_is_torchs_causal_one():
    """A fresh sequence: torch's grouped conv1d with left padding, cut to the rows."""
    g = torch.Generator().manual_seed(1)
    for W in (2, 3, 4):
        x = torch.randn(11, 6, generator=g, dtype=torch.float64)
        w = torch.randn(6, W, generator=g, dtype=torch.float64)
        b = torch.randn(6, generator=g, dtype=torch.float64)
        y, pool, _ = layer.conv(x, w, b, "silu", pool=torch.full((1, W - 1, 6), math.nan),
                                init=[False], nseqs=1, cu=torch.tensor([0, 11]), prompt=True)
        ref = torch.nn.functional.conv1d(x.t()[None], w[:, None], b, padding=W - 1, groups=6)
        ref = torch.nn.functional.silu(ref)[0, :, :11].t()
        np.testing.assert_allclose(y, ref.numpy(), rtol=1e-12, atol=1e-12)
        assert np.array_equal(pool[0], x[11 - (W - 1):].numpy())


def test_convolution_in_pieces_is_the_whole():
    g = torch.Generator().manual_seed(2)
    x = torch.randn(9, 5, generator=g, dtype=torch.float64)
    w = torch.randn(5, 4, generator=g, dtype=torch.float64)
    whole, end, _ = layer.conv(x, w, pool=torch.zeros(1, 3, 5), nseqs=1, cu=torch.tensor([0, 9]),
                               prompt=True)
    pool = torch.zeros(1, 3, 5, dtype=torch.float64)
    got = []
    for a, b in ((0, 1), (1, 2), (2, 7), (7, 9)):   # pieces shorter than the window too
        y, p, _ = layer.conv(x[a:b], w, pool=pool, nseqs=1, cu=torch.tensor([0, b - a]),
                             prompt=True)
        pool = torch.from_numpy(p)
        got.append(y)
    np.testing.assert_array_equal(np.concatenate(got), whole)
    np.testing.assert_array_equal(pool.numpy(), end)


def test_scan_with_a_constant_along_dstate_is_the_state_update(oracle_mod):
    """A[c, n] = A[c]: the C oracle's one-token update with one channel per head."""
    g = torch.Generator().manual_seed(3)
    batch, dim, N = 3, 8, 16
    state = torch.randn(4, dim, N, generator=g)
    x = torch.randn(batch, dim, generator=g).bfloat16()
    z = torch.randn(batch, dim, generator=g).bfloat16()
    dt = torch.randn(batch, dim, generator=g)
    B = torch.randn(batch, 2, N, generator=g).bfloat16()
    C = torch.randn(batch, 2, N, generator=g).bfloat16()
    A, D, bias = -torch.rand(dim, generator=g), torch.rand(dim, generator=g), torch.randn(dim, generator=g)
    slots = torch.tensor([2, 0, -1])
    y, _, pool, _, written = layer.scan(x, dt, A[:, None].expand(dim, N), B, C, D=D, z=z,
                                        dt_bias=bias, softplus=True, pool=state, nseqs=batch,
                                        src=slots[:, None])
    s2 = state.clone().reshape(4, dim, 1, N).contiguous()
    ref = oracle_mod.ssu_update(s2, x[:, :, None], dt, A, B, C, D=D, z=z[:, :, None], dt_bias=bias,
                                dt_softplus=True, state_batch_indices=slots)
    np.testing.assert_allclose(y, ref.reshape(batch, dim).numpy(), rtol=1e-10, atol=1e-12)
    assert written == {0, 2}
    np.testing.assert_allclose(pool, s2.reshape(4, dim, N).double().numpy(), rtol=1e-6, atol=1e-7)


def test_scan_of_a_constant_input_is_a_geometric_sum():
    T, A, d = 40, -0.7, 0.3
    x, dt = torch.ones(T, 1), torch.full((T, 1), d)
    one = torch.ones(T, 1, 1)
    y, bound, pool, _, _ = layer.scan(x, dt, torch.tensor([[A]]), one, one, pool=torch.ones(1, 1, 1),
                                      nseqs=1, cu=torch.tensor([0, T]), prompt=True)
    a = math.exp(float(torch.tensor(A)) * float(torch.tensor(d)))
    b = float(torch.tensor(d))
    want = [a ** (t + 1) + b * (1 - a ** (t + 1)) / (1 - a) for t in range(T)]
    np.testing.assert_allclose(y[:, 0], want, rtol=1e-12)
    assert pool[0, 0, 0] == y[-1, 0]
    assert (bound > 0).all() and (bound < 1e-3).all()


def test_the_error_bound_holds_for_fp32():
    """The scan carried out in numpy's fp32 stays inside the oracle's bound."""
    g = np.random.default_rng(5)
    T, dim, N = 300, 4, 16
    x, dt = g.normal(size=(T, dim)), g.normal(size=(T, dim)) * 0.5 - 2.0
    A = -np.arange(1, N + 1) * g.uniform(0.5, 1.5, (dim, N))
    B, C = g.normal(size=(T, N)), g.normal(size=(T, N))
    t32 = [torch.from_numpy(v.astype(np.float32)) for v in (x, dt, A, B, C)]
    y, bound, _, _, _ = layer.scan(*t32, softplus=True, nseqs=1, cu=torch.tensor([0, T]),
                                   prompt=True)
    h = np.zeros((dim, N), np.float32)
    for t in range(T):
        d = np.logaddexp(np.float32(0), t32[1].numpy()[t])
        h = np.exp(t32[2].numpy() * d[:, None]) * h + (d * t32[0].numpy()[t])[:, None] * t32[3].numpy()[t]
        v = (h * t32[4].numpy()[t]).sum(-1)
        assert v.dtype == np.float32
        assert (np.abs(v - y[t]) <= bound[t]).all()


def test_sequences_rules():
    """Empty sequences are left out, ranges clamped, a pad read slot writes nothing."""
    got = list(layer.sequences(7, 5, nseqs=4, cu=torch.tensor([0, 0, 3, 4, 9]),
                               src=torch.tensor([1, 2, -1, 4]), prompt=True))
    assert got == [(1, 0, 3, 2, [None, None, 2]), (2, 3, 1, None, [None]),
                   (3, 4, 3, 4, [None, None, 4])]
    table = torch.tensor([[0, 1], [2, 9], [3, 4]])
    got = list(layer.sequences(6, 5, nseqs=3, steps=2, accepted=torch.tensor([2, 1, 3]), src=table))
    assert got == [(0, 0, 2, 1, [0, 1]), (1, 2, 2, 2, [2, None]), (2, 4, 2, None, [None, None])]


def test_compaction_keeps_order_and_fills_the_front():
    table, m, moves = layer.compact([[9, -1, 2], [7, 2, 0]], 10)
    assert (m, moves) == (4, {7: 1, 9: 3})
    assert table.tolist() == [[3, -1, 2], [1, 2, 0]]


@pytest.mark.parametrize("seed", range(4))
def test_compaction_is_a_bijection_onto_the_front(seed):
    g = np.random.default_rng(seed)
    slots = int(g.integers(1, 60))
    t = g.integers(-2, slots + 3, size=int(g.integers(0, 50)))
    new, m, moves = layer.compact(t, slots)
    live = {v for v in t.tolist() if 0 <= v < slots}
    assert {n for o, n in zip(t.tolist(), new.tolist()) if o in live} == set(range(m))
    assert all(n < m <= o for o, n in moves.items())
