"""Pins of the oracle of linear attention, verification, maps and slot assignment
(oracle/serving.py)."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from oracle import serving

F64 = torch.float64


def test_linear_attention_is_its_quadratic_form():
    """o_t = scale sum over s <= t of exp(ld_{s+1} + .. + ld_t) (q_t . k_s) v_s."""
    g = torch.Generator().manual_seed(1)
    T, H, G, dk, dv = 9, 4, 2, 5, 3
    q, k = (torch.randn(T, G, dk, generator=g, dtype=F64) for _ in range(2))
    v = torch.randn(T, H, dv, generator=g, dtype=F64)
    ld = -torch.rand(T, H, generator=g, dtype=F64)
    o = serving.linattn(q, k, v, ld, 0.5, nseqs=1, cu=torch.tensor([0, T]), prompt=True)[0]
    for h in range(H):
        a = ld[:, h].cumsum(0)
        w = torch.exp(a[:, None] - a[None]).tril() * (q[:, h // 2] @ k[:, h // 2].t())
        np.testing.assert_allclose(o[:, h], (0.5 * w @ v[:, h]).numpy(), rtol=1e-12, atol=1e-13)


def test_linear_attention_in_pieces_is_the_whole():
    g = torch.Generator().manual_seed(2)
    T, H, d = 7, 2, 4
    q, k, v = (torch.randn(T, H, d, generator=g, dtype=F64) for _ in range(3))
    ld = -torch.rand(H, generator=g, dtype=F64)
    whole, _, _, end, _, _ = serving.linattn(q, k, v, ld, pool=torch.zeros(1, H, d, d), nseqs=1,
                                             cu=torch.tensor([0, T]), prompt=True)
    pool, got = torch.zeros(1, H, d, d, dtype=F64), []
    for a, b in ((0, 1), (1, 5), (5, 7)):
        o, _, _, p, _, _ = serving.linattn(q[a:b], k[a:b], v[a:b], ld, pool=pool, nseqs=1,
                                           cu=torch.tensor([0, b - a]), prompt=True)
        pool = torch.from_numpy(p)
        got.append(o)
    np.testing.assert_allclose(np.concatenate(got), whole, rtol=1e-12, atol=1e-13)
    np.testing.assert_allclose(pool.numpy(), end, rtol=1e-12, atol=1e-13)


def test_the_bound_covers_fp32_arithmetic():
    g = torch.Generator().manual_seed(3)
    T, H, d = 200, 2, 8
    q, k, v = (torch.randn(T, H, d, generator=g) for _ in range(3))
    ld = -torch.rand(T, H, generator=g) / 8
    o, bound, *_ = serving.linattn(q, k, v, ld, 0.3, nseqs=1, cu=torch.tensor([0, T]), prompt=True)
    S = torch.zeros(H, d, d)
    for t in range(T):
        S = torch.exp(ld[t])[:, None, None] * S + v[t][:, :, None] * k[t][:, None]
        got = 0.3 * (S * q[t][:, None]).sum(-1)
        assert (np.abs(got.double().numpy() - o[t]) <= bound[t]).all()


def test_a_draft_is_taken_with_the_ratio_and_the_rest_is_drawn():
    p = torch.tensor([[0.5, 0.25, 0.25], [0.0, 0.0, 1.0]])
    q = torch.tensor([[[0.25, 0.5, 0.25]]])
    # draft 1: taken while u q < p, so for u < 1/2
    for u, want in ((0.49, [1, 2]), (0.5, [0, -1])):   # p - q is left of token 0 alone
        tokens, n = serving.verify(p, torch.tensor([[1]]), torch.tensor([[u, 0.999]]), q)
        assert tokens == [want] and n == [2 - (want[1] < 0)]
    # a certain draft: what is left is p without it
    tokens, n = serving.verify(p, torch.tensor([[1]]), torch.tensor([[0.3, 0.7]]))
    assert tokens == [[2, -1]] and n == [1]
    tokens, n = serving.verify(p, torch.tensor([[1]]), torch.tensor([[0.3, 0.6]]))
    assert tokens == [[0, -1]] and n == [1]


def test_tokens_are_distributed_as_the_targets():
    """Over a grid of random numbers, the first token comes up as often as the target
    says, whatever the drafts came from."""
    p = torch.tensor([[0.5, 0.125, 0.375], [1.0, 0.0, 0.0]])
    q = torch.tensor([0.25, 0.5, 0.25])
    N, hits = 64, np.zeros(3)
    grid = (np.arange(N) + 0.5) / N
    for d in range(3):
        for a in grid:
            us = torch.tensor([[a, b] for b in grid], dtype=torch.float32)
            tokens, _ = serving.verify(p.repeat(N, 1), torch.full((N, 1), d), us,
                                       q.expand(N, 1, 3))
            for t in tokens:
                hits[t[0]] += float(q[d]) / N / N
    np.testing.assert_allclose(hits, p[0].numpy(), atol=1.0 / N)


def test_nothing_left_and_greedy():
    p = torch.tensor([[0.5, 0.5], [0.25, 0.75]])
    tokens, n = serving.verify(p, torch.tensor([[5]]), torch.tensor([[0.0, 0.6]]), p[None, :1])
    assert tokens == [[1, -1]] and n == [1]          # a draft outside; p - p is nothing: p itself
    tokens, n = serving.verify(torch.zeros(1, 3), torch.zeros(1, 0, dtype=torch.int64),
                               torch.tensor([[0.5]]))
    assert tokens == [[-1]] and n == [1]
    tokens, n = serving.verify(p, torch.tensor([[0]]), torch.tensor([[0.0, 0.0]]),
                               greedy=[True])
    assert tokens == [[0, 1]] and n == [2]           # the lowest of equal ones


def test_maps_by_hand():
    got = serving.prompt_maps([5, 0, 3], 4, 10, context=[0, 2, 3], most=8)
    assert got == [[0, 5, 5, 8],
                   [0, 4, 5, 5, 6, 8, 8, 8, 8],     # 3 tokens before: the first one closes a chunk
                   [0, 0, 1, 2, 2, 2, 2, 2], [1, 2, 4], [False, True, True], [5],
                   [0] * 5 + [2] * 3 + [-1, -1], [0, 1, 2, 3, 4, 3, 4, 5, -1, -1]]
    assert serving.prompt_maps([], 4, 2)[:3] == [[0], [0], []]


def test_assignment_by_hand():
    out, fresh, missing = serving.assign([[3, -1], [0, 5], [9, 1]], [2, 1, 2], 4)
    assert out == [[3, 2], [0, -1], [-1, 1]] and fresh == [[-1, 2], [-1, -1], [-1, -1]]
    assert missing == 1
    assert serving.assign([[0, 7]], [2], 4, pad=0)[0] == [[1, 2]]


@pytest.mark.parametrize("seed", range(3))
def test_assignment_gives_each_slot_once(seed):
    r = np.random.default_rng(seed)
    ids = r.permutation(30)
    table = [[int(ids[i * 3 + t]) if r.random() < 0.5 else -1 for t in range(3)] for i in range(8)]
    counts = [int(r.integers(0, 4)) for _ in range(8)]
    out, fresh, missing = serving.assign(table, counts, 26)
    flat = [v for row in out for v in row if v >= 0]
    assert len(flat) == len(set(flat)) and max(flat) < 26
    assert sum(v >= 0 for v in flat) + missing == sum(counts)
