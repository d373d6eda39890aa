"""Plain fp64 oracle of the calls around the state update: the causal
convolution, the selective scan with a full A, and the moves of slots.

TEST INFRASTRUCTURE ONLY: like the rest of this package it is imported by the
tests and the smoke run; no product code uses it.  It shares no code with the
CUDA library.  Everything is written row by row from the definitions:

    convolution   y[t, c] = act(bias[c] + sum_j w[c, j] xs[t - (W - 1) + j, c]),
                  xs the slot's W - 1 rows followed by the sequence's
    scan          dt' = softplus(dt + bias);  h <- exp(A dt') h + dt' x B;
                  y = (h . C + D x) silu(z)

``scan`` also returns, for each value, a bound on what fp32 arithmetic may be
off by: a step multiplies what was carried by an exponential with a relative
error of at most EPS (1 + |A dt'|) and adds a product with one of at most EPS,
so the error e of h follows e <- exp(A dt') e + EPS ((1 + |A dt'|) exp(A dt') m
+ |dt' x B|) with m the same recurrence over magnitudes.  Where m or the exponential leaves fp32's
range there is no bound (inf).

Pins: tests/test_oracle_layer.py.
"""
from __future__ import annotations

import numpy as np

F32_MAX = 2.0 ** 127
EPS = 2.0 ** -20   # a few fp32 roundings, a fast exponential and a softplus


def _f64(t):
    if t is None:
        return None
    if hasattr(t, "detach"):
        import torch
        return t.detach().cpu().to(torch.float64).numpy()
    return np.asarray(t, dtype=np.float64)


def _ints(t):
    return None if t is None else np.asarray(t.detach().cpu().numpy(), dtype=np.int64)


def silu(v):
    with np.errstate(over="ignore"):
        return v / (1.0 + np.exp(-v))


def sequences(rows, slots, *, nseqs, cu=None, steps=1, accepted=None, src=None, dst=None, pad=-1,
              prompt=False):
    """(first row, length, read slot or None, write slot or None of each row) of
    every sequence that has rows.  ``prompt``: src and dst are one slot per
    sequence and only the last row writes; else they are [S, T] tables, or flat
    ones whose entry (s, t) is s + t."""
    cu, accepted, src, dst = _ints(cu), _ints(accepted), _ints(src), _ints(dst)

    def entry(t, s, p):
        if t is None:
            return s
        if t.ndim == 2:
            return int(t[s, p]) if 0 <= p < t.shape[1] else None
        return int(t[s + p]) if p >= 0 and s + p < len(t) else None

    def valid(v):
        return v if v is not None and v != pad and 0 <= v < slots else None

    for s in range(nseqs):
        b, e = (int(cu[s]), int(cu[s + 1])) if cu is not None else (s * steps, (s + 1) * steps)
        b, e = max(b, 0), min(e, rows)
        if e <= b:
            continue
        if prompt:
            read = valid(s if src is None else int(src[s]))
            to = valid(read if dst is None else int(dst[s]))
            write = [None] * (e - b - 1) + [to]
        else:
            read = valid(entry(src, s, 0 if accepted is None else int(accepted[s]) - 1))
            table = dst if dst is not None else src
            write = [valid(entry(table, s, t)) for t in range(e - b)]
        if read is None:
            write = [None] * (e - b)
        yield s, b, e - b, read, write


def conv(x, weight, bias=None, act=None, pool=None, init=None, write=True, **seqs):
    """(y [rows, C] with NaN where no sequence has the row, the pool, the sum of
    magnitudes behind every y)."""
    x, w, b = _f64(x), _f64(weight), _f64(bias)
    rows, C = x.shape
    W = w.shape[1]
    before = np.zeros((0, W - 1, C)) if pool is None else _f64(pool)
    after = before.copy()
    y, mag = np.full((rows, C), np.nan), np.zeros((rows, C))
    for s, r0, n, read, to in sequences(rows, len(before), **seqs):
        old = np.zeros((W - 1, C))
        if read is not None and (init is None or bool(init[s])):
            old = before[read]
        line = np.concatenate([old, x[r0:r0 + n]])
        for t in range(n):
            v = np.zeros(C) if b is None else b.copy()
            m = np.abs(v)
            for j in range(W):
                v = v + w[:, j] * line[t + j]
                m = m + np.abs(w[:, j] * line[t + j])
            y[r0 + t], mag[r0 + t] = (silu(v) if act == "silu" else v), m
            if write and to[t] is not None:
                after[to[t]] = line[t + 1:t + W]
    return y, after, mag


@np.errstate(over="ignore", invalid="ignore")
def scan(x, dt, A, B, C, D=None, z=None, dt_bias=None, softplus=False, pool=None, init=None,
         write=True, **seqs):
    """(y [rows, dim], NaN where no sequence has the row; its error bound; the
    pool; its error bound; the slots written)."""
    x, dt, A, B, C = _f64(x), _f64(dt), _f64(A), _f64(B), _f64(C)
    D, z, dt_bias = _f64(D), _f64(z), _f64(dt_bias)
    rows, dim = x.shape
    if B.ndim == 2:
        B, C = B[:, None], C[:, None]
    N = A.shape[1]
    group = np.arange(dim) // (dim // B.shape[1])
    before = np.zeros((0, dim, N)) if pool is None else _f64(pool)
    after, off = before.copy(), np.zeros_like(before)
    y, bound = np.full((rows, dim), np.nan), np.zeros((rows, dim))
    written = set()
    for s, r0, n, read, to in sequences(rows, len(before), **seqs):
        h = np.zeros((dim, N))
        if read is not None and (init is None or bool(init[s])):
            h = before[read]
        m, e = np.abs(h), np.zeros((dim, N))
        for t in range(n):
            r = r0 + t
            d = dt[r] + (0.0 if dt_bias is None else dt_bias)
            if softplus:
                d = np.logaddexp(0.0, d)
            arg = A * d[:, None]
            dA = np.exp(arg)
            new = (d * x[r])[:, None] * B[r][group]
            e = dA * e + EPS * ((1.0 + np.abs(arg)) * dA * m + np.abs(new))
            m = dA * m + np.abs(new)
            h = dA * h + new
            e = np.where((m > F32_MAX) | (dA > F32_MAX), np.inf, e)
            Ct = C[r][group]
            v = (h * Ct).sum(-1)
            size = (m * np.abs(Ct)).sum(-1)
            err = np.where(size > F32_MAX, np.inf, (e * np.abs(Ct)).sum(-1) + EPS * size)
            if D is not None:
                v, err = v + D * x[r], err + EPS * np.abs(D * x[r])
            if z is not None:
                g = silu(z[r])
                err = err * np.abs(g) + EPS * (1.0 + np.abs(z[r])) * np.abs(v * g)
                v = v * g
            y[r], bound[r] = v, err + EPS * np.abs(v)
            if write and to[t] is not None:
                after[to[t]], off[to[t]] = h, e
                written.add(to[t])
    return y, bound, after, off, written


def compact(table, slots, pad=-1):
    """(new table, live slots, {old slot: new slot} of those that move)."""
    flat = [int(v) for v in np.asarray(table).reshape(-1)]
    live = sorted({v for v in flat if v != pad and 0 <= v < slots})
    m = len(live)
    free = [i for i in range(m) if i not in set(live)]
    moves = dict(zip([v for v in live if v >= m], free))
    return np.array([moves.get(v, v) for v in flat]).reshape(np.asarray(table).shape), m, moves
