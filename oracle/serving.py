"""Plain oracle of linear attention with a decay for each head, the verification
of drafted tokens, the maps of a batch and the assignment of slots.

TEST INFRASTRUCTURE ONLY, like the rest of this package; it shares no code with
the CUDA library.  Everything is written from the definitions:

    linear attention   S <- exp(ld) S + v k^T;  o = scale S q   (row by row, fp64)
    verification       draft by draft, then one draw from what is left of a row
    maps               sequence by sequence, chunk by chunk, row by row
    assignment         entry by entry, the lowest slot that is free

``linattn`` also returns what fp32 arithmetic may be off by: a step multiplies
what was carried by a decay with a relative error of at most eps (1 + |ld|) and
adds a product with one of at most eps, so the error e of S follows e <- exp(ld)
e + eps ((1 + |ld|) exp(ld) m + |v k|) with m the same recurrence over
magnitudes.  Where m leaves fp32's range there is no bound (inf).

Pins: tests/test_oracle_serving.py.
"""
from __future__ import annotations

import math
from fractions import Fraction

import numpy as np

from .layer import F32_MAX, _f64, _ints, sequences


@np.errstate(over="ignore", invalid="ignore")
def linattn(q, k, v, log_decay=None, scale=1.0, pool=None, init=None, write=True, eps=2.0 ** -20,
            **seqs):
    """(o [rows, H, dv], NaN where no sequence has the row; its error bound; the
    magnitude behind it; the pool; its error bound; the slots written)."""
    q, k, v, ld = _f64(q), _f64(k), _f64(v), _f64(log_decay)
    rows, H, dv = v.shape
    dk = q.shape[2]
    group = np.arange(H) // (H // q.shape[1])
    before = np.zeros((0, H, dv, dk)) if pool is None else _f64(pool)
    after, off = before.copy(), np.zeros_like(before)
    o, bound, size = np.full((rows, H, dv), np.nan), np.zeros((rows, H, dv)), np.zeros((rows, H, dv))
    written = set()
    for s, r0, n, read, to in sequences(rows, len(before), **seqs):
        S = np.zeros((H, dv, dk))
        if read is not None and (init is None or bool(init[s])):
            S = before[read].copy()
        m, e = np.abs(S), np.zeros_like(S)
        for t in range(n):
            r = r0 + t
            l = np.zeros(H) if ld is None else ld if ld.ndim == 1 else ld[r]
            d = np.exp(l)[:, None, None]
            # a decay of zero forgets, whatever its logarithm
            slack = np.where(d > 0, 1.0 + np.abs(l)[:, None, None], 1.0) * d
            new = v[r][:, :, None] * k[r][group][:, None, :]
            e = d * e + eps * (slack * m + np.abs(new))
            m = d * m + np.abs(new)
            S = d * S + new
            e = np.where(m > F32_MAX, np.inf, e)
            qt = q[r][group][:, None, :]
            o[r] = scale * (S * qt).sum(-1)
            size[r] = abs(scale) * (m * np.abs(qt)).sum(-1)
            bound[r] = abs(scale) * (e * np.abs(qt)).sum(-1) + eps * size[r]
            bound[r][size[r] > F32_MAX] = np.inf
            if write and to[t] is not None:
                after[to[t]], off[to[t]] = S, e
                written.add(to[t])
    return o, bound, size, after, off, written


def _best(row):
    """The largest value's lowest place; NaN is never it (-1: there is nothing else)."""
    numbers = np.flatnonzero(~np.isnan(row))
    return int(numbers[row[numbers].argmax()]) if len(numbers) else -1


def verify(p, drafts, u, q=None, cu=None, greedy=None):
    """(tokens [S, K + 1], how many of them) as lists of ints."""
    p = p.detach().cpu().float().numpy()
    drafts, u = _ints(drafts), u.detach().cpu().numpy().astype(np.float32)
    q = None if q is None else q.detach().cpu().float().numpy()
    S, K = drafts.shape
    V = p.shape[1]
    starts = [s * (K + 1) for s in range(S + 1)] if cu is None else [int(c) for c in cu]
    out, counts = [], []
    for s in range(S):
        r0, r1 = max(0, min(starts[s], len(p))), max(0, min(starts[s + 1], len(p)))
        n = min(r1 - r0 - 1, K)
        if n < 0:
            out.append([-1] * (K + 1))
            counts.append(0)
            continue
        taken, token = [], None
        while token is None:
            j = len(taken)
            row = p[r0 + j]
            d = int(drafts[s, j]) if j < n else -1
            inside = 0 <= d < V
            if greedy is not None and bool(greedy[s]):
                best = _best(row)
                if j < n and best == d and inside:
                    taken.append(d)
                else:
                    token = best
                continue
            # products of two fp32 numbers are whole in fp64
            at = 1.0 if q is None or not inside else float(q[s, j, d])
            if j < n and inside and float(u[s, j]) * at < float(row[d]):
                taken.append(d)
                continue
            left = row.copy()
            if j < n and q is not None:
                left = row - q[s, j]
            elif j < n and inside:
                left[d] = 0.0
            for rest in (left, row):
                with np.errstate(invalid="ignore"):
                    w = np.where(rest > 0, np.minimum(rest, np.float32(1.0)), 0.0).astype(np.float64)
                w = [int(x) for x in np.rint(w * 2.0 ** 44)]
                total = sum(w)
                if total:
                    break
            token = -1
            if total:
                draw = float(u[s, K]) if u[s, K] == u[s, K] else 0.0
                mark = min(math.floor(Fraction(min(max(draw, 0.0), 1.0)) * total), total - 1)
                run = 0
                for i, x in enumerate(w):
                    run += x
                    if run > mark:
                        token = i
                        break
        counts.append(len(taken) + 1)
        out.append((taken + [token] + [-1] * (K + 1))[:K + 1])
    return out, counts


def prompt_maps(lens, chunk, rows, context=None, most=None):
    """The eight maps as lists, in the order of the call's results."""
    lens = [max(int(n), 0) for n in lens]
    S = len(lens)
    context = [0] * S if context is None else [max(int(c), 0) for c in context]
    if most is None:
        most = rows // chunk + (2 if any(context) else 1) * S
    cu, starts, owner, last = [0], [], [], []
    row_seq, row_pos = [-1] * rows, [-1] * rows
    for s in range(S):
        b, e = cu[-1], min(cu[-1] + lens[s], rows)
        cu.append(e)
        at, first = b, True
        while first or at < e:
            starts.append(at)
            owner.append(s)
            room = chunk - (context[s] + at - b) % chunk   # to the end of the chunk of `at`
            at, first = min(at + room, e), False
        last.append(len(starts) - 1)
        for r in range(b, e):
            row_seq[r], row_pos[r] = s, context[s] + r - b
    used = len(starts)
    starts += [cu[-1]] * (most + 1 - used)
    owner += [max(S - 1, 0)] * (most - used)
    return [cu, starts, owner, last, [c > 0 for c in context], [used], row_seq, row_pos]


def assign(table, counts, slots, pad=-1):
    """(new table, slots newly given, entries that got none)."""
    table = [[int(v) for v in row] for row in table]
    keep = [[t < int(n) and v != pad and 0 <= v < slots for t, v in enumerate(row)]
            for row, n in zip(table, counts)]
    held = {v for row, k in zip(table, keep) for v, stays in zip(row, k) if stays} | {pad}
    free = [i for i in range(slots) if i not in held]
    out, fresh, missing = [], [], 0
    for row, k, n in zip(table, keep, counts):
        new, given = [], []
        for t, v in enumerate(row):
            got = pad
            if t < int(n) and not k[t]:
                if free:
                    got = free.pop(0)
                else:
                    missing += 1
            new.append(v if k[t] else got)
            given.append(got)
        out.append(new)
        fresh.append(given)
    return out, fresh, missing
