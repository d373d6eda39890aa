"""GPU parity of the layer calls where values, memory and streams come to their
edges: infinite and huge A, sequences split over a cluster in every form,
operands that overlap, results on another stream than the current one.

Tolerances as in test_layer_gpu.py: the oracle's running bound for the scan, and
half a unit in the last place of what is stored in 16 bits.
"""
from __future__ import annotations

import math

import pytest
import torch

import mamba2_ssm_decode_gb300 as ssu
from oracle import layer

from .test_layer_gpu import (BF16, DEV, F16, F32, OPERANDS, _built, conv_check, conv_inputs,  # noqa: F401
                             cu_of, cuda, gen, same_bits, scan_check, scan_inputs, scan_prompt)

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# values at the edges of their range
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("lens", [[1, 2, 7, 16, 33, 0, 61], [401], [1203]])
@pytest.mark.parametrize("io", [BF16, F32])
@pytest.mark.parametrize("N", [16, 32, 64, 128, 256])
def test_scan_columns_that_forget_at_once(N, io, lens):
    """A = -inf: exp(A dt') is 0 for every dt' > 0, whatever the sequence's length.
    The oracle has -1e30 there, whose exponentials are 0 as well."""
    S, dim = len(lens), 24
    i = scan_inputs(sum(lens), dim, N, S + 1, 1, io, F32, F32, seed=N)
    forget = torch.rand(dim, N, generator=gen(1)) < 0.3
    i["A"][forget] = -1e30
    slots = torch.randperm(S + 1, generator=gen(2))[:S]
    ref = dict(i, A=i["A"].clone())
    i["A"][forget] = -math.inf
    got, pool = scan_prompt(i, lens, slots)
    scan_check(ref, got, pool, "prompts", pool=i["pool"], nseqs=S, cu=cu_of(lens), src=slots, prompt=True)
    # ... and one row at a time
    d = dict(zip(OPERANDS, cuda(i, *OPERANDS)))
    pool, cu = i["pool"].to(DEV), cu_of([min(n, 5) for n in lens])
    T = int(cu[-1])
    d = {k: v[:T] if k in ("x", "dt", "z", "B", "C") else v for k, v in d.items()}
    ref.update({k: ref[k][:T] for k in ("x", "dt", "z", "B", "C")})
    table = slots[:, None].repeat(1, 5)
    got = ssu.scan_update_varlen(pool, d["x"], d["dt"], d["A"], d["B"], d["C"], D=d["D"], z=d["z"],
                                 dt_bias=d["dt_bias"], dt_softplus=True, cu_seqlens=cu.to(DEV),
                                 state_batch_indices=table.int().to(DEV))
    scan_check(ref, got, pool, "rows", pool=i["pool"], nseqs=S, cu=cu, src=table)


@pytest.mark.parametrize("lens", [[1, 7, 16, 33], [401]])
@pytest.mark.parametrize("N", [16, 64, 256])
def test_scan_huge_rates_and_steps_of_zero(N, lens):
    """|A| up to the largest fp32 (A log2 e is beyond it) with steps of exactly 0,
    which change nothing; a NaN in A stays in its column."""
    S, dim, T = len(lens), 24, sum(lens)
    i = scan_inputs(T, dim, N, S, 1, BF16, F32, F32, seed=N)
    i["A"][torch.rand(dim, N, generator=gen(1)) < 0.3] = -3.4e38
    i["dt"] = i["dt"].abs() * 0.1 * (torch.rand(T, dim, generator=gen(2)) < 0.5)
    i["dt_bias"] = None
    got, pool = scan_prompt(i, lens, softplus=False)
    scan_check(i, got, pool, "prompts", softplus=False, pool=i["pool"], nseqs=S, cu=cu_of(lens), prompt=True)
    d = dict(zip(OPERANDS, cuda(i, *OPERANDS)))
    rows = [d[k][:S] if k != "A" else d[k] for k in ("x", "dt", "A", "B", "C")]
    pool = i["pool"].to(DEV)
    got = ssu.scan_update(pool, *rows, D=d["D"], z=d["z"][:S])
    i.update({k: i[k][:S] for k in ("x", "dt", "z", "B", "C")})
    scan_check(i, got, pool, "rows", softplus=False, pool=i["pool"], nseqs=S)
    d["A"][3, 5] = math.nan
    pool = i["pool"].to(DEV)
    got = ssu.scan_update(pool, *rows, D=d["D"], z=d["z"][:S])
    bad = torch.isnan(pool)
    assert bool(bad[:, 3, 5].all()) and int(bad.sum()) == S and bool(torch.isnan(got[:, 3]).all())
    held = i["pool"].to(DEV)
    got = ssu.scan_fwd_varlen(*rows, cu_of([S]).to(DEV), D=d["D"], z=d["z"][:S], state=held)
    bad = torch.isnan(held)
    assert bool(bad[0, 3, 5]) and int(bad.sum()) == 1 and bool(torch.isnan(got[:, 3]).all())


@pytest.mark.parametrize("N", [16, 32, 64, 128, 256])
def test_scan_split_states_at_the_ends_of_the_range(N):
    """A long prompt split into pieces whose decay alone leaves fp32's range where the
    state does not: from 0, from tiny states that grow and from large ones that decay."""
    T, dim = 1203, 24
    i = scan_inputs(T, dim, N, 1, 1, BF16, F32, F32, seed=N)
    i["x"].zero_()
    i["dt"].zero_()
    i["dt_bias"] = None
    for c in range(dim):   # 20 steps of 5: a sum of 100 nats inside one piece for most channels
        i["dt"][30 + 48 * c:50 + 48 * c, c] = 5.0
        i["pool"][0, c] *= (0.0, 1e-35, 1e30)[c % 3]
        i["A"][c] = (1.0, 1.0, -1.0)[c % 3] * (0.9 + 0.1 * torch.rand(N, generator=gen(c)))
    got, pool = scan_prompt(i, [T], softplus=False)
    has = scan_check(i, got, pool, "pieces", softplus=False, pool=i["pool"], nseqs=1, cu=cu_of([T]),
                     prompt=True)
    assert has.all() and bool((pool[0, 0::3] == 0).all()) and bool((pool[0, 1::3] != 0).all())
    assert bool(torch.isfinite(pool).all()) and bool((pool[0, 2::3] != 0).all())


def test_scan_split_keeps_rows_of_zeros():
    """Leading rows of zeros under growing factors, then rows that count."""
    T, dim, N = 1203, 24, 16
    i = scan_inputs(T, dim, N, 1, 1, BF16, F32, F32, seed=2)
    i["x"][:-40] = 0.0
    i["A"], i["dt"], i["dt_bias"] = torch.rand(dim, N, generator=gen(1)), torch.full((T, dim), 2.0), None
    i["pool"].zero_()
    got, pool = scan_prompt(i, [T], softplus=False)
    assert bool(torch.isfinite(pool).all()) and bool((got[:-40] == 0).all())
    scan_check(i, got, pool, "zeros", softplus=False, pool=i["pool"], nseqs=1, cu=cu_of([T]), prompt=True)


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("name", ["x", "dt", "z", "B", "C"])
@pytest.mark.parametrize("lens,at", [([9, 21, 5], 17), ([700, 401, 333], 950), ([700, 401, 333], 1100)])
def test_scan_bad_values_stay_where_they_belong(lens, at, name, bad):
    """A NaN or an infinity in one row, whole sequences and split ones, the last row of
    one among them: earlier rows, other channels (groups for B and C) and other
    sequences keep their bits."""
    dim, N, G, S = 48, 16, 2, len(lens)
    i = scan_inputs(sum(lens), dim, N, S, G, BF16, F32, F32, seed=4)
    clean, held = scan_prompt(i, lens)
    i[name] = i[name].clone()
    c = 7
    if name in ("B", "C"):
        i[name][at, 1, 3] = bad
        touched = torch.arange(dim) >= dim // 2
    else:
        i[name][at, c] = bad
        touched = torch.arange(dim) == c
    got, pool = scan_prompt(i, lens)
    q = next(s for s in range(S) if sum(lens[:s + 1]) > at)
    end = sum(lens[:q + 1]) if name in ("x", "dt", "B") else at + 1   # z and C: that row alone
    hit = torch.zeros(got.shape, dtype=torch.bool)
    hit[at:end, touched] = True
    same_bits(got.cpu()[~hit], clean.cpu()[~hit])
    assert not torch.equal(got.cpu()[hit], clean.cpu()[hit])
    hit = torch.zeros(pool.shape, dtype=torch.bool)
    if name in ("x", "dt", "B"):
        hit[q, touched] = True
        assert not torch.equal(pool.cpu()[hit], held.cpu()[hit])
    same_bits(pool.cpu()[~hit], held.cpu()[~hit])


@pytest.mark.parametrize("C", [64, 37])
def test_conv_bad_values_stay_where_they_belong(C):
    """NaN in one element: its channel's next W rows of the same sequence, no others."""
    lens, at, W = [40, 90, 5], 127, 4
    i = conv_inputs(sum(lens), C, W, 3, seed=4)
    cu = cu_of(lens).to(DEV)
    x, w, b, held = cuda(i, "x", "weight", "bias", "pool")
    clean = ssu.conv_fwd_varlen(x, w, cu, bias=b, conv_state=held)
    x[at, 5] = math.nan
    pool = i["pool"].to(DEV)
    got = ssu.conv_fwd_varlen(x, w, cu, bias=b, conv_state=pool)
    bad = torch.isnan(got)
    assert bad.nonzero().tolist() == [[r, 5] for r in range(at, 130)]
    same_bits(got[~bad], clean[~bad])
    bad = torch.isnan(pool)
    assert bad.nonzero().tolist() == [[1, 0, 5]]
    same_bits(pool[~bad], held[~bad])


# ---------------------------------------------------------------------------
# sequences split over the CTAs of a cluster
# ---------------------------------------------------------------------------

# a mean of 505 rows and few channels select the split for every dstate; the
# cluster's 16 CTAs then take 16 pieces of some sequences, fewer of others, and
# one alone takes those of a few tiles
SPLIT = [900, 1, 0, 333, 1100, 700]


@pytest.mark.parametrize("io,dt,state", [(BF16, BF16, F32), (BF16, F32, BF16), (F16, F16, F16),
                                         (F16, F32, F32), (F32, F32, F32), (F32, F32, BF16)])
@pytest.mark.parametrize("N,dim,G", [(16, 160, 1), (16, 75, 3), (32, 72, 2), (64, 40, 4),
                                     (128, 24, 1), (256, 12, 3)])
def test_split_prompts(io, dt, state, N, dim, G):
    """Every type, dstate and number of groups; half the sequences are fresh, in slots
    that hold NaN."""
    S, T = len(SPLIT), sum(SPLIT)
    i = scan_inputs(T, dim, N, S + 2, G, io, dt, state, seed=N + dim)
    slots = torch.randperm(S + 2, generator=gen(1))[:S]
    init = torch.tensor([s % 2 == 1 for s in range(S)])
    clean = i["pool"].clone()
    for s in range(S):
        if not init[s] and SPLIT[s]:
            i["pool"][slots[s]] = math.nan
    got, pool = scan_prompt(i, SPLIT, slots, init)
    i["pool"] = clean
    scan_check(i, got, pool, "split", pool=clean, init=init, nseqs=S, cu=cu_of(SPLIT), src=slots,
               prompt=True)


@pytest.mark.parametrize("variant", ["no_pool", "no_z", "no_D", "no_bias", "raw_steps", "dst", "pads",
                                     "int64", "out_f32", "strided", "odd_strides", "two_d",
                                     "no_table", "gaps", "big_steps"])
@pytest.mark.parametrize("dim,N", [(48, 16), (29, 16), (24, 128)])
def test_split_prompt_variants(variant, dim, N):
    S, T = len(SPLIT), sum(SPLIT)
    i = scan_inputs(T, dim, N, S + 2, 1, seed=21)
    kw, softplus, cu = {}, True, cu_of(SPLIT)
    slots, init = torch.tensor([5, 0, 3, 1, 6, 2]), torch.tensor([True, False, True, True, False, True])
    if variant in ("no_z", "no_D", "no_bias"):
        i[{"no_z": "z", "no_D": "D", "no_bias": "dt_bias"}[variant]] = None
    if variant == "raw_steps":
        softplus, i["dt"], i["dt_bias"] = False, i["dt"].abs() * 0.1, i["dt_bias"].abs() * 0.01
    if variant == "big_steps":
        i["dt"] = (40.0 * torch.randn(T, dim, generator=gen(2))).to(BF16)
    if variant == "pads":
        slots = torch.tensor([5, -1, 3, 99, -1, 2])
    if variant == "gaps":
        cu = torch.tensor([3, 880, 880, 900, 1300, 2400, T - 4])
    if variant in ("strided", "odd_strides"):
        pad = 16 if variant == "strided" else 5
        for k in ("x", "z", "dt", "A"):
            i[k] = torch.cat([i[k], i[k][:, :pad]], 1)[:, :i[k].shape[1]]
        for k in ("B", "C"):
            i[k] = torch.cat([i[k], i[k][:, :, :pad]], 2)[:, :, :N]
    if variant == "two_d":
        i["B"], i["C"] = i["B"][:, 0], i["C"][:, 0]
    seqs = dict(nseqs=S, cu=cu, prompt=True)
    if variant == "no_pool":
        i["pool"] = None
    else:
        seqs.update(pool=i["pool"], init=init)
        kw["has_initial_state"] = init.to(DEV)
        idx = torch.int64 if variant == "int64" else torch.int32
        if variant != "no_table":
            seqs["src"] = slots
            kw["state_batch_indices"] = slots.to(idx).to(DEV)
        if variant == "dst":
            seqs["dst"] = torch.tensor([6, 4, 2, -1, 0, 7])
            kw["dst_state_batch_indices"] = seqs["dst"].int().to(DEV)
    if variant == "out_f32":
        kw["out_dtype"] = F32
    else:
        kw["out"] = torch.full((T, dim), 7.0, dtype=BF16, device=DEV)
    d = dict(zip(OPERANDS, cuda(i, *OPERANDS)))
    pool = None if i["pool"] is None else i["pool"].to(DEV)
    meta = torch.int64 if variant == "int64" else torch.int32
    got = ssu.scan_fwd_varlen(d["x"], d["dt"], d["A"], d["B"], d["C"], cu.to(meta).to(DEV), D=d["D"],
                              z=d["z"], dt_bias=d["dt_bias"], dt_softplus=softplus, state=pool, **kw)
    scan_check(i, got, pool, variant, softplus=softplus, **seqs)
    if variant == "gaps":   # rows of no sequence
        assert bool((got[:3] == 7.0).all()) and bool((got[-4:] == 7.0).all())


# ---------------------------------------------------------------------------
# streams
# ---------------------------------------------------------------------------

def _stream_calls():
    """name: (inputs, call(inputs, stream) -> results; the pools are results too)."""
    T, S, dim, N = 70, 3, 64, 16
    c, i = conv_inputs(T, dim, 4, 8, seed=1), scan_inputs(T, dim, N, 8, seed=1)
    d = {**{k: v for k, v in i.items() if k != "pool"}, "state": i["pool"], "conv": c["pool"],
         "w": c["weight"], "cb": c["bias"], "cu": cu_of([40, 5, 25]),
         "table": torch.tensor([6, 0, 3], dtype=torch.int32)}
    scan = lambda d, n: ([d[k][:n] if k != "A" else d[k] for k in ("x", "dt", "A", "B", "C")],  # noqa: E731
                         dict(D=d["D"], z=d["z"][:n], dt_bias=d["dt_bias"], dt_softplus=True,
                              state_batch_indices=d["table"]))

    def scan_call(f, n, pool_first, **extra):
        def call(d, stream):
            args, kw = scan(d, n)
            if pool_first:
                return f(d["state"], *args, **kw, **{k: d[v] for k, v in extra.items()}, stream=stream)
            return f(*args, d["cu"], state=d["state"], **kw, stream=stream)
        return call

    pools = lambda d: [d["state"], d["conv"]]  # noqa: E731
    return d, {
        "conv_update": lambda d, s: ssu.conv_update(d["conv"], d["x"][:S], d["w"], bias=d["cb"],
                                                    state_batch_indices=d["table"], stream=s),
        "conv_update_varlen": lambda d, s: ssu.conv_update_varlen(
            d["conv"], d["x"], d["w"], bias=d["cb"], cu_seqlens=d["cu"],
            state_batch_indices=d["table"], stream=s),
        "conv_fwd_varlen": lambda d, s: ssu.conv_fwd_varlen(
            d["x"], d["w"], d["cu"], bias=d["cb"], conv_state=d["conv"],
            state_batch_indices=d["table"], stream=s),
        "scan_update": scan_call(ssu.scan_update, S, True),
        "scan_update_varlen": scan_call(ssu.scan_update_varlen, T, True, cu_seqlens="cu"),
        "scan_fwd_varlen": scan_call(ssu.scan_fwd_varlen, T, False),
        "slots_copy": lambda d, s: ssu.slots_copy(pools(d), d["table"][:2], d["table"][1:], stream=s),
        "slots_clear": lambda d, s: ssu.slots_clear(pools(d), d["table"], stream=s),
        "slots_compact": lambda d, s: ssu.slots_compact(pools(d), d["table"], stream=s),
        "slots_compact in place": lambda d, s: ssu.slots_compact(pools(d), d["table"], out=d["table"],
                                                                 stream=s)}


@pytest.mark.parametrize("how", ["argument", "current"])
@pytest.mark.parametrize("name", list(_stream_calls()[1]))
def test_calls_follow_the_work_of_their_stream(name, how):
    """The inputs get their values on a side stream, behind work of some 10 ms; nothing
    between that and the call waits for the GPU.  The call, with `stream=` while another
    stream is current or with the side stream current, sees those values."""
    d, calls = _stream_calls()
    call = calls[name]
    flat = lambda r: [] if r is None else list(r) if isinstance(r, tuple) else [r]  # noqa: E731
    late = {k: v.to(DEV) for k, v in d.items()}
    want_in = {k: v.clone() for k, v in late.items()}
    want = flat(call(want_in, None)) + [want_in["state"], want_in["conv"]]
    early = {k: torch.zeros_like(v) for k, v in late.items()}
    early["table"].fill_(-1)
    busy = torch.zeros(1 << 28, device=DEV)
    side = torch.cuda.Stream()
    call({k: v.clone() for k, v in early.items()}, side)   # everything loaded
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(30):
            busy.add_(1.0)
        for k in early:
            early[k].copy_(late[k])
        waiting = torch.cuda.Event()
        waiting.record()
        got = call(early, None) if how == "current" else None
    if how == "argument":
        got = call(early, side)
    assert not waiting.query(), "the work in front was over before the call: nothing shown"
    side.synchronize()
    got = flat(got) + [early["state"], early["conv"]]
    assert len(got) == len(want)
    for a, b in zip(got, want):
        same_bits(a, b)


def test_results_are_not_memory_in_use_on_the_current_stream():
    """With `stream=`, a result must not be a block that was just freed on the
    current stream: work queued there may still be using it."""
    d, calls = _stream_calls()
    d = {k: v.to(DEV) for k, v in d.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for name in ("conv_fwd_varlen", "scan_fwd_varlen", "conv_update_varlen", "scan_update_varlen"):
        freed = [torch.empty_like(d["x"]) for _ in range(8)]
        places = {t.data_ptr() for t in freed}
        del freed
        got = calls[name](d, side)
        assert got.data_ptr() not in places, name
    side.synchronize()


# ---------------------------------------------------------------------------
# memory shared by out and operands
# ---------------------------------------------------------------------------

def test_out_in_the_columns_beside_its_operands():
    """x, z, dt, B, C and out as columns of one tensor: no element is shared."""
    T, dim, N = 70, 64, 16
    c, i = conv_inputs(T, dim, 4, 2, seed=1), scan_inputs(T, dim, N, 2, seed=1)
    w, b, pool = cuda(c, "weight", "bias", "pool")
    wide = torch.empty(T, 2 * dim, dtype=BF16, device=DEV)
    wide[:, :dim] = c["x"].to(DEV)
    cu = cu_of([40, 30])
    got = ssu.conv_fwd_varlen(wide[:, :dim], w, cu.to(DEV), bias=b, conv_state=pool, out=wide[:, dim:])
    conv_check(c, got, pool, "silu", "columns", pool=c["pool"], nseqs=2, cu=cu, prompt=True)
    d = dict(zip(OPERANDS, cuda(i, *OPERANDS)))
    names, at = ("x", "z", "dt", "B", "C", "out"), 0
    wide = torch.empty(T, 4 * dim + 2 * N, dtype=BF16, device=DEV)
    for k in names:
        n = N if k in ("B", "C") else dim
        part = wide[:, at:at + n]
        if k != "out":
            part.copy_(d[k].view(T, n))
        d[k] = part.unsqueeze(1) if k in ("B", "C") else part
        at += n
    pool = i["pool"].to(DEV)
    got = ssu.scan_fwd_varlen(d["x"], d["dt"], d["A"], d["B"], d["C"], cu.to(DEV), D=d["D"], z=d["z"],
                              dt_bias=d["dt_bias"], dt_softplus=True, state=pool, out=d["out"])
    scan_check(i, got, pool, "columns", pool=i["pool"], nseqs=2, cu=cu, prompt=True)


@pytest.mark.parametrize("name", ["x", "z", "dt"])
def test_scan_tokens_into_an_operand(name):
    i = scan_inputs(5, 75, 16, 5, 3, seed=3)
    d = dict(zip(OPERANDS, cuda(i, *OPERANDS)))
    pool = i["pool"].to(DEV)
    got = ssu.scan_update(pool, d["x"], d["dt"], d["A"], d["B"], d["C"], D=d["D"], z=d["z"],
                          dt_bias=d["dt_bias"], dt_softplus=True, out=d[name])
    assert got is d[name]
    scan_check(i, got, pool, "in place", pool=i["pool"], nseqs=5)


def test_overlapping_views_are_refused():
    T, dim, N = 6, 32, 16
    c, i = conv_inputs(T, dim, 4, 6), scan_inputs(T, dim, N, 6)
    w, pool = cuda(c, "weight", "pool")
    d = dict(zip(OPERANDS, cuda(i, *OPERANDS)))
    sp, cu = i["pool"].to(DEV), cu_of([2, 4]).to(DEV)
    buf = torch.zeros(T + 1, dim, dtype=BF16, device=DEV)
    shifted = torch.zeros(T, dim + 8, dtype=BF16, device=DEV)
    for x, out in ((buf[:-1], buf[1:]), (buf[1:], buf[:-1]), (shifted[:, :dim], shifted[:, 8:])):
        with pytest.raises(ValueError, match="overlap x"):
            ssu.conv_fwd_varlen(x, w, cu, out=out)
        with pytest.raises(ValueError, match="overlap x"):
            ssu.conv_update(pool, x, w, out=out)
        for k in ("x", "dt", "z"):
            e = {**d, k: x}
            with pytest.raises(ValueError, match=f"overlap {k}"):
                ssu.scan_fwd_varlen(e["x"], e["dt"], e["A"], e["B"], e["C"], cu, z=e["z"], out=out)
            with pytest.raises(ValueError, match=f"overlap {k}"):
                ssu.scan_update(sp, e["x"], e["dt"], e["A"], e["B"], e["C"], z=e["z"], out=out)
    for k in ("B", "C"):
        both = torch.zeros(T, dim, dtype=BF16, device=DEV)
        e = {**d, k: both[:, None, 16:]}
        with pytest.raises(ValueError, match=f"overlap {k}"):
            ssu.scan_fwd_varlen(e["x"], e["dt"], e["A"], e["B"], e["C"], cu, out=both)
        with pytest.raises(ValueError, match=f"overlap {k}"):
            ssu.scan_update(sp, e["x"], e["dt"], e["A"], e["B"], e["C"], out=both)


@pytest.mark.parametrize("slots", [40, 5000])
def test_compaction_into_a_view_of_its_table(slots):
    held = torch.randperm(slots, generator=gen(slots))[:17].int()
    want, m, moves = layer.compact(held.numpy(), slots)
    pool = torch.arange(slots, dtype=torch.int32)
    p, t = pool.to(DEV), held.to(DEV)
    out, live = ssu.slots_compact([p], t, out=t.view(17))
    assert t.tolist() == want.tolist() and int(live) == m and out.data_ptr() == t.data_ptr()
    for a, b in moves.items():
        pool[b] = a
    same_bits(p, pool)


def test_flags_without_a_truth_value():
    """The caller's own error, and nothing runs."""
    c, i = conv_inputs(3, 32, 4, 3), scan_inputs(3, 32, 16, 3)
    x, w, pool = cuda(c, "x", "weight", "pool")
    d = dict(zip(OPERANDS, cuda(i, *OPERANDS)))
    args, sp = [d[k] for k in ("x", "dt", "A", "B", "C")], i["pool"].to(DEV)

    class Neither:
        def __bool__(self):
            raise KeyError("neither")

    for call in (lambda v: ssu.conv_update(pool, x, w, disable_state_update=v),
                 lambda v: ssu.scan_update(sp, *args, disable_state_update=v),
                 lambda v: ssu.scan_update(sp, *args, dt_softplus=v)):
        with pytest.raises(KeyError, match="neither"):
            call(Neither())
    same_bits(pool, c["pool"])
    same_bits(sp, i["pool"])
